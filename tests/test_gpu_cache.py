"""The 8-bit key/value cache against the fp64 oracle: quantising as it is written,
reading back, and attention over it, at the sizes, layouts and masks where they
can go wrong.

Append and read are exact by definition (power-of-two scales, one rounding to
the nearest code), so codes and scales are compared bit for bit.

Attention's bar is derived element by element.  With A = sum_j P_j |v_j| and
S = the largest sum_c |scale q_c k_c| of the row's visible keys, n visible keys,
u = 2^-24 (half a step of fp32):
  a score's error is at most (d + 8) u S: d products summed in fp32, then the
  factors scale, log2(e) and the block's scale; the exponent's error is that
  plus 4 u |score| <= 4 u S for the shift by the maximum, plus 2^-22 for ex2;
  the sums add n u;
  a weight is rounded to fp16, half a step being 2^-11 of it: 2^-11 A (the weights
  below fp16's normal range, under 2^-22 of the largest, are off by 2^-33 of it);
  the result is rounded to bf16, half a step being 2^-8 of the value.
  |O - O_ref| <= 2^-8 |O_ref| + A (2^-11 + 2 eps),  eps = (d + 12) u S + n u + 2^-21
  |LSE - LSE_ref| <= eps + 2^-22 (1 + |LSE_ref|)
"""
import numpy as np
import pytest
import torch

from online_softmax_08_gb300 import fattn
from oracle import cache as oc

pytestmark = pytest.mark.gpu

TYPES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _no_device_error():
    fattn.fattn_device_error()
    yield
    torch.cuda.synchronize()
    assert fattn.fattn_device_error() == 0


def _bf16(rng, shape, scale=1.0):
    return torch.tensor(rng.standard_normal(shape) * scale, dtype=torch.float32).bfloat16()


class Case:
    """A cache with garbage everywhere, and a batch over scattered blocks of it.
    pairs: (n_b, tokens before them) of each sequence."""

    def __init__(self, pairs, H, d, bs, fmt="e4m3", seed=0, spare=3, pad_tokens=0, nan_slots=True):
        rng = self.rng = np.random.default_rng(seed)
        self.H, self.d, self.bs, self.fmt, self.pairs = H, d, bs, fmt, pairs
        lens = [n + p for n, p in pairs]
        need = [-(-x // bs) for x in lens]
        nb = sum(need) + spare
        order = rng.permutation(nb).tolist()
        width = max(max(need), 1) + 1
        # entries behind a sequence's blocks are out of range and must not be looked at
        table = np.full((len(pairs), width), 2 ** 30, dtype=np.int32)
        for b, n in enumerate(need):
            table[b, :n] = [order.pop() for _ in range(n)]
        self.table, self.lens = table, np.array(lens, dtype=np.int32)
        self.cu = np.concatenate([[0], np.cumsum([n for n, _ in pairs])]).astype(np.int32)
        self.T = int(self.cu[-1]) + pad_tokens
        codes = rng.integers(0, 256, (2, nb, H, bs, d)).astype(np.uint8)
        if not nan_slots:
            codes[~np.isfinite(oc.code_values(fmt)[codes])] = 0
        scale = 2.0 ** rng.integers(-9, -5, (2, nb, H))
        if fmt == "e5m2":
            scale *= 2.0 ** -7
        self.cache = {"k": codes[0], "v": codes[1], "k_scale": scale[0], "v_scale": scale[1]}

    def fill(self, nan=None):
        """Finite codes of normal values in every visible slot; the rest stays garbage."""
        for side in ("k", "v"):
            for b, length in enumerate(self.lens):
                for p in range(0, int(length), self.bs):
                    blk, c = self.table[b, p // self.bs], min(self.bs, int(length) - p)
                    x = self.rng.standard_normal((self.H, c, self.d))
                    top = oc.FORMATS[self.fmt][2]
                    for h in range(self.H):
                        s = oc.scale_for(np.abs(x[h]).max(), self.fmt)
                        self.cache[side + "_scale"][blk, h] = s
                        self.cache[side][blk, h, :c] = oc.round_codes(
                            np.clip(x[h] / s, -top, top), self.fmt)
        return self

    @property
    def batch(self):
        return self.table, self.lens, self.cu

    def on_device(self):
        c = self.cache
        dev = lambda a: torch.tensor(a, device=DEV)
        cache = fattn.KVCache(dev(c["k"]).view(TYPES[self.fmt]), dev(c["v"]).view(TYPES[self.fmt]),
                              dev(c["k_scale"].astype(np.float32)),
                              dev(c["v_scale"].astype(np.float32)))
        batch = fattn.CacheBatch(dev(self.table), dev(self.lens), dev(self.cu), self.T,
                                 max([n for n, _ in self.pairs] + [0]))
        return cache, batch


def _host(cache):
    return {"k": cache.k.view(torch.uint8).cpu().numpy(), "v": cache.v.view(torch.uint8).cpu().numpy(),
            "k_scale": cache.k_scale.cpu().double().numpy(),
            "v_scale": cache.v_scale.cpu().double().numpy()}


def _assert_cache(got, want, fmt):
    got = _host(got)
    values = oc.code_values(fmt)
    for name in ("k_scale", "v_scale"):
        np.testing.assert_array_equal(got[name], want[name])
    for name in ("k", "v"):
        nan = np.isnan(values[want[name]])
        np.testing.assert_array_equal(np.isnan(values[got[name]]), nan)  # any NaN code is NaN
        np.testing.assert_array_equal(got[name][~nan], want[name][~nan])


def _strided(x, layout):
    """x [T, heads, d] on the device as: its own tensor, a slice of a wider one, head-major."""
    x = x.to(DEV)
    if layout == "slice":
        big = torch.zeros((x.shape[0], x.shape[1] + 5, x.shape[2]), dtype=x.dtype, device=DEV)
        big[:, 2:2 + x.shape[1]] = x
        return big[:, 2:2 + x.shape[1]]
    if layout == "heads":
        return x.transpose(0, 1).contiguous().transpose(0, 1)
    return x.contiguous()


APPEND = [
    # (pairs, H, d, bs, fmt, layout)
    ([(1, 0)], 1, 64, 16, "e4m3", "own"),
    ([(1, 15), (1, 16), (1, 17), (1, 0)], 3, 128, 16, "e4m3", "slice"),
    ([(5, 11), (0, 7), (40, 3), (0, 0), (17, 31)], 2, 128, 32, "e5m2", "heads"),
    ([(300, 0), (1, 129), (64, 64), (65, 63)], 2, 64, 64, "e4m3", "slice"),
    ([(259, 77)], 1, 128, 128, "e4m3", "own"),
    ([(130, 0), (127, 1)], 2, 64, 128, "e5m2", "own"),
    ([(1, 3 * i) for i in range(37)], 2, 64, 16, "e4m3", "slice"),
    ([(i % 5, i) for i in range(1100)], 1, 64, 16, "e4m3", "own"),
]


@pytest.mark.parametrize("pairs,H,d,bs,fmt,layout", APPEND)
def test_append_then_read(pairs, H, d, bs, fmt, layout):
    c = Case(pairs, H, d, bs, fmt, seed=len(pairs) * 100 + d + bs, pad_tokens=3, nan_slots=False)
    size = np.exp(c.rng.standard_normal((c.T, 1, 1)))
    k = (_bf16(c.rng, (c.T, H, d)).float() * torch.tensor(size)).bfloat16()
    v = (_bf16(c.rng, (c.T, H, d)).float() * torch.tensor(1 / size)).bfloat16()
    cache, batch = c.on_device()
    want = oc.append(c.cache, fmt, c.batch, k.double().numpy(), v.double().numpy())
    for _ in range(2):  # the second call changes nothing
        fattn.cache_append(_strided(k, layout), _strided(v, layout), cache, batch)
        _assert_cache(cache, want, fmt)
    # read back into tensors of the same layout whose other elements stay as they were
    outs = []
    for _ in range(2):
        base = torch.full((c.T, H + 4, d), 7.0, dtype=torch.bfloat16, device=DEV)
        outs.append((base, base[:, 1:1 + H]))
    got = fattn.cache_read(cache, batch, out=(outs[0][1], outs[1][1]))
    n = int(c.cu[-1])
    for (base, part), g, ref in zip(outs, got, oc.read(want, fmt, c.batch)):
        np.testing.assert_array_equal(part[:n].cpu().double().numpy(), ref)
        base[:n, 1:1 + H] = 7.0
        assert bool((base == 7.0).all())


@pytest.mark.parametrize("bs,d", [(64, 128), (16, 64)])
def test_append_of_more_than_the_caches_hold(bs, d):
    """A prompt whose codes exceed half of L2, written in one call and block by block."""
    H, T, steps = 32, 20480 * 128 // d, 8
    g = torch.Generator(device=DEV).manual_seed(6)
    k, v = (torch.randn((T, H, d), generator=g, device=DEV).bfloat16() for _ in range(2))
    table = torch.randperm(T // bs, generator=g, device=DEV).int()[None].contiguous()
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)
    one, many = (fattn.new_cache(T // bs, H, bs, d, device=DEV) for _ in range(2))
    fattn.cache_append(k, v, one, fattn.CacheBatch(table, i32(T), i32(0, T), T, T))
    n = T // steps
    for i in range(steps):
        part = slice(i * n, (i + 1) * n)
        fattn.cache_append(k[part], v[part], many,
                           fattn.CacheBatch(table, i32((i + 1) * n), i32(0, n), n, n))
    for a, b in zip(one, many):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    # and against the definition, in 64 bits: a block's values are off by half a step
    rk, _ = fattn.cache_read(one, fattn.CacheBatch(table, i32(T), i32(0, T), T, T))
    err = (rk.double() - k.double()).abs()
    floor = one.k_scale[table[0].long()].repeat_interleave(bs, 0)[:, :, None].double() * 2.0 ** -10
    assert bool((err <= 2.0 ** -4 * k.double().abs() + floor).all())


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_append_special_values(fmt):
    """Zeros, NaN, infinities, subnormals, the largest bf16, and values at the
    border between two scales."""
    H, d, bs = 2, 64, 16
    c = Case([(16, 0), (16, 0), (16, 0), (16, 0), (16, 0), (7, 9)], H, d, bs, fmt, nan_slots=False)
    top = oc.FORMATS[fmt][2]
    k = _bf16(c.rng, (c.T, H, d))
    v = _bf16(c.rng, (c.T, H, d))
    k[0:16] = 0.0
    v[0:16] *= 1e-37
    k[16:32, 0, 3] = float("nan")
    k[16:32, 1, 5] = float("-inf")
    v[16:32] = float("inf")
    k[32:48] *= 2.0 ** 126 / 8
    v[32:48] = k[32:48]
    v[32, 0, 0] = 3.3895313892515355e38  # the largest bf16
    k[48:64] = 0.25
    k[48, 0, 0], k[48, 1, 0] = top / 64, top / 32
    v[48:64] = 1e-40
    k[64:80] = -0.0
    v[80:, 0, 1] = float("nan")
    cache, batch = c.on_device()
    want = oc.append(c.cache, fmt, c.batch, k.double().numpy(), v.double().numpy())
    fattn.cache_append(k.to(DEV), v.to(DEV), cache, batch)
    _assert_cache(cache, want, fmt)


@pytest.mark.parametrize("fmt,bs,d", [("e4m3", 16, 128), ("e5m2", 64, 64), ("e4m3", 128, 128)])
def test_token_by_token_growth(fmt, bs, d):
    """One token a call, each larger than the last: the block's scale grows and its
    earlier codes are rewritten, again and again."""
    H, steps = 2, 70
    c = Case([(1, steps), (1, 5)], H, d, bs, fmt, nan_slots=False)
    cache, batch = c.on_device()
    want = c.cache
    for i in range(steps):
        lens = np.array([i + 1, 1], dtype=np.int32)
        k, v = (_bf16(c.rng, (2, H, d), s) for s in (1.25 ** i, 0.9 ** i))
        want = oc.append(want, fmt, (c.table, lens, c.cu), k.double().numpy(), v.double().numpy())
        fattn.cache_append(k.to(DEV), v.to(DEV), cache, batch._replace(
            lens=torch.tensor(lens, device=DEV)))
    _assert_cache(cache, want, fmt)


def _check_forward(c, q, scale, causal, o, lse, rows=None):
    """Against the oracle; rows of the packed batch are checked whole."""
    n = int(c.cu[-1])
    ref, lse_ref, A, S, seen = oc.forward(c.cache, c.fmt, c.batch, q.double().numpy()[:n], scale,
                                          causal, d_error=True)
    u = 2.0 ** -24
    eps = (c.d + 12) * u * S + seen[None, :] * u + 2.0 ** -21  # [Hq, T]
    got, got_lse = o[:n].cpu().double().numpy(), lse[:, :n].cpu().double().numpy()
    bar = 2.0 ** -8 * np.abs(ref) + A * (2.0 ** -11 + 2 * eps.T[:, :, None])
    assert np.all(np.abs(got - ref) <= bar), np.nanmax(np.abs(got - ref) / np.maximum(bar, 1e-300))
    np.testing.assert_array_equal(np.isneginf(got_lse), np.isneginf(lse_ref))
    f = np.isfinite(lse_ref)
    assert np.all(np.abs(got_lse[f] - lse_ref[f]) <= (eps + 2.0 ** -22 * (1 + np.abs(lse_ref)))[f])


FORWARD = [
    # (pairs, H, G, d, bs, fmt, causal)
    ([(1, 0)], 1, 1, 64, 16, "e4m3", True),
    ([(1, 16)], 2, 1, 128, 16, "e4m3", True),
    ([(1, 1), (1, 14), (1, 15), (1, 126), (1, 127), (1, 128), (1, 300)], 2, 4, 128, 16, "e4m3", True),
    ([(1, 700), (1, 0), (1, 2100)], 2, 7, 64, 32, "e5m2", True),
    ([(1, 999)], 2, 8, 128, 128, "e4m3", False),
    ([(1, 511), (1, 33)], 1, 16, 128, 64, "e4m3", True),
    ([(1, 200)], 1, 33, 64, 64, "e4m3", True),
    ([(4, 60), (0, 9), (3, 0), (7, 250), (0, 0)], 2, 3, 128, 32, "e4m3", True),
    ([(5, 500), (5, 3)], 2, 8, 64, 16, "e5m2", True),
    ([(2, 77), (8, 1)], 2, 5, 64, 128, "e4m3", False),
    ([(40, 0), (17, 100), (1, 64)], 2, 2, 128, 64, "e4m3", True),
    ([(130, 0)], 2, 1, 64, 64, "e4m3", True),
    ([(129, 200), (1, 90), (65, 0)], 1, 4, 128, 16, "e4m3", True),
    ([(128, 128), (300, 1)], 1, 2, 64, 32, "e5m2", True),
    ([(260, 13)], 1, 3, 128, 128, "e4m3", False),
    ([(257, 130)], 1, 1, 128, 64, "e5m2", True),
    # groups larger than a row block of either kernel, and ones that do not divide it
    ([(1, 50), (3, 40)], 1, 300, 64, 16, "e4m3", True),
    ([(2, 30), (1, 77)], 1, 256, 64, 32, "e4m3", True),
    ([(3, 30)], 1, 129, 128, 16, "e5m2", True),
    ([(5, 200)], 2, 100, 64, 64, "e4m3", True),
    # more than 32 sequences, of which every kernel's search takes two steps
    ([(i % 4, 5 * i) for i in range(70)], 2, 2, 64, 16, "e4m3", True),
    ([(1 if i % 9 else 40, 2 * i + 1) for i in range(60)], 1, 2, 128, 32, "e4m3", True),
    ([(i % 2, i % 50) for i in range(1100)], 1, 1, 64, 16, "e5m2", True),
    # a unit of the 256-row kernel cut into pieces
    ([(130, 3000), (1, 70), (70, 5000)], 1, 1, 64, 64, "e4m3", True),
    ([(33, 2600)], 1, 3, 128, 16, "e4m3", False),
    # more than 256 sequences or row blocks for its plan, whole and with one that is cut
    ([(40, i % 90) for i in range(300)], 1, 1, 64, 16, "e4m3", True),
    ([(600, 2000)] + [(40 if i % 3 else 1, i) for i in range(280)], 1, 1, 64, 32, "e5m2", True),
    ([(520, 7)], 1, 128, 64, 64, "e4m3", True),
]


@pytest.mark.parametrize("pairs,H,G,d,bs,fmt,causal", FORWARD)
@pytest.mark.parametrize("layout", ["own", "slice", "heads"])
def test_forward_matches_oracle(pairs, H, G, d, bs, fmt, causal, layout):
    c = Case(pairs, H, d, bs, fmt, seed=d + bs + G + len(pairs), pad_tokens=2).fill()
    q = _bf16(c.rng, (c.T, H * G, d), 1.5)
    cache, batch = c.on_device()
    base = torch.full((c.T, H * G + 3, d), 7.0, dtype=torch.bfloat16, device=DEV)
    scale = d ** -0.5
    o, lse = fattn.cache_forward(_strided(q, layout), cache, batch, scale, causal,
                                 out=base[:, 1:1 + H * G])
    _check_forward(c, q, scale, causal, o, lse)
    base[:int(c.cu[-1]), 1:1 + H * G] = 7.0  # padded rows and neighbouring heads untouched
    assert bool((base == 7.0).all())


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,length,G", [(5, 2, 2), (3, 0, 1), (40, 7, 4), (300, 20, 1)])
def test_rows_that_see_nothing(n, length, G, causal):
    """More queries than tokens: with the causal mask the first ones see no key."""
    H, d = 2, 64
    c = Case([(1, 40), (n, length - n), (1, 3)], H, d, 16).fill()
    q = _bf16(c.rng, (c.T, H * G, d))
    cache, batch = c.on_device()
    o, lse = fattn.cache_forward(q.to(DEV), cache, batch, 0.125, causal)
    _check_forward(c, q, 0.125, causal, o, lse)
    blind = int(max(0, n - length)) if causal else (n if length == 0 else 0)
    rows = slice(1, 1 + blind)
    assert bool((o[rows] == 0).all()) and bool(torch.isneginf(lse[:, rows]).all())


@pytest.mark.parametrize("n,G", [(4, 2), (20, 4), (150, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_nan_in_values_a_query_does_not_see(n, G, d):
    """A token whose keys and values are NaN, in the causal part: the queries before
    it stay finite and right, it and the ones behind it become NaN."""
    H, bs, prior = 2, 16, 37
    c = Case([(n, prior)], H, d, bs, seed=n + d).fill()
    bad = prior + n // 2
    c.cache["v"][c.table[0, bad // bs], 1, bad % bs, 3] = 0xff
    q = _bf16(c.rng, (c.T, H * G, d))
    cache, batch = c.on_device()
    o, lse = fattn.cache_forward(q.to(DEV), cache, batch, d ** -0.5, True)
    got = o.cpu().double().numpy()
    nan = np.zeros(got.shape, dtype=bool)
    nan[n // 2:, G:, 3] = True
    np.testing.assert_array_equal(np.isnan(got), nan)
    # the rest as if the value were zero: compare where it is finite
    c.cache["v"][c.table[0, bad // bs], 1, bad % bs, 3] = 0
    ref = o.clone()
    ref[torch.tensor(nan, device=DEV)] = 0
    r, lse_ref, A, S, seen = oc.forward(c.cache, c.fmt, c.batch, q.double().numpy(), d ** -0.5, True,
                                        d_error=True)
    r[nan], A[nan] = 0, 0
    eps = (d + 12) * 2.0 ** -24 * S + seen[None] * 2.0 ** -24 + 2.0 ** -21
    bar = 2.0 ** -8 * np.abs(r) + A * (2.0 ** -11 + 2 * eps.T[:, :, None])
    assert np.all(np.abs(ref.cpu().double().numpy() - r) <= bar)
    # a NaN key makes NaN of every column of the rows that see it, and of no other
    c.cache["k"][c.table[0, bad // bs], 0, bad % bs, 1] = 0x7f
    cache, batch = c.on_device()
    o, lse = fattn.cache_forward(q.to(DEV), cache, batch, d ** -0.5, True)
    nan = np.zeros(got.shape, dtype=bool)
    nan[n // 2:, :G] = True
    np.testing.assert_array_equal(np.isnan(o.cpu().double().numpy()), nan)
    np.testing.assert_array_equal(np.isnan(lse.cpu().numpy()), nan[:, :, 0].T)


@pytest.mark.parametrize("n", [1, 6, 140])
def test_logits_scales_and_zero_blocks(n):
    """Large logits whose maximum rises late, blocks whose values differ by 2^20 or
    are all zero (the smallest scale), and queries far from one in size."""
    H, G, d, bs = 2, 2, 128, 16
    c = Case([(n, 300), (n, 64)], H, d, bs, seed=n).fill()
    for b in range(2):
        for j in range(3):
            c.cache["v_scale"][c.table[b, j]] *= 2.0 ** (10 * j - 10)
        c.cache["v"][c.table[b, 3]] = 0
        c.cache["v_scale"][c.table[b, 3]] = 2.0 ** -100
        c.cache["k_scale"][c.table[b, 2]] *= 8.0
    q = _bf16(c.rng, (c.T, H * G, d), 3.0)
    q[:, 1] *= 2.0 ** 30
    cache, batch = c.on_device()
    for scale in (d ** -0.5, 2.0 ** -33):
        o, lse = fattn.cache_forward(q.to(DEV), cache, batch, scale, True)
        _check_forward(c, q, scale, True, o, lse)


def test_values_of_any_size():
    """Values around 2^-60 and 2^100: the result scales with them."""
    H, G, d, bs = 1, 2, 64, 16
    c = Case([(2, 100)], H, d, bs).fill()
    q = _bf16(c.rng, (c.T, H * G, d))
    base = c.cache["v_scale"].copy()
    for e in (-60, 0, 100):
        c.cache["v_scale"] = base * 2.0 ** e
        cache, batch = c.on_device()
        o, lse = fattn.cache_forward(q.to(DEV), cache, batch, 0.125, True)
        _check_forward(c, q, 0.125, True, o, lse)


def test_scales_that_are_no_powers_of_two():
    H, G, d, bs = 2, 3, 64, 32
    c = Case([(1, 200), (9, 70)], H, d, bs).fill()
    for side in ("k_scale", "v_scale"):
        c.cache[side] = (c.cache[side] * c.rng.uniform(0.5, 1.5, c.cache[side].shape)) \
            .astype(np.float32).astype(np.float64)
    q = _bf16(c.rng, (c.T, H * G, d))
    cache, batch = c.on_device()
    o, lse = fattn.cache_forward(q.to(DEV), cache, batch, 0.125, True)
    _check_forward(c, q, 0.125, True, o, lse)
    for got, ref in zip(fattn.cache_read(cache, batch), oc.read(c.cache, c.fmt, c.batch)):
        assert np.all(np.abs(got.cpu().double().numpy() - ref) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(ref))


def _torch_reference(c, cache, q, scale, causal):
    """O, LSE, A, S and the visible keys as oc.forward gives them, in 64 bits on the device."""
    k = cache.k.view(torch.uint8).view(TYPES[c.fmt]).double() * cache.k_scale.double()[..., None, None]
    v = cache.v.view(torch.uint8).view(TYPES[c.fmt]).double() * cache.v_scale.double()[..., None, None]
    T, Hq, d = q.shape
    G = Hq // c.H
    out = [torch.zeros((T, Hq, d)).double(), torch.full((Hq, T), -np.inf).double(),
           torch.zeros((T, Hq, d)).double(), torch.zeros((Hq, T)).double(), np.zeros(T, dtype=int)]
    for b, length in enumerate(c.lens):
        lo, n = int(c.cu[b]), int(c.cu[b + 1] - c.cu[b])
        rows = torch.tensor(c.table[b][:-(-int(length) // c.bs)].astype(np.int64), device=DEV)
        kb = k[rows].transpose(0, 1).reshape(c.H, -1, d)[:, :length]
        vb = v[rows].transpose(0, 1).reshape(c.H, -1, d)[:, :length]
        at = torch.arange(int(length), device=DEV)
        for i in range(n):
            lim = int(length) - n + i + 1 if causal else int(length)
            x = q[lo + i].double().reshape(c.H, G, d)
            s = scale * x @ kb.transpose(1, 2)
            s = s.masked_fill(at >= lim, -np.inf)
            w = torch.softmax(s, 2)
            out[0][lo + i] = (w @ vb).reshape(Hq, d).cpu()
            out[1][:, lo + i] = torch.logsumexp(s, 2).reshape(Hq).cpu()
            out[2][lo + i] = (w @ vb.abs()).reshape(Hq, d).cpu()
            out[3][:, lo + i] = (scale * x.abs() @ kb.abs().transpose(1, 2)).masked_fill(
                at >= lim, 0).amax(2).reshape(Hq).cpu()
            out[4][lo + i] = lim
    return [x if isinstance(x, np.ndarray) else x.numpy() for x in out]


@pytest.mark.parametrize("pairs,H,G,d,bs,fmt", [
    ([(1, 9000), (2, 17000), (1, 300)], 40, 1, 128, 16, "e4m3"),
    ([(1, 20000), (3, 30000)], 48, 2, 64, 64, "e4m3"),
    ([(9, 7000), (12, 900)], 16, 1, 128, 128, "e5m2"),
])
def test_long_shares(pairs, H, G, d, bs, fmt):
    """Enough keys that every CTA's share runs through several sets of 32 tiles, and
    through whole units and pieces of them."""
    c = Case(pairs, H, d, bs, fmt, nan_slots=False)
    g = torch.Generator(device=DEV).manual_seed(4)
    q = _bf16(c.rng, (c.T, H * G, d)).to(DEV)
    cache, batch = c.on_device()
    for codes, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        x = torch.randn(codes.shape, generator=g, device=DEV)
        codes.copy_((x * 8).to(codes.dtype))
        scale.fill_(0.125)
    o, lse = fattn.cache_forward(q, cache, batch, d ** -0.5, True)
    ref, lse_ref, A, S, seen = _torch_reference(c, cache, q, d ** -0.5, True)
    u = 2.0 ** -24
    eps = (d + 12) * u * S + seen[None, :] * u + 2.0 ** -21
    bar = 2.0 ** -8 * np.abs(ref) + A * (2.0 ** -11 + 2 * eps.T[:, :, None])
    assert np.all(np.abs(o.cpu().double().numpy() - ref) <= bar)
    assert np.all(np.abs(lse.cpu().double().numpy() - lse_ref) <= eps + 2.0 ** -22 * (1 + np.abs(lse_ref)))


@pytest.mark.parametrize("d", [64, 128])
def test_nan_in_a_unit_cut_into_pieces(d):
    H, bs, n, prior = 1, 32, 80, 3000
    c = Case([(n, prior)], H, d, bs, seed=d).fill()
    q = _bf16(c.rng, (n, H, d))
    bad = prior + 41
    c.cache["v"][c.table[0, bad // bs], 0, bad % bs, 7] = 0x7f
    early = 500  # seen by every row, in another piece
    c.cache["v"][c.table[0, early // bs], 0, early % bs, 9] = 0xff
    cache, batch = c.on_device()
    o, _ = fattn.cache_forward(q.to(DEV), cache, batch, d ** -0.5, True)
    nan = np.zeros((n, H, d), dtype=bool)
    nan[41:, :, 7] = True
    nan[:, :, 9] = True
    np.testing.assert_array_equal(np.isnan(o.cpu().double().numpy()), nan)


@pytest.mark.parametrize("d,fmt", [(64, "e5m2"), (128, "e4m3")])
@pytest.mark.parametrize("n,G", [(65, 1), (41, 3), (128, 1)])
def test_units_of_at_most_128_rows(n, G, d, fmt):
    """The second subtile has no rows, or few: one tile to many, whole and cut, with an odd
    and an even number of tiles, ends inside a tile, and the first rows blind."""
    lens = [n // 2, n, 128, 129, 256, 300, 385, 640, 900, 1025, 3001]
    c = Case([(n, length - n) for length in lens], 1, d, 32, fmt, seed=n + d).fill()
    q = _bf16(c.rng, (c.T, G, d), 1.5)
    cache, batch = c.on_device()
    for causal in (True, False):
        o, lse = fattn.cache_forward(q.to(DEV), cache, batch, d ** -0.5, causal)
        _check_forward(c, q, d ** -0.5, causal, o, lse)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tile", [0, 1, 2, 3])
def test_nan_in_values_of_no_weight(d, tile):
    """A value that is NaN reaches every row that sees it, even one whose weight of that
    tile is zero: the keys of one tile win by more than fp32 holds."""
    n, bs = 100, 16
    c = Case([(n, 500)], 1, d, bs, seed=d + tile).fill()
    for i in range(128 // bs):  # of the neighbouring tile
        block = c.table[0, (tile ^ 1) * 128 // bs + i]
        c.cache["k"][block] = 0x70  # 128
        c.cache["k_scale"][block] = 1.0
    at = tile * 128 + 5
    c.cache["v"][c.table[0, at // bs], 0, at % bs, 11] = 0x7f
    q = torch.ones((n, 1, d), dtype=torch.bfloat16)
    cache, batch = c.on_device()
    o, lse = fattn.cache_forward(q.to(DEV), cache, batch, 1.0, True)
    nan = np.zeros((n, 1, d), dtype=bool)
    nan[:, :, 11] = True
    np.testing.assert_array_equal(np.isnan(o.cpu().double().numpy()), nan)
    assert bool(torch.isfinite(lse).all())


def test_graph_of_a_mixed_batch():
    """Pieces of prompts and single tokens captured together; lengths and offsets move
    between replays, and a replay with fewer tokens leaves the rows behind them alone."""
    H, G, d, bs = 2, 4, 64, 16
    c = Case([(100, 30), (1, 400), (20, 60), (1, 9)], H, d, bs, nan_slots=False).fill()
    q = _bf16(c.rng, (c.T, H * G, d))
    cache, batch = c.on_device()
    qd = q.to(DEV)
    out = torch.full_like(qd, 7.0)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fattn.cache_forward(qd, cache, batch, 0.125, True)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        _, lse = fattn.cache_forward(qd, cache, batch, 0.125, True, out=out)
    for n, lens in (((100, 1, 20, 1), (130, 401, 80, 10)), ((2, 70, 0, 5), (100, 390, 80, 10)),
                    ((1, 1, 1, 1), (130, 401, 80, 10)), ((90, 1, 30, 1), (130, 300, 30, 1))):
        c.lens = np.array(lens, dtype=np.int32)
        c.cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        batch.lens.copy_(torch.tensor(c.lens))
        batch.cu_seqlens.copy_(torch.tensor(c.cu))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        _check_forward(c, q, 0.125, True, out, lse)
        assert bool((out[int(c.cu[-1]):] == 7.0).all())


def test_offsets_that_do_not_ascend():
    """Nothing is written out of place, and the word is set."""
    H, G, d, bs = 1, 2, 64, 16
    c = Case([(40, 30), (50, 40), (60, 50), (1, 3)], H, d, bs).fill()
    q = _bf16(c.rng, (c.T, H * G, d)).to(DEV)
    x = _bf16(c.rng, (c.T, H, d)).to(DEV)
    cache, batch = c.on_device()
    for cu in ([0, 60, 0, 60, 0], [0, 40, 90, 40, 151], [5, 5, 2 ** 31 - 1, 90, -7],
               [0, 60, 10, 70, 20]):
        bad = batch._replace(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV))
        base = torch.full((c.T + 2, H * G, d), 7.0, dtype=torch.bfloat16, device=DEV)
        fattn.cache_forward(q, cache, bad, 0.125, True, out=base[1:-1])
        assert fattn.fattn_device_error() != 0
        assert bool((base[0] == 7.0).all()) and bool((base[-1] == 7.0).all())
        kv = [torch.full((c.T + 2, H, d), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        fattn.cache_read(cache, bad, out=(kv[0][1:-1], kv[1][1:-1]))
        assert fattn.fattn_device_error() != 0
        for t in kv:
            assert bool((t[0] == 7.0).all()) and bool((t[-1] == 7.0).all())
        fattn.cache_append(x, x, cache, bad)
        assert fattn.fattn_device_error() != 0


def test_nothing_to_do():
    c = Case([(0, 40), (0, 0)], 2, 64, 16).fill()
    cache, batch = c.on_device()
    q = torch.empty((0, 4, 64), dtype=torch.bfloat16, device=DEV)
    x = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    before = _host(cache)
    o, lse = fattn.cache_forward(q, cache, batch, 0.1, True)
    assert o.shape == (0, 4, 64) and lse.shape == (4, 0)
    fattn.cache_append(x, x, cache, batch)
    assert fattn.cache_read(cache, batch)[0].shape == (0, 2, 64)
    after = _host(cache)
    for name in before:
        np.testing.assert_array_equal(before[name], after[name])
    # padded rows only
    c = Case([(0, 40), (0, 5)], 2, 64, 16, pad_tokens=3).fill()
    cache, batch = c.on_device()
    out = torch.full((3, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    for most in (0, 3):
        fattn.cache_forward(torch.zeros_like(out), cache, batch._replace(max_seqlen=most), 0.1, True,
                            out=out)
    assert bool((out == 7.0).all())


def test_shared_prefix():
    """Two sequences whose first blocks are the same ones."""
    H, G, d, bs = 2, 2, 64, 16
    c = Case([(1, 70), (3, 70)], H, d, bs).fill()
    c.table[1, :4] = c.table[0, :4]
    q = _bf16(c.rng, (c.T, H * G, d))
    cache, batch = c.on_device()
    o, lse = fattn.cache_forward(q.to(DEV), cache, batch, 0.125, True)
    _check_forward(c, q, 0.125, True, o, lse)


def test_long_context_and_far_blocks():
    """One sequence of 70000 tokens; codes beyond 2^32 bytes from the pool's start."""
    H, G, d, bs = 1, 4, 128, 128
    nb = (1 << 32) // (bs * d) + 600
    k, v = (torch.zeros((nb, H, bs, d), dtype=torch.uint8, device=DEV) for _ in range(2))
    g = torch.Generator(device=DEV).manual_seed(1)
    n = 70000
    need = -(-n // bs)
    table = torch.arange(nb - need, nb, dtype=torch.int32, device=DEV)[None]
    for x in (k, v):
        x[nb - need:] = torch.randn((need, H, bs, d), generator=g, device=DEV).to(
            torch.float8_e4m3fn).view(torch.uint8)
    ones = torch.ones((nb, H), device=DEV)
    cache = fattn.KVCache(k.view(TYPES["e4m3"]), v.view(TYPES["e4m3"]), ones, ones)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)
    batch = fattn.CacheBatch(table, i32(n), i32(0, 2), 2, 2)
    q = torch.randn((2, H * G, d), generator=g, device=DEV).bfloat16()
    o, lse = fattn.cache_forward(q, cache, batch, d ** -0.5, True)
    kk = k[nb - need:].view(TYPES["e4m3"]).double().reshape(-1, d)
    vv = v[nb - need:].view(TYPES["e4m3"]).double().reshape(-1, d)
    for i in range(2):
        lim = n - 1 + i
        s = q[i].double() @ kk[:lim].t() * d ** -0.5
        p = torch.softmax(s, 1)
        ref, A = p @ vv[:lim], p @ vv[:lim].abs()
        S = (q[i].double().abs() @ kk[:lim].abs().t() * d ** -0.5).amax(1, keepdim=True)
        eps = (d + 12) * 2.0 ** -24 * S + n * 2.0 ** -24 + 2.0 ** -21
        assert bool(((o[i].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + A * (2.0 ** -11 + 2 * eps)).all())
        want = torch.logsumexp(s, 1)
        assert bool(((lse[:, i].double() - want).abs() <= eps[:, 0] + 2.0 ** -22 * (1 + want.abs())).all())
    # and the writer and reader there
    x = torch.randn((2, H, d), generator=g, device=DEV).bfloat16()
    fattn.cache_append(x, x, cache, batch)
    rk, rv = fattn.cache_read(cache, batch)
    torch.testing.assert_close(rk, x, rtol=2.0 ** -4, atol=2.0 ** -9)
    assert torch.equal(rk, rv)


def test_bad_entries_are_skipped_and_reported():
    H, G, d, bs = 2, 2, 64, 16
    c = Case([(2, 30), (3, 40), (2, 50)], H, d, bs).fill()
    q = _bf16(c.rng, (c.T, H * G, d))
    cache, batch = c.on_device()
    before = _host(cache)
    x = _bf16(c.rng, (c.T, H, d)).to(DEV)
    o = torch.full((c.T, H * G, d), 7.0, dtype=torch.bfloat16, device=DEV)
    good, _ = fattn.cache_forward(q.to(DEV), cache, batch, 0.125, True)
    width = batch.block_table.shape[1]
    for lens in ([32, 1000000, 52], [32, -1, 52], [32, width * bs + 1, 52]):
        bad = batch._replace(lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
        o.fill_(7.0)
        fattn.cache_forward(q.to(DEV), cache, bad, 0.125, True, out=o)
        assert fattn.fattn_device_error() == 0x460
        assert torch.equal(o[:2], good[:2]) and torch.equal(o[5:], good[5:])
        assert bool((o[2:5] == 7.0).all())
    for lens, cu in (([32, 2, 52], [0, 2, 5, 7]), ([32, 43, 52], [0, 2, 100, 7]),
                     ([32, 43, 52], [0, 2, -1, 7])):
        bad = batch._replace(lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
                             cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV))
        fattn.cache_append(x, x, cache, bad)
        assert fattn.fattn_device_error() == 0x440
        after = _host(cache)
        for b in (1,):
            for j in range(3):
                np.testing.assert_array_equal(after["k"][c.table[b, j]], before["k"][c.table[b, j]])
        fattn.cache_read(cache, bad)
        assert fattn.fattn_device_error() == 0x450
    # a block number out of range: its tokens are dropped
    for page in (-1, cache.k.shape[0], 2 ** 31 - 1):
        c2 = Case([(2, 30), (3, 40)], H, d, bs, seed=9).fill()
        q2 = _bf16(c2.rng, (c2.T, H * G, d))
        cache2, batch2 = c2.on_device()
        batch2.block_table[1, 1] = page
        o2, _ = fattn.cache_forward(q2.to(DEV), cache2, batch2, 0.125, True)
        assert fattn.fattn_device_error() == 0x461
        # as if the block's keys were not there: the same attention without them
        keep = np.r_[0:16, 32:43]
        kk = oc.tokens(c2.cache, "e4m3", c2.table[1], "k", 0, 43)
        vv = oc.tokens(c2.cache, "e4m3", c2.table[1], "v", 0, 43)
        for i in range(3):
            see = keep[keep <= 40 + i]
            for hq in range(H * G):
                s = 0.125 * kk[see, hq // G] @ q2[2 + i, hq].double().numpy()
                w = np.exp(s - s.max())
                w /= w.sum()
                ref, A = w @ vv[see, hq // G], w @ np.abs(vv[see, hq // G])
                err = np.abs(o2[2 + i, hq].cpu().double().numpy() - ref)
                assert np.all(err <= 2.0 ** -8 * np.abs(ref) + A * 2.0 ** -10)
        batch2.block_table[1, 1] = int(c2.table[1, 1])
        batch2.block_table[1, 2] = page
        x2 = _bf16(c2.rng, (c2.T, H, d)).to(DEV)
        fattn.cache_append(x2, x2, cache2, batch2)
        assert fattn.fattn_device_error() == 0x441
        rk, rv = fattn.cache_read(cache2, batch2)
        assert fattn.fattn_device_error() == 0x451
        assert bool((rk[2:] == 0).all()) and bool((rv[2:] == 0).all()) and bool((rk[:2] != 0).any())


def test_serving_run():
    """A prompt in two pieces, then tokens one by one: append, attend and read back as
    a server does, eagerly and replayed from a captured graph."""
    H, G, d, bs, B = 2, 3, 64, 16, 3
    rng = np.random.default_rng(11)
    cache = fattn.new_cache(24, H, bs, d, device=DEV)
    table = torch.tensor(rng.permutation(24).reshape(B, 8).astype(np.int32), device=DEV)
    host = {n: a.copy() for n, a in _host(cache).items()}
    tab = table.cpu().numpy()
    done = np.zeros(B, dtype=np.int32)

    def batch_of(n):
        cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        return cu, fattn.CacheBatch(table, torch.tensor(done + n, dtype=torch.int32, device=DEV),
                                    torch.tensor(cu, device=DEV), int(cu[-1]), int(max(n)))

    def step(n, run):
        nonlocal host, done
        n = np.array(n, dtype=np.int32)
        cu, batch = batch_of(n)
        T = int(cu[-1])
        q, k, v = _bf16(rng, (T, H * G, d)), _bf16(rng, (T, H, d)), _bf16(rng, (T, H, d))
        o, lse = run(q.to(DEV), k.to(DEV), v.to(DEV), batch)
        done = done + n
        host = oc.append(host, "e4m3", (tab, done, cu), k.double().numpy(), v.double().numpy())
        _assert_cache(cache, host, "e4m3")
        c = Case.__new__(Case)
        c.cache, c.fmt, c.table, c.lens, c.cu, c.d = host, "e4m3", tab, done, cu, d
        _check_forward(c, q, 0.125, True, o, lse)

    def eager(q, k, v, batch):
        fattn.cache_append(k, v, cache, batch)
        return fattn.cache_forward(q, cache, batch, 0.125, True)

    step([20, 45, 1], eager)
    step([33, 0, 7], eager)
    step([1, 1, 1], eager)

    # one token a step, captured once; lengths move on the device
    sq = torch.zeros((B, H * G, d), dtype=torch.bfloat16, device=DEV)
    sk, sv = (torch.zeros((B, H, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    _, batch = batch_of(np.ones(B, dtype=np.int32))
    so = torch.empty_like(sq)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        fattn.cache_append(sk, sv, cache, batch)
        _, slse = fattn.cache_forward(sq, cache, batch, 0.125, True, out=so)

    def replayed(q, k, v, b):
        sq.copy_(q), sk.copy_(k), sv.copy_(v), batch.lens.copy_(b.lens)
        graph.replay()
        return so, slse

    for _ in range(18):
        step([1, 1, 1], replayed)
    total = int(done.sum())
    cu = np.concatenate([[0], np.cumsum(done)]).astype(np.int32)
    whole = fattn.CacheBatch(table, torch.tensor(done, device=DEV), torch.tensor(cu, device=DEV),
                             total, int(done.max()))
    for got, ref in zip(fattn.cache_read(cache, whole), oc.read(host, "e4m3", (tab, done, cu))):
        np.testing.assert_array_equal(got.cpu().double().numpy(), ref)


def test_other_stream_and_repeatability():
    """Work on a stream of the caller's, and the same bits on every call."""
    H, G, d = 2, 4, 128
    c = Case([(1, 900), (1, 2000), (30, 77)], H, d, 64).fill()
    q = _bf16(c.rng, (c.T, H * G, d)).to(DEV)
    cache, batch = c.on_device()
    o, lse = fattn.cache_forward(q, cache, batch, 0.1, True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (s, s.cuda_stream):
        for _ in range(3):
            o2, lse2 = fattn.cache_forward(q, cache, batch, 0.1, True, stream=stream)
            s.synchronize()
            assert torch.equal(o, o2) and torch.equal(lse, lse2)
        k, v = fattn.cache_read(cache, batch, stream=stream)
        s.synchronize()
        k2, v2 = fattn.cache_read(cache, batch)
        assert torch.equal(k, k2) and torch.equal(v, v2)


def test_workspaces_that_are_refused():
    c = Case([(1, 20)], 1, 64, 16).fill()
    q = _bf16(c.rng, (c.T, 2, 64)).to(DEV)
    cache, batch = c.on_device()
    big = torch.empty((2, 64 << 20), dtype=torch.uint8, device=DEV)
    for ws in (torch.empty(64 << 20, dtype=torch.uint8), big[:, ::2]):
        with pytest.raises(ValueError):
            fattn.cache_forward(q, cache, batch, 0.125, True, workspace=ws)
    with pytest.raises(fattn.FattnError):
        fattn.cache_forward(q, cache, batch, 0.125, True, workspace=big[0, :256])
    o, lse = fattn.cache_forward(q, cache, batch, 0.125, True, workspace=big[0])
    _check_forward(c, q.cpu(), 0.125, True, o, lse)


def test_workspace_inside_sentinels():
    H, G, d = 2, 4, 128
    c = Case([(1, 900), (5, 300), (70, 10)], H, d, 64).fill()
    q = _bf16(c.rng, (c.T, H * G, d))
    cache, batch = c.on_device()
    cc, bb = fattn._cache_args(cache, batch)[:2]
    need = int(fattn.load().fattn_cache_fwd_workspace_bytes(cc, bb, H * G))
    buf = torch.full((need + 1024,), 0xa5, dtype=torch.uint8, device=DEV)
    ws = buf[512:512 + need]
    with pytest.raises(fattn.FattnError):
        fattn.cache_forward(q.to(DEV), cache, batch, 0.1, True, workspace=buf[512:512 + need - 1])
    o, lse = fattn.cache_forward(q.to(DEV), cache, batch, 0.1, True, workspace=ws)
    _check_forward(c, q, 0.1, True, o, lse)
    assert bool((buf[:512] == 0xa5).all()) and bool((buf[512 + need:] == 0xa5).all())
