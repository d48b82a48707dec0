"""The 4-bit key/value cache against the fp64 oracle: quantising as it is written, reading
back, and attention over it, at the sizes, layouts and masks where they can go wrong.

Append and read are exact by definition (the scale's one rounding to e5m2, the code's one to a
whole number, ties to even; a value has at most 7 significant bits), so codes, scales and values
are compared bit for bit.  Attention's bar is that of the 8-bit cache, derived element by element
in test_gpu_cache.py: the values are exact in fp16 there as here, and the further factor of a
block's scale is 1 here.  That bar leaves out what it states of the smallest weights; here, where
a channel can be zero in every key but one, they count.  The largest weight of a row is held as
2^8 or more, half a step of fp16's subnormal range is 2^-25, so a weight is off by up to 2^-33 of
the largest one, which is at most 1: 2^-33 sum_j |v_j| more, over the visible keys.
"""
import numpy as np
import pytest
import torch

import test_gpu_cache as base
from online_softmax_08_gb300 import fattn
from oracle import cache4 as oc4

pytestmark = pytest.mark.gpu

DEV = base.DEV
_bf16, _strided = base._bf16, base._strided


@pytest.fixture(autouse=True)
def _no_device_error():
    fattn.fattn_device_error()
    yield
    torch.cuda.synchronize()
    assert fattn.fattn_device_error() == 0


class Case(base.Case):
    """A 4-bit cache with garbage everywhere (scales that are infinite or NaN among it), and a
    batch over scattered blocks of it."""

    def __init__(self, pairs, H, d, bs, seed=0, spare=3, pad_tokens=0):
        super().__init__(pairs, H, d, bs, "e4m3", seed, spare, pad_tokens)
        nb = self.cache["k"].shape[0]
        byte = lambda n: self.rng.integers(0, 256, (nb, H, bs, n)).astype(np.uint8)
        self.cache = {"k": byte(d // 2), "v": byte(d // 2), "k_scale": byte(d // 16),
                      "v_scale": byte(d // 16)}

    def fill(self, size=1.0):
        """Tokens of normal values in every visible slot; the rest stays garbage."""
        for side in ("k", "v"):
            for b, length in enumerate(self.lens):
                p = np.arange(int(length))
                at = (self.table[b, p // self.bs], slice(None), p % self.bs)
                x = self.rng.standard_normal((len(p), self.H, self.d)) * size
                x[..., :16] *= 8.0
                self.cache[side][at], self.cache[side + "_scale"][at] = oc4.quantise(x)
        return self

    def on_device(self):
        c = self.cache
        dev = lambda a: torch.tensor(a, device=DEV)
        cache = fattn.KVCache(dev(c["k"]), dev(c["v"]), dev(c["k_scale"]).view(torch.float8_e5m2),
                              dev(c["v_scale"]).view(torch.float8_e5m2))
        batch = fattn.CacheBatch(dev(self.table), dev(self.lens), dev(self.cu), self.T,
                                 max([n for n, _ in self.pairs] + [0]))
        return cache, batch


def _assert_cache(got, want):
    for name in want:
        np.testing.assert_array_equal(getattr(got, name).view(torch.uint8).cpu().numpy(), want[name])


@pytest.mark.parametrize("pairs,H,d,bs,layout", [a[:4] + a[5:] for a in base.APPEND])
def test_append_then_read(pairs, H, d, bs, layout):
    c = Case(pairs, H, d, bs, seed=len(pairs) * 100 + d + bs, pad_tokens=3)
    size = np.exp(c.rng.standard_normal((c.T, 1, 1)))
    k = (_bf16(c.rng, (c.T, H, d)).float() * torch.tensor(size)).bfloat16()
    v = (_bf16(c.rng, (c.T, H, d)).float() * torch.tensor(1 / size)).bfloat16()
    cache, batch = c.on_device()
    want = oc4.append(c.cache, c.batch, k.double().numpy(), v.double().numpy())
    for _ in range(2):  # the second call changes nothing
        fattn.cache_append(_strided(k, layout), _strided(v, layout), cache, batch)
        _assert_cache(cache, want)
    outs = []
    for _ in range(2):
        whole = torch.full((c.T, H + 4, d), 7.0, dtype=torch.bfloat16, device=DEV)
        outs.append((whole, whole[:, 1:1 + H]))
    got = fattn.cache_read(cache, batch, out=(outs[0][1], outs[1][1]))
    n = int(c.cu[-1])
    for (whole, part), g, ref in zip(outs, got, oc4.read(want, c.batch)):
        np.testing.assert_array_equal(part[:n].cpu().double().numpy(), ref)
        whole[:n, 1:1 + H] = 7.0
        assert bool((whole == 7.0).all())


def test_append_special_values():
    """Zeros, NaN, infinities, subnormals, the largest bf16, ties between codes and between
    scales, and groups whose largest magnitude comes with both signs."""
    H, d, bs = 2, 64, 16
    c = Case([(16, 0)] * 9, H, d, bs)
    k, v = _bf16(c.rng, (c.T, H, d)), _bf16(c.rng, (c.T, H, d))
    k[0:16] = 0.0
    v[0:16] *= 1e-37
    k[16:32, 0, 3] = float("nan")
    k[16:32, 1, 5] = float("-inf")
    v[16:32] = float("inf")
    k[32:48] *= 2.0 ** 126 / 8
    v[32:48] = k[32:48]
    v[32, 0, 0] = 3.3895313892515355e38
    k[48:64, :, ::16] = 8.0  # scale -1: halves are ties
    k[48:64, :, 1::16] = -8.0
    k[48:64, :, 2:16] = torch.arange(-7, 7)[None, None] + 0.5
    v[48:64, :, ::16] = -10.0  # scale 1.25: multiples of 0.625
    v[48:64, :, 1:16] = (torch.arange(-7, 8)[None, None]) * 0.625
    k[64:80] = -0.0
    k[80:96, :, 7] = 9.0  # a / 8 = 1.125, halfway between two scales
    v[80:96, :, 7] = -11.0
    k[96:112] *= 2.0 ** -13
    v[96:112] *= 2.0 ** -16
    k[112:128] = float("nan")
    v[112:128, :, 9] = 57344.0
    v[128:] = 2.0 ** -14 * torch.arange(64)[None, None]
    cache, batch = c.on_device()
    want = oc4.append(c.cache, c.batch, k.double().numpy(), v.double().numpy())
    fattn.cache_append(k.to(DEV), v.to(DEV), cache, batch)
    got = {n: getattr(cache, n).view(torch.uint8).cpu().numpy() for n in cache._fields}
    for side in ("k", "v"):
        scale, ref = got[side + "_scale"], want[side + "_scale"]
        zero = (ref & 0x7f) == 0  # the sign of a scale of zero does not matter
        np.testing.assert_array_equal(scale[~zero], ref[~zero])
        assert not np.any(scale[zero] & 0x7f)
        np.testing.assert_array_equal(got[side], want[side])


def test_append_error_bound():
    """Every value that is written is off by at most half a scale, or what the range cuts."""
    g = torch.Generator(device=DEV).manual_seed(5)
    T, H, d = 4096, 4, 128
    k, v = (torch.randn((T, H, d), generator=g, device=DEV).bfloat16() for _ in range(2))
    cache = fattn.new_cache(T // 64, H, 64, d, dtype=torch.uint8, device=DEV)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)
    batch = fattn.CacheBatch(torch.randperm(T // 64, generator=g, device=DEV).int()[None].contiguous(),
                             i32(T), i32(0, T), T, T)
    fattn.cache_append(k, v, cache, batch)
    for x, y in zip((k, v), fattn.cache_read(cache, batch)):
        a = x.double().unflatten(-1, (-1, 16))
        top = a.abs().amax(dim=-1, keepdim=True)
        s = (top / 8) / (8 / 9)  # the scale lies within a ninth of a / 8
        same = a.sign() == (torch.where((a == top).any(dim=-1, keepdim=True), 1.0, -1.0))
        cut = torch.where(same, 1.0, 2.0)
        bar = torch.where(a.abs() > 6.5 * top / 8 * (8 / 9), cut, 0.5) * s
        assert bool(((y.double().unflatten(-1, (-1, 16)) - a).abs() <= bar).all())


def _sum_of_values(c, causal, G):
    """sum_j |v_j| over the keys that each query sees, [T, Hq, d]."""
    out = np.zeros((int(c.cu[-1]), c.H * G, c.d))
    for b, length in enumerate(c.lens):
        n, length = int(c.cu[b + 1] - c.cu[b]), int(length)
        v = np.abs(oc4.tokens(c.cache, None, c.table[b], "v", 0, length))
        upto = np.concatenate([np.zeros((1, c.H, c.d)), np.cumsum(v, axis=0)])
        seen = [max(0, length - n + i + 1) if causal else length for i in range(n)]
        out[c.cu[b]:c.cu[b + 1]] = np.repeat(upto[seen], G, axis=1)
    return out


def _check_forward(c, q, scale, causal, o, lse):
    n = int(c.cu[-1])
    ref, lse_ref, A, S, seen = oc4.forward(c.cache, c.batch, q.double().numpy()[:n], scale, causal,
                                           d_error=True)
    u = 2.0 ** -24
    eps = (c.d + 12) * u * S + seen[None, :] * u + 2.0 ** -21
    got, got_lse = o[:n].cpu().double().numpy(), lse[:, :n].cpu().double().numpy()
    bar = 2.0 ** -8 * np.abs(ref) + A * (2.0 ** -11 + 2 * eps.T[:, :, None])
    bar += 2.0 ** -33 * _sum_of_values(c, causal, q.shape[1] // c.H)
    assert np.all(np.abs(got - ref) <= bar), np.nanmax(np.abs(got - ref) / np.maximum(bar, 1e-300))
    np.testing.assert_array_equal(np.isneginf(got_lse), np.isneginf(lse_ref))
    f = np.isfinite(lse_ref)
    assert np.all(np.abs(got_lse[f] - lse_ref[f]) <= (eps + 2.0 ** -22 * (1 + np.abs(lse_ref)))[f])


@pytest.mark.parametrize("layout", ["own", "slice", "heads"])
@pytest.mark.parametrize("pairs,H,G,d,bs,causal", [a[:5] + a[6:] for a in base.FORWARD])
def test_forward_matches_oracle(pairs, H, G, d, bs, causal, layout):
    c = Case(pairs, H, d, bs, seed=d + bs + G + len(pairs), pad_tokens=2).fill()
    q = _bf16(c.rng, (c.T, H * G, d), 1.5)
    cache, batch = c.on_device()
    whole = torch.full((c.T, H * G + 3, d), 7.0, dtype=torch.bfloat16, device=DEV)
    scale = d ** -0.5
    o, lse = fattn.cache_forward(_strided(q, layout), cache, batch, scale, causal,
                                 out=whole[:, 1:1 + H * G])
    _check_forward(c, q, scale, causal, o, lse)
    whole[:int(c.cu[-1]), 1:1 + H * G] = 7.0  # padded rows and neighbouring heads untouched
    assert bool((whole == 7.0).all())


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,length,G", [(5, 2, 2), (3, 0, 1), (40, 7, 4), (300, 20, 1)])
def test_rows_that_see_nothing(n, length, G, causal):
    H, d = 2, 64
    c = Case([(1, 40), (n, length - n), (1, 3)], H, d, 16).fill()
    q = _bf16(c.rng, (c.T, H * G, d))
    cache, batch = c.on_device()
    o, lse = fattn.cache_forward(q.to(DEV), cache, batch, 0.125, causal)
    _check_forward(c, q, 0.125, causal, o, lse)
    blind = int(max(0, n - length)) if causal else (n if length == 0 else 0)
    rows = slice(1, 1 + blind)
    assert bool((o[rows] == 0).all()) and bool(torch.isneginf(lse[:, rows]).all())


@pytest.mark.parametrize("size", [2.0 ** -10, 2.0 ** 8])
@pytest.mark.parametrize("n", [1, 6, 140])
def test_large_logits_and_sizes(n, size):
    """Logits in the hundreds, values near the smallest scales and far from one."""
    H, G, d, bs = 2, 2, 128, 16
    c = Case([(n, 200), (n, 64)], H, d, bs, seed=n).fill(size)
    q = _bf16(c.rng, (c.T, H * G, d), 3.0)
    q[:, 1] *= 2.0 ** 20
    cache, batch = c.on_device()
    for scale in (d ** -0.5 / size, 2.0 ** -30):
        o, lse = fattn.cache_forward(q.to(DEV), cache, batch, scale, True)
        _check_forward(c, q, scale, True, o, lse)


@pytest.mark.parametrize("n,G", [(4, 2), (20, 4), (150, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_scales_that_are_none_stay_with_the_rows_that_see_them(n, G, d):
    """An infinite, a NaN and a too large scale in the causal part: the queries before the token
    stay right."""
    H, bs, prior = 2, 16, 37
    c = Case([(n, prior)], H, d, bs, seed=n + d).fill()
    bad = prior + n // 2
    at = (c.table[0, bad // bs], 1, bad % bs)
    c.cache["v_scale"][at + (0,)], c.cache["v_scale"][at + (1,)] = 0x7c, 0xff
    c.cache["v_scale"][at + (2,)], c.cache["k_scale"][at + (1,)] = 0x7a, 0xfc
    q = _bf16(c.rng, (c.T, H * G, d))
    cache, batch = c.on_device()
    o, lse = fattn.cache_forward(q.to(DEV), cache, batch, d ** -0.5, True)
    first = n // 2
    c.pairs, c.cu = [(first, prior)], np.array([0, first], dtype=np.int32)
    c.lens = np.array([prior + first], dtype=np.int32)
    _check_forward(c, q[:first], d ** -0.5, True, o, lse)


def test_offsets_past_32_bits_and_the_last_block():
    """A pool of more than 2^32 bytes of codes, whose last blocks are used."""
    H, d, bs = 8, 128, 128
    nb = (1 << 32) // (H * bs * d // 2) + 3
    cache = fattn.new_cache(nb, H, bs, d, dtype=torch.uint8, device=DEV)
    c = Case([(1, 200), (140, 30)], H, d, bs, spare=0)
    small, batch = c.on_device()
    k, v = (_bf16(c.rng, (170, H, d)).to(DEV) for _ in range(2))
    q = _bf16(c.rng, (c.T, H * 2, d)).to(DEV)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)
    # the same tokens in a small pool and in the last blocks of the large one
    moved = batch._replace(block_table=torch.where(batch.block_table < nb, nb - 1 - batch.block_table,
                                                   batch.block_table).contiguous())
    got = []
    for pool, b in ((small, batch), (cache, moved)):
        write = b._replace(cu_seqlens=i32(0, 0, 170), total=170, max_seqlen=170)
        fattn.cache_append(k, v, pool, write)
        first = fattn.CacheBatch(b.block_table[:1].contiguous(), i32(201), i32(0, 201), 201, 201)
        fattn.cache_append(k[:1].expand(201, H, d), v[:1].expand(201, H, d), pool, first)
        got.append(fattn.cache_forward(q, pool, b, 0.1, True) + fattn.cache_read(pool, b))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    del cache
    torch.cuda.empty_cache()


def test_bad_entries_are_reported_and_skipped():
    """Wrong lengths, offsets and block numbers: reported, and the other sequences are served."""
    H, G, d, bs = 2, 2, 64, 16
    c = Case([(3, 20), (2, 30), (0, 5), (4, 9), (1, 50)], H, d, bs, seed=4).fill()
    q, k, v = _bf16(c.rng, (c.T, H * G, d)), _bf16(c.rng, (c.T, H, d)), _bf16(c.rng, (c.T, H, d))
    for change, code in (("len", 0), ("page", 1), ("empty", 0)):
        lens, table = c.lens.copy(), c.table.copy()
        if change == "len":
            lens[1] = 1000000
        elif change == "empty":
            lens[2] = -3
        else:
            table[1, :] = 2 ** 29
        cache, batch = c.on_device()
        batch = batch._replace(lens=torch.tensor(lens, device=DEV),
                               block_table=torch.tensor(table, device=DEV))
        fattn.fattn_device_error()
        fattn.cache_append(k.to(DEV), v.to(DEV), cache, batch)
        assert fattn.fattn_device_error() == 0x440 + code
        good = [b for b in range(5) if not (change != "empty" and b == 1)]
        want = oc4.append(c.cache, (c.table, c.lens, c.cu), k.double().numpy(), v.double().numpy())
        if change != "empty":
            for blk in c.table[1][:2]:
                for name in want:
                    want[name][blk] = c.cache[name][blk]
        _assert_cache(cache, want)
        rk, rv = fattn.cache_read(cache, batch)
        assert fattn.fattn_device_error() == 0x450 + code
        for got, ref in zip((rk, rv), oc4.read(want, c.batch)):
            for b in good:
                z = slice(c.cu[b], c.cu[b + 1])
                np.testing.assert_array_equal(got[z].cpu().double().numpy(), ref[z])
        if change == "page":
            assert bool((rk[c.cu[1]:c.cu[2]] == 0).all()) and bool((rv[c.cu[1]:c.cu[2]] == 0).all())
        o, lse = fattn.cache_forward(q.to(DEV), cache, batch, 0.125, True)
        assert fattn.fattn_device_error() == 0x460 + code
        saved, c.cache = c.cache, want
        ref, lse_ref = oc4.forward(want, c.batch, q.double().numpy(), 0.125, True)
        c.cache = saved
        for b in good:
            z = slice(c.cu[b], c.cu[b + 1])
            assert np.abs(o[z].cpu().double().numpy() - ref[z]).max(initial=0) <= 2e-2 * 8


def test_graph_capture_and_another_stream():
    """Append, attention and read captured once and replayed with other lengths, and the calls on
    a stream of their own."""
    H, G, d, bs, T = 2, 4, 128, 32, 6
    c = Case([(2, 50), (3, 40), (1, 90)], H, d, bs, seed=8, spare=0).fill()
    cache, batch = c.on_device()
    lens = batch.lens.clone()
    q, k, v = (torch.zeros((T, h, d), dtype=torch.bfloat16, device=DEV) for h in (H * G, H, H))
    ws = torch.empty(1 << 26, dtype=torch.uint8, device=DEV)
    out = torch.zeros_like(q)

    def step():
        fattn.cache_append(k, v, cache, batch)
        o, lse = fattn.cache_forward(q, cache, batch, 0.1, True, out=out, workspace=ws)
        return (lse,) + fattn.cache_read(cache, batch)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            lse, rk, rv = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    host = {n: getattr(cache, n).view(torch.uint8).cpu().numpy() for n in cache._fields}
    for i in range(2):
        batch.lens.copy_(lens - 2 * i)
        c.lens = (lens - 2 * i).cpu().numpy()
        for x in (q, k, v):
            x.copy_(_bf16(c.rng, tuple(x.shape)))
        graph.replay()
        torch.cuda.synchronize()
        host = oc4.append(host, c.batch, k.cpu().double().numpy(), v.cpu().double().numpy())
        c.cache = host
        _assert_cache(cache, host)
        _check_forward(c, q.cpu(), 0.1, True, out, lse)
        for got, ref in zip((rk, rv), oc4.read(host, c.batch)):
            np.testing.assert_array_equal(got.cpu().double().numpy(), ref)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    fattn.cache_append(k, v, cache, batch, stream=other)
    o, lse2 = fattn.cache_forward(q, cache, batch, 0.1, True, stream=other)
    other.synchronize()
    assert torch.equal(o, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("offset,pad", [(8, 0), (16, 8), (0, 8), (0, 16)])
@pytest.mark.parametrize("d", [64, 128])
def test_read_into_rows_of_any_alignment(d, offset, pad):
    """Outputs whose rows start on 16-byte boundaries that are none of 32 bytes, and on those."""
    H, bs = 3, 16
    c = Case([(40, 3), (1, 9)], H, d, bs).fill()
    cache, batch = c.on_device()
    ref = oc4.read(c.cache, c.batch)
    outs = []
    for _ in range(2):
        flat = torch.full((offset + c.T * (H * d + pad) + 64,), 7.0, dtype=torch.bfloat16, device=DEV)
        outs.append((flat, flat[offset:].as_strided((c.T, H, d), (H * d + pad, d, 1))))
    got = fattn.cache_read(cache, batch, out=(outs[0][1], outs[1][1]))
    for (flat, part), g, r in zip(outs, got, ref):
        np.testing.assert_array_equal(g.cpu().double().numpy(), r)
        part.fill_(7.0)
        assert bool((flat == 7.0).all())


def test_append_of_many_heads_and_tokens():
    """A prompt large enough for several heads a warp, heads that do not divide among them."""
    H, T, d, bs = 37, 16500, 64, 128
    g = torch.Generator(device=DEV).manual_seed(9)
    k, v = (torch.randn((T, H, d), generator=g, device=DEV).bfloat16() for _ in range(2))
    nb = -(-T // bs)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)
    one, many = (fattn.new_cache(nb, H, bs, d, dtype=torch.uint8, device=DEV) for _ in range(2))
    table = torch.randperm(nb, generator=g, device=DEV).int()[None].contiguous()
    fattn.cache_append(k, v, one, fattn.CacheBatch(table, i32(T), i32(0, T), T, T))
    for a in range(0, T, 500):  # in pieces too small for that
        n = min(500, T - a)
        fattn.cache_append(k[a:a + n], v[a:a + n], many,
                           fattn.CacheBatch(table, i32(a + n), i32(0, n), n, n))
    for x, y in zip(one, many):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layout", ["own", "slice"])
def test_read_of_any_scale(d, layout):
    """Every scale there is, infinities and NaN among them: (c - 8) inf is an infinity, 0 inf NaN."""
    H, bs = 3, 32
    c = Case([(70, 0), (200, 30)], H, d, bs, seed=d)
    assert len(np.unique(c.cache["k_scale"])) == 256
    cache, batch = c.on_device()
    whole = torch.full((2, c.T, H + 1, d + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    out = whole[:, :, :H, 8:] if layout == "slice" else torch.empty((2, c.T, H, d), dtype=torch.bfloat16,
                                                                    device=DEV)
    got = fattn.cache_read(cache, batch, out=(out[0], out[1]))
    with np.errstate(invalid="ignore"):
        want = oc4.read(c.cache, c.batch)
    for g, ref in zip(got, want):
        assert np.isinf(ref).any() and np.isnan(ref).any()
        np.testing.assert_array_equal(g.cpu().double().numpy(), ref)
