"""The attention weights of cached keys, and eviction by them, against the fp64 oracle.

Bar of a weight, for what the queries add to it: a term exp(s - lse) has the score's error,
(d + 12) u S as in test_gpu_cache.py, that of taking s - lse to base 2 in fp32, 4 u (S + |lse|),
and 2^-22 of ex2, all relative to it; the terms are positive, so n of them summed in fp32 add
n u.  With Z the largest S + |lse| of the rows that see the key and n rows:
  |W - W_ref| <= new ((d + 16) u Z + n u + 2^-21) + u |W_ref|,
u = 2^-24, the last term the sum with the weight from before; terms below 2^-126 are flushed:
n 2^-126 more.  Eviction copies: positions, weights, codes and scales are compared bit for bit.
"""
import numpy as np
import pytest
import torch

import test_gpu_cache as base8
import test_gpu_cache4 as base4
from online_softmax_08_gb300 import fattn
from oracle import cache as oc
from oracle import evict as oe

pytestmark = pytest.mark.gpu

DEV = base8.DEV
_bf16, _strided = base8._bf16, base8._strided


@pytest.fixture(autouse=True)
def _no_device_error():
    fattn.fattn_device_error()
    yield
    torch.cuda.synchronize()
    assert fattn.fattn_device_error() == 0


def _case(pairs, H, d, bs, fmt, **kw):
    if fmt == "int4":
        return base4.Case(pairs, H, d, bs, **kw)
    return base8.Case(pairs, H, d, bs, fmt, nan_slots=False, **kw)


def _check_weights(c, fmt, q, lse, scale, causal, before, was, got):
    n = int(c.cu[-1])
    ref, Z = oe.weights(c.cache, fmt, c.batch, q.double().cpu().numpy()[:n],
                        lse.double().cpu().numpy()[:, :n], scale, causal, before, was)
    zero = None if before is None else np.zeros_like(before)
    new, _ = oe.weights(c.cache, fmt, c.batch, q.double().cpu().numpy()[:n],
                        lse.double().cpu().numpy()[:, :n], scale, causal, zero, np.zeros_like(was))
    rows = max(a for a, _ in c.pairs) * (q.shape[1] // c.H)
    u = 2.0 ** -24
    touched = np.zeros(ref.shape, dtype=bool)
    for b, length in enumerate(c.lens):
        if c.cu[b + 1] > c.cu[b]:
            touched[b, :, :length] = True
    bar = new * ((c.d + 16) * u * Z + rows * u + 2.0 ** -21) + u * np.abs(ref) + rows * 2.0 ** -126
    err = np.abs(got.double().cpu().numpy() - ref)
    assert np.all(err[touched] <= bar[touched]), (err / bar)[touched].max()
    assert np.all(err[~touched] == 0)


WEIGHTS = [
    # (pairs, H, G, d, bs, fmt, causal)
    ([(1, 0)], 1, 1, 64, 16, "int4", True),
    ([(1, 16)], 2, 1, 128, 16, "e4m3", True),
    ([(1, 1), (1, 14), (1, 127), (1, 128), (1, 300)], 2, 4, 128, 16, "int4", True),
    ([(1, 700), (1, 0), (1, 2100)], 2, 7, 64, 32, "e5m2", True),
    ([(1, 999)], 2, 8, 128, 128, "int4", False),
    ([(1, 200)], 1, 33, 64, 64, "e4m3", True),
    ([(4, 60), (0, 9), (3, 0), (7, 250), (0, 0)], 2, 3, 128, 32, "int4", True),
    ([(40, 0), (17, 100), (1, 64)], 2, 2, 128, 64, "e4m3", True),
    ([(130, 0)], 2, 1, 64, 64, "int4", True),
    ([(32, 100), (31, 97)], 1, 1, 128, 16, "int4", True),
    ([(129, 200), (1, 90), (65, 0)], 1, 4, 128, 16, "int4", True),
    ([(260, 13)], 1, 3, 128, 128, "e5m2", False),
    ([(1, 50), (3, 40)], 1, 300, 64, 16, "e4m3", True),
    ([(i % 4, 5 * i) for i in range(70)], 2, 2, 64, 16, "int4", True),
    ([(i % 2, i % 50) for i in range(1100)], 1, 1, 64, 16, "int4", True),
    # the tcgen05 kernel: groups that divide its tiles and that do not, units cut by the shares,
    # second tiles of keys with and without tokens, mixed with sequences of few rows
    ([(33, 0)], 1, 1, 128, 16, "int4", True),
    ([(600, 3000)], 2, 4, 128, 64, "e4m3", True),
    ([(100, 0), (1, 50), (513, 200), (0, 40)], 1, 5, 64, 16, "int4", True),
    ([(9, 300)], 1, 128, 128, 32, "int4", True),
    ([(300, 600), (33, 1), (40, 216)], 2, 3, 128, 128, "e5m2", False),
    ([(35 + i, 90 * i) for i in range(40)], 1, 2, 64, 32, "e4m3", True),
    ([(1 if i % 3 else 129, 7 * i) for i in range(70)], 3, 1, 128, 16, "int4", True),
    ([(257, 5000)], 1, 7, 64, 64, "int4", False),
]


@pytest.mark.parametrize("layout", ["own", "slice", "heads"])
@pytest.mark.parametrize("pairs,H,G,d,bs,fmt,causal", WEIGHTS)
def test_weights_match_oracle(pairs, H, G, d, bs, fmt, causal, layout):
    c = _case(pairs, H, d, bs, fmt, seed=d + bs + G + len(pairs), pad_tokens=2).fill()
    q = _bf16(c.rng, (c.T, H * G, d), 1.5)
    cache, batch = c.on_device()
    scale = d ** -0.5
    dq = _strided(q, layout)
    _, lse = fattn.cache_forward(dq, cache, batch, scale, causal)
    B, width = len(pairs), int(c.lens.max()) + 5
    # new, added to what was there, in place, and into rows apart
    new = fattn.cache_weights(dq, lse, cache, batch, scale, causal)
    assert new.shape == (B, H, batch.block_table.shape[1] * bs)
    _check_weights(c, fmt, q, lse, scale, causal, None, np.zeros(new.shape), new)
    before = torch.tensor(c.rng.uniform(0, 3, (H, B, width)), dtype=torch.float32, device=DEV).transpose(0, 1)
    keep = before.clone()
    whole = torch.full((B, H + 2, width + 3), 7.0, device=DEV)
    out = fattn.cache_weights(dq, lse, cache, batch, scale, causal, before, out=whole[:, 1:1 + H, 1:])
    assert torch.equal(before, keep)
    was = np.full((B, H, width + 2), 7.0)
    padded = np.concatenate([keep.cpu().numpy(), np.zeros((B, H, 2))], axis=2)
    _check_weights(c, fmt, q, lse, scale, causal, padded, was, out)
    whole[:, 1:1 + H, 1:] = 7.0
    assert bool((whole == 7.0).all())
    again = fattn.cache_weights(dq, lse, cache, batch, scale, causal, before)
    assert again is before
    _check_weights(c, fmt, q, lse, scale, causal, keep.cpu().numpy(), keep.cpu().numpy(), before)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,length,G", [(5, 2, 2), (3, 0, 1), (40, 7, 4), (300, 20, 1)])
def test_weights_of_more_queries_than_tokens(n, length, G, causal):
    H, d = 2, 64
    c = _case([(1, 40), (n, length - n), (1, 3)], H, d, 16, "int4").fill()
    q = _bf16(c.rng, (c.T, H * G, d)).to(DEV)
    cache, batch = c.on_device()
    _, lse = fattn.cache_forward(q, cache, batch, 0.125, causal)
    w = fattn.cache_weights(q, lse, cache, batch, 0.125, causal)
    _check_weights(c, "int4", q, lse, 0.125, causal, None, np.zeros(w.shape), w)
    # every row that sees something gives one in all
    total = w.sum(dim=2).cpu().double()
    live = n if length > 0 and not causal else min(n, length)
    assert abs(float(total[1, 0]) - live * G) <= 1e-4 * max(1, live * G)


@pytest.mark.parametrize("n,G", [(3, 2), (50, 3)])
def test_weights_of_a_broadcast_query(n, G):
    """One query for all tokens, and one for all heads, by strides of zero."""
    H, d = 2, 64
    c = _case([(n, 70), (1, 20)], H, d, 16, "int4").fill()
    cache, batch = c.on_device()
    row = _bf16(c.rng, (1, H * G, d)).to(DEV)
    for q in (row.expand(n + 1, H * G, d), row[:, :1].expand(n + 1, H * G, d),
              _bf16(c.rng, (n + 1, 1, d)).to(DEV).expand(n + 1, H * G, d)):
        _, lse = fattn.cache_forward(q, cache, batch, 0.125, True)
        got = fattn.cache_weights(q, lse, cache, batch, 0.125, True)
        _check_weights(c, "int4", q.contiguous(), lse, 0.125, True, None, np.zeros(got.shape), got)


def test_nan_queries_stay_with_their_sequence():
    """Rows of the next sequence, which a tile of queries may hold as well, do not count."""
    H, G, d = 1, 2, 128
    c = _case([(50, 30), (40, 20)], H, d, 16, "e4m3").fill()
    cache, batch = c.on_device()
    q = _bf16(c.rng, (90, G, d)).to(DEV)
    _, lse = fattn.cache_forward(q, cache, batch, 0.1, True)
    ref = fattn.cache_weights(q, lse, cache, batch, 0.1, True)
    q[50:] = float("nan")
    got = fattn.cache_weights(q, lse, cache, batch, 0.1, True)
    assert torch.equal(got[0], ref[0])


def test_nan_key_and_repeated_calls():
    """A NaN key of one head makes NaN of the weights of the keys that its queries see, and of no
    other head's or sequence's.  Repeated calls agree bit for bit."""
    H, G, d, bs = 2, 2, 128, 16
    c = _case([(3, 50), (40, 20)], H, d, bs, "e4m3").fill()
    q = _bf16(c.rng, (c.T, H * G, d)).to(DEV)
    cache, batch = c.on_device()
    _, lse = fattn.cache_forward(q, cache, batch, 0.1, True)
    w = fattn.cache_weights(q, lse, cache, batch, 0.1, True)
    assert torch.equal(w, fattn.cache_weights(q, lse, cache, batch, 0.1, True))
    c.cache["k"][c.table[0, 3], 0, 4, 7] = 0x7f  # position 52, which the last query sees
    cache, batch = c.on_device()
    _, lse = fattn.cache_forward(q, cache, batch, 0.1, True)
    got = fattn.cache_weights(q, lse, cache, batch, 0.1, True)
    assert torch.equal(got[0, 1], w[0, 1]) and torch.equal(got[1], w[1])
    assert bool(torch.isnan(got[0, 0, :53]).all()) and bool((got[0, 0, 53:] == 0).all())


def _scatter(c, new, bs):
    """A table of blocks that no sequence has, for `new` tokens each; the pool grows by them."""
    need = [-(-x // bs) for x in new]
    nb = c.cache["k"].shape[0]
    for name, a in c.cache.items():
        more = c.rng.integers(0, 100, (sum(need),) + a.shape[1:])
        c.cache[name] = np.concatenate([a, more.astype(a.dtype)])
    order = (nb + c.rng.permutation(sum(need))).tolist()
    table = np.full((len(new), max(max(need), 1) + 1), 2 ** 30, dtype=np.int32)
    for b, n in enumerate(need):
        table[b, :n] = [order.pop() for _ in range(n)]
    return table


EVICT = [
    # (lens, H, d, bs, fmt, keep, recent)
    ([1], 1, 64, 16, "int4", 1, 0),
    ([2, 3], 1, 128, 16, "int4", 1, 1),
    ([17, 16, 15, 0, 40], 2, 64, 16, "int4", 16, 4),
    ([1000, 3, 500, 257], 3, 128, 64, "int4", 100, 30),
    ([1025, 2049, 64], 2, 128, 32, "int4", 1024, 0),
    ([5000, 4999], 1, 64, 128, "int4", 1500, 1500),
    ([300, 77], 2, 128, 16, "e4m3", 50, 10),
    ([300, 77, 512], 1, 64, 64, "e5m2", 200, 100),
    ([400, 90], 2, 64, 128, "e4m3", 129, 0),
    ([i * 7 % 200 for i in range(150)], 2, 64, 16, "int4", 33, 5),
]


def _weights_for(c, lens, H, kind):
    w = c.rng.exponential(1.0, (len(lens), H, max(max(lens), 1) + 3)) ** 3
    if kind == "ties":
        w = np.floor(w * 2) / 2
    if kind == "special":
        w = w * 10.0 ** c.rng.integers(-40, 30, w.shape)
        r = c.rng.random(w.shape)
        w[r < 0.02] = np.inf
        w[(r > 0.02) & (r < 0.04)] = np.nan
        w[(r > 0.04) & (r < 0.06)] = -np.inf
        w[(r > 0.1) & (r < 0.4)] *= -1.0
        w[(r > 0.4) & (r < 0.5)] = 0.0
        w[(r > 0.5) & (r < 0.6)] = -0.0
    return w.astype(np.float32)


@pytest.mark.parametrize("kind", ["plain", "ties", "special"])
@pytest.mark.parametrize("lens,H,d,bs,fmt,keep,recent", EVICT)
def test_evict_matches_oracle(lens, H, d, bs, fmt, keep, recent, kind):
    c = _case([(0, x) for x in lens], H, d, bs, fmt, seed=len(lens) + keep).fill()
    new = [min(x, keep) for x in lens]
    table_out = _scatter(c, new, bs)
    w = _weights_for(c, lens, H, kind)
    want, kept, new = oe.evict(c.cache, fmt, c.table, c.lens, w, table_out, keep, recent)
    cache, batch = c.on_device()
    dev = lambda a: torch.tensor(a, device=DEV)
    whole = torch.full((len(lens), H + 1, keep + 2), 7.0, device=DEV)
    out = whole[:, 1:, 2:]
    for _ in range(2):  # the second call changes nothing
        got_lens, got_kept, got_w = fattn.cache_evict(cache, dev(w), batch.block_table, batch.lens,
                                                      dev(table_out), keep, recent, out=out)
        np.testing.assert_array_equal(got_lens.cpu().numpy(), new)
        for b in range(len(lens)):
            for h in range(H):
                k = got_kept[b, h].cpu().numpy()
                np.testing.assert_array_equal(k[:new[b]], kept[b][h])
                assert np.all(k[new[b]:] == -1)
                x = got_w[b, h].cpu().numpy()
                np.testing.assert_array_equal(x[:new[b]], w[b, h, kept[b][h]])
                assert np.all(x[new[b]:] == 7.0)
        if fmt == "int4":
            base4._assert_cache(cache, want)
        else:
            base8._assert_cache(cache, want, fmt)
    whole[:, 1:, 2:] = 7.0
    assert bool((whole == 7.0).all())


def test_evict_of_a_long_sequence():
    """More tokens than any pass holds at once, nearly all weights alike in their upper digits."""
    H, d, bs, L, keep, recent = 2, 64, 128, 150001, 70000, 123
    g = torch.Generator(device=DEV).manual_seed(1)
    w = (1.0 + torch.rand((1, H, L), generator=g, device=DEV) * 2.0 ** -12)
    w[:, 1] = 0.5
    nb = -(-L // bs)
    cache = fattn.new_cache(nb + -(-keep // bs), H, bs, d, dtype=torch.uint8, device=DEV)
    for x in (cache.k, cache.v, cache.k_scale.view(torch.uint8)):
        x.copy_(torch.randint(0, 256, x.shape, generator=g, device=DEV))
    i32 = dict(dtype=torch.int32, device=DEV)
    table = torch.randperm(nb, generator=g, device=DEV).int()[None].contiguous()
    out_table = torch.arange(nb, nb + -(-keep // bs), **i32)[None].contiguous()
    lens, kept, moved = fattn.cache_evict(cache, w, table, torch.tensor([L], **i32), out_table, keep,
                                          recent)
    assert int(lens[0]) == keep
    order = torch.sort(w[0, :, :L - recent].double(), dim=1, descending=True, stable=True).indices
    want = torch.cat((order[:, :keep - recent].sort(dim=1).values,
                      torch.arange(L - recent, L, device=DEV).expand(H, -1)), dim=1)
    assert torch.equal(kept[0].long(), want)
    assert torch.equal(moved[0], w[0].gather(1, want))
    for x in (cache.k, cache.v, cache.k_scale.view(torch.uint8)):
        src = x[table[0].long()].transpose(0, 1).reshape(H, -1, x.shape[-1])
        dst = x[out_table[0].long()].transpose(0, 1).reshape(H, -1, x.shape[-1])[:, :keep]
        at = want[..., None].expand(-1, -1, x.shape[-1])
        assert torch.equal(dst, src.gather(1, at))


@pytest.mark.parametrize("B,L,keep,recent", [(80, 40000, 999, 10), (40, 70001, 40000, 1),
                                             (1, 300001, 150000, 0), (200, 33333, 5, 5)])
def test_evict_of_rows_read_in_parts(B, L, keep, recent):
    """More weights than the CTAs of a row hold, many of them equal, in one to eight CTAs a row."""
    d, bs = 64, 128
    g = torch.Generator(device=DEV).manual_seed(B)
    w = torch.floor(torch.rand((B, 1, L), generator=g, device=DEV) * 500) / 256
    w[:, :, ::7] = 0.0
    nb, nk = -(-L // bs), -(-keep // bs)
    cache = fattn.new_cache(nb + B * nk, 1, bs, d, dtype=torch.uint8, device=DEV)
    cache.k.copy_(torch.randint(0, 256, cache.k.shape, generator=g, device=DEV))
    i32 = dict(dtype=torch.int32, device=DEV)
    table = torch.arange(nb, **i32).expand(B, nb).contiguous()  # all of them share their blocks
    out_table = torch.arange(nb, nb + B * nk, **i32).reshape(B, nk)
    lens = torch.full((B,), L, **i32)
    lens[0] = L - 3
    new, kept, moved = fattn.cache_evict(cache, w, table, lens, out_table, keep, recent)
    assert new.tolist() == [keep] * B
    for b in (0, B // 2, B - 1):
        n = int(lens[b]) - recent
        order = torch.sort(w[b, 0, :n].double(), descending=True, stable=True).indices
        want = torch.cat((order[:keep - recent].sort().values, torch.arange(n, n + recent, device=DEV)))
        assert torch.equal(kept[b, 0].long(), want)
        assert torch.equal(moved[b, 0], w[b, 0][want])
        src = cache.k[:nb, 0].reshape(-1, d // 2)
        assert torch.equal(cache.k[out_table[b].long(), 0].reshape(-1, d // 2)[:keep], src[want])


def test_evict_to_its_own_blocks():
    """A sequence that is short enough may be given its own blocks: it stays as it is."""
    c = _case([(0, 30), (0, 100)], 2, 64, 16, "e4m3").fill()
    table_out = _scatter(c, [0, 40], 16)
    table_out[0, :2] = c.table[0, :2]
    w = _weights_for(c, [30, 100], 2, "plain")
    want, kept, new = oe.evict(c.cache, "e4m3", c.table, c.lens, w, table_out, 40, 8)
    cache, batch = c.on_device()
    dev = lambda a: torch.tensor(a, device=DEV)
    fattn.cache_evict(cache, dev(w), batch.block_table, batch.lens, dev(table_out), 40, 8)
    base8._assert_cache(cache, want, "e4m3")


def test_bad_entries_are_reported():
    H, d, bs = 2, 64, 16
    c = _case([(1, 30), (2, 50), (1, 20)], H, d, bs, "int4").fill()
    q = _bf16(c.rng, (c.T, H, d)).to(DEV)
    cache, batch = c.on_device()
    _, lse = fattn.cache_forward(q, cache, batch, 0.1, True)
    ref = fattn.cache_weights(q, lse, cache, batch, 0.1, True)
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)
    lens = batch.lens.clone()
    lens[1] = 10 ** 6
    w = torch.full_like(ref, 7.0)
    fattn.cache_weights(q, lse, cache, batch._replace(lens=lens), 0.1, True, out=w)
    assert fattn.fattn_device_error() == 0x470
    assert torch.equal(w[0, :, :31], ref[0, :, :31]) and torch.equal(w[2, :, :21], ref[2, :, :21])
    assert bool((w[1] == 7.0).all())
    narrow = torch.zeros((3, H, 40), device=DEV)  # no room for sequence 1
    fattn.cache_weights(q, lse, cache, batch, 0.1, True, out=narrow)
    assert fattn.fattn_device_error() == 0x470 and bool((narrow[1] == 0).all())
    table = batch.block_table.clone()
    table[1, 1] = -5
    got = fattn.cache_weights(q, lse, cache, batch._replace(block_table=table), 0.1, True)
    assert fattn.fattn_device_error() == 0x471
    assert bool((got[1, :, 16:32] == 0).all()) and torch.equal(got[1, :, :16], ref[1, :, :16])
    # eviction
    table_out = dev(_scatter(c, [10, 10, 10], bs))
    cache, batch = c.on_device()
    w = torch.rand((3, H, 60), device=DEV)
    good = fattn.cache_evict(cache, w, batch.block_table, batch.lens, table_out, 10, 2)
    bad_lens = fattn.cache_evict(cache, w, batch.block_table, lens, table_out, 10, 2)
    assert fattn.fattn_device_error() == 0x480 and bad_lens[0].tolist() == [10, 0, 10]
    assert torch.equal(bad_lens[1][0], good[1][0]) and bool((bad_lens[1][1] == -1).all())
    fattn.cache_evict(cache, w, table, batch.lens, table_out, 10, 2)
    assert fattn.fattn_device_error() in (0, 0x481)
    wrong = table_out.clone()
    wrong[2, 0] = 10 ** 8
    fattn.cache_evict(cache, w, batch.block_table, batch.lens, wrong, 10, 2)
    assert fattn.fattn_device_error() == 0x481


@pytest.mark.parametrize("n", [1, 70])
def test_captured_and_on_another_stream(n):
    """Weights and eviction captured once and replayed with other lengths, queries and weights;
    on a stream of their own; and two at a time."""
    H, G, d, bs, keep = 2, 4, 128, 32, 40
    c = _case([(n, 130), (n, 20), (n, 300)], H, d, bs, "e4m3", seed=n).fill()
    table_out = _scatter(c, [keep] * 3, bs)
    cache, batch = c.on_device()
    table_out = torch.tensor(table_out, device=DEV)
    lens = batch.lens.clone()
    q = _bf16(c.rng, (c.T, H * G, d)).to(DEV)
    w = torch.zeros((3, H, 384), device=DEV)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device=DEV)
    w_out = torch.zeros((3, H, keep), device=DEV)

    def step():
        o, lse = fattn.cache_forward(q, cache, batch, 0.1, True, workspace=ws)
        fattn.cache_weights(q, lse, cache, batch, 0.1, True, None, out=w)
        new, kept, _ = fattn.cache_evict(cache, w, batch.block_table, batch.lens, table_out, keep,
                                         7, out=w_out)
        return lse, new, kept

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()
        with torch.cuda.graph(graph, stream=side):
            lse, new, kept = step()
    torch.cuda.synchronize()
    for i in range(2):
        batch.lens.copy_(lens - 11 * i)
        c.lens = (lens - 11 * i).cpu().numpy()
        q.copy_(_bf16(c.rng, tuple(q.shape)))
        w.zero_()
        w_out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        _check_weights(c, "e4m3", q, lse, 0.1, True, None, np.zeros(w.shape), w)
        host = {name: getattr(cache, name).cpu() for name in cache._fields}
        want, chosen, count = oe.evict(
            {name: (a.view(torch.uint8) if a.element_size() == 1 else a).numpy()
             for name, a in host.items()}, "e4m3", c.table, c.lens, w.cpu().numpy(),
            table_out.cpu().numpy(), keep, 7)
        np.testing.assert_array_equal(new.cpu().numpy(), count)
        for b in range(3):
            for h in range(H):
                np.testing.assert_array_equal(kept[b, h, :count[b]].cpu().numpy(), chosen[b][h])
        base8._assert_cache(cache, want, "e4m3")
    # two streams at once, each its own outputs
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(w) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, x in zip(streams, outs):
            fattn.cache_weights(q, lse, cache, batch, 0.1, True, None, out=x, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], w) and torch.equal(outs[1], w)
    other = fattn.cache_evict(cache, w, batch.block_table, batch.lens, table_out, keep, 7,
                              stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(other[0], new) and torch.equal(other[1], kept) and torch.equal(other[2], w_out)


def test_weights_and_eviction_past_32_bits():
    """A pool of more than 2^32 bytes of codes, whose last blocks are used."""
    H, d, bs, keep = 8, 128, 128, 100
    nb = (1 << 32) // (H * bs * d // 2) + 8
    c = _case([(1, 200), (140, 30)], H, d, bs, "int4", spare=0).fill()
    table_out = _scatter(c, [keep, keep], bs)
    small, batch = c.on_device()
    cache = fattn.new_cache(nb, H, bs, d, dtype=torch.uint8, device=DEV)
    used = small.k.shape[0]
    for name in cache._fields:
        getattr(cache, name).view(torch.uint8)[-used:] = getattr(small, name).view(torch.uint8)
    move = lambda t: torch.where((t >= 0) & (t < used), t + (nb - used), t).contiguous()
    moved = batch._replace(block_table=move(batch.block_table))
    table_out = torch.tensor(table_out, device=DEV)
    q = _bf16(c.rng, (c.T, H * 2, d)).to(DEV)
    _, lse = fattn.cache_forward(q, small, batch, 0.1, True)
    got = []
    for pool, b, to in ((small, batch, table_out), (cache, moved, move(table_out))):
        w = fattn.cache_weights(q, lse, pool, b, 0.1, True)
        got.append((w,) + fattn.cache_evict(pool, w, b.block_table, b.lens, to, keep, 9))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    for name in cache._fields:
        assert torch.equal(getattr(cache, name).view(torch.uint8)[-used:],
                           getattr(small, name).view(torch.uint8))
    del cache
    torch.cuda.empty_cache()


@pytest.mark.parametrize("fmt,n", [("int4", 1), ("e4m3", 1), ("int4", 70), ("e5m2", 70)])
def test_missing_large_block(fmt, n):
    """A bad number of a block that holds several warps' keys: they get 0, the others what they
    get without it, whatever lies in the pool's first block."""
    H, G, d, bs = 2, 2, 128, 64
    c = _case([(n, 300), (1, 90)], H, d, bs, fmt, seed=3, spare=40).fill()
    assert 0 not in c.table
    for name in ("k", "k_scale"):
        a = c.cache[name]
        a[0] = np.nan if a.dtype.kind == "f" else 0xff if name == "k" else 0x7f
    q = _bf16(c.rng, (c.T, H * G, d)).to(DEV)
    cache, batch = c.on_device()
    _, lse = fattn.cache_forward(q, cache, batch, 0.1, True)
    ref = fattn.cache_weights(q, lse, cache, batch, 0.1, True)
    for bad in (-1, 10 ** 6):
        table = batch.block_table.clone()
        table[0, 2] = bad
        got = fattn.cache_weights(q, lse, cache, batch._replace(block_table=table), 0.1, True)
        assert fattn.fattn_device_error() == 0x471
        assert bool((got[0, :, 128:192] == 0).all())
        for part in (slice(0, 128), slice(192, None)):
            assert torch.equal(got[0, :, part], ref[0, :, part])
        assert torch.equal(got[1], ref[1])


def test_serving_run():
    """What they are for, together: queries and keys are turned, the keys and values go into the
    4-bit cache, the queries attend and weigh the keys, the cache is cut to its most attended
    tokens in other blocks, and the next step, captured in a graph, goes on from there."""
    H, G, d, bs, n = 2, 4, 128, 16, 200
    keep, recent, steps = 64, 16, 3
    rng = np.random.default_rng(7)
    scale = d ** -0.5
    table = fattn.rope_table(d, 1e4, "yarn", 4.0, 64, device=DEV)
    pool = fattn.new_cache(60, H, bs, d, dtype=torch.uint8, device=DEV)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)
    blocks = torch.arange(40, dtype=torch.int32, device=DEV).flip(0).reshape(2, 20).contiguous()
    others = torch.arange(40, 60, dtype=torch.int32, device=DEV).reshape(2, 10).contiguous()
    lens = i32(n, n - 30)
    batch = fattn.CacheBatch(blocks, lens, i32(0, n, 2 * n - 30), 2 * n - 30, n)
    pos = torch.cat((torch.arange(n), torch.arange(n - 30))).int().to(DEV)
    x = _bf16(rng, (2 * n - 30, H * (G + 2), d)).to(DEV)
    q, k = fattn.rope(x[:, :H * G], x[:, H * G:H * (G + 1)], pos, table)
    fattn.cache_append(k, x[:, H * (G + 1):], pool, batch)
    o, lse = fattn.cache_forward(q, pool, batch, scale, True)
    w = fattn.cache_weights(q, lse, pool, batch, scale, True)
    rows = torch.tensor([n, n - 30], device=DEV) * G
    assert torch.allclose(w.sum(dim=2), rows[:, None].float().expand(2, H), rtol=1e-4)
    before = fattn.cache_read(pool, batch)
    lens2, kept, w2 = fattn.cache_evict(pool, w, blocks, lens, others, keep, recent)
    w2 = torch.cat((w2, torch.zeros((2, H, 96), device=DEV)), dim=2).contiguous()
    after = fattn.cache_read(pool, fattn.CacheBatch(others, lens2, i32(0, keep, 2 * keep), 2 * keep, keep))
    for a, b in zip(before, after):
        for s, first in enumerate((0, n)):
            for h in range(H):
                assert torch.equal(b[s * keep:(s + 1) * keep, h], a[first + kept[s, h].long(), h])
    # single tokens on what is left
    step = fattn.CacheBatch(others, lens2, i32(0, 1, 2), 2, 1)
    place = i32(n, n - 30)
    xs = torch.zeros((2, H * (G + 2), d), dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device=DEV)

    def one():
        lens2.add_(1)
        q, k = fattn.rope(xs[:, :H * G], xs[:, H * G:H * (G + 1)], place, table)
        fattn.cache_append(k, xs[:, H * (G + 1):], pool, step)
        o, lse = fattn.cache_forward(q, pool, step, scale, True, workspace=ws)
        fattn.cache_weights(q, lse, pool, step, scale, True, w2)
        place.add_(1)
        return q, o, lse

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            q1, o1, lse1 = one()
    torch.cuda.synchronize()
    for i in range(steps):
        xs.copy_(_bf16(rng, tuple(xs.shape)))
        old = w2.clone()
        graph.replay()
        torch.cuda.synchronize()
        # in 64 bits, of the cache's own values
        L = keep + i + 1
        kv = fattn.cache_read(pool, fattn.CacheBatch(others, lens2, i32(0, L, 2 * L), 2 * L, L))
        for s in range(2):
            ks, vs = (t[s * L:(s + 1) * L].double().transpose(0, 1) for t in kv)  # [H, L, d]
            z = scale * torch.einsum("hgd,hld->hgl", q1[s].double().reshape(H, G, d), ks)
            p = torch.softmax(z, dim=2)
            ref = torch.einsum("hgl,hld->hgd", p, vs).reshape(H * G, d)
            assert float((o1[s].double() - ref).abs().max()) <= 2e-2
            want = old[s, :, :L].double()
            want[:, L - 1] = 0.0
            want += p.sum(dim=1)
            assert float((w2[s, :, :L].double() - want).abs().max()) <= 1e-4
            assert torch.equal(w2[s, :, L:], old[s, :, L:])


def test_evict_keeps_infinities():
    """e5m2: an infinite code stays one, whatever scale its block gets; NaN stays NaN."""
    d, bs, keep = 64, 16, 16
    cache = fattn.new_cache(4, 1, bs, d, dtype=torch.float8_e5m2, device=DEV)
    for side, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        side.view(torch.uint8)[:2] = 0x3c  # 1.0
        side.view(torch.uint8)[0, 0, :, 5] = 0x7c
        side.view(torch.uint8)[0, 0, :, 6] = 0xfc
        side.view(torch.uint8)[0, 0, :, 7] = 0x7e
        side.view(torch.uint8)[0, 0, :, 8] = 0x7b  # the largest finite one
        scale[0], scale[1] = 2.0, 8.0
    i32 = dict(dtype=torch.int32, device=DEV)
    w = torch.ones((1, 1, 32), device=DEV)
    w[..., 8:24] = 2.0  # half of either block
    table, table_out = torch.tensor([[0, 1]], **i32), torch.tensor([[3]], **i32)
    _, kept, _ = fattn.cache_evict(cache, w, table, torch.tensor([32], **i32), table_out, keep)
    assert kept[0, 0].tolist() == list(range(8, 24))
    for side, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        assert float(scale[3]) == 8.0
        got = side.view(torch.uint8)[3, 0]
        assert bool((got[:8, 5] == 0x7c).all()) and bool((got[:8, 6] == 0xfc).all())
        assert bool(torch.isnan(side[3, 0, :8, 7].float()).all())
        assert bool((got[:8, 8] == 0x73).all())  # a quarter of 57344
        assert bool((got[:8, 9:] == 0x34).all()) and bool((got[:8, :5] == 0x34).all())
        assert bool((got[8:] == 0x3c).all())


@pytest.mark.parametrize("B", [1, 20])
def test_evict_of_the_longest_rows(B):
    """As many tokens as a table row may name, in eight and in four CTAs a row: the number of the
    weight behind the last segment does not fit 32 bits."""
    d, bs, keep, recent = 64, 128, 1000, 9
    L = (1 << 31) - 65536
    i32 = dict(dtype=torch.int32, device=DEV)
    nb, nk = 50, -(-keep // bs)
    cache = fattn.new_cache(nb + B * nk, 1, bs, d, dtype=torch.uint8, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(3)
    cache.k.copy_(torch.randint(0, 256, cache.k.shape, generator=g, device=DEV))
    # weights of zero but for some, the last ones among them; zeros fill up from the front
    some = torch.cat((torch.arange(300, device=DEV) * 7000001 + 5,
                      L - recent - 1 - torch.arange(200, device=DEV)))
    w = torch.zeros((1, 1, L), device=DEV)
    w[0, 0, some] = 1.0 + torch.rand((500,), generator=g, device=DEV)
    table = (torch.arange(L // bs, **i32) % nb).expand(B, -1).contiguous()
    table_out = torch.arange(nb, nb + B * nk, **i32).reshape(B, nk)
    lens = torch.full((B,), L, **i32)
    new, kept, moved = fattn.cache_evict(cache, w.expand(B, 1, L), table, lens, table_out, keep, recent)
    assert new.tolist() == [keep] * B
    chosen = some.tolist()
    first = [j for j in range(keep) if j not in chosen][:keep - recent - 500]
    want = torch.tensor(sorted(chosen + first) + list(range(L - recent, L)), device=DEV)
    src = cache.k[:nb, 0].reshape(-1, d // 2)
    for b in range(B):
        assert torch.equal(kept[b, 0].long(), want) and torch.equal(moved[b, 0], w[0, 0, want])
        assert torch.equal(cache.k[table_out[b].long(), 0].reshape(-1, d // 2)[:keep],
                           src[want % (nb * bs)])


@pytest.mark.parametrize("keep", [(1 << 31) - 1, (1 << 31) - 1024])
def test_evict_that_keeps_all(keep):
    """The largest `keep`, whose places behind the last token are filled, and nothing behind them."""
    c = _case([(0, 21)], 1, 64, 16, "int4").fill()
    table_out = torch.tensor(_scatter(c, [21], 16), device=DEV)
    cache, batch = c.on_device()
    w = torch.rand((1, 1, 21), device=DEV)
    out = torch.full((1, 1, 25), 7.0, device=DEV)
    lens_out = torch.empty((1,), dtype=torch.int32, device=DEV)
    whole = torch.full((keep + 4096,), 7, dtype=torch.int32, device=DEV)
    pool, dev, _, _ = fattn._pool_args(cache)
    b = fattn._pack_batch(batch.block_table.data_ptr(), batch.lens.data_ptr(), batch.lens.data_ptr(), 1,
                          batch.block_table.shape[1], 0, 0)
    st = fattn.load().fattn_cache_evict(pool, b, w.data_ptr(), 0, 0, 21, table_out.data_ptr(),
                                        table_out.shape[1], keep, 3, lens_out.data_ptr(),
                                        whole[1024:].data_ptr(), out.data_ptr(), 0, 0, 25,
                                        torch.cuda.current_stream().cuda_stream)
    assert st == 0 and lens_out.tolist() == [21]
    assert whole[1024:1045].tolist() == list(range(21)) and torch.equal(out[..., :21], w)
    assert bool((out[..., 21:] == 7.0).all())
    low, high = torch.aminmax(whole[1045:1024 + keep])
    assert int(low) == -1 and int(high) == -1
    assert bool((whole[:1024] == 7).all()) and bool((whole[1024 + keep:] == 7).all())


def test_evict_of_weights_that_change():
    """Weights that change while a row is read (here: its own results, written over weights that are
    still to be read, which the call does not allow) may leave places without a token.  What lies
    there is no block's number: such a token becomes zeros and is reported, nothing else changes."""
    L, keep, many, d, bs, nb = 600000, 76712, 75712, 64, 128, 50
    i32 = dict(dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(5)
    nk = -(-keep // bs)
    cache = fattn.new_cache(nb + nk + 7, 1, bs, d, dtype=torch.uint8, device=DEV)
    for x in (cache.k, cache.v, cache.k_scale.view(torch.uint8), cache.v_scale.view(torch.uint8)):
        x.copy_(torch.randint(0, 112, x.shape, generator=g, device=DEV))
    old = [x.view(torch.uint8).clone() for x in cache]
    # the first 1000 tokens are kept, of many that are equal, and the last 75712; the first ones'
    # weights then take the places of some of the last ones'
    buf = torch.zeros((1, 1, 700000), device=DEV)
    buf[..., :262144] = 1.0
    buf[..., L - many:L] = 2.0
    table = (torch.arange(-(-L // bs), **i32) % nb)[None].contiguous()
    table_out = torch.arange(nb, nb + nk, **i32)[None].contiguous()
    lens, lens_out = torch.tensor([L], **i32), torch.empty((1,), **i32)
    kept = torch.full((keep,), 1 << 30, **i32)
    kept[1::2] = -5
    blank = kept.clone()
    pool = fattn._pool_args(cache)[0]
    b = fattn._pack_batch(table.data_ptr(), lens.data_ptr(), lens.data_ptr(), 1, table.shape[1], 0, 0)
    st = fattn.load().fattn_cache_evict(pool, b, buf.data_ptr(), 0, 0, L, table_out.data_ptr(), nk, keep,
                                        0, lens_out.data_ptr(), kept.data_ptr(),
                                        buf[..., 550000:].data_ptr(), 0, 0, keep,
                                        torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    none = kept == blank
    assert bool(none.any()) and not bool(none[:1000].any())
    assert fattn.fattn_device_error() == 0x481
    at = torch.where(none, 0, kept).long()
    for x, was, empty in zip(cache, old, (0x88, 0x88, 0, 0)):
        x = x.view(torch.uint8)
        assert torch.equal(x[:nb], was[:nb]) and torch.equal(x[nb + nk:], was[nb + nk:])
        src = was[:nb].reshape(nb * bs, -1)
        want = torch.where(none[:, None], torch.full_like(src[:1], empty), src[at % (nb * bs)])
        assert torch.equal(x[nb:nb + nk].reshape(nk * bs, -1)[:keep], want)


@pytest.mark.parametrize("bad", [-1, 1000, 2 ** 30])
@pytest.mark.parametrize("fmt", ["int4", "e4m3", "e5m2"])
def test_evict_of_missing_blocks(fmt, bad):
    """Kept tokens whose block number is bad become zeros (8 bits: of the scale that the others
    give, 2^-100 where there are none); a bad number to write to drops its tokens alone."""
    H, d, bs, keep = 2, 64, 16, 48
    lens = [160, 100]
    c = _case([(0, x) for x in lens], H, d, bs, fmt).fill()
    table_out = _scatter(c, [keep, keep], bs)
    w = np.zeros((2, H, 160), dtype=np.float32)
    # head 0: a part of two destination blocks is missing; head 1: the whole second one
    first = [list(range(8)) + list(range(16, 32)) + list(range(40, 64)),
             list(range(32)) + list(range(64, 80))]
    for h in range(H):
        w[0, h, first[h]] = 1.0
        w[1, h, 30 + h:30 + h + keep] = 1.0
    # the oracle's: a block of nothing in the place of the missing one
    missing = int(c.table[0, 1])
    nothing = {n: a.copy() for n, a in c.cache.items()}
    for side in ("k", "v"):
        nothing[side][missing] = 0x88 if fmt == "int4" else 0
        nothing[side + "_scale"][missing] = 0 if fmt == "int4" else 2.0 ** -100
    want, kept, new = oe.evict(nothing, fmt, c.table, c.lens, w, table_out, keep, 0)
    assert kept[0][0].tolist() == first[0] and kept[0][1].tolist() == first[1]
    for n in want:
        want[n][missing] = c.cache[n][missing]
    check = lambda cache: base4._assert_cache(cache, want) if fmt == "int4" else \
        base8._assert_cache(cache, want, fmt)
    dev = lambda a: torch.tensor(a, device=DEV)
    table = c.table.copy()
    table[0, 1] = bad
    cache, batch = c.on_device()
    got = fattn.cache_evict(cache, dev(w), dev(table), batch.lens, dev(table_out), keep)
    assert fattn.fattn_device_error() == 0x481
    assert got[0].tolist() == [keep, keep]
    np.testing.assert_array_equal(got[1].cpu().numpy(), np.array(kept))
    np.testing.assert_array_equal(got[2].cpu().numpy(), np.take_along_axis(w, np.array(kept), axis=2))
    check(cache)
    # a bad number to write to: as if nothing had been written there
    want, _, _ = oe.evict(c.cache, fmt, c.table, c.lens, w, table_out, keep, 0)
    for n in want:
        want[n][table_out[1, 1]] = c.cache[n][table_out[1, 1]]
    wrong = table_out.copy()
    wrong[1, 1] = bad
    cache, batch = c.on_device()
    fattn.cache_evict(cache, dev(w), batch.block_table, batch.lens, dev(wrong), keep)
    assert fattn.fattn_device_error() == 0x481
    check(cache)


@pytest.mark.parametrize("n", [1, 70])
@pytest.mark.parametrize("byte", [0x70, 0x78, 0x7c, 0xfc, 0x7f])
def test_weights_beside_scales_out_of_range(n, byte):
    """A scale of 4 bits beyond what the attention takes (8192, 32768, infinities, NaN): the weights
    of other heads and other sequences are what they are without it."""
    H, G, d, bs = 2, 2, 128, 16
    c = _case([(n, 50), (n, 33)], H, d, bs, "int4", seed=9).fill()
    q = _bf16(c.rng, (c.T, H * G, d)).to(DEV)
    got = []
    for scale in (None, byte):
        if scale is not None:
            c.cache["k_scale"][c.table[0, 1], 0, 3, 2] = scale
        cache, batch = c.on_device()
        _, lse = fattn.cache_forward(q, cache, batch, 0.1, True)
        got.append(fattn.cache_weights(q, lse, cache, batch, 0.1, True))
    assert torch.equal(got[0][0, 1], got[1][0, 1]) and torch.equal(got[0][1], got[1][1])
