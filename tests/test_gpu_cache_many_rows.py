"""Edge cases of the 8-bit cache's attention with enough rows per key/value head for the
256-row kernel (and calls that mix both kernels, streams and graphs), against the fp64
oracle with the bar of test_gpu_cache.py."""
import numpy as np
import pytest
import torch

from online_softmax_08_gb300 import fattn
from oracle import cache as oc
from test_gpu_cache import (DEV, TYPES, Case, _bf16, _check_forward,  # noqa: F401
                            _no_device_error, _torch_reference)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [70, 140])
def test_bad_lengths_beside_good_sequences(n):
    H, G, d, bs = 2, 2, 64, 16
    c = Case([(n, 30), (n + 10, 40), (n + 20, 300), (1, 50)], H, d, bs).fill()
    q = _bf16(c.rng, (c.T, H * G, d)).to(DEV)
    cache, batch = c.on_device()
    good, good_lse = fattn.cache_forward(q, cache, batch, 0.125, True)
    _check_forward(c, q.cpu(), 0.125, True, good, good_lse)
    o = torch.empty_like(q)
    bad_rows = slice(int(c.cu[1]), int(c.cu[2]))
    for length in (1000000, -1, batch.block_table.shape[1] * bs + 1, 2 ** 31 - 1):
        lens = c.lens.copy()
        lens[1] = length
        bad = batch._replace(lens=torch.tensor(lens, device=DEV))
        o.fill_(7.0)
        fattn.cache_forward(q, cache, bad, 0.125, True, out=o)
        assert fattn.fattn_device_error() == 0x460
        assert bool((o[bad_rows] == 7.0).all())
        o[bad_rows] = good[bad_rows]
        assert torch.equal(o, good)


def _without(c, q, scale, causal, gone, G):
    """O, LSE, A, S and the visible keys of sequence 0 without the keys in `gone`."""
    n, length = int(c.cu[1]), int(c.lens[0])
    keep = np.array([j not in gone for j in range(length)])
    T, Hq, d = q.shape
    out = [np.zeros((n, Hq, d)), np.full((Hq, n), -np.inf), np.zeros((n, Hq, d)), np.zeros((Hq, n)),
           np.zeros(n, dtype=int)]
    k, v = (oc.tokens(c.cache, c.fmt, c.table[0], side, 0, length) for side in ("k", "v"))
    for i in range(n):
        lim = length - n + i + 1 if causal else length
        see = np.flatnonzero(keep[:lim])
        out[4][i] = len(see)
        for hq in range(Hq if len(see) else 0):
            h = hq // G
            s = scale * (k[see, h] @ q[i, hq])
            e = np.exp(s - s.max())
            w = e / e.sum()
            out[0][i, hq], out[1][hq, i] = w @ v[see, h], s.max() + np.log(e.sum())
            out[2][i, hq] = w @ np.abs(v[see, h])
            out[3][hq, i] = (scale * (np.abs(k[see, h]) @ np.abs(q[i, hq]))).max()
    return out


@pytest.mark.parametrize("d,bs,fmt", [(64, 16, "e4m3"), (128, 64, "e5m2")])
@pytest.mark.parametrize("blocks", ["first", "tile", "last", "all"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n", [3, 140])
def test_block_numbers_out_of_range(n, d, bs, fmt, blocks, causal):
    """Their keys are not there: the first block, a whole tile of 128 keys, the last block,
    all of them (no row sees anything)."""
    H, G = 2, 1
    c = Case([(n, 300)], H, d, bs, fmt, seed=n + d).fill()
    q = _bf16(c.rng, (n, H * G, d))
    need = -(-int(c.lens[0]) // bs)
    at = {"first": [0], "tile": list(range(128 // bs, 256 // bs)), "last": [need - 1],
          "all": list(range(need))}[blocks]
    gone = {j for b in at for j in range(b * bs, (b + 1) * bs)}
    ref, lse_ref, A, S, seen = _without(c, q.double().numpy(), d ** -0.5, causal, gone, G)
    for page in (-1, c.cache["k"].shape[0], 2 ** 31 - 1, -2 ** 31):
        cache, batch = c.on_device()
        batch.block_table[0, at] = page
        o, lse = fattn.cache_forward(q.to(DEV), cache, batch, d ** -0.5, causal)
        assert fattn.fattn_device_error() == 0x461
        u = 2.0 ** -24
        eps = (d + 12) * u * S + seen[None] * u + 2.0 ** -21
        bar = 2.0 ** -8 * np.abs(ref) + A * (2.0 ** -11 + 2 * eps.T[:, :, None])
        assert np.all(np.abs(o.cpu().double().numpy() - ref) <= bar)
        got = lse.cpu().double().numpy()
        np.testing.assert_array_equal(np.isneginf(got), np.isneginf(lse_ref))
        f = np.isfinite(lse_ref)
        assert np.all(np.abs(got[f] - lse_ref[f]) <= (eps + 2.0 ** -22 * (1 + np.abs(lse_ref)))[f])


@pytest.mark.parametrize("d", [64, 128])
def test_values_of_any_size(d):
    H, G = 1, 2
    c = Case([(140, 100), (70, 500)], H, d, 16).fill()
    q = _bf16(c.rng, (c.T, H * G, d))
    base = c.cache["v_scale"].copy()
    for e in (-60, 0, 100):
        c.cache["v_scale"] = base * 2.0 ** e
        cache, batch = c.on_device()
        o, lse = fattn.cache_forward(q.to(DEV), cache, batch, 0.125, True)
        _check_forward(c, q, 0.125, True, o, lse)


@pytest.mark.parametrize("d,fmt", [(64, "e5m2"), (128, "e4m3")])
def test_scales_that_are_no_powers_of_two(d, fmt):
    H, G = 2, 3
    c = Case([(70, 200), (90, 70)], H, d, 32, fmt).fill()
    for side in ("k_scale", "v_scale"):
        c.cache[side] = (c.cache[side] * c.rng.uniform(0.5, 1.5, c.cache[side].shape)) \
            .astype(np.float32).astype(np.float64)
    q = _bf16(c.rng, (c.T, H * G, d))
    cache, batch = c.on_device()
    o, lse = fattn.cache_forward(q.to(DEV), cache, batch, 0.125, True)
    _check_forward(c, q, 0.125, True, o, lse)


def test_shared_prefix():
    H, G, d, bs = 2, 2, 128, 16
    c = Case([(70, 300), (100, 170), (1, 200)], H, d, bs).fill()
    c.table[1, :10] = c.table[0, :10]
    c.table[2, :10] = c.table[0, :10]
    q = _bf16(c.rng, (c.T, H * G, d))
    cache, batch = c.on_device()
    o, lse = fattn.cache_forward(q.to(DEV), cache, batch, 0.125, True)
    _check_forward(c, q, 0.125, True, o, lse)


@pytest.mark.parametrize("bs,d", [(128, 128), (16, 64)])
def test_blocks_beyond_four_gigabytes(bs, d):
    """Codes beyond 2^32 bytes from the pool's start."""
    H, G = 1, 2
    nb = (1 << 32) // (bs * d) + 600
    k, v = (torch.zeros((nb, H, bs, d), dtype=torch.uint8, device=DEV) for _ in range(2))
    g = torch.Generator(device=DEV).manual_seed(1)
    c = Case([(100, 5000)], H, d, bs, nan_slots=False)
    need = -(-5100 // bs)
    c.table = np.arange(nb - need, nb, dtype=np.int32)[None].copy()
    for x in (k, v):
        x[nb - need:] = torch.randn((need, H, bs, d), generator=g, device=DEV).to(
            torch.float8_e4m3fn).view(torch.uint8)
    ones = torch.ones((nb, H), device=DEV)
    cache = fattn.KVCache(k.view(TYPES["e4m3"]), v.view(TYPES["e4m3"]), ones, ones)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)
    batch = fattn.CacheBatch(i32(c.table), i32(c.lens), i32(c.cu), 100, 100)
    q = torch.randn((100, H * G, d), generator=g, device=DEV).bfloat16()
    o, lse = fattn.cache_forward(q, cache, batch, d ** -0.5, True)
    tail = fattn.KVCache(cache.k[nb - need:], cache.v[nb - need:], ones[:need], ones[:need])
    c.table = np.arange(need, dtype=np.int32)[None].copy()
    ref, lse_ref, A, S, seen = _torch_reference(c, tail, q, d ** -0.5, True)
    u = 2.0 ** -24
    eps = (d + 12) * u * S + seen[None, :] * u + 2.0 ** -21
    bar = 2.0 ** -8 * np.abs(ref) + A * (2.0 ** -11 + 2 * eps.T[:, :, None])
    assert np.all(np.abs(o.cpu().double().numpy() - ref) <= bar)
    assert np.all(np.abs(lse.cpu().double().numpy() - lse_ref)
                  <= eps + 2.0 ** -22 * (1 + np.abs(lse_ref)))


@pytest.mark.parametrize("pairs", [[(1, 900), (3, 40), (1, 5000)], [(140, 300), (1, 60), (70, 4000)]])
def test_result_in_place_of_the_queries(pairs):
    """out may be q itself: every row is read before it is written."""
    H, G, d = 2, 2, 128
    c = Case(pairs, H, d, 64, nan_slots=False).fill()
    q = _bf16(c.rng, (c.T, H * G, d)).to(DEV)
    cache, batch = c.on_device()
    want, want_lse = fattn.cache_forward(q, cache, batch, 0.1, True)
    for _ in range(3):
        x = q.clone()
        o, lse = fattn.cache_forward(x, cache, batch, 0.1, True, out=x)
        assert torch.equal(x, want) and torch.equal(lse, want_lse)


def test_queries_of_one_token_for_all():
    """A token stride of zero: every token asks the same."""
    H, G, d = 2, 2, 64
    c = Case([(70, 200), (1, 40)], H, d, 32).fill()
    one = _bf16(c.rng, (1, H * G, d))
    cache, batch = c.on_device()
    o, lse = fattn.cache_forward(one.to(DEV).expand(c.T, -1, -1), cache, batch, 0.125, True)
    _check_forward(c, one.expand(c.T, -1, -1), 0.125, True, o, lse)


def test_two_streams_and_two_graphs_at_once():
    """Calls that overlap, eagerly and replayed: each has its own workspace."""
    d, runs = 64, []
    for i, pairs in enumerate([[(140, 3000), (1, 700)], [(1, 5000), (90, 100), (2, 800)]]):
        c = Case(pairs, 2, d, 32, seed=i, nan_slots=False).fill()
        q = _bf16(c.rng, (c.T, 4, d)).to(DEV)
        cache, batch = c.on_device()
        want = fattn.cache_forward(q, cache, batch, 0.125, True)
        runs.append((q, cache, batch, want, torch.cuda.Stream(), torch.cuda.CUDAGraph()))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (q, cache, batch, _, stream, _) in enumerate(runs):
            got[i].append(fattn.cache_forward(q, cache, batch, 0.125, True, stream=stream))
    torch.cuda.synchronize()
    for i, (q, cache, batch, want, stream, graph) in enumerate(runs):
        assert all(torch.equal(a, b) for pair in got[i] for a, b in zip(pair, want))
        with torch.cuda.graph(graph, stream=stream):
            got[i] = [fattn.cache_forward(q, cache, batch, 0.125, True)]
    for _ in range(20):
        for *_, stream, graph in runs:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for i, (*_, want, _, _) in enumerate(runs):
        assert all(torch.equal(a, b) for pair in got[i] for a, b in zip(pair, want))


@pytest.mark.parametrize("n", [6, 140])
def test_more_tokens_than_the_stated_bound(n):
    """A sequence of more new tokens than max_seqlen is skipped and reported."""
    H, G, d, bs = 2, 2, 64, 16
    c = Case([(n, 30), (n + 1, 40), (n, 90)], H, d, bs, nan_slots=False).fill()
    q = _bf16(c.rng, (c.T, H * G, d)).to(DEV)
    cache, batch = c.on_device()
    want, _ = fattn.cache_forward(q, cache, batch, 0.125, True)
    few = batch._replace(max_seqlen=n)
    skipped = slice(n, 2 * n + 1)
    o = torch.full_like(q, 7.0)
    fattn.cache_forward(q, cache, few, 0.125, True, out=o)
    assert fattn.fattn_device_error() == 0x460
    assert bool((o[skipped] == 7.0).all())
    o[skipped] = want[skipped]
    # other splits of the keys: each is within 2^-8 |O| + 2^-11 A of the value, A = sum_j P_j |v_j|
    # below 6 for values of the normal distribution
    torch.testing.assert_close(o, want, rtol=2.0 ** -7, atol=6 * 2.0 ** -10)
    k, v = fattn.cache_read(cache, batch)
    out = [torch.full_like(k, 7.0) for _ in range(2)]
    fattn.cache_read(cache, few, out=out)
    assert fattn.fattn_device_error() == 0x450
    for got, ref in zip(out, (k, v)):
        assert bool((got[skipped] == 7.0).all())
        got[skipped] = ref[skipped]
        assert torch.equal(got, ref)
    before = [x.view(torch.uint8).clone() for x in cache]
    fattn.cache_append(k, v, cache, few)
    assert fattn.fattn_device_error() == 0x440
    mine = torch.tensor(c.table[1, :-(-int(c.lens[1]) // bs)].astype(np.int64), device=DEV)
    for a, b in zip(cache, before):
        assert torch.equal(a.view(torch.uint8)[mine], b[mine])
