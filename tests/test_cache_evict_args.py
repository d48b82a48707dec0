"""Weights of cached keys and eviction without a GPU: argument checks that come before any device
call, and the oracle's own properties."""
import numpy as np
import pytest
import torch

from online_softmax_08_gb300 import build as fbuild
from online_softmax_08_gb300 import fattn
from oracle import cache as oc
from oracle import evict as oe
from test_cache_args import A, CUDA, INVALID, UNSUPPORTED, _batch, _cache


@pytest.fixture(scope="module")
def lib():
    fbuild.build()
    return fattn.load()


def _weights(lib, c, b, q=A, qst=512, qsh=64, lse=A, Hq=8, scale=0.1, w=A, wb=400, wh=100, o=2 * A,
             ob=400, oh=100, width=100):
    return lib.fattn_cache_weights(c, b, q, qst, qsh, lse, Hq, scale, 1, w, wb, wh, o, ob, oh, width,
                                   None)


def _evict(lib, c, b, w=A, wb=400, wh=100, width=100, table=A, twidth=4, keep=50, recent=10, lens=2 * A,
           kept=3 * A, o=4 * A, ob=400, oh=100, owidth=64):
    return lib.fattn_cache_evict(c, b, w, wb, wh, width, table, twidth, keep, recent, lens, kept, o, ob,
                                 oh, owidth, None)


@pytest.mark.parametrize("fmt", [0, 1, 4])
def test_weights_arguments(lib, fmt):
    c, b = _cache(format=fmt), _batch()
    for kw in (dict(q=None), dict(q=A + 8), dict(lse=None), dict(lse=A + 2), dict(Hq=6), dict(scale=0.0),
               dict(scale=float("nan")), dict(w=A + 2), dict(o=None), dict(o=A + 1), dict(wb=-1),
               dict(oh=-4), dict(qst=12), dict(width=-1), dict(ob=399), dict(oh=99), dict(ob=0),
               dict(ob=100, oh=100), dict(wb=1 << 39), dict(o=A, ob=800)):
        assert _weights(lib, c, b, **kw) == INVALID, kw
    for kw, status in ((dict(d=80), UNSUPPORTED), (dict(k=0), INVALID), (dict(block_size=4), UNSUPPORTED)):
        assert _weights(lib, _cache(**dict(dict(format=fmt), **kw)), b) == status
    assert _weights(lib, None, b) == _weights(lib, c, None) == INVALID
    assert _weights(lib, c, _batch(total=0, max_seqlen=0)) == 0
    if not torch.cuda.is_available():  # accepted: the calls go on to the device
        for kw in (dict(), dict(w=None, wb=-3), dict(o=A), dict(ob=100, oh=200), dict(wb=0, wh=0)):
            assert _weights(lib, c, b, **kw) == CUDA, kw


@pytest.mark.parametrize("fmt", [0, 1, 4])
def test_evict_arguments(lib, fmt):
    c, b = _cache(format=fmt), _batch(cu_seqlens=0, total=-7, max_seqlen=99)  # not looked at
    for kw in (dict(w=None), dict(w=A + 2), dict(width=0), dict(table=None), dict(table=A + 1),
               dict(twidth=3), dict(keep=0), dict(recent=-1), dict(recent=51), dict(lens=None), dict(lens=A),
               dict(kept=None), dict(o=None), dict(o=A), dict(owidth=49), dict(oh=49), dict(ob=49),
               dict(wb=-1)):
        assert _evict(lib, c, b, **kw) == INVALID, kw
    assert _evict(lib, c, _batch(lens=0)) == _evict(lib, c, _batch(block_table=0)) == INVALID
    assert _evict(lib, _cache(format=fmt, d=32), b) == UNSUPPORTED
    assert _evict(lib, None, b) == _evict(lib, c, None) == INVALID
    assert _evict(lib, c, _batch(B=1 << 24), width=1 << 30, keep=1 << 20, twidth=1 << 20,
                  owidth=1 << 20, ob=1 << 30, oh=1 << 20) == INVALID
    if not torch.cuda.is_available():
        for kw in (dict(), dict(keep=1 << 30, owidth=100, twidth=7), dict(ob=50, oh=100)):
            assert _evict(lib, c, b, **kw) == CUDA, kw


def test_binding_refuses_wrong_tensors():
    cache = fattn.new_cache(6, 2, 16, 64, dtype=torch.uint8, device="cpu")
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32)
    with pytest.raises(ValueError):  # (on no CUDA device)
        fattn.cache_evict(cache, torch.zeros((2, 2, 32)), i32([0, 1], [2, 3]), i32(20, 9),
                          i32([4], [5]), 10)
    batch = fattn.CacheBatch(i32([0, 1], [2, 3]), i32(20, 9), i32(0, 3, 5), 5, 3)
    with pytest.raises(ValueError):
        fattn.cache_weights(torch.zeros((5, 4, 64), dtype=torch.bfloat16), torch.zeros((4, 5)), cache,
                            batch, 0.1, True)


def test_oracle_chooses_as_defined():
    w = np.array([3.0, 1.0, 3.0, np.nan, -0.0, 0.0, 2.0, 9.0])
    np.testing.assert_array_equal(oe.choose(w, 8, 8, 0), np.arange(8))
    np.testing.assert_array_equal(oe.choose(w, 8, 1, 0), [3])
    np.testing.assert_array_equal(oe.choose(w, 8, 3, 1), [0, 3, 7])
    np.testing.assert_array_equal(oe.choose(w, 7, 5, 0), [0, 1, 2, 3, 6])
    np.testing.assert_array_equal(oe.choose(w, 7, 6, 0), [0, 1, 2, 3, 4, 6])  # -0 equals 0: the first
    np.testing.assert_array_equal(oe.choose(w, 8, 2, 2), [6, 7])


def test_oracle_weights_sum_to_the_queries():
    rng = np.random.default_rng(2)
    codes = rng.integers(0, 112, (2, 4, 1, 16, 64)).astype(np.uint8)
    cache = {"k": codes[0], "v": codes[1], "k_scale": np.full((4, 1), 2.0 ** -6),
             "v_scale": np.ones((4, 1))}
    batch = (np.array([[2, 0, 3]]), np.array([40]), np.array([0, 7]))
    q = rng.standard_normal((7, 2, 64))
    _, lse = oc.forward(cache, "e4m3", batch, q, 0.1, True)
    before = rng.uniform(0, 1, (1, 1, 44))
    w, _ = oe.weights(cache, "e4m3", batch, q, lse, 0.1, True, before, np.full((1, 1, 44), 7.0))
    np.testing.assert_allclose(w[0, 0, :40].sum() - before[0, 0, :33].sum(), 14.0, rtol=1e-12)
    assert np.all(w[0, 0, 40:] == 7.0)


def test_weights_refuse_more_rows_than_are_counted(lib):
    """The kernels step through a sequence's query rows 32 or 256 at a time, in 32 bits."""
    c = _cache(H=1)
    call = lambda n, total=(1 << 31) - 1: _weights(lib, c, _batch(total=total, max_seqlen=n), qst=0,
                                                   qsh=0, Hq=1)
    for n in ((1 << 31) - 1, (1 << 31) - 65535):
        assert call(n) == INVALID, n
    assert _weights(lib, c, _batch(total=(1 << 28) - 1, max_seqlen=(1 << 28) - 1), qst=0,
                    qsh=0, Hq=8) == INVALID
    if not torch.cuda.is_available():
        assert call((1 << 31) - 65536) == CUDA
