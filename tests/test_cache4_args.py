"""The 4-bit cache without a GPU: argument checks that come before any device call, and the
oracle's quantisation."""
import numpy as np
import pytest
import torch

from online_softmax_08_gb300 import build as fbuild
from online_softmax_08_gb300 import fattn
from oracle import cache4 as oc4
from test_cache_args import A, CUDA, INVALID, UNSUPPORTED, _append, _batch, _cache, _fwd, _read


@pytest.fixture(scope="module")
def lib():
    fbuild.build()
    return fattn.load()


@pytest.mark.parametrize("call", [_append, _read, _fwd])
def test_bad_descriptors(lib, call):
    for kw, status in [(dict(k=0), INVALID), (dict(k=A + 8), INVALID), (dict(k_scale=A + 4), INVALID),
                       (dict(v_scale=A + 8), INVALID), (dict(v_scale=0), INVALID),
                       (dict(d=96), UNSUPPORTED), (dict(d=32), UNSUPPORTED),
                       (dict(block_size=8), UNSUPPORTED)]:
        assert call(lib, _cache(format=4, **kw), _batch()) == status, kw
    for fmt in (3, 5, -1):
        assert call(lib, _cache(format=fmt), _batch()) == UNSUPPORTED
    assert call(lib, _cache(format=4), _batch(total=0, max_seqlen=0)) == 0
    if not torch.cuda.is_available():  # accepted: the calls go on to the device
        assert call(lib, _cache(format=4), _batch()) == CUDA


def test_binding_refuses_wrong_tensors():
    cache = fattn.new_cache(6, 2, 16, 64, dtype=torch.uint8, device="cpu")
    assert cache.k.shape == (6, 2, 16, 32) and cache.k_scale.shape == (6, 2, 16, 4)
    assert bool((cache.k == 0x88).all()) and cache.v_scale.dtype is torch.float8_e5m2
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32)
    batch = fattn.CacheBatch(i32([0, 1], [2, 3]), i32(20, 9), i32(0, 3, 5), 5, 3)
    x = torch.zeros((5, 2, 64), dtype=torch.bfloat16)
    for c in (cache._replace(v=cache.v[:5]), cache._replace(v=cache.v.view(torch.float8_e5m2)),
              cache._replace(k_scale=cache.k_scale.view(torch.uint8)),
              cache._replace(k_scale=torch.ones((6, 2))),
              cache._replace(v_scale=cache.v_scale[..., :3]),
              cache._replace(v_scale=cache.v_scale.transpose(1, 2)),
              cache):  # (on no CUDA device)
        with pytest.raises(ValueError):
            fattn.cache_append(x, x, c, batch)
    with pytest.raises(ValueError):
        fattn.new_cache(6, 2, 16, 40, dtype=torch.uint8, device="cpu")


def _group(x):
    codes, byte = oc4.quantise_groups(np.asarray(x)[None])
    return codes[0].astype(int), byte[0]


def test_oracle_quantises_as_defined():
    x = np.arange(16.0)  # +15 is the largest: scale -(15 / 8 -> 2, a tie to the even)
    codes, byte = _group(x)
    assert oc4.E5M2[byte] == -2.0
    np.testing.assert_array_equal((codes - 8) * -2.0,
                                  [0, 0, 2, 4, 4, 4, 6, 8, 8, 8, 10, 12, 12, 12, 14, 16])
    codes, byte = _group(-x)
    assert oc4.E5M2[byte] == 2.0
    codes, byte = _group(np.full(16, np.nan))
    assert byte & 0x7f == 0 and np.all(codes == 8)
    codes, byte = _group(np.array([np.inf, -np.inf] + [1.0] * 14))
    assert oc4.E5M2[byte] == -7168.0 and list(codes[:3]) == [0, 15, 8]
    # brute force: no other code of the chosen scale is nearer
    rng = np.random.default_rng(3)
    for _ in range(200):
        x = rng.standard_normal(16)
        codes, byte = _group(x)
        s = oc4.E5M2[byte]
        all_values = (np.arange(16) - 8) * s
        best = np.abs(x[:, None] - all_values).min(axis=1)
        np.testing.assert_allclose(np.abs((codes - 8) * s - x), best, rtol=0, atol=0)
        assert abs(abs(s) - np.abs(x).max() / 8) <= np.abs(x).max() / 8 / 8


def test_oracle_packs_and_reads_back():
    rng = np.random.default_rng(4)
    x = rng.standard_normal((5, 3, 64))
    codes, scale = oc4.quantise(x)
    assert codes.shape == (5, 3, 32) and scale.shape == (5, 3, 4)
    y = oc4.values(codes, scale)
    again, scale2 = oc4.quantise(y)
    assert np.abs(y - x).max() <= 2.3 * np.abs(x).max() / 8
    np.testing.assert_array_equal(codes[0, 0, 0] & 15, _group(x[0, 0, :16])[0][0])
    np.testing.assert_array_equal(codes[0, 0, 0] >> 4, _group(x[0, 0, :16])[0][1])
