"""The fp64 oracle of the 8-bit cache, pinned on the CPU: the code tables and
rounding against torch's own 8-bit types, the scales by their definition, and
attention over the cache against the dense oracle on the values read back."""
import numpy as np
import pytest
import torch

import oracle
from oracle import cache as oc

TYPES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_code_values_and_rounding_match_torch(fmt):
    codes = torch.arange(256, dtype=torch.uint8)
    np.testing.assert_array_equal(oc.code_values(fmt), codes.view(TYPES[fmt]).double().numpy())
    g = torch.Generator().manual_seed(3)
    top = oc.FORMATS[fmt][2]
    x = torch.cat([torch.randn(20000, generator=g) * top / 8,
                   torch.randn(20000, generator=g) * 2.0 ** -8,
                   torch.tensor([0.0, -0.0, top, -top])])
    v = oc.code_values(fmt)[:120]
    mid = torch.tensor((v[1:] + v[:-1]) / 2, dtype=torch.float32)  # ties
    x = torch.cat([x, mid, -mid]).clamp(-top, top)
    want = x.to(TYPES[fmt]).view(torch.uint8).numpy()
    np.testing.assert_array_equal(oc.round_codes(x.double().numpy(), fmt), want)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_scale_is_the_smallest_that_holds_the_largest_value(fmt):
    top = oc.FORMATS[fmt][2]
    for a in (0.0, 1e-38, 0.3, 1.0, top, np.nextafter(top, np.inf), 3.0 * top, 3e38):
        s = oc.scale_for(a, fmt)
        assert a <= top * s and np.log2(s) == round(np.log2(s))
        assert s == 2.0 ** oc.E_MIN or a > top * s / 2


def test_growing_block_and_forward():
    rng = np.random.default_rng(5)
    H, bs, d, G = 2, 16, 64, 3
    cache = {"k": np.zeros((6, H, bs, d), np.uint8), "v": np.zeros((6, H, bs, d), np.uint8),
             "k_scale": np.zeros((6, H)), "v_scale": np.zeros((6, H))}
    table = np.array([[4, 1, 2]])
    xs = []
    for step, n in enumerate((5, 1, 20, 1)):
        x = rng.standard_normal((2, n, H, d)) * 4.0 ** step
        xs.append(x)
        length = sum(a.shape[1] for a in xs)
        cache = oc.append(cache, "e4m3", (table, [length], [0, n]), x[0], x[1])
    k, v = oc.read(cache, "e4m3", (table, [27], [0, 27]))
    want = np.concatenate(xs, axis=1)
    # half a step of a 3-bit mantissa, and of the smallest code of the block's scale
    floor = np.repeat(cache["k_scale"][table[0]], bs, axis=0)[:27, :, None] * 2.0 ** -10
    assert np.all(np.abs(k - want[0]) <= 2.0 ** -4 * np.abs(want[0]) * (1 + 2.0 ** -4) + 2 * floor)
    q = rng.standard_normal((27, H * G, d))
    o, lse = oc.forward(cache, "e4m3", (table, [27], [0, 27]), q, 0.125, True)
    dense = lambda x: np.ascontiguousarray(np.repeat(x, G, axis=1).transpose(1, 0, 2))[None]
    o_ref, lse_ref = oracle.attention_fwd(np.ascontiguousarray(q.transpose(1, 0, 2))[None],
                                          dense(k), dense(v), 0.125, True)
    np.testing.assert_allclose(o.transpose(1, 0, 2), o_ref[0], rtol=1e-9, atol=1e-9)
    np.testing.assert_allclose(lse, lse_ref[0], rtol=1e-12, atol=1e-12)
