"""Attention over the 8-bit cache where the blocks of one sequence differ much in the
size of their values: blocks of zeros (the smallest scale, 2^-100) beside others, small
values beside large ones that are zero in some columns.

The bar is that of test_gpu_cache.py, with the rounding of the weights below fp16's
normal range spelled out.  A key's weight times its scale is held in fp16 against a
reference that leaves the largest such product of 2^8 or more; keys share a reference
only with smaller ones and ones up to 2^20 larger in scale.  Half of fp16's smallest
step is 2^-25, so with W_j the largest P_i vs_i of the keys i with vs_i <= 2^20 vs_j
  |O - O_ref| <= 2^-8 |O_ref| + A (2^-11 + 2 eps) + sum_j 2^-33 W_j |code_j|.
"""
import numpy as np
import pytest
import torch

from online_softmax_08_gb300 import fattn
from oracle import cache as oc
from test_gpu_cache import DEV, Case, _bf16, _no_device_error  # noqa: F401

pytestmark = pytest.mark.gpu


def _check(c, q, scale, causal, o, lse):
    got, got_lse = o.cpu().double().numpy(), lse.cpu().double().numpy()
    q = q.double().numpy()
    G = q.shape[1] // c.H
    for b, length in enumerate(c.lens):
        length, n = int(length), int(c.cu[b + 1] - c.cu[b])
        k, v = (oc.tokens(c.cache, c.fmt, c.table[b], side, 0, length) for side in ("k", "v"))
        at = c.table[b, np.arange(length) // c.bs]
        for h in range(c.H):
            vs = c.cache["v_scale"][at, h]
            code = np.abs(v[:, h]) / vs[:, None]
            sizes, which = np.unique(vs, return_inverse=True)
            shares = sizes[None, :] <= 2.0 ** 20 * sizes[:, None]
            for i in range(n):
                lim, t = length - n + i + 1 if causal else length, int(c.cu[b]) + i
                if lim <= 0:
                    assert np.all(got[t, h * G:(h + 1) * G] == 0)
                    assert np.all(np.isneginf(got_lse[h * G:(h + 1) * G, t]))
                    continue
                for hq in range(h * G, (h + 1) * G):
                    s = scale * (k[:lim, h] @ q[t, hq])
                    e = np.exp(s - s.max())
                    P = e / e.sum()
                    ref, A = P @ v[:lim, h], P @ np.abs(v[:lim, h])
                    largest = np.zeros(len(sizes))
                    np.maximum.at(largest, which[:lim], P * vs[:lim])
                    W = np.where(shares, largest[None, :], 0.0).max(1)[which[:lim]]
                    S = (scale * (np.abs(k[:lim, h]) @ np.abs(q[t, hq]))).max()
                    eps = (c.d + 12) * 2.0 ** -24 * S + lim * 2.0 ** -24 + 2.0 ** -21
                    bar = 2.0 ** -8 * np.abs(ref) + A * (2.0 ** -11 + 2 * eps) + \
                        2.0 ** -33 * (W @ code[:lim])
                    assert np.all(np.abs(got[t, hq] - ref) <= bar), \
                        (b, i, hq, np.nanmax(np.abs(got[t, hq] - ref) / np.maximum(bar, 1e-300)))
                    want = s.max() + np.log(e.sum())
                    assert abs(got_lse[hq, t] - want) <= eps + 2.0 ** -22 * (1 + abs(want)), (b, i, hq)


def _run(c, G, causal=True):
    q = _bf16(c.rng, (c.T, c.H * G, c.d))
    cache, batch = c.on_device()
    o, lse = fattn.cache_forward(q.to(DEV), cache, batch, c.d ** -0.5, causal)
    _check(c, q, c.d ** -0.5, causal, o, lse)


FEW, MANY = [1, 6], [140]  # tokens: the few-row kernel, the 256-row one


def _zero_blocks(n, d, size, zeros, fmt):
    c = Case([(n, 330), (n, 70)], 2, d, 16, fmt, seed=n + d + size).fill()
    c.cache["v_scale"] = c.cache["v_scale"] * 2.0 ** size
    for b in range(2):
        blocks = c.table[b, :-(-int(c.lens[b]) // 16)]
        for blk in {"first": blocks[:1], "inside": blocks[2:3], "most": np.r_[blocks[:1], blocks[2:]],
                    "all": blocks}[zeros]:
            c.cache["v"][blk], c.cache["v_scale"][blk] = 0, 2.0 ** -100
    _run(c, 2)


ZEROS = [(size, zeros) for size in (0, 30, 70, 110) for zeros in ("first", "inside", "most")]
ZEROS += [(0, "all")]


@pytest.mark.parametrize("n", FEW)
@pytest.mark.parametrize("d,fmt", [(64, "e5m2"), (128, "e4m3")])
@pytest.mark.parametrize("size,zeros", ZEROS)
def test_blocks_of_zeros_few_rows(n, d, fmt, size, zeros):
    _zero_blocks(n, d, size, zeros, fmt)


def _small_and_large(n, d, levels, order, fmt):
    """Blocks of several sizes; but for the smallest, they are zero in half of the columns."""
    H, bs = 2, 16
    c = Case([(n, 400), (n, 90)], H, d, bs, fmt, seed=n + d + levels[-1]).fill()
    for b in range(2):
        blocks = c.table[b, :-(-int(c.lens[b]) // bs)]
        which = {"alternating": np.arange(len(blocks)) % len(levels),
                 "rising": np.minimum(np.arange(len(blocks)) // 2, len(levels) - 1)[::-1],
                 "falling": np.minimum(np.arange(len(blocks)) // 2, len(levels) - 1)}[order]
        for blk, i in zip(blocks, which):
            c.cache["v_scale"][blk] *= 2.0 ** -levels[i]
            if i < len(levels) - 1:
                c.cache["v"][blk][..., ::2] = 0
    _run(c, 2)


LEVELS = [(0, 19), (0, 24), (0, 34), (0, 40), (0, 25, 50), (0, 8, 16, 24)]


@pytest.mark.parametrize("n", FEW)
@pytest.mark.parametrize("d,fmt", [(64, "e4m3"), (128, "e5m2")])
@pytest.mark.parametrize("levels", LEVELS, ids=str)
@pytest.mark.parametrize("order", ["alternating", "rising", "falling"])
def test_small_values_beside_large_few_rows(n, d, fmt, levels, order):
    _small_and_large(n, d, levels, order, fmt)


def _many_keys(pairs, H, d, bs, fmt):
    """Codes below 2 in size; a block's values are ordinary, 2^30 smaller or zero."""
    c = Case(pairs, H, d, bs, fmt, seed=d + bs, nan_slots=False)
    c.cache["k"] &= 0xbf
    c.cache["v"] &= 0xbf
    c.cache["k_scale"][:] = 0.5
    kind = c.rng.integers(0, 3, c.cache["v_scale"].shape)
    c.cache["v_scale"] = np.choose(kind, [1.0, 2.0 ** -30, 2.0 ** -100])
    c.cache["v"][kind == 2] &= 0x80
    c.cache["v"][kind == 0, :, ::3] = 0
    return c


@pytest.mark.parametrize("d,bs,fmt", [(64, 16, "e5m2"), (128, 32, "e4m3")])
def test_long_shares_of_many_sizes(d, bs, fmt):
    """Shares of several sets of 32 tiles that begin and end inside units."""
    _run(_many_keys([(1, 8000 + 37 * i) for i in range(4)], 32, d, bs, fmt), 1)


def _nan_among_zeros(n, d, fmt):
    """A NaN in a block that is zero otherwise: for the rows that see it, in its column."""
    c = Case([(n, 100)], 2, d, 16, fmt, seed=n + d).fill()
    nan = np.zeros((n, 4, d), dtype=bool)
    for at, col in ((35, 5), (100 + n // 2, 9)):
        blk = c.table[0, at // 16]
        c.cache["v"][blk], c.cache["v_scale"][blk] = 0, 2.0 ** -100
        c.cache["v"][blk, 1, at % 16, col] = 0x7f
        nan[max(0, at - 100):, 2:, col] = True
    q = _bf16(c.rng, (n, 4, d))
    cache, batch = c.on_device()
    o, lse = fattn.cache_forward(q.to(DEV), cache, batch, d ** -0.5, True)
    np.testing.assert_array_equal(np.isnan(o.cpu().double().numpy()), nan)
    assert bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("n", FEW)
@pytest.mark.parametrize("d,fmt", [(64, "e5m2"), (128, "e4m3")])
def test_nan_among_zeros_few_rows(n, d, fmt):
    _nan_among_zeros(n, d, fmt)


def _lse_error(n, G, zero):
    """Mean error of LSE over many rows, with ordinary values or a first block of zeros."""
    c = Case([(n, 300)] * (600 if n == 1 else 3), 1, 64, 16, seed=n).fill()
    if zero:
        for blk in c.table[:, 0]:
            c.cache["v"][blk], c.cache["v_scale"][blk] = 0, 2.0 ** -100
    q = _bf16(c.rng, (c.T, G, 64))
    cache, batch = c.on_device()
    _, lse = fattn.cache_forward(q.to(DEV), cache, batch, 0.125, True)
    _, ref = oc.forward(c.cache, c.fmt, c.batch, q.double().numpy(), 0.125, True)
    return np.abs(lse.cpu().double().numpy() - ref).mean()


def test_lse_beside_a_block_of_zeros_few_rows():
    """LSE does not depend on the values, so its error may not either (a factor of two for
    the places where the sums round)."""
    assert _lse_error(1, 2, True) <= 2 * _lse_error(1, 2, False)


@pytest.mark.parametrize("n", MANY)
@pytest.mark.parametrize("d,fmt", [(64, "e5m2"), (128, "e4m3")])
@pytest.mark.parametrize("size,zeros", ZEROS)
def test_blocks_of_zeros_many_rows(n, d, fmt, size, zeros):
    _zero_blocks(n, d, size, zeros, fmt)


@pytest.mark.parametrize("n", MANY)
@pytest.mark.parametrize("d,fmt", [(64, "e4m3"), (128, "e5m2")])
@pytest.mark.parametrize("levels", LEVELS, ids=str)
@pytest.mark.parametrize("order", ["alternating", "rising", "falling"])
def test_small_values_beside_large_many_rows(n, d, fmt, levels, order):
    _small_and_large(n, d, levels, order, fmt)


def test_lse_beside_a_block_of_zeros_many_rows():
    assert _lse_error(140, 1, True) <= 2 * _lse_error(140, 1, False)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d,bs,fmt", [(64, 16, "e5m2"), (128, 32, "e4m3")])
def test_cut_units_of_many_sizes(d, bs, fmt, causal):
    """Units in pieces of 8 tiles; rows that fill one subtile, and two; the first rows of one
    sequence see nothing."""
    _run(_many_keys([(70, 5000), (200, 90), (130, -40)], 1, d, bs, fmt), 1, causal)


@pytest.mark.parametrize("d,bs,fmt", [(64, 64, "e4m3"), (128, 16, "e5m2")])
def test_long_units_of_many_sizes(d, bs, fmt):
    """Units of 19 tiles: their scales are fetched 16 tiles at a time."""
    _run(_many_keys([(33, 2300)] * 3, 64, d, bs, fmt), 1)


@pytest.mark.parametrize("n", MANY)
@pytest.mark.parametrize("d,fmt", [(64, "e5m2"), (128, "e4m3")])
def test_nan_among_zeros_many_rows(n, d, fmt):
    _nan_among_zeros(n, d, fmt)
