"""The paged 4-bit key/value cache in numpy, fp64: the definition of quantising, reading back
and attending, token by token and group by group.  TEST INFRASTRUCTURE ONLY; shares no code
with the library.

A cache is a dict of numpy arrays: k, v uint8 [num_blocks, H, bs, d / 2], two codes a byte, the
even channel in the low half, and k_scale, v_scale uint8 [num_blocks, H, bs, d / 16], e5m2.  A
batch is (table [B, width], lens [B], cu [B + 1]) as the library takes it.
"""
import numpy as np

from . import cache as _cache

E5M2 = _cache.code_values("e5m2")
LARGEST = 57344.0


def quantise_groups(x):
    """Codes (0 to 15) and scale bytes of groups of 16 values, x [n, 16]."""
    x = np.where(np.isnan(x), 0.0, np.clip(x, -LARGEST, LARGEST))
    a = np.abs(x).max(axis=1, keepdims=True)
    byte = _cache.round_codes(a / 8.0, "e5m2")
    byte = np.where(np.any(x == a, axis=1, keepdims=True), byte | 0x80, byte)
    s = E5M2[byte]
    c = np.rint(x / np.where(s == 0.0, 1.0, s)) + 8
    return np.where(s == 0.0, 8, np.clip(c, 0, 15)).astype(np.uint8), byte[:, 0].astype(np.uint8)


def quantise(x):
    """Packed codes [..., d / 2] and scale bytes [..., d / 16] of x [..., d]."""
    codes, scales = quantise_groups(x.reshape(-1, 16))
    codes = codes.reshape(x.shape)
    return codes[..., 0::2] | codes[..., 1::2] << 4, scales.reshape(x.shape[:-1] + (x.shape[-1] // 16,))


def values(codes, scales):
    """The values [..., d] of packed codes and scale bytes."""
    c = np.stack((codes & 15, codes >> 4), axis=-1).reshape(codes.shape[:-1] + (2 * codes.shape[-1],))
    c = c.astype(float)
    return (c - 8.0) * np.repeat(E5M2[scales], 16, axis=-1)


def append(cache, batch, k, v):
    """The cache after the call; k, v float64 [total, H, d]."""
    out = {name: a.copy() for name, a in cache.items()}
    table, lens, cu = batch
    bs = out["k"].shape[2]
    for b in range(len(lens)):
        n = int(cu[b + 1] - cu[b])
        for i in range(n):
            p = int(lens[b]) - n + i
            blk, row = table[b, p // bs], p % bs
            for side, x in (("k", k), ("v", v)):
                out[side][blk, :, row], out[side + "_scale"][blk, :, row] = quantise(x[cu[b] + i])
    return out


def tokens(cache, fmt, table_row, side, lo, hi):
    """Values [hi - lo, H, d] of tokens [lo, hi) of a sequence (fmt: not used)."""
    codes, scale = cache[side], cache[side + "_scale"]
    p = np.arange(lo, hi)
    blk, row = np.asarray(table_row)[p // codes.shape[2]], p % codes.shape[2]
    return values(codes[blk, :, row], scale[blk, :, row])


def read(cache, batch):
    table, lens, cu = batch
    return tuple(np.concatenate([tokens(cache, None, table[b], side,
                                        int(lens[b] - (cu[b + 1] - cu[b])), int(lens[b]))
                                 for b in range(len(lens))]) for side in ("k", "v"))


def forward(cache, batch, q, scale, causal, d_error=False):
    """As oracle.cache.forward."""
    return _cache.forward(cache, None, batch, q, scale, causal, d_error, tokens)
