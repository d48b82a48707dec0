"""The paged 8-bit key/value cache in numpy, fp64: the definition of quantising,
reading back and attending, sequence by sequence and block by block.  TEST
INFRASTRUCTURE ONLY; shares no code with the library.

A cache is a dict of numpy arrays: k, v uint8 codes [num_blocks, H, bs, d],
k_scale, v_scale float64 [num_blocks, H].  A batch is (table [B, width], lens
[B], cu [B + 1]) as the library takes it.
"""
import numpy as np

# format -> (exponent bits, mantissa bits, largest finite value)
FORMATS = {"e4m3": (4, 3, 448.0), "e5m2": (5, 2, 57344.0)}
E_MIN = -100


def code_values(fmt):
    """The value of each of the 256 codes (NaN and infinities included)."""
    ebits, mbits, _ = FORMATS[fmt]
    bias = 2 ** (ebits - 1) - 1
    out = np.empty(256)
    for c in range(256):
        sign = -1.0 if c & 0x80 else 1.0
        e, m = (c >> mbits) & (2 ** ebits - 1), c & (2 ** mbits - 1)
        if fmt == "e4m3" and (c & 0x7f) == 0x7f:
            x = np.nan
        elif fmt == "e5m2" and e == 31:
            x = np.nan if m else np.inf
        elif e == 0:
            x = m * 2.0 ** (1 - bias - mbits)
        else:
            x = (1.0 + m * 2.0 ** -mbits) * 2.0 ** (e - bias)
        out[c] = sign * x
    return out


def round_codes(x, fmt):
    """Codes of the nearest representable values (ties to the even code); NaN for
    NaN, the sign of a zero kept.  |x| must not exceed the largest value."""
    values = code_values(fmt)
    pos = values[:128]
    n = int(np.sum(np.isfinite(pos)))  # codes 0 .. n - 1 ascend
    a = np.abs(x)
    up = np.clip(np.searchsorted(pos[:n], a), 0, n - 1)
    down = np.maximum(up - 1, 0)
    below, above = a - pos[down], pos[up] - a
    pick = np.where(below < above, down, up)
    pick = np.where(below == above, np.where(down % 2 == 0, down, up), pick)
    code = np.where(np.isnan(x), 0x7f, pick).astype(np.uint8)
    return np.where(np.signbit(x), code | 0x80, code).astype(np.uint8)


def scale_for(amax, fmt):
    """The smallest power of two 2^e, e >= E_MIN, with amax <= largest * 2^e."""
    e = E_MIN
    while amax > FORMATS[fmt][2] * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(cache, fmt, batch, k, v):
    """The cache after the call; k, v float64 [total, H, d] (infinities and NaN allowed)."""
    out = {name: a.copy() for name, a in cache.items()}
    table, lens, cu = batch
    bs = out["k"].shape[2]
    for b in range(len(lens)):
        n = int(cu[b + 1] - cu[b])
        start = int(lens[b]) - n
        for side, x in (("k", k), ("v", v)):
            codes, scale = out[side], out[side + "_scale"]
            p = start
            while p < lens[b]:
                blk, row = table[b, p // bs], p % bs
                count = min(bs - row, int(lens[b]) - p)
                for h in range(codes.shape[1]):
                    new = x[cu[b] + p - start:cu[b] + p - start + count, h]
                    new = np.where(np.isfinite(new), new, np.copysign(np.nan, new))
                    a = np.abs(new[np.isfinite(new)])
                    s = scale_for(a.max() if a.size else 0.0, fmt)
                    if row > 0 and scale[blk, h] > s:
                        s = scale[blk, h]
                    if row > 0 and s > scale[blk, h]:
                        old = code_values(fmt)[codes[blk, h, :row]]
                        codes[blk, h, :row] = round_codes(old * (scale[blk, h] / s), fmt)
                    codes[blk, h, row:row + count] = round_codes(new / s, fmt)
                    scale[blk, h] = s
                p += count
    return out


def tokens(cache, fmt, table_row, side, lo, hi):
    """Values [hi - lo, H, d] of tokens [lo, hi) of a sequence."""
    values, codes, scale = code_values(fmt), cache[side], cache[side + "_scale"]
    bs = codes.shape[2]
    rows = [values[codes[table_row[p // bs], :, p % bs]] * scale[table_row[p // bs]][:, None]
            for p in range(lo, hi)]
    return np.stack(rows) if rows else np.zeros((0, codes.shape[1], codes.shape[3]))


def read(cache, fmt, batch):
    table, lens, cu = batch
    return tuple(np.concatenate([tokens(cache, fmt, table[b], side,
                                        int(lens[b] - (cu[b + 1] - cu[b])), int(lens[b]))
                                 for b in range(len(lens))]) for side in ("k", "v"))


def forward(cache, fmt, batch, q, scale, causal, d_error=False, tokens=tokens):
    """O [T, Hq, d], LSE [Hq, T] of q [T, Hq, d]; with d_error also A [T, Hq, d] =
    sum_j P_j |v_j|, S [Hq, T] = the largest scale * sum_c |q_c k_c| of a visible
    key, and the number of visible keys [T].  tokens: how the cache's values are read."""
    table, lens, cu = batch
    T, Hq, d = q.shape
    H = cache["k"].shape[1]
    o, lse = np.zeros((T, Hq, d)), np.full((Hq, T), -np.inf)
    A, S, seen = np.zeros((T, Hq, d)), np.zeros((Hq, T)), np.zeros(T, dtype=int)
    for b in range(len(lens)):
        length, n = int(lens[b]), int(cu[b + 1] - cu[b])
        if n == 0 or length == 0:
            continue
        k = tokens(cache, fmt, table[b], "k", 0, length)
        v = tokens(cache, fmt, table[b], "v", 0, length)
        for i in range(n):
            lim = length - n + i + 1 if causal else length
            if lim <= 0:
                continue
            t = int(cu[b]) + i
            seen[t] = lim
            for hq in range(Hq):
                h = hq // (Hq // H)
                s = scale * (k[:lim, h] @ q[t, hq])
                m = s.max()
                e = np.exp(s - m)
                lse[hq, t] = m + np.log(e.sum())
                w = e / e.sum()
                o[t, hq] = w @ v[:lim, h]
                A[t, hq] = w @ np.abs(v[:lim, h])
                S[hq, t] = (scale * (np.abs(k[:lim, h]) @ np.abs(q[t, hq]))).max()
    return (o, lse, A, S, seen) if d_error else (o, lse)
