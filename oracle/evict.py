"""The attention weight of cached keys, and the eviction by it, in numpy, fp64.  TEST
INFRASTRUCTURE ONLY; shares no code with the library."""
import numpy as np

from . import cache as _cache
from . import cache4 as _cache4


def _tokens(fmt):
    return _cache4.tokens if fmt == "int4" else _cache.tokens


def weights(cache, fmt, batch, q, lse, scale, causal, before, out):
    """The weights [B, H, width] after the call (`out` before it), and for every element a bound
    of the relative error of what the queries add: the largest sum_c |scale q_c k_c| + |lse|."""
    table, lens, cu = batch
    H, Hq = cache["k"].shape[1], q.shape[1]
    out, size = np.array(out, dtype=np.float64), np.zeros(out.shape)
    for b, length in enumerate(lens):
        n, length = int(cu[b + 1] - cu[b]), int(length)
        if n == 0:
            continue
        start = max(0, length - n)
        out[b, :, start:length] = 0.0
        out[b, :, :start] = 0.0 if before is None else before[b, :, :start]
        k = _tokens(fmt)(cache, fmt, table[b], "k", 0, length)
        t = np.arange(int(cu[b]), int(cu[b + 1]))
        at = np.arange(length)
        sees = at[None, :] <= (length - n + np.arange(n))[:, None] if causal else \
            np.ones((n, length), dtype=bool)
        for hq in range(Hq):
            h = hq // (Hq // H)
            rows = lse[hq, t] != -np.inf
            see = sees[rows]
            x, l = q[t[rows], hq], lse[hq, t[rows]][:, None]
            with np.errstate(invalid="ignore", over="ignore"):
                out[b, h, :length] += np.where(see, np.exp(scale * (x @ k[:, h].T) - l), 0.0).sum(axis=0)
            s = np.where(see, scale * (np.abs(x) @ np.abs(k[:, h].T)) + np.abs(l), 0.0)
            size[b, h, :length] = np.maximum(size[b, h, :length], s.max(axis=0, initial=0.0))
    return out, size


def choose(w, length, keep, recent):
    """Positions that a head keeps, ascending."""
    if length <= keep:
        return np.arange(length)
    old = length - recent
    x = np.where(np.isnan(w[:old]), np.inf, w[:old])
    nan = np.isnan(w[:old])
    # largest first: NaN, then by weight, then by position
    order = sorted(range(old), key=lambda j: (not nan[j], -x[j], j))
    return np.array(sorted(order[:keep - recent]) + list(range(old, length)), dtype=int)


def evict(cache, fmt, table, lens, w, table_out, keep, recent):
    """The pool after the call, the kept positions [B][H] and the new lengths."""
    out = {name: a.copy() for name, a in cache.items()}
    bs, H = cache["k"].shape[2], cache["k"].shape[1]
    kept = [[choose(w[b, h], int(lens[b]), keep, recent) for h in range(H)] for b in range(len(lens))]
    for b in range(len(lens)):
        for h in range(H):
            pos = kept[b][h]
            for j0 in range(0, len(pos), bs):
                to, part = table_out[b, j0 // bs], pos[j0:j0 + bs]
                blk, row = table[b][part // bs], part % bs
                for side in ("k", "v"):
                    scale = side + "_scale"
                    if fmt == "int4":
                        out[side][to, h, :len(part)] = cache[side][blk, h, row]
                        out[scale][to, h, :len(part)] = cache[scale][blk, h, row]
                        continue
                    old = cache[scale][blk, h]
                    new = old.max()
                    codes = cache[side][blk, h, row]
                    x = _cache.code_values(fmt)[codes] * (old / new)[:, None]
                    with np.errstate(invalid="ignore"):
                        moved = np.where((old == new)[:, None], codes, _cache.round_codes(x, fmt))
                    out[side][to, h, :len(part)] = moved
                    out[scale][to, h] = new
    return out, kept, np.minimum(lens, keep)
