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
        for i in range(n):
            lim = max(0, length - n + i + 1) if causal else length
            t = int(cu[b]) + i
            for hq in range(Hq):
                h = hq // (Hq // H)
                if lse[hq, t] == -np.inf:
                    continue
                out[b, h, :lim] += np.exp(scale * (k[:lim, h] @ q[t, hq]) - lse[hq, t])
                s = scale * (np.abs(k[:lim, h]) @ np.abs(q[t, hq])) + abs(lse[hq, t])
                size[b, h, :lim] = np.maximum(size[b, h, :lim], s)
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
