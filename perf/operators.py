"""Cases that measure the operators of the paged 8-bit key/value cache: writing new tokens into it
(append), reading tokens back (read), and attention over it (forward).

The cache is a pool of blocks.  A block holds `bs` tokens of one sequence, for each of H heads, as
8-bit floating codes, with one fp32 scale (a power of two) per block and head, for keys and values
apart.  Sequence b has `lens[b]` tokens; token p of it is row p % bs of block table[b, p // bs].  A
call works on the last n_b tokens of every sequence, packed token by token ([total, heads, d],
sequence b at rows [cu[b], cu[b+1])).
"""
import math
import random

import torch

own = False

DEV = "cuda"
# format -> (torch type, largest value's exponent as frexp gives it; both largest values are 0.875 * 2^x)
FORMATS = {"e4m3": (torch.float8_e4m3fn, 9), "e5m2": (torch.float8_e5m2, 16)}
E_MIN = -100  # the smallest scale's exponent (a block of zeros)


# ------------------------------------------------------------------ cases

def _case(name, op, B, n, prior, H, d, bs, G=1, fmt="e4m3", causal=True, fused=False):
    """n, prior: (lowest, highest) new tokens per sequence and tokens before them."""
    c = {"name": name, "op": op, "B": B, "n_lo": n[0], "n_hi": n[1], "prior_lo": prior[0],
         "prior_hi": prior[1], "H": H, "G": G, "d": d, "bs": bs, "fmt": fmt, "causal": causal,
         "fused": fused}
    if name is None:
        del c["name"]
    return c


def listed():
    return [
        # one decoding step's new token of a small batch: latency
        _case("append_step_b4", "append", 4, (1, 1), (200, 2000), 8, 128, 16),
        # one decoding step of a large batch, keys and values cut from the fused projection's output
        _case("append_step_b256", "append", 256, (1, 1), (100, 2000), 8, 128, 64, G=4, fused=True),
        # a whole long prompt written at once
        _case("append_prompt_32768", "append", 1, (32768, 32768), (0, 0), 16, 128, 64),
        # ragged pieces of prompts that begin and end inside blocks, d = 64
        _case("append_ragged_d64", "append", 16, (1, 2000), (3, 1500), 4, 64, 32, fmt="e5m2"),
        # a short shared prefix read back: latency
        _case("read_prefix_777", "read", 1, (777, 777), (0, 0), 8, 128, 16),
        # whole ragged sequences read back
        _case("read_ragged", "read", 16, (512, 8192), (0, 0), 16, 128, 64),
        # one decoding step of one sequence with grouped heads: latency
        _case("forward_step_b1", "forward", 1, (1, 1), (999, 999), 8, 128, 16, G=4),
        # one decoding step of a ragged batch with grouped heads
        _case("forward_step_ragged", "forward", 32, (1, 1), (511, 8191), 8, 128, 64, G=4, fused=True),
        # one decoding step against long contexts, as many key heads as query heads
        _case("forward_step_long", "forward", 4, (1, 1), (32767, 32767), 32, 128, 128),
        # a few drafted tokens of each sequence checked at once, d = 64
        _case("forward_draft_d64", "forward", 24, (5, 5), (100, 4000), 2, 64, 32, G=8, fmt="e5m2"),
        # one piece of a long prompt, after 8192 tokens of it
        _case("forward_chunk_2048", "forward", 1, (2048, 2048), (8192, 8192), 8, 128, 64, G=4),
        # a mixed batch: single tokens and pieces of prompts in one call, d = 64
        _case("forward_mixed_d64", "forward", 16, (1, 1000), (300, 7000), 16, 64, 32),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        m = most.setdefault(c["op"], [0, 0])
        m[0], m[1] = max(m[0], w["bytes"]), max(m[1], w["flops"])
    while True:
        op = rng.choice(["append", "read", "forward", "forward"])
        d, bs = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
        fmt, fused = rng.choice(["e4m3", "e4m3", "e5m2"]), rng.random() < 0.5
        G = rng.choice([1, 1, 2, 3, 4, 5, 7, 8]) if op == "forward" or fused else 1
        H = rng.choice([1, 2, 3, 4, 8, 16]) if G > 1 else rng.choice([1, 4, 8, 16, 32])
        B = _log_int(rng, 1, 256)
        kind = rng.choice(["step", "draft", "chunk"])
        if op == "read" and kind == "draft":
            kind = "chunk"
        n_hi = 1 if kind == "step" and op != "read" else _log_int(rng, 2, 8) if kind == "draft" \
            else _log_int(rng, 9, 8192)
        n_lo = rng.choice([n_hi, max(1, n_hi // 7), 1])
        prior_hi = _log_int(rng, 1, 32768)
        prior_lo = rng.choice([prior_hi, max(1, prior_hi // 10)])
        c = _case(None, op, B, (n_lo, n_hi), (prior_lo, prior_hi), H, d, bs, G, fmt,
                  rng.random() < 0.8, fused)
        w = work(c)
        pairs = _sizes(c)
        pool = sum(n + p for n, p in pairs) * H * d
        square = B * H * G * max(n for n, _ in pairs) * max(n + p for n, p in pairs)
        if w["bytes"] <= most[op][0] and w["flops"] <= max(most[op][1], 1) and pool <= 3e8 \
                and B * max(n + p for n, p in pairs) * H * d <= 6e8 \
                and (op != "forward" or square <= 1.5e9):
            return c


def _sizes(case):
    """(new tokens, tokens before them) of each sequence, spread over their ranges' logarithms."""
    B = case["B"]
    step = next(s for s in (7, 5, 3, 1) if math.gcd(s, B) == 1)

    def at(lo, hi, i):
        if lo == hi or B == 1:
            return hi
        return int(round(max(lo, 0.5) * (hi / max(lo, 0.5)) ** (i / (B - 1))))

    return [(max(1, at(case["n_lo"], case["n_hi"], i)),
             at(case["prior_lo"], case["prior_hi"], (i * step) % B)) for i in range(B)]


def work(case):
    H, G, d, bs = (case[k] for k in ("H", "G", "d", "bs"))
    pairs = _sizes(case)
    T = sum(n for n, _ in pairs)
    blocks = sum((n + p + bs - 1) // bs - p // bs for n, p in pairs)
    if case["op"] in ("append", "read"):
        # bf16 keys and values on one side, codes and scales on the other
        return {"bytes": T * H * d * (4 + 2) + blocks * H * 8, "flops": 0}
    length = sum(n + p for n, p in pairs)
    seen = sum(n * (n + p) - (n * (n - 1) // 2 if case["causal"] else 0) for n, p in pairs)
    blocks = sum((n + p + bs - 1) // bs for n, p in pairs)
    return {"bytes": length * H * d * 2 + blocks * (H * 8 + 4) + T * H * G * (4 * d + 4),
            "flops": 4 * seen * H * G * d}


# ------------------------------------------------------------------ inputs

def _pool(gen, blocks, H, bs, d, fmt, key):
    """Codes and scales of `blocks` blocks as a model leaves them: keys with a few strong channels,
    values whose size varies from block to block."""
    dt, top = FORMATS[fmt]
    size = torch.exp(0.7 * torch.randn((blocks, H, 1, 1), generator=gen, device=DEV))
    chan = torch.ones((1, H, 1, d), device=DEV)
    if key:
        chan = torch.where(torch.rand((1, H, 1, d), generator=gen, device=DEV) < 0.04, 6.0, 0.8)
        size = torch.ones_like(size)
    codes = torch.empty((blocks, H, bs, d), dtype=dt, device=DEV)
    scale = torch.empty((blocks, H), device=DEV)
    part = max(1, (1 << 27) // (H * bs * d))
    for a in range(0, blocks, part):
        z = slice(a, min(blocks, a + part))
        x = torch.randn((z.stop - a, H, bs, d), generator=gen, device=DEV) * chan * size[z]
        s = _scale_of(x.abs().amax(dim=(2, 3)), top)
        codes[z] = (x / s[:, :, None, None]).to(dt)
        scale[z] = s
    return codes, scale


def prepare(case, seed):
    B, H, G, d, bs, fmt = (case[k] for k in ("B", "H", "G", "d", "bs", "fmt"))
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rng = random.Random(seed)
    pairs = _sizes(case)
    rng.shuffle(pairs)
    n = [a for a, _ in pairs]
    lens = [a + p for a, p in pairs]
    need = [(x + bs - 1) // bs for x in lens]
    blocks = sum(need) + 3
    order = list(range(blocks))
    rng.shuffle(order)
    table = [[0] * max(need) for _ in range(B)]
    for b in range(B):
        table[b][:need[b]] = [order.pop() for _ in range(need[b])]
    k, k_scale = _pool(gen, blocks, H, bs, d, fmt, True)
    v, v_scale = _pool(gen, blocks, H, bs, d, fmt, False)
    T, Hq = sum(n), H * G
    # the projections' output: one tensor of queries, keys and values, or one for each
    if case["fused"]:
        x = torch.randn((T, Hq + 2 * H, d), generator=gen, device=DEV).bfloat16()
        q, kn, vn = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
    else:
        q, kn, vn = (torch.randn((T, h, d), generator=gen, device=DEV).bfloat16()
                     for h in (Hq, H, H))
    if case["op"] == "append":  # tokens of different size, so that some blocks' scales grow
        kn.mul_(torch.exp(0.5 * torch.randn((T, 1, 1), generator=gen, device=DEV)).bfloat16())
        vn.mul_(torch.exp(0.7 * torch.randn((T, 1, 1), generator=gen, device=DEV)).bfloat16())
    cu = [0]
    for a in n:
        cu.append(cu[-1] + a)
    i32 = dict(dtype=torch.int32, device=DEV)
    s = {"case": dict(case), "k": k, "v": v, "k_scale": k_scale, "v_scale": v_scale,
         "table": torch.tensor(table, **i32), "lens": torch.tensor(lens, **i32),
         "cu": torch.tensor(cu, **i32), "total": T, "max_n": max(n), "max_len": max(lens)}
    if case["op"] == "append":
        s["kn"], s["vn"] = kn, vn
    if case["op"] == "forward":
        s["q"] = q
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    c = state["case"]
    if own:
        from online_softmax_08_gb300 import fattn
        cache = fattn.KVCache(state["k"], state["v"], state["k_scale"], state["v_scale"])
        batch = fattn.CacheBatch(state["table"], state["lens"], state["cu"], state["total"],
                                 state["max_n"])
        if c["op"] == "append":
            fattn.cache_append(state["kn"], state["vn"], cache, batch)
            return _whole(state)
        if c["op"] == "read":
            k, v = fattn.cache_read(cache, batch)
            return {"k": k, "v": v}
        o, lse = fattn.cache_forward(state["q"], cache, batch, c["d"] ** -0.5, c["causal"])
        return {"o": o, "lse": lse}
    return {"append": _append, "read": _read, "forward": _forward}[c["op"]](state)


def _whole(state):
    return {name: state[name] for name in ("k", "v", "k_scale", "v_scale")}


def _scale_of(amax, top):
    """2^e with the smallest e >= E_MIN for which amax <= 0.875 * 2^top * 2^e."""
    m, x = torch.frexp(amax)
    e = torch.clamp(x - top + (m > 0.875).to(x.dtype), min=E_MIN)
    e = torch.where(amax > 0, e, torch.full_like(e, E_MIN))
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _tokens(state):
    """Of every packed token: its sequence, and its position in it."""
    n = state["cu"].diff()
    seq = torch.repeat_interleave(torch.arange(n.numel(), device=DEV), n, output_size=state["total"])
    i = torch.arange(state["total"], device=DEV) - state["cu"][seq]
    return seq, i + (state["lens"] - n)[seq]


def _append(state):
    bs, (dt, top) = state["case"]["bs"], FORMATS[state["case"]["fmt"]]
    seq, pos = _tokens(state)
    blk, row = state["table"][seq, pos // bs].long(), pos % bs
    n = state["cu"].diff()
    start = state["lens"] - n
    first = state["table"][torch.arange(n.numel(), device=DEV), start // bs].long()
    held = torch.arange(bs, device=DEV)[None, :] < (start % bs)[:, None]  # rows written before
    for new, codes, scale in ((state["kn"], state["k"], state["k_scale"]),
                              (state["vn"], state["v"], state["v_scale"])):
        x = new.float()
        amax = torch.zeros_like(scale)
        amax.scatter_reduce_(0, blk[:, None].expand(-1, x.shape[1]), x.abs().amax(dim=2), "amax")
        need = _scale_of(amax, top)
        before = scale[first]
        after = torch.where((start % bs > 0)[:, None], torch.maximum(need[first], before),
                            need[first])
        scale[blk] = need[blk]
        scale[first] = after
        raw = codes.view(torch.uint8)
        old = codes.view(torch.uint8)[first].view(dt).float()
        moved = (old * (before / after)[:, :, None, None]).to(dt).view(torch.uint8)
        raw[first] = torch.where(held[:, None, :, None], moved, raw[first])
        raw[blk, :, row] = (x / scale[blk][:, :, None]).to(dt).view(torch.uint8)
    return _whole(state)


def _read(state):
    bs, dt = state["case"]["bs"], state["k"].dtype
    seq, pos = _tokens(state)
    blk, row = state["table"][seq, pos // bs].long(), pos % bs

    def back(codes, scale):
        x = codes.view(torch.uint8)[blk, :, row].view(dt).float()
        return (x * scale[blk][:, :, None]).bfloat16()

    return {"k": back(state["k"], state["k_scale"]), "v": back(state["v"], state["v_scale"])}


def _forward(state):
    c = state["case"]
    H, G, d, bs = (c[k] for k in ("H", "G", "d", "bs"))
    B, N, L, dt = state["table"].shape[0], state["max_n"], state["max_len"], state["k"].dtype
    table = state["table"].long()

    def whole(codes, scale):  # [B, H, L, d]
        x = codes.view(torch.uint8)[table].view(dt).float() * scale[table][..., None, None]
        return x.transpose(1, 2).reshape(B, H, -1, d)[:, :, :L]

    seq, pos = _tokens(state)
    i = torch.arange(state["total"], device=DEV) - state["cu"][seq]
    q = torch.zeros((B, N, H * G, d), device=DEV)
    q[seq, i] = state["q"].float()
    q = q.reshape(B, N, H, G, d).permute(0, 2, 3, 1, 4).reshape(B, H, G * N, d)
    s = torch.matmul(q, whole(state["k"], state["k_scale"]).transpose(2, 3)) * d ** -0.5
    at = torch.arange(L, device=DEV)
    seen = (at[None, :] < state["lens"][:, None])[:, None, :].expand(B, N, L)
    if c["causal"]:
        where = (state["lens"] - state["cu"].diff())[:, None] + torch.arange(N, device=DEV)
        seen = seen & (at <= where[:, :, None])
    s = s.reshape(B, H, G, N, L).masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    p = s.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    total = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p.reshape(B, H, G * N, L), whole(state["v"], state["v_scale"]))
    o = o.reshape(B, H, G, N, d) / torch.where(total > 0, total, 1.0)
    lse = (m + total.log())[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, N, H * G, d)[seq, i].bfloat16()
    lse = lse.permute(0, 3, 1, 2).reshape(B, N, H * G)[seq, i].t().contiguous()
    return {"o": o, "lse": lse}


# ------------------------------------------------------------------ the definition in 64 bits

def _pow2(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _round8(x, fmt):
    """x rounded to the nearest value of the format (ties to even), in 64 bits."""
    bits, low = (3, -6) if fmt == "e4m3" else (2, -14)
    _, e = torch.frexp(x)
    step = _pow2(torch.clamp(e - 1, min=low) - bits)
    return torch.round(x / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    H, G, d, bs, fmt = (case[k] for k in ("H", "G", "d", "bs", "fmt"))
    if work(case)["flops"] > 4e12:
        return None
    table, lens, cu = s["table"].tolist(), s["lens"].tolist(), s["cu"].tolist()
    largest = 448.0 if fmt == "e4m3" else 57344.0
    if case["op"] == "append":
        out = {}
        for name, new in (("k", s["kn"]), ("v", s["vn"])):
            codes, scale = s[name].double(), s[name + "_scale"].double()
            for b, length in enumerate(lens):
                start = length - (cu[b + 1] - cu[b])
                for j in range(start // bs, (length - 1) // bs + 1):
                    blk, lo, hi = table[b][j], max(start, j * bs), min(length, (j + 1) * bs)
                    x = new[cu[b] + lo - start:cu[b] + hi - start].double().transpose(0, 1)
                    a = x.abs().amax(dim=(1, 2))
                    m, e = torch.frexp(a / largest)  # m in [0.5, 1): 2^(e - 1) when m = 0.5
                    e = torch.where(a > 0, e - (m == 0.5).int(), E_MIN).clamp(min=E_MIN)
                    s_new = _pow2(e)
                    if lo % bs:
                        s_new = torch.maximum(s_new, scale[blk])
                        old = codes[blk, :, :lo % bs] * (scale[blk] / s_new)[:, None, None]
                        codes[blk, :, :lo % bs] = _round8(old, fmt)
                    codes[blk, :, lo % bs:lo % bs + hi - lo] = _round8(x / s_new[:, None, None], fmt)
                    scale[blk] = s_new
            out[name], out[name + "_scale"] = codes, scale
        return out

    def tokens(name, b, lo, hi):  # [H, hi - lo, d]
        rows = torch.tensor(table[b][lo // bs:(hi - 1) // bs + 1], device=DEV)
        x = s[name].view(torch.uint8)[rows].view(s[name].dtype).double()
        x = x * s[name + "_scale"][rows].double()[:, :, None, None]
        x = x.transpose(0, 1).reshape(H, -1, d)
        return x[:, lo % bs:lo % bs + hi - lo]

    if case["op"] == "read":
        return {name: torch.cat([tokens(name, b, length - (cu[b + 1] - cu[b]), length).transpose(0, 1)
                                 for b, length in enumerate(lens)]) for name in ("k", "v")}
    o = torch.empty((s["total"], H * G, d), dtype=torch.float64, device=DEV)
    lse = torch.empty((H * G, s["total"]), dtype=torch.float64, device=DEV)
    for b, length in enumerate(lens):
        n = cu[b + 1] - cu[b]
        k, v = tokens("k", b, 0, length), tokens("v", b, 0, length)
        hide = torch.arange(length, device=DEV)[None, :] > \
            torch.arange(length - n, length, device=DEV)[:, None]
        for h in range(H * G):
            t = s["q"][cu[b]:cu[b + 1], h].double() @ k[h // G].t() / math.sqrt(d)
            if case["causal"]:
                t = t.masked_fill(hide, -math.inf)
            l = torch.logsumexp(t, dim=1)
            lse[h, cu[b]:cu[b + 1]] = l
            o[cu[b]:cu[b + 1], h] = torch.exp(t - l[:, None]) @ v[h // G]
    return {"o": o, "lse": lse}
