"""Cases that measure the operators around the paged key/value cache in 4 bits: writing tokens into it
and reading them back (write), attention over it (forward), the rotary positions that queries and keys
get before (rope), the attention weight that every cached key has received (weights), and the copy of
a cache's most attended tokens into a shorter one (evict).

The cache is a pool of blocks of `bs` tokens of one sequence, for each of H heads.  In 4 bits
("int4"), 16 neighbouring channels of a token share a scale s, an 8-bit float of 2 mantissa bits
(e5m2), and are codes c from 0 to 15 with the value (c - 8) s, two codes a byte, the even channel in
the low half.  With a the group's largest magnitude, |s| is a / 8 rounded to e5m2, and s is negative if
the group holds +a, so that this value gets the code 0, else positive; c - 8 is x / s rounded to the
nearest whole number (ties to even) within [-8, 7].  In 8 bits ("e4m3", "e5m2") a block and head has
one fp32 scale.  Sequence b has `lens[b]` tokens; token p of it is row p % bs of block
table[b, p // bs].  Packed tensors are [total, heads, d], sequence b at rows [cu[b], cu[b + 1]).
"""
import math
import random

import torch

own = False

DEV = "cuda"
FLOATS = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = 57344.0  # the largest magnitude that int4 keeps: 8 times the scale 7168
PI2 = 2.0 * math.pi


# ------------------------------------------------------------------ cases

def _case(name, op, B, n, prior, H, d, bs=64, G=1, fmt="int4", causal=True, fused=False, **more):
    """n, prior: (lowest, highest) new tokens per sequence and tokens before them.  evict: keep and
    recent; rope: rot, layout, kind, factor, length, base, back, far."""
    c = {"name": name, "op": op, "B": B, "n_lo": n[0], "n_hi": n[1], "prior_lo": prior[0],
         "prior_hi": prior[1], "H": H, "G": G, "d": d, "bs": bs, "fmt": fmt, "causal": causal,
         "fused": fused}
    c.update(more)
    if name is None:
        del c["name"]
    return c


def listed():
    return [
        # the new tokens of a small batch's decoding step, written and read back: latency
        _case("write_step_b4", "write", 4, (1, 1), (200, 2000), 8, 128, 16, G=4, fused=True),
        # a whole long prompt written, and read back for a stage that takes bf16
        _case("write_prompt_32768", "write", 1, (32768, 32768), (0, 0), 16, 128, 64),
        # one decoding step of one sequence with grouped heads: latency
        _case("forward_step_b1", "forward", 1, (1, 1), (999, 999), 8, 128, 16, G=4),
        # one decoding step against long contexts, as many key heads as query heads
        _case("forward_step_long", "forward", 4, (1, 1), (32767, 32767), 32, 128, 128),
        # a mixed batch: single tokens and pieces of prompts in one call, d = 64
        _case("forward_mixed_d64", "forward", 16, (1, 1000), (300, 7000), 16, 64, 32),
        # one piece of a long prompt, after 8192 tokens of it
        _case("forward_chunk_2048", "forward", 1, (2048, 2048), (8192, 8192), 8, 128, 64, G=4),
        # one decoding step of a batch: positions for its queries and keys, scaled for long contexts
        _case("rope_step_b64", "rope", 64, (1, 1), (100, 120000), 8, 128, G=4, fused=True, rot=128,
              layout="half", kind="yarn", factor=16.0, length=8192, base=10000.0, back=False, far=0),
        # the gradients of a training step's queries and keys, pairs of neighbours in half of the head
        _case("rope_grad_16384", "rope", 8, (2048, 2048), (0, 0), 8, 128, G=4, rot=64,
              layout="interleaved", kind="none", factor=1.0, length=0, base=10000.0, back=True, far=0),
        # one decoding step of a ragged batch: its weights join those of the steps before
        _case("weights_step_ragged", "weights", 32, (1, 1), (511, 8191), 8, 128, 64, G=4),
        # the last 512 tokens of a prompt, which say what to keep of it, over an 8-bit cache
        _case("weights_window_512", "weights", 1, (512, 512), (16384, 16384), 8, 128, 64, G=4, fmt="e4m3"),
        # one long sequence cut to 2048 tokens, and the kept ones read back
        _case("evict_b1_to_2048", "evict", 1, (0, 0), (16384, 16384), 8, 128, 64, keep=2048, recent=512),
        # a batch of long sequences cut to 8192 tokens each, 8 bits
        _case("evict_b8_to_8192_e4m3", "evict", 8, (0, 0), (9000, 32768), 8, 128, 64, fmt="e4m3",
              keep=8192, recent=1024),
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
        op = rng.choice(["write", "forward", "forward", "rope", "weights", "evict"])
        d, bs = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
        fused, causal = rng.random() < 0.5, rng.random() < 0.8
        G = rng.choice([1, 1, 2, 3, 4, 5, 7, 8])
        H = rng.choice([1, 2, 3, 4, 8, 16]) if G > 1 else rng.choice([1, 4, 8, 16, 32])
        B = _log_int(rng, 1, 256)
        kind = rng.choice(["step", "draft", "chunk"])
        n_hi = 1 if kind == "step" else _log_int(rng, 2, 8) if kind == "draft" \
            else _log_int(rng, 9, 8192)
        n_lo = rng.choice([n_hi, max(1, n_hi // 7), 1])
        prior_hi = _log_int(rng, 1, 32768)
        prior_lo = rng.choice([prior_hi, max(1, prior_hi // 10)])
        fmt, more = "int4", {}
        if op in ("weights", "evict"):
            fmt = rng.choice(["int4", "int4", "e4m3", "e5m2"])
        if op == "evict":
            n_lo = n_hi = 0
            more["keep"] = _log_int(rng, 1, prior_hi)
            more["recent"] = rng.choice([0, more["keep"] // 4, more["keep"]])
        if op == "rope":
            how = rng.choice(["none", "linear", "base", "yarn", "bands"])
            more = {"rot": rng.choice([16, 32, 48, 64]) if d == 64 else rng.choice([16, 32, 64, 112, 128]),
                    "layout": rng.choice(["half", "interleaved"]), "kind": how,
                    "factor": 1.0 if how == "none" else rng.choice([2.0, 8.0, 32.0, 40.0]),
                    "length": rng.choice([2048, 4096, 8192]), "base": rng.choice([1e4, 5e5, 1e6]),
                    "back": rng.random() < 0.4, "far": rng.choice([0, 0, 1000000])}
        c = _case(None, op, B, (n_lo, n_hi), (prior_lo, prior_hi), H, d, bs, G, fmt, causal, fused,
                  **more)
        w = work(c)
        pairs = _sizes(c)
        longest = max(n + p for n, p in pairs)
        square = B * H * G * max(n for n, _ in pairs) * longest
        if w["bytes"] <= most[op][0] and w["flops"] <= max(most[op][1], 1) \
                and (op == "rope" or sum(n + p for n, p in pairs) * H * d <= 5.5e8) \
                and (op == "rope" or B * longest * H * d <= 6e8) \
                and (op not in ("forward", "weights") or square <= 1.5e9):
            return c


def _sizes(case):
    """(new tokens, tokens before them) of each sequence, spread over their ranges' logarithms."""
    B = case["B"]
    step = next(s for s in (7, 5, 3, 1) if math.gcd(s, B) == 1)

    def at(lo, hi, i):
        if lo == hi or B == 1:
            return hi
        return int(round(max(lo, 0.5) * (hi / max(lo, 0.5)) ** (i / (B - 1))))

    least = 0 if case["op"] == "evict" else 1
    return [(max(least, at(case["n_lo"], case["n_hi"], i)),
             at(case["prior_lo"], case["prior_hi"], (i * step) % B)) for i in range(B)]


def _token_bytes(case):
    """Bytes of one token's codes, of one head's keys or values (8 bits: the scales come by block)."""
    d = case["d"]
    return d // 2 + d // 16 if case["fmt"] == "int4" else d


def work(case):
    H, G, d, bs, op = (case[k] for k in ("H", "G", "d", "bs", "op"))
    pairs, one = _sizes(case), _token_bytes(case)
    T, length = sum(n for n, _ in pairs), sum(n + p for n, p in pairs)
    blocks = sum((n + p + bs - 1) // bs for n, p in pairs)
    scales = 0 if case["fmt"] == "int4" else blocks * H * 4  # of keys or values
    seen = sum(n * (n + p) - (n * (n - 1) // 2 if case["causal"] else 0) for n, p in pairs)
    if op == "write":  # bf16 keys and values read and written, codes written
        return {"bytes": T * H * (4 * d + 4 * d + 2 * one), "flops": 0}
    if op == "rope":  # bf16 in and out; four products and two sums for each pair of channels
        return {"bytes": T * H * (G + 1) * 4 * d + 4 * T, "flops": 3 * T * H * (G + 1) * case["rot"]}
    if op == "forward":
        return {"bytes": length * H * 2 * one + blocks * 4 + T * H * G * (4 * d + 4),
                "flops": 4 * seen * H * G * d}
    if op == "weights":  # keys, old and new weights, queries and their log-sum-exp
        return {"bytes": length * H * (one + 8) + scales + blocks * 4 + T * H * G * (2 * d + 4),
                "flops": 2 * seen * H * G * d}
    kept = [min(p, case["keep"]) for _, p in pairs]
    m = sum(kept)
    # weights looked at; kept tokens read and written, their positions and weights written
    total = sum(p * 4 for (_, p), k in zip(pairs, kept) if k < p) * H + m * H * (4 * one + 12)
    if case["fmt"] == "int4":
        total += m * H * 4 * d  # and read back as bf16
    else:
        total += 2 * scales + 2 * 4 * H * sum((k + bs - 1) // bs for k in kept)
    return {"bytes": total, "flops": 0}


# ------------------------------------------------------------------ the formats, in the plain form

def _int4(x):
    """Codes (0 to 15) and scales (e5m2) of x [..., d]; 64 bits, so that ties are ties."""
    g = x.reshape(*x.shape[:-1], -1, 16).double()
    top = g.amax(dim=-1)
    a = torch.maximum(top, -g.amin(dim=-1)).clamp(max=TOP)
    s = (a / 8).float().to(torch.float8_e5m2)
    s = torch.where(top >= a, -s.float(), s.float()).to(torch.float8_e5m2)
    w = s.double()[..., None]
    c = torch.round(g / torch.where(w == 0, 1.0, w)).clamp(-8, 7)
    c = torch.where(w == 0, 0.0, c).to(torch.int32) + 8
    return c.reshape(x.shape), s


def _pack(c):
    return (c[..., 0::2] | c[..., 1::2] << 4).to(torch.uint8)


def _from_int4(codes, scale):
    """Values, in 32 bits (exact), of packed codes [..., d / 2] and scales [..., d / 16]."""
    w = codes.to(torch.int32)
    c = torch.stack((w & 15, w >> 4), dim=-1).reshape(*codes.shape[:-1], -1)
    return (c - 8).float() * scale.float().repeat_interleave(16, dim=-1)


def _blocks(state, side, pages):
    """Values [..., H, bs, d], in 32 bits, of the blocks `pages`."""
    codes, scale = state[side], state[side + "_scale"]
    if state["case"]["fmt"] == "int4":
        return _from_int4(codes[pages], scale.view(torch.uint8)[pages].view(torch.float8_e5m2))
    return codes.view(torch.uint8)[pages].view(codes.dtype).float() * scale[pages][..., None, None]


def _inverse_frequencies(case):
    """Angles in radians per position, 64 bits, and what the rotated channels are multiplied by."""
    rot, base, kind, f, length = (case[k] for k in ("rot", "base", "kind", "factor", "length"))
    i = torch.arange(rot // 2, dtype=torch.float64)
    if kind == "base":
        base = base * f ** (rot / (rot - 2)) if rot > 2 else base
    w = base ** (-2.0 * i / rot)
    if kind == "linear":
        return w / f, 1.0
    if kind == "yarn":
        def turning(n):  # the channel that makes n turns over the original length
            return rot * math.log(length / (n * PI2)) / (2.0 * math.log(base))
        lo, hi = max(math.floor(turning(32.0)), 0), min(math.ceil(turning(1.0)), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        return w * (1.0 - ramp) + w / f * ramp, 0.1 * math.log(f) + 1.0
    if kind == "bands":
        turns = length * w / PI2  # over the original length
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        return w * keep + w / f * (1.0 - keep), 1.0
    return w, 1.0


# ------------------------------------------------------------------ inputs

def _pool(gen, blocks, H, bs, d, fmt, key):
    """Codes and scales of `blocks` blocks as a model leaves them: keys with a few strong channels,
    values whose size varies from block to block."""
    size = torch.exp(0.7 * torch.randn((blocks, H, 1, 1), generator=gen, device=DEV))
    chan = torch.ones((1, H, 1, d), device=DEV)
    if key:
        chan = torch.where(torch.rand((1, H, 1, d), generator=gen, device=DEV) < 0.04, 6.0, 0.8)
        size = torch.ones_like(size)
    if fmt == "int4":
        codes = torch.empty((blocks, H, bs, d // 2), dtype=torch.uint8, device=DEV)
        scale = torch.empty((blocks, H, bs, d // 16), dtype=torch.float8_e5m2, device=DEV)
    else:
        codes = torch.empty((blocks, H, bs, d), dtype=FLOATS[fmt], device=DEV)
        scale = torch.empty((blocks, H), device=DEV)
        largest = torch.finfo(FLOATS[fmt]).max
    part = max(1, (1 << 26) // (H * bs * d))
    for a in range(0, blocks, part):
        z = slice(a, min(blocks, a + part))
        x = torch.randn((z.stop - a, H, bs, d), generator=gen, device=DEV) * chan * size[z]
        if fmt == "int4":
            c, s = _int4(x.bfloat16())
            codes[z], scale[z] = _pack(c), s
            continue
        s = torch.exp2(torch.ceil(torch.log2(x.abs().amax(dim=(2, 3)) / largest)))
        codes[z] = (x / s[:, :, None, None]).clamp(-largest, largest).to(FLOATS[fmt])
        scale[z] = s
    return codes, scale


def prepare(case, seed):
    B, H, G, d, bs, fmt, op = (case[k] for k in ("B", "H", "G", "d", "bs", "fmt", "op"))
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rng = random.Random(seed)
    pairs = _sizes(case)
    rng.shuffle(pairs)
    n = [a for a, _ in pairs]
    lens = [a + p for a, p in pairs]
    T, Hq = sum(n), H * G
    cu = [0]
    for a in n:
        cu.append(cu[-1] + a)
    i32 = dict(dtype=torch.int32, device=DEV)
    s = {"case": dict(case), "lens": torch.tensor(lens, **i32), "cu": torch.tensor(cu, **i32),
         "total": T, "max_n": max(n), "max_len": max(lens)}
    # the projections' output: one tensor of queries, keys and values, or one for each
    if op != "evict":
        if case["fused"]:
            x = torch.randn((T, Hq + 2 * H, d), generator=gen, device=DEV).bfloat16()
            q, kn, vn = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
        else:
            q, kn, vn = (torch.randn((T, h, d), generator=gen, device=DEV).bfloat16()
                         for h in (Hq, H, H))
    if op == "rope":
        seq, pos = _tokens(s)
        s["q"], s["k"] = q, kn
        s["positions"] = (pos + case["far"]).to(torch.int32)
        s["w"], s["magnitude"] = _inverse_frequencies(case)
        s["w"] = s["w"].to(DEV)
        if own:
            from online_softmax_08_gb300 import fattn
            s["rope"] = fattn.rope_table(case["rot"], case["base"], case["kind"], case["factor"],
                                         case["length"], device=DEV)
        return s
    after = [min(x, case["keep"]) for x in lens] if op == "evict" else []
    need = [(x + bs - 1) // bs for x in lens]
    need_after = [(x + bs - 1) // bs for x in after]
    blocks = sum(need) + sum(need_after) + 3
    order = list(range(blocks))
    rng.shuffle(order)

    def table_of(need):
        t = torch.zeros((B, max(need)), dtype=torch.int32)
        for b in range(B):
            t[b, :need[b]] = torch.tensor([order.pop() for _ in range(need[b])], dtype=torch.int32)
        return t.to(DEV)

    s["table"] = table_of(need)
    s["k"], s["k_scale"] = _pool(gen, blocks, H, bs, d, fmt, True)
    s["v"], s["v_scale"] = _pool(gen, blocks, H, bs, d, fmt, False)
    if op == "write":  # tokens of different size
        kn.mul_(torch.exp(0.5 * torch.randn((T, 1, 1), generator=gen, device=DEV)).bfloat16())
        vn.mul_(torch.exp(0.7 * torch.randn((T, 1, 1), generator=gen, device=DEV)).bfloat16())
        s["kn"], s["vn"] = kn, vn
    if op in ("forward", "weights"):
        s["q"] = q
    if op in ("weights", "evict"):
        # what the steps before left: few keys have most of the weight, many next to none
        w = torch.exp(2.0 * torch.randn((B, H, s["max_len"]), generator=gen, device=DEV) - 4.0)
        s["weights"] = torch.where(w < 0.01, 0.0, w)
        s["weights_out"] = torch.zeros((B, H, s["max_len"] if op == "weights" else max(after)),
                                       device=DEV)
    if op == "weights":
        s["lse"] = _forward(s, values=False)["lse"]
    if op == "evict":
        s["table_out"] = table_of(need_after)
        cu = [0]
        for a in after:
            cu.append(cu[-1] + a)
        s["cu_after"], s["total_after"] = torch.tensor(cu, **i32), cu[-1]
        s["max_after"] = max(after)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    c = state["case"]
    if own:
        from online_softmax_08_gb300 import fattn
        if c["op"] == "rope":
            turn = fattn.rope_backward if c["back"] else fattn.rope
            q, k = turn(state["q"], state["k"], state["positions"], state["rope"], c["layout"])
            return {"q": q, "k": k}
        cache = fattn.KVCache(state["k"], state["v"], state["k_scale"], state["v_scale"])
        batch = fattn.CacheBatch(state["table"], state["lens"], state["cu"], state["total"],
                                 state["max_n"])
        if c["op"] == "write":
            fattn.cache_append(state["kn"], state["vn"], cache, batch)
            k, v = fattn.cache_read(cache, batch)
            return {"k": k, "v": v}
        if c["op"] == "forward":
            o, lse = fattn.cache_forward(state["q"], cache, batch, c["d"] ** -0.5, c["causal"])
            return {"o": o, "lse": lse}
        if c["op"] == "weights":
            w = fattn.cache_weights(state["q"], state["lse"], cache, batch, c["d"] ** -0.5,
                                    c["causal"], state["weights"], out=state["weights_out"])
            return {"weights": w}
        lens, kept, w = fattn.cache_evict(cache, state["weights"], state["table"], state["lens"],
                                          state["table_out"], c["keep"], c["recent"],
                                          out=state["weights_out"])
        out = {"lens": lens, "kept": kept, "weights": w}
        if c["fmt"] != "int4":
            return dict(out, **{n: state[n] for n in ("k", "v", "k_scale", "v_scale")})
        out["k"], out["v"] = fattn.cache_read(cache, fattn.CacheBatch(
            state["table_out"], lens, state["cu_after"], state["total_after"], state["max_after"]))
        return out
    return {"write": _write, "forward": _forward, "rope": _rope, "weights": _weights,
            "evict": _evict}[c["op"]](state)


def _tokens(state):
    """Of every packed token: its sequence, and its position in it."""
    n = state["cu"].diff()
    seq = torch.repeat_interleave(torch.arange(n.numel(), device=DEV), n, output_size=state["total"])
    i = torch.arange(state["total"], device=DEV) - state["cu"][seq]
    return seq, i + (state["lens"] - n)[seq]


def _write(state):
    bs = state["case"]["bs"]
    seq, pos = _tokens(state)
    blk, row = state["table"][seq, pos // bs].long(), pos % bs
    out = {}
    for side in ("k", "v"):
        c, s = _int4(state[side + "n"])
        scale = state[side + "_scale"].view(torch.uint8)
        state[side][blk, :, row] = _pack(c)
        scale[blk, :, row] = s.view(torch.uint8)
        out[side] = _from_int4(state[side][blk, :, row],
                               scale[blk, :, row].view(torch.float8_e5m2)).bfloat16()
    return out


def _whole(state, side):  # [B, H, L, d]
    x = _blocks(state, side, state["table"].long()).transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[4])[:, :, :state["max_len"]]


def _scores(state):
    """Scores [B, H, G, N, L] of the padded queries, those of unseen keys -inf."""
    c = state["case"]
    H, G, d = c["H"], c["G"], c["d"]
    B, N, L = state["table"].shape[0], state["max_n"], state["max_len"]
    seq, pos = _tokens(state)
    i = torch.arange(state["total"], device=DEV) - state["cu"][seq]
    q = torch.zeros((B, N, H * G, d), device=DEV)
    q[seq, i] = state["q"].float()
    q = q.reshape(B, N, H, G, d).permute(0, 2, 3, 1, 4).reshape(B, H, G * N, d)
    s = torch.matmul(q, _whole(state, "k").transpose(2, 3)) * d ** -0.5
    at = torch.arange(L, device=DEV)
    seen = (at[None, :] < state["lens"][:, None])[:, None, :].expand(B, N, L)
    n = state["cu"].diff()
    seen = seen & (torch.arange(N, device=DEV)[None, :] < n[:, None])[:, :, None]
    if c["causal"]:
        where = (state["lens"] - n)[:, None] + torch.arange(N, device=DEV)
        seen = seen & (at <= where[:, :, None])
    return s.reshape(B, H, G, N, L).masked_fill_(~seen[:, None, None], -math.inf), seq, i


def _forward(state, values=True):
    c = state["case"]
    H, G, d = c["H"], c["G"], c["d"]
    B, N, L = state["table"].shape[0], state["max_n"], state["max_len"]
    s, seq, i = _scores(state)
    m = s.amax(dim=-1, keepdim=True)
    p = s.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    total = p.sum(dim=-1, keepdim=True)
    lse = (m + total.log())[..., 0]
    lse = lse.permute(0, 3, 1, 2).reshape(B, N, H * G)[seq, i].t().contiguous()
    if not values:
        return {"lse": lse}
    o = torch.matmul(p.reshape(B, H, G * N, L), _whole(state, "v"))
    o = o.reshape(B, H, G, N, d) / torch.where(total > 0, total, 1.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, N, H * G, d)[seq, i].bfloat16()
    return {"o": o, "lse": lse}


def _rope(state):
    c = state["case"]
    rot, half = c["rot"], c["rot"] // 2
    angle = state["positions"].double()[:, None] * state["w"]  # far positions need 64 bits
    cos = (torch.cos(angle) * state["magnitude"]).float()[:, None]
    sin = (torch.sin(angle) * state["magnitude"]).float()[:, None]
    if c["back"]:
        sin = -sin

    def turn(x):
        y = x.float()
        if c["layout"] == "half":
            a, b = y[..., :half], y[..., half:rot]
            r = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
        else:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            r = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
        return torch.cat((r, y[..., rot:]), dim=-1).bfloat16()

    return {"q": turn(state["q"]), "k": turn(state["k"])}


def _weights(state):
    c = state["case"]
    H, G = c["H"], c["G"]
    B, N, L = state["table"].shape[0], state["max_n"], state["max_len"]
    s, seq, i = _scores(state)
    lse = torch.zeros((B, N, H * G), device=DEV)
    lse[seq, i] = state["lse"].t()
    lse = lse.reshape(B, N, H, G).permute(0, 2, 3, 1)[..., None]
    new = s.sub_(lse).exp_().sum(dim=(2, 3))  # [B, H, L]
    at = torch.arange(L, device=DEV)
    before = (state["lens"] - state["cu"].diff())[:, None]
    total = torch.where((at < before)[:, None], state["weights"] + new, new)
    out = state["weights_out"]
    inside = (at < state["lens"][:, None])[:, None].expand(B, H, L)
    out.copy_(torch.where(inside, total, out))
    return {"weights": out}


def _evict(state):
    c = state["case"]
    keep, recent, bs, H = c["keep"], c["recent"], c["bs"], c["H"]
    B, L = state["table"].shape[0], state["max_len"]
    lens = state["lens"].long()
    at = torch.arange(L, device=DEV)
    # the last ones come first, then the rest by weight, ties by position, what is no token last
    w = state["weights"].clone()
    w.masked_fill_((at >= lens[:, None])[:, None], -math.inf)
    w.masked_fill_(((at >= lens[:, None] - recent) & (at < lens[:, None]))[:, None], math.inf)
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :keep]
    new = torch.clamp(lens, max=keep)
    M = state["max_after"]
    j = torch.arange(order.shape[-1], device=DEV)
    order = torch.where(j < new[:, None, None], order, L).sort(dim=-1).values  # ascending positions
    inside = j < new[:, None, None]
    kept = torch.full((B, H, keep), -1, dtype=torch.int32, device=DEV)
    kept[..., :order.shape[-1]] = torch.where(inside, order, -1)
    order = torch.where(inside, order, 0)[..., :M]
    inside = inside[..., :M].expand(B, H, M)
    moved = state["weights"].gather(2, order)
    out = state["weights_out"]
    out.copy_(torch.where(inside, moved, out))
    result = {"lens": new.to(torch.int32), "kept": kept, "weights": out}
    b, h, to = torch.nonzero(inside, as_tuple=True)
    src = order[inside]
    from_blk, from_row = state["table"][b, src // bs].long(), src % bs
    to_blk, to_row = state["table_out"][b, to // bs].long(), to % bs
    for side in ("k", "v"):
        raw, scale = state[side].view(torch.uint8), state[side + "_scale"]
        if c["fmt"] == "int4":
            s8 = scale.view(torch.uint8)
            raw[to_blk, h, to_row] = raw[from_blk, h, from_row]
            s8[to_blk, h, to_row] = s8[from_blk, h, from_row]
            continue
        old = scale[from_blk, h]
        new_scale = torch.zeros_like(scale).view(-1)
        new_scale = new_scale.scatter_reduce_(0, to_blk * H + h, old, "amax").view_as(scale)
        scale.copy_(torch.where(new_scale > 0, new_scale, scale))
        dt = FLOATS[c["fmt"]]
        part = 1 << 21
        for a in range(0, b.numel(), part):
            z = slice(a, a + part)
            x = raw[from_blk[z], h[z], from_row[z]].view(dt).float()
            x = x * (old[z] / scale[to_blk[z], h[z]])[:, None]
            raw[to_blk[z], h[z], to_row[z]] = x.to(dt).view(torch.uint8)
    if c["fmt"] != "int4":
        return dict(result, **{n: state[n] for n in ("k", "v", "k_scale", "v_scale")})
    n = state["cu_after"].diff()
    seq = torch.repeat_interleave(torch.arange(B, device=DEV), n, output_size=state["total_after"])
    pos = torch.arange(state["total_after"], device=DEV) - state["cu_after"][seq]
    blk, row = state["table_out"][seq, pos // bs].long(), pos % bs
    for side in ("k", "v"):
        s8 = state[side + "_scale"].view(torch.uint8)[blk, :, row].view(torch.float8_e5m2)
        result[side] = _from_int4(state[side][blk, :, row], s8).bfloat16()
    return result


# ------------------------------------------------------------------ the definition in 64 bits

def _decode(codes, scale, fmt):
    """[n, H, bs, d] in 64 bits of whole blocks."""
    if fmt != "int4":
        return codes.double() * scale.double()[:, :, None, None]
    lo, hi = codes.long() % 16, codes.long() // 16
    both = torch.empty((*codes.shape[:-1], 2 * codes.shape[-1]), dtype=torch.float64, device=DEV)
    both[..., 0::2], both[..., 1::2] = lo.double() - 8, hi.double() - 8
    g = both.unflatten(-1, (-1, 16)) * scale.double()[..., None]
    return g.flatten(-2)


def _near_e5m2(x):
    """Positive x to the nearest value of 3 significant bits (ties to even, steps of 2^-16 at least)."""
    _, e = torch.frexp(x)
    step = ((torch.clamp(e - 3, min=-16).long() + 1023) << 52).view(torch.float64)  # 2^that
    return torch.round(x / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    H, G, d, bs, fmt, op = (case[k] for k in ("H", "G", "d", "bs", "fmt", "op"))
    if work(case)["flops"] > 4e12:
        return None
    lens, cu = s["lens"].tolist(), s["cu"].tolist()
    if op == "rope":
        w, rot = s["w"], case["rot"]
        z = torch.polar(torch.full_like(w, s["magnitude"]).expand(s["total"], -1).contiguous(),
                        s["positions"].double()[:, None] * w * (-1.0 if case["back"] else 1.0))[:, None]
        out = {}
        for name in ("q", "k"):
            y = s[name].double()
            if case["layout"] == "half":
                r = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * z
                y[..., :rot // 2], y[..., rot // 2:rot] = r.real, r.imag
            else:
                r = torch.view_as_complex(y[..., :rot].reshape(*y.shape[:2], rot // 2, 2)) * z
                y[..., :rot] = torch.view_as_real(r).flatten(-2)
            out[name] = y
        return out
    if op == "write":
        out = {}
        for name in ("k", "v"):
            x = s[name + "n"].double().unflatten(-1, (-1, 16)).clamp(-TOP, TOP)
            a, where = x.abs().max(dim=-1, keepdim=True)
            first = (x == a).any(dim=-1, keepdim=True)
            step = _near_e5m2(a / 8) * torch.where(first, -1.0, 1.0)
            c = torch.where(step == 0, 0.0, torch.round(x / step)).clamp(-8, 7)
            out[name] = torch.where(step == 0, 0.0, c * step).flatten(-2)
        return out
    table = s["table"].tolist()

    def tokens(side, b, length):  # [H, length, d]
        rows = torch.tensor(table[b][:(length + bs - 1) // bs], dtype=torch.long, device=DEV)
        c, z = s[side], s[side + "_scale"]
        c = c.view(torch.uint8)[rows].view(c.dtype)
        z = z.view(torch.uint8)[rows].view(z.dtype) if fmt == "int4" else z[rows]
        return _decode(c, z, fmt).transpose(0, 1).reshape(H, -1, d)[:, :length]

    if op in ("forward", "weights"):
        o = torch.empty((s["total"], H * G, d), dtype=torch.float64, device=DEV)
        lse = torch.empty((H * G, s["total"]), dtype=torch.float64, device=DEV)
        if op == "weights":
            weights = s["weights_out"].double()
        for b, length in enumerate(lens):
            n = cu[b + 1] - cu[b]
            k = tokens("k", b, length)
            v = tokens("v", b, length) if op == "forward" else None
            hide = torch.arange(length, device=DEV)[None, :] > \
                torch.arange(length - n, length, device=DEV)[:, None]
            if op == "weights":
                weights[b, :, :length - n] = s["weights"][b, :, :length - n].double()
            for h in range(H * G):
                t = s["q"][cu[b]:cu[b + 1], h].double() @ k[h // G].t() / math.sqrt(d)
                if case["causal"]:
                    t = t.masked_fill(hide, -math.inf)
                if op == "weights":
                    weights[b, h // G, :length] += torch.exp(
                        t - s["lse"][h, cu[b]:cu[b + 1], None].double()).sum(dim=0)
                    continue
                l = torch.logsumexp(t, dim=1)
                lse[h, cu[b]:cu[b + 1]] = l
                o[cu[b]:cu[b + 1], h] = torch.exp(t - l[:, None]) @ v[h // G]
        return {"weights": weights} if op == "weights" else {"o": o, "lse": lse}

    # evict, a sequence and head at a time; in 8 bits a block's scale is its tokens' largest
    keep, recent = case["keep"], case["recent"]
    new = [min(x, keep) for x in lens]
    kept = torch.full((len(lens), H, keep), -1, dtype=torch.int32, device=DEV)
    moved = s["weights_out"].double()
    k_out, v_out = [], []
    for b, length in enumerate(lens):
        m = new[b]
        old = length if length <= keep else length - recent  # those that compete
        for h in range(H):
            w = s["weights"][b, h, :old]
            place = torch.argsort(-w.double(), stable=True)[:m - (length - old)]
            rest = torch.arange(old, length, device=DEV)
            kept[b, h, :m] = torch.cat((torch.sort(place).values, rest)).int()
            moved[b, h, :m] = s["weights"][b, h, kept[b, h, :m].long()].double()
        if fmt == "int4":
            at = kept[b, :, :m].long()[..., None].expand(H, m, d)
            k_out.append(tokens("k", b, length).gather(1, at).transpose(0, 1))
            v_out.append(tokens("v", b, length).gather(1, at).transpose(0, 1))
    out = {"lens": torch.tensor(new, dtype=torch.int32, device=DEV), "kept": kept, "weights": moved}
    if fmt == "int4":
        return dict(out, k=torch.cat(k_out), v=torch.cat(v_out))
    for side in ("k", "v"):
        codes, scale = s[side].clone(), s[side + "_scale"].double()
        for b, m in enumerate(new):
            at = kept[b, :, :m].long()
            from_blk = s["table"][b].long()[at // bs]
            heads = torch.arange(H, device=DEV)[:, None]
            was = s[side + "_scale"][from_blk, heads].double()
            x = s[side].view(torch.uint8)[from_blk, heads, at % bs].view(codes.dtype)
            for j in range(0, m, bs):
                blk = int(s["table_out"][b, j // bs])
                z = slice(j, min(m, j + bs))
                scale[blk] = was[:, z].amax(dim=1)
                y = x[:, z].double() * (was[:, z] / scale[blk][:, None])[..., None]
                codes.view(torch.uint8)[blk, :, :z.stop - j] = \
                    y.float().to(codes.dtype).view(torch.uint8)  # (exact in 32 bits)
        # (in 32 bits: a pool's codes, each of which is one of the format's values)
        out[side], out[side + "_scale"] = codes.float(), scale
    return out
