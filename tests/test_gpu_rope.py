"""Rotary positions against the fp64 oracle.

Bar, for a pair (a, b), magnitude m and position p: the angle is a 32-bit fraction of a turn
(2 pi 2^-33), rounded to fp32 (at most pi 2^-25), the sine and cosine are off by 2^-23 each
(two units of the last place below 1), their product with m and the two products and the sum by
2^-24 each: below 2^-21 (|a| + |b|) m in all; the oracle's own angle is off by 2 pi 2^-52 |p|; the
result is rounded to bf16, half a step being 2^-8 of it (or of what it should be, plus the rest).
"""
import numpy as np
import pytest
import torch

from online_softmax_08_gb300 import fattn
from oracle import rope as orope
from test_gpu_cache import DEV, _bf16, _strided

pytestmark = pytest.mark.gpu


def _check(got, x, pos, w, m, layout, backward):
    x = x.double().cpu().numpy()
    ref = orope.turn(x, pos, w, m, layout, backward)
    n = len(w)
    size = np.zeros_like(ref)
    if layout == "half":
        size[..., :n] = size[..., n:2 * n] = np.abs(x[..., :n]) + np.abs(x[..., n:2 * n])
    else:
        size[..., 0:2 * n:2] = size[..., 1:2 * n:2] = np.abs(x[..., 0:2 * n:2]) + np.abs(x[..., 1:2 * n:2])
    angle = 2 * np.pi * 2.0 ** -52 * np.abs(np.asarray(pos, dtype=np.float64))[:, None, None]
    inner = m * size * (2.0 ** -21 + angle)
    bar = inner + 2.0 ** -8 * (np.abs(ref) + inner)
    bar[..., 2 * n:] = 0.0  # copied
    err = np.abs(got.double().cpu().numpy() - ref)
    assert np.all(err <= bar), (err / np.maximum(bar, 1e-30)).max()


CASES = [
    # (T, Hq, Hk, d, rot, kind)
    (1, 1, 1, 64, 16, "none"), (1, 32, 8, 128, 128, "yarn"), (3, 5, 0, 64, 64, "linear"),
    (5, 0, 7, 128, 112, "base"), (67, 8, 2, 128, 64, "bands"), (130, 3, 3, 64, 48, "yarn"),
    (1000, 16, 1, 128, 16, "none"), (4099, 9, 2, 64, 32, "bands"), (7, 130, 9, 128, 96, "none"),
]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("strides", ["own", "slice", "heads"])
@pytest.mark.parametrize("T,Hq,Hk,d,rot,kind", CASES)
def test_matches_oracle(T, Hq, Hk, d, rot, kind, strides, layout):
    rng = np.random.default_rng(T + Hq)
    q, k = _bf16(rng, (T, Hq, d), 2.0), _bf16(rng, (T, Hk, d))
    pos = rng.integers(-1000, 200000, T)
    pos[0], pos[-1] = 2 ** 31 - 1, -2 ** 31
    args = (rot, 1e4, kind, 1.0 if kind == "none" else 8.0, 4096)
    table = fattn.rope_table(*args, device=DEV)
    w, m = orope.frequencies(*args)
    dpos = torch.tensor(pos, dtype=torch.int32, device=DEV)
    for call, backward in ((fattn.rope, False), (fattn.rope_backward, True)):
        base = torch.full((T, Hq + Hk + 3, d), 7.0, dtype=torch.bfloat16, device=DEV)
        gq, gk = call(_strided(q, strides), _strided(k, strides) if Hk else None, dpos, table, layout,
                      out=(base[:, 1:1 + Hq], base[:, 2 + Hq:2 + Hq + Hk]))
        _check(gq, q, pos, w, m, layout, backward)
        if Hk:
            _check(gk, k, pos, w, m, layout, backward)
        base[:, 1:1 + Hq] = 7.0
        base[:, 2 + Hq:2 + Hq + Hk] = 7.0
        assert bool((base == 7.0).all())


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_in_place_and_own_outputs(layout):
    rng = np.random.default_rng(2)
    T, d = 33, 128
    x = _bf16(rng, (T, 12, d)).to(DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    table = fattn.rope_table(64, device=DEV)
    q, k = fattn.rope(x[:, :8], x[:, 8:10], pos, table, layout)
    y = x.clone()
    fattn.rope(y[:, :8], y[:, 8:10], pos, table, layout, out=(y[:, :8], y[:, 8:10]))
    assert torch.equal(y[:, :8], q) and torch.equal(y[:, 8:10], k) and torch.equal(y[:, 10:], x[:, 10:])
    q2, none = fattn.rope(x[:, :8], None, pos, table, layout)
    assert none is None and torch.equal(q2, q)
    back, _ = fattn.rope_backward(q, None, pos, table, layout)  # magnitude 1: the inverse
    assert float((back.float() - x[:, :8].float()).abs().max()) <= 2.0 ** -6 * float(x.abs().max())


def test_gradient_by_differences():
    """sum(dy rope(x)) changes along x by what rope_backward gives: the map is linear, so a
    difference of two calls is exact but for the roundings to bf16 (2^-8 each)."""
    rng = np.random.default_rng(3)
    T, H, d = 9, 2, 64
    table = fattn.rope_table(32, 1e4, "yarn", 4.0, 2048, device=DEV)
    pos = torch.tensor(rng.integers(0, 5000, T), dtype=torch.int32, device=DEV)
    dy, e = _bf16(rng, (T, H, d)).to(DEV), _bf16(rng, (T, H, d)).to(DEV)
    for layout in ("half", "interleaved"):
        g, _ = fattn.rope_backward(dy, None, pos, table, layout)
        plus, _ = fattn.rope(e, None, pos, table, layout)
        minus, _ = fattn.rope(-e, None, pos, table, layout)
        change = (dy.double() * (plus.double() - minus.double())).sum() / 2
        size = (dy.double().abs() * plus.double().abs()).sum() + (g.double().abs() * e.double().abs()).sum()
        assert float((change - (g.double() * e.double()).sum()).abs()) <= 2.0 ** -8 * float(size)


def test_captured_and_empty_and_refused():
    T, d = 4, 128
    table = fattn.rope_table(128, device=DEV)
    x = torch.randn((T, 6, d), device=DEV).bfloat16()
    pos = torch.zeros(T, dtype=torch.int32, device=DEV)
    out = (torch.zeros((T, 4, d), dtype=torch.bfloat16, device=DEV),
           torch.zeros((T, 2, d), dtype=torch.bfloat16, device=DEV))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fattn.rope(x[:, :4], x[:, 4:], pos, table, out=out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            fattn.rope(x[:, :4], x[:, 4:], pos, table, out=out)
    torch.cuda.synchronize()
    for p in (3, 70000):
        pos.fill_(p)
        graph.replay()
        q, k = fattn.rope(x[:, :4], x[:, 4:], pos, table, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out[0], q) and torch.equal(out[1], k)
    q, k = fattn.rope(x[:0, :4], x[:0, 4:], pos[:0], table)
    assert q.shape == (0, 4, d) and k.shape == (0, 2, d)
    for bad in (pos.long(), pos[:2], pos.cpu(), torch.stack((pos, pos), 1)[:, 0]):
        with pytest.raises(ValueError):
            fattn.rope(x[:, :4], x[:, 4:], bad, table)
    with pytest.raises(ValueError):
        fattn.rope(x.float(), None, pos, table)
    with pytest.raises(fattn.FattnError):
        fattn.rope(x, None, pos, fattn.rope_table(24, device=DEV))


@pytest.mark.parametrize("layout,rot", [("half", 64), ("interleaved", 32)])
def test_training_run(layout, rot):
    """Queries and keys of the dense layout turned (by strides), attention and its backward pass,
    and the gradients turned back, against 64-bit differentiation of the whole.  The bars are the
    attention's own: 2e-2 for the result and the gradients (values of size 1)."""
    H, N, d = 2, 150, 64
    rng = np.random.default_rng(11)
    q, k, v, do = (_bf16(rng, (1, H, N, d)).to(DEV) for _ in range(4))
    pos = torch.arange(N, dtype=torch.int32, device=DEV)
    table = fattn.rope_table(rot, device=DEV)
    rows = lambda x: x[0].transpose(0, 1)  # [N, H, d] over the dense tensor
    qr, kr, dq, dk = (torch.empty_like(q) for _ in range(4))
    fattn.rope(rows(q), rows(k), pos, table, layout, out=(rows(qr), rows(kr)))
    o, lse = fattn.forward(qr, kr, v, d ** -0.5, True)
    dqr, dkr, dv = fattn.backward(qr, kr, v, o, lse, do, d ** -0.5, True)
    fattn.rope_backward(rows(dqr), rows(dkr), pos, table, layout, out=(rows(dq), rows(dk)))

    w, _ = orope.frequencies(rot)
    angle = pos.double()[:, None] * torch.tensor(w, device=DEV)
    cos, sin = torch.cos(angle), torch.sin(angle)

    def turn(x):
        a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if layout == "half" else \
            (x[..., 0:rot:2], x[..., 1:rot:2])
        y = (a * cos - b * sin, a * sin + b * cos)
        y = torch.cat(y, -1) if layout == "half" else torch.stack(y, -1).flatten(-2)
        return torch.cat((y, x[..., rot:]), -1)

    q64, k64, v64 = (x.double().requires_grad_() for x in (q, k, v))
    s = turn(q64) @ turn(k64).transpose(2, 3) * d ** -0.5
    s = s.masked_fill(torch.ones((N, N), dtype=torch.bool, device=DEV).triu(1), -np.inf)
    ref = torch.softmax(s, dim=-1) @ v64
    ref.backward(do.double())
    for got, want in ((o, ref), (dq, q64.grad), (dk, k64.grad), (dv, v64.grad)):
        assert float((got.double() - want.detach()).abs().max()) <= 2e-2 * max(1.0, float(want.detach().abs().max()))
