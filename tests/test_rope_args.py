"""Rotary positions without a GPU: the frequency table, the oracle's own properties, and argument
checks that come before any device call."""
import ctypes

import numpy as np
import pytest
import torch

from online_softmax_08_gb300 import build as fbuild
from online_softmax_08_gb300 import fattn
from oracle import rope as orope

A = 1 << 20  # 256-byte aligned, never dereferenced
INVALID, UNSUPPORTED, CUDA = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    fbuild.build()
    return fattn.load()


TABLES = [(128, 1e4, "none", 1.0, 0), (64, 5e5, "linear", 4.0, 0), (48, 1e4, "base", 8.0, 0),
          (128, 1e4, "yarn", 16.0, 4096), (32, 1e6, "yarn", 40.0, 2048), (16, 100.0, "yarn", 1.0, 7),
          (128, 5e5, "bands", 8.0, 8192), (2, 1e4, "base", 3.0, 0), (64, 1e4, "bands", 2.0, 64)]


@pytest.mark.parametrize("rot,base,kind,factor,length", TABLES)
def test_table_holds_the_frequencies(lib, rot, base, kind, factor, length):
    table = fattn.rope_table(rot, base, kind, factor, length, device="cpu")
    w, m = orope.frequencies(rot, base, kind, factor, length)
    got = table.turns.numpy().view(np.uint64).astype(np.float64) * 2.0 ** -64
    # a few roundings of 2^-53 of the value, and the one to 2^-64
    np.testing.assert_allclose(got, w / (2 * np.pi), rtol=2.0 ** -48, atol=2.0 ** -62)
    assert abs(table.magnitude - m) <= 2.0 ** -23 * m


def test_oracle_turns():
    rng = np.random.default_rng(1)
    w, _ = orope.frequencies(16)
    x, dy = rng.standard_normal((2, 5, 3, 64))
    pos = np.array([0, 1, 2, 1000, -7])
    for layout in ("half", "interleaved"):
        y = orope.turn(x, pos, w, 1.5, layout)
        np.testing.assert_array_equal(y[0, :, 16:], x[0, :, 16:])
        np.testing.assert_allclose(y[0, :, :16], 1.5 * x[0, :, :16])
        # scores depend on the distance alone
        a = orope.turn(x, pos, w, 1.0, layout)
        b = orope.turn(x, pos + 11, w, 1.0, layout)
        np.testing.assert_allclose(a[:1] * 0 + np.einsum("thc,uhc->htu", a, a).sum(),
                                   np.einsum("thc,uhc->htu", b, b).sum() + a[:1] * 0)
        # the gradient, by differences of sum(dy * turn(x))
        g = orope.turn(dy, pos, w, 1.5, layout, backward=True)
        for at in ((0, 0, 0), (3, 1, 5), (4, 2, 15), (1, 0, 40)):
            e = np.zeros_like(x)
            e[at] = 1e-3
            d = (orope.turn(x + e, pos, w, 1.5, layout) - orope.turn(x - e, pos, w, 1.5, layout)) / 2e-3
            assert abs((dy * d).sum() - g[at]) <= 1e-9


def _rope(lib, q=A, qst=512, qsh=128, qo=2 * A, qost=512, qosh=128, Hq=4, k=A, kst=256, ksh=128,
          ko=3 * A, kost=256, kosh=128, Hk=2, pos=A, turns=A, m=1.0, T=5, d=128, rot=64, layout=0):
    return lib.fattn_rope(q, qst, qsh, qo, qost, qosh, Hq, k, kst, ksh, ko, kost, kosh, Hk, pos, turns,
                          m, T, d, rot, layout, 0, None)


def test_bad_arguments(lib):
    for kw in (dict(q=None), dict(qo=A + 8), dict(k=A + 2), dict(ko=None), dict(pos=None),
               dict(pos=A + 2), dict(turns=None), dict(turns=A + 4), dict(m=0.0),
               dict(m=float("nan")), dict(m=float("inf")), dict(T=-1), dict(Hq=0, Hk=0), dict(Hq=-1),
               dict(Hk=70000), dict(T=1 << 30), dict(rot=0), dict(rot=8), dict(rot=144),
               dict(qst=516), dict(ksh=4), dict(qst=-512), dict(qost=128), dict(kosh=64),
               dict(q=A, qo=A, qost=1024), dict(k=A, ko=A, kosh=256, kost=512)):
        assert _rope(lib, **kw) == INVALID, kw
    for kw in (dict(d=96), dict(rot=24), dict(rot=20), dict(layout=2)):
        assert _rope(lib, **kw) == UNSUPPORTED, kw
    assert _rope(lib, T=0) == 0
    assert _rope(lib, T=0, q=None) == 0
    if not torch.cuda.is_available():  # accepted: the calls go on to the device
        for kw in (dict(), dict(qo=A), dict(Hk=0, k=None, ko=None), dict(Hq=0, q=None, qo=None),
                   dict(qst=0, qsh=0)):
            assert _rope(lib, **kw) == CUDA, kw


def test_bad_tables(lib):
    buf, m = (ctypes.c_uint64 * 64)(), ctypes.c_float()
    call = lambda rot=64, base=1e4, kind=3, factor=4.0, length=4096, fast=32.0, slow=1.0, t=buf: \
        lib.fattn_rope_turns(t, ctypes.byref(m), rot, base, kind, factor, length, fast, slow)
    assert call() == 0
    for kw in (dict(t=None), dict(rot=0), dict(rot=3), dict(base=1.0), dict(base=float("inf")),
               dict(base=float("nan")), dict(factor=0.0), dict(factor=float("nan")), dict(length=0),
               dict(slow=0.0), dict(fast=1.0), dict(factor=0.5), dict(kind=2, factor=1e-300)):
        assert call(**kw) == INVALID, kw
    for kind in (-1, 5):
        assert call(kind=kind) == UNSUPPORTED
    with pytest.raises(ValueError):
        fattn.rope_table(64, kind="other", device="cpu")
    with pytest.raises(fattn.FattnError):
        fattn.rope_table(63, device="cpu")
    table = fattn.rope_table(64, device="cpu")
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fattn.rope(x, x, torch.zeros(3, dtype=torch.int32), table)  # (on no CUDA device)
    with pytest.raises(ValueError):
        fattn.rope(x, x, torch.zeros(3, dtype=torch.int32), table, layout="quarter")


def test_most_rows(lib):
    one = dict(k=None, ko=None, Hk=0, Hq=1, qst=0, qsh=0, d=64)
    for T in ((1 << 31) - 1, (1 << 31) - 3):
        assert _rope(lib, T=T, **one) == INVALID, T
    if not torch.cuda.is_available():  # accepted
        assert _rope(lib, T=(1 << 31) - 4, **one) == CUDA


def test_frequencies_that_overflow(lib):
    """A factor whose inverse is no finite number: the first pair's frequency would be none."""
    buf, m = (ctypes.c_uint64 * 32)(*([7] * 32)), ctypes.c_float(-1.0)
    for kind in (1, 4):
        assert lib.fattn_rope_turns(buf, ctypes.byref(m), 64, 1e4, kind, 1e-310, 64, 4.0, 1.0) == INVALID
        assert list(buf) == [7] * 32 and m.value == -1.0
    assert lib.fattn_rope_turns(buf, ctypes.byref(m), 64, 1e4, 1, 1e-300, 64, 4.0, 1.0) == 0
