"""Rotary positions in numpy, fp64: the frequencies, their scalings and the turn of pairs of
channels.  TEST INFRASTRUCTURE ONLY; shares no code with the library."""
import math

import numpy as np


def frequencies(rot, base=10000.0, kind="none", factor=1.0, length=0, fast=None, slow=None):
    """w_i in radians per position, and the magnitude."""
    i = np.arange(rot // 2)
    if kind == "base" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    w = np.array([base ** (-2.0 * k / rot) for k in i])
    if kind in ("none", "base"):
        return w, 1.0
    if kind == "linear":
        return w / factor, 1.0
    turns = length * w / (2 * math.pi)
    if kind == "bands":
        fast, slow = (4.0 if fast is None else fast), (1.0 if slow is None else slow)
        share = np.clip((turns - slow) / (fast - slow), 0, 1)
        return share * w + (1 - share) * w / factor, 1.0
    fast, slow = (32.0 if fast is None else fast), (1.0 if slow is None else slow)
    # the (fractional) pair whose frequency makes n turns: length base^(-2 i / rot) = 2 pi n
    pair = lambda n: rot / 2 * math.log(length / (2 * math.pi * n), base)
    lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rot - 1)
    share = 1 - np.clip((i - lo) / max(hi - lo, 0.001), 0, 1)
    return share * w + (1 - share) * w / factor, 1 + 0.1 * math.log(factor)


def turn(x, positions, w, magnitude=1.0, layout="half", backward=False):
    """x [T, heads, d] with its first 2 len(w) channels turned."""
    n = len(w)
    angle = np.asarray(positions, dtype=np.float64)[:, None] * w
    z = magnitude * np.exp(1j * (-angle if backward else angle))[:, None]
    out = np.array(x, dtype=np.float64)
    if layout == "half":
        y = (x[..., :n] + 1j * x[..., n:2 * n]) * z
        out[..., :n], out[..., n:2 * n] = y.real, y.imag
    else:
        y = (x[..., 0:2 * n:2] + 1j * x[..., 1:2 * n:2]) * z
        out[..., 0:2 * n:2], out[..., 1:2 * n:2] = y.real, y.imag
    return out
