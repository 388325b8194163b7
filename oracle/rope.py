"""Rotary positions in fp64, and their fp32 step-by-step form.

A pair (a, b) of a row at position n, pair index i, turns by the angle
n f_i, f_i = base^(-2 i / rot): (a c - b s, b c + a s).  Pairs are elements
(i, i + rot / 2), or (2 i, 2 i + 1) when interleaved; elements from ``rot``
on pass through.  Stretching for longer contexts changes only f_i (and, by
parts, the magnitude of c and s).
"""
from __future__ import annotations

import math

import numpy as np


def frequencies(rot, base=10000.0, scaling="none", factor=1.0, original_max=0, slow_turns=1.0, fast_turns=32.0):
    """f_i in fp64, [rot / 2]."""
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = np.float64(base) ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / factor
    if scaling == "by_parts":
        turns = original_max * f / (2.0 * math.pi)
        g = np.clip((turns - slow_turns) / (fast_turns - slow_turns), 0.0, 1.0)
        return (1.0 - g) * f / factor + g * f
    return f


def table(max_positions, rot, magnitude=None, **kw):
    """cos, sin [max_positions, rot / 2] in fp64."""
    f = frequencies(rot, **kw)
    if magnitude is None:
        magnitude = 0.1 * math.log(kw.get("factor", 1.0)) + 1.0 if kw.get("scaling") == "by_parts" else 1.0
    angle = np.arange(max_positions, dtype=np.float64)[:, None] * f
    return magnitude * np.cos(angle), magnitude * np.sin(angle)


def rotate(x, cos, sin, rot, interleaved):
    """Rows x [t, heads, d] turned by cos, sin [t, rot / 2], in x's precision, one operation at a time."""
    x = np.asarray(x)
    c, s = cos[:, None, :].astype(x.dtype), sin[:, None, :].astype(x.dtype)
    y = x.copy()
    first = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    second = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    a, b = x[..., first], x[..., second]
    y[..., first] = a * c - b * s
    y[..., second] = b * c + a * s
    return y
