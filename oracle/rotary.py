"""Rotary positions in float64. Test infrastructure: only tests and the smoke check use it.

The first R dimensions of a row turn by its position: pair (a, b) = (i, i + R/2), or
(2i, 2i + 1), by the angle p f_i. A bf16 row's values are rounded to float32 and from
there to bf16, as include/pkv.h states.
"""

from __future__ import annotations

import math

import numpy as np


def frequencies(dim, base, kind="plain", stretch=1.0, original_context=0.0, low_turns=0.0, high_turns=0.0):
    """Angles per position, from the statements of include/pkv.h, one number at a time."""
    found = []
    if kind == "base":
        base = base * stretch ** (dim / (dim - 2))
    for i in range(dim // 2):
        f = math.exp(-2 * i / dim * math.log(base))
        if kind == "linear":
            f = f / stretch
        elif kind == "turns":
            n = original_context * f / (2 * math.pi)
            if n <= low_turns:
                f = f / stretch
            elif n < high_turns:
                part = (n - low_turns) / (high_turns - low_turns)
                f = part * f + (1 - part) * f / stretch
        elif kind == "ramp":
            def at(turns):
                return dim / 2 * math.log(original_context / (2 * math.pi * turns)) / math.log(base)
            first, last = max(math.floor(at(high_turns)), 0), min(math.ceil(at(low_turns)), dim - 1)
            part = min(max((i - first) / max(last - first, 1e-3), 0), 1)
            f = (1 - part) * f + part * f / stretch
        found.append(f)
    return np.array(found)


def table(freq, positions, factor=1.0):
    """float64 [positions][2 * len(freq)]: factor * cosines, then sines."""
    angle = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(freq, dtype=np.float64)
    return factor * np.concatenate([np.cos(angle), np.sin(angle)], 1)


def turn(x, rows, interleaved):
    """x [tokens][heads][d] float64 turned by table rows [tokens][R]."""
    x, rows = np.asarray(x, dtype=np.float64), np.asarray(rows, dtype=np.float64)
    half = rows.shape[1] // 2
    y = x.copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = rows[:, None, i], rows[:, None, half + i]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y
