"""CPU oracle of the attention-side operators (numpy, float64 or wider):
rotary positions, head norms with the rotation, and scored attention with its
gradients.  Test infrastructure only; written from the formulas, head by head
and pair by pair, with nothing of the library in it."""

from __future__ import annotations

import math

import numpy as np


# ------------------------------------------------------------------- rotary
def rope_frequencies(r, base, scaling="none", factor=1.0, original_len=0.0, low=1.0, high=4.0):
    """Angle per position of each of the r/2 pairs (long double)."""
    ld = np.longdouble
    base, factor = ld(base), ld(factor)
    if scaling == "base" and r > 2:
        base = base * factor ** (ld(r) / ld(r - 2))
    out = []
    for i in range(r // 2):
        w = base ** (ld(-2 * i) / ld(r))
        if scaling == "linear":
            w = w / factor
        elif scaling == "bands":
            turns = ld(original_len) * w / (2 * ld(np.pi))
            if turns <= low:
                w = w / factor
            elif turns < high:
                s = (turns - ld(low)) / (ld(high) - ld(low))
                w = w * s + w / factor * (1 - s)
        elif scaling == "ramp":
            def index(n):
                return r * math.log(original_len / (2 * math.pi * n)) / (2 * math.log(float(base)))
            first, last = max(math.floor(index(high)), 0), min(math.ceil(index(low)), r - 1)
            span = last - first if last > first else 0.001
            g = min(1.0, max(0.0, (i - first) / span))
            w = w * ld(1 - g) + w / factor * ld(g)
        out.append(w)
    return np.array(out, dtype=np.longdouble)


def rope_rotate(x, positions, freqs, layout="half", amplitude=1.0, inverse=False):
    """x [T, heads, D] -> each head's pairs turned by position * freq."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    two_pi = 2 * np.longdouble("3.14159265358979323846264338327950288")
    n = len(freqs)
    for i in range(n):
        a, b = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
        f = np.mod(np.asarray(positions).astype(np.longdouble) * freqs[i], two_pi)
        c, s = np.cos(f).astype(np.float64), np.sin(f).astype(np.float64)
        if inverse:
            s = -s
        c, s = amplitude * c[:, None], amplitude * s[:, None]
        y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
    return y


def head_norm(x, w, eps):
    """x [T, heads, D]: x / rms(x) * w over the last dimension."""
    x = np.asarray(x, np.float64)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 if w is None else w)


def head_norm_backward(x, w, g, eps):
    """(dx, dw) of head_norm for the upstream gradient g."""
    x, g = np.asarray(x, np.float64), np.asarray(g, np.float64)
    rms = np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xhat = x / rms
    dw = (g * xhat).sum((0, 1))
    gw = g * (1.0 if w is None else w)
    return (gw - xhat * (gw * xhat).mean(-1, keepdims=True)) / rms, dw
