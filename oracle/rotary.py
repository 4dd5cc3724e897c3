"""Float64 oracle of rotary positions.

Test infrastructure: only ``tests/``, ``__graft_entry__.smoke()`` and
``bench.py`` may import this module. It shares no code with the CUDA library.

Pair k of a head's first ``rot`` dimensions turns by position * rate[k]; pairs are
(2k, 2k+1) (interleaved) or (k, k + rot/2) (half); later dimensions pass through.
"""
from __future__ import annotations

import math

import numpy as np

from .temporal_conv import _f64


def rotary_rates(rot: int, base: float = 10000.0, scaling=None) -> np.ndarray:
    kind = scaling[0] if scaling else None
    out = []
    for k in range(rot // 2):
        b = base
        if kind == "base" and rot > 2:
            b = base * scaling[1] ** (rot / (rot - 2))
        f = b ** (-2.0 * k / rot)
        if kind == "linear":
            f /= scaling[1]
        elif kind == "parts":
            _, factor, length, slow, fast = scaling
            w = min(1.0, max(0.0, (length * f / (2 * math.pi) - slow) / (fast - slow)))
            f = f * w + f / factor * (1 - w)
        out.append(f)
    return np.array(out)


def rotary(X, positions, rot: int, layout: str = "half", base: float = 10000.0, scaling=None,
           mscale: float = 1.0, inverse: bool = False) -> np.ndarray:
    """X [B, N, H, D]; positions [N] or [B, N]."""
    x = _f64(X)
    y = x.copy()
    t = np.asarray(positions, dtype=np.float64)[..., None] * rotary_rates(rot, base, scaling)
    if t.ndim == 2:
        t = t[None]
    c, s = np.cos(t)[:, :, None] * mscale, np.sin(t)[:, :, None] * mscale * (-1 if inverse else 1)
    k = np.arange(rot // 2)
    i, j = (2 * k, 2 * k + 1) if layout == "interleaved" else (k, k + rot // 2)
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., i] * s + x[..., j] * c
    return y
