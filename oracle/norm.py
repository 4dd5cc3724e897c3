"""Float64 oracle of the gated residual with the norms before and after a block.

Test infrastructure: only ``tests/``, ``__graft_entry__.smoke()`` and
``bench.py`` may import this module. It shares no code with the CUDA library.

    u = f, or RMSNorm(f) w_post
    h = x + alpha gate_b u
    y = n w_pre (1 + mod_scale_b) + mod_shift_b,  n the RMS or layer norm of h

x, f [B, N, C]; gate, mod_* [B, C]; w_* [C].
"""
from __future__ import annotations

import numpy as np

from .temporal_conv import _f64


def _get(t, fill, wide):
    if t is None:
        return np.float64(fill)
    return _f64(t)[:, None] if wide else _f64(t)


def gate_residual_norm(x, f=None, gate=None, w_post=None, w_pre=None, mod_scale=None, mod_shift=None,
                       norm="layer", eps=1e-6, alpha=1.0):
    h = _f64(x)
    if f is not None:
        u = _f64(f)
        if w_post is not None:
            u = u / np.sqrt((u * u).mean(-1, keepdims=True) + eps) * _f64(w_post)
        h = h + alpha * _get(gate, 1.0, True) * u
    a = h - h.mean(-1, keepdims=True) if norm == "layer" else h
    n = a / np.sqrt((a * a).mean(-1, keepdims=True) + eps)
    y = n * _get(w_pre, 1.0, False) * (1 + _get(mod_scale, 0.0, True)) + _get(mod_shift, 0.0, True)
    return h, y


def gate_residual_norm_backward(x, f, dy, dh, gate=None, w_post=None, w_pre=None, mod_scale=None,
                                norm="layer", eps=1e-6, alpha=1.0):
    """dict of the gradients of every parameter (given or not), dx and df."""
    hx = _f64(x)
    C = hx.shape[-1]
    u = un = np.zeros_like(hx) if f is None else _f64(f)
    rf = 1.0
    if w_post is not None:
        rf = 1 / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
        un = u * rf
        u = un * _f64(w_post)
    hx = hx + alpha * _get(gate, 1.0, True) * u
    a = hx - hx.mean(-1, keepdims=True) if norm == "layer" else hx
    rh = 1 / np.sqrt((a * a).mean(-1, keepdims=True) + eps)
    n = a * rh
    gy = np.zeros_like(hx) if dy is None else _f64(dy)
    g = np.zeros_like(hx) if dh is None else _f64(dh)
    wi, ms = _get(w_pre, 1.0, False), 1 + _get(mod_scale, 0.0, True)
    t = gy * wi * ms
    back = t - n * (t * n).mean(-1, keepdims=True)
    if norm == "layer":
        back = back - t.mean(-1, keepdims=True)
    g = g + rh * back
    du = alpha * _get(gate, 1.0, True) * g
    df = du
    if w_post is not None:
        t2 = du * _f64(w_post)
        df = rf * (t2 - un * (t2 * un).mean(-1, keepdims=True))
    assert un.shape[-1] == C
    return {"x": g, "f": df, "gate": alpha * (u * g).sum(1), "w_post": (du * un).sum((0, 1)),
            "w_pre": (gy * ms * n).sum((0, 1)), "mod_scale": (gy * n * wi).sum(1), "mod_shift": gy.sum(1)}
