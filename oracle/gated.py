"""Float64 oracle of gated linear attention, token by token.

Test infrastructure: only ``tests/``, ``__graft_entry__.smoke()`` and
``bench.py`` may import this module. It shares no code with the CUDA library.

    S_n = exp(g_n) S_{n-1} + k_n^T v_n,   o_n = scale q_n S_n

Q, K, V [B, N, H, D], G [B, N, H] log gates (-inf: nothing passes), S [B, H, D, D].
"""
from __future__ import annotations

from typing import Optional, Tuple

import numpy as np

from .temporal_conv import _f64


def _decays(G) -> np.ndarray:
    with np.errstate(over="ignore"):
        return np.exp(_f64(G))


def gated_attention(Q, K, V, G, S_in=None, scale: float = 1.0) -> Tuple[np.ndarray, np.ndarray]:
    """O and the last state."""
    q, k, v, a = _f64(Q), _f64(K), _f64(V), _decays(G)
    B, N, H, D = q.shape
    S = np.zeros((B, H, D, D)) if S_in is None else _f64(S_in).copy()
    O = np.empty_like(q)
    for n in range(N):
        S = a[:, n, :, None, None] * S + k[:, n, :, :, None] * v[:, n, :, None, :]
        O[:, n] = scale * np.einsum("bhd,bhde->bhe", q[:, n], S)
    return O, S


def gated_bruteforce(Q, K, V, G, S_in=None, scale: float = 1.0) -> np.ndarray:
    """O as the masked quadratic form: each weight is the product of the gates between
    the two tokens, multiplied out one by one."""
    q, k, v, a = _f64(Q), _f64(K), _f64(V), _decays(G)
    B, N, H, D = q.shape
    O = np.zeros_like(q)
    for b in range(B):
        for h in range(H):
            for i in range(N):
                w = 1.0
                for j in range(i, -1, -1):
                    O[b, i, h] += scale * w * (q[b, i, h] @ k[b, j, h]) * v[b, j, h]
                    w *= a[b, j, h]
                if S_in is not None:
                    O[b, i, h] += scale * w * (q[b, i, h] @ _f64(S_in)[b, h])
    return O


def gated_attention_backward(Q, K, V, G, dO, S_in=None, dS_out=None, scale: float = 1.0):
    """dQ, dK, dV, dG, dS_in: the adjoint recurrence."""
    q, k, v, a, do = _f64(Q), _f64(K), _f64(V), _decays(G), scale * _f64(dO)
    B, N, H, D = q.shape
    past = np.empty((N + 1, B, H, D, D))
    past[0] = 0.0 if S_in is None else _f64(S_in)
    for n in range(N):
        past[n + 1] = a[:, n, :, None, None] * past[n] + k[:, n, :, :, None] * v[:, n, :, None, :]
    dQ, dK, dV, dG = np.empty_like(q), np.empty_like(q), np.empty_like(q), np.empty_like(a)
    U = np.zeros((B, H, D, D)) if dS_out is None else _f64(dS_out).copy()
    for n in range(N - 1, -1, -1):
        U = U + q[:, n, :, :, None] * do[:, n, :, None, :]
        dQ[:, n] = np.einsum("bhde,bhe->bhd", past[n + 1], do[:, n])
        dK[:, n] = np.einsum("bhde,bhe->bhd", U, v[:, n])
        dV[:, n] = np.einsum("bhde,bhd->bhe", U, k[:, n])
        U = a[:, n, :, None, None] * U
        dG[:, n] = (U * past[n]).sum((-1, -2))
    return dQ, dK, dV, dG, U


def gated_magnitudes(Q, K, V, G, dO=None, S_in=None, dS_out=None, scale: float = 1.0,
                     window: int = 256):
    """Sums of the absolute values of all terms: (O, S) or, with dO, (dQ, dK, dV, dG, dS_in).
    dG's counts what a sum over up to ``window`` later tokens of q . dq - k . dk adds up."""
    p = [np.abs(_f64(x)) for x in (Q, K, V)]
    S: Optional[np.ndarray] = None if S_in is None else np.abs(_f64(S_in))
    if dO is None:
        return gated_attention(*p, G, S, abs(scale))
    dS = None if dS_out is None else np.abs(_f64(dS_out))
    dQ, dK, dV, dG, dS0 = gated_attention_backward(*p, G, np.abs(_f64(dO)), S, dS, abs(scale))
    rows = (p[0] * dQ).sum(-1) + (p[1] * dK).sum(-1)                       # [B, N, H]
    total = np.concatenate([np.zeros_like(rows[:, :1]), rows.cumsum(1)], 1)
    N = rows.shape[1]
    end = np.minimum(np.arange(N) + window, N)
    # the anchor at the window's end is a gate's gradient itself; past the last token it is
    # <dS_out, S_N>, no larger than its terms
    last = 0.0
    if dS is not None:
        SN = gated_attention(*p, G, S, 1.0)[1]
        last = (dS * SN).sum((-1, -2))[:, None]
    at_end = dG.max(1, keepdims=True)
    return dQ, dK, dV, dG + (total[:, end] - total[:, :N]) + at_end + last, dS0


def gated_window_errors(dG, ref, window: int = 256) -> np.ndarray:
    """Relative 2-norm error of dG [B, N, H] in every head's windows of ``window`` tokens,
    [B, windows, H]. A last window shorter than 32 tokens counts with the one before."""
    got, ref = _f64(dG), _f64(ref)
    N = ref.shape[1]
    starts = list(range(0, N, window))
    if len(starts) > 1 and N - starts[-1] < 32:
        starts.pop()
    sums = [np.add.reduceat(x * x, starts, axis=1) for x in (got - ref, ref)]
    return np.sqrt(sums[0] / np.maximum(sums[1], 1e-300))
