"""ReLU linear attention on B200 (sm_100a): a thin ctypes binding of ``libla_b200.so``.

The functions below carry the names of the C ABI in ``include/la.h`` and only
marshal arguments (tensor pointers, sizes, the stream) into it; every step of
the computation runs in the library's CUDA kernels. There is no CPU path:
importing this package fails if the library has not been built
(``python linear_attention_diffusion_b200/build.py``).
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libla_b200.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python linear_attention_diffusion_b200/build.py`"
        " (this package has no CPU fallback)")

_lib = ctypes.CDLL(LIB_PATH)

LA_OK = 0
LA_ERR_INVALID_ARG = 1
LA_ERR_UNSUPPORTED = 2
LA_ERR_WORKSPACE = 3
LA_ERR_CUDA = 4
LA_IO_BF16 = 0
LA_IO_F32 = 1
HEAD_DIM = 32


class LaShape(ctypes.Structure):
    """Mirror of ``la_shape`` in include/la.h."""

    _fields_ = [
        ("B", ctypes.c_int), ("N", ctypes.c_int), ("H", ctypes.c_int), ("D", ctypes.c_int),
        ("io_dtype", ctypes.c_int), ("rope", ctypes.c_int),
        ("T", ctypes.c_int), ("Hh", ctypes.c_int), ("W", ctypes.c_int),
        ("t_offset", ctypes.c_int), ("rope_base", ctypes.c_double), ("eps", ctypes.c_float),
    ]


class LaConvShape(ctypes.Structure):
    """Mirror of ``la_conv_shape`` in include/la.h."""

    _fields_ = [
        ("B", ctypes.c_int), ("T", ctypes.c_int), ("Hh", ctypes.c_int), ("W", ctypes.c_int),
        ("C", ctypes.c_int), ("io_dtype", ctypes.c_int),
    ]


class LaGatedShape(ctypes.Structure):
    """Mirror of ``la_gated_shape`` in include/la.h."""

    _fields_ = [
        ("B", ctypes.c_int), ("N", ctypes.c_int), ("H", ctypes.c_int), ("D", ctypes.c_int),
        ("io_dtype", ctypes.c_int), ("scale", ctypes.c_float),
    ]


class LaRotaryShape(ctypes.Structure):
    """Mirror of ``la_rotary_shape`` in include/la.h."""

    _fields_ = [(n, ctypes.c_int) for n in (
        "B", "N", "H", "Hk", "D", "rot", "io_dtype", "half", "scaling", "inverse", "pos_rows",
        "pos_offset")] + [(n, ctypes.c_double) for n in (
            "base", "factor", "original_length", "slow", "fast", "mscale")]


class LaNormShape(ctypes.Structure):
    """Mirror of ``la_norm_shape`` in include/la.h."""

    _fields_ = [
        ("B", ctypes.c_int), ("N", ctypes.c_int), ("C", ctypes.c_int), ("io_dtype", ctypes.c_int),
        ("norm", ctypes.c_int), ("eps", ctypes.c_float), ("alpha", ctypes.c_float),
    ]


class LaError(RuntimeError):
    def __init__(self, status: int, func: str):
        self.status = status
        detail = la_last_error()
        super().__init__(f"{func}: {la_status_string(status)}" + (f" -- {detail}" if detail else ""))


_vp = ctypes.c_void_p
_sz = ctypes.c_size_t
_i = ctypes.c_int
_shape_p = ctypes.POINTER(LaShape)

_lib.la_workspace_bytes.argtypes = [_shape_p]
_lib.la_workspace_bytes.restype = _sz
_lib.la_causal_workspace_bytes.argtypes = [_shape_p]
_lib.la_causal_workspace_bytes.restype = _sz
_lib.la_state_reduce.argtypes = [_shape_p, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.la_state_reduce.restype = _i
_lib.la_state_reduce_static.argtypes = [_shape_p, _vp, _vp, _vp, _vp, _vp]
_lib.la_state_reduce_static.restype = _i
_lib.la_apply.argtypes = [_shape_p, _vp, _vp, _vp, _vp, _vp]
_lib.la_apply.restype = _i
_lib.la_attention.argtypes = [_shape_p, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.la_attention.restype = _i
_lib.la_block_causal_step.argtypes = [_shape_p, _vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _sz, _vp]
_lib.la_block_causal_step.restype = _i
_lib.la_attention_backward.argtypes = [_shape_p] + [_vp] * 11 + [_vp, _sz, _vp]
_lib.la_attention_backward.restype = _i
_lib.la_causal_attention.argtypes = [_shape_p, _vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _sz, _vp]
_lib.la_causal_attention.restype = _i
_lib.la_temporal_conv.argtypes = [ctypes.POINTER(LaConvShape), _vp, _vp, _vp, _vp, _vp, _vp, _vp]
_lib.la_temporal_conv.restype = _i
_lib.la_qkv_workspace_bytes.argtypes = [_shape_p, _i]
_lib.la_qkv_workspace_bytes.restype = _sz
_lib.la_qkv_state.argtypes = [_shape_p, _i] + [_vp] * 7 + [_sz, _vp]
_lib.la_qkv_state.restype = _i
_gated_p = ctypes.POINTER(LaGatedShape)
_lib.la_gated_workspace_bytes.argtypes = [_gated_p, _i]
_lib.la_gated_workspace_bytes.restype = _sz
_lib.la_gated_launches.argtypes = [_gated_p, _i]
_lib.la_gated_launches.restype = _i
_lib.la_gated_attention.argtypes = [_gated_p] + [_vp] * 8 + [_sz, _vp]
_lib.la_gated_attention.restype = _i
_lib.la_gated_attention_backward.argtypes = [_gated_p] + [_vp] * 13 + [_sz, _vp]
_lib.la_gated_attention_backward.restype = _i
_lib.la_rotary.argtypes = [ctypes.POINTER(LaRotaryShape)] + [_vp] * 6
_lib.la_rotary.restype = _i
_norm_p = ctypes.POINTER(LaNormShape)
_lib.la_gate_residual_norm.argtypes = [_norm_p] + [_vp] * 10
_lib.la_gate_residual_norm.restype = _i
_lib.la_norm_workspace_bytes.argtypes = [_norm_p]
_lib.la_norm_workspace_bytes.restype = _sz
_lib.la_gate_residual_norm_backward.argtypes = [_norm_p] + [_vp] * 16 + [_sz, _vp]
_lib.la_gate_residual_norm_backward.restype = _i
_lib.la_state_reset.argtypes = [_vp, _vp, _i, _i, _i, _vp]
_lib.la_state_reset.restype = _i
_lib.la_status_string.argtypes = [_i]
_lib.la_status_string.restype = ctypes.c_char_p
_lib.la_last_error.argtypes = []
_lib.la_last_error.restype = ctypes.c_char_p
_lib.la_attention_launches.argtypes = [_shape_p]
_lib.la_attention_launches.restype = _i
_lib.la_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint), _i]
_lib.la_wait_selftest.argtypes = [ctypes.c_uint, _vp]
_lib.la_wait_selftest.restype = _i
_lib.la_device_error.restype = _i


def make_shape(B: int, N: int, H: int, D: int = HEAD_DIM, io_dtype: str = "bf16",
               rope: bool = False, T: int = 0, Hh: int = 0, W: int = 0,
               t_offset: int = 0, rope_base: float = 10000.0, eps: float = 1e-6) -> LaShape:
    io = {"bf16": LA_IO_BF16, "f32": LA_IO_F32, "float32": LA_IO_F32}[io_dtype]
    return LaShape(int(B), int(N), int(H), int(D), io, int(bool(rope)), int(T), int(Hh),
                   int(W), int(t_offset), float(rope_base), float(eps))


def _ptr(x) -> Optional[int]:
    """Device address of a tensor (or an int address); None for NULL."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if not x.is_cuda:
        raise ValueError("tensor arguments must live on a CUDA device")
    if not x.is_contiguous():
        raise ValueError("tensor arguments must be contiguous")
    return x.data_ptr()


def _nbytes(x) -> int:
    return 0 if x is None else x.numel() * x.element_size()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, func: str) -> None:
    if status != LA_OK:
        raise LaError(status, func)


def la_workspace_bytes(shape: LaShape) -> int:
    return int(_lib.la_workspace_bytes(ctypes.byref(shape)))


def la_causal_workspace_bytes(shape: LaShape) -> int:
    return int(_lib.la_causal_workspace_bytes(ctypes.byref(shape)))


def la_state_reduce(shape: LaShape, K, V, S, z, ws, stream=None) -> None:
    _check(_lib.la_state_reduce(ctypes.byref(shape), _ptr(K), _ptr(V), _ptr(S), _ptr(z),
                                _ptr(ws), _nbytes(ws), _stream(stream)), "la_state_reduce")


def la_state_reduce_static(shape: LaShape, K, V, S, z, stream=None) -> None:
    """la_state_reduce without a workspace: the scratch is the library's own
    fixed device array (for callers that cannot allocate; see include/la.h)."""
    _check(_lib.la_state_reduce_static(ctypes.byref(shape), _ptr(K), _ptr(V), _ptr(S), _ptr(z),
                                       _stream(stream)), "la_state_reduce_static")


def la_apply(shape: LaShape, Q, S, z, O, stream=None) -> None:
    _check(_lib.la_apply(ctypes.byref(shape), _ptr(Q), _ptr(S), _ptr(z), _ptr(O),
                         _stream(stream)), "la_apply")


def la_attention(shape: LaShape, Q, K, V, S, z, O, ws, stream=None) -> None:
    _check(_lib.la_attention(ctypes.byref(shape), _ptr(Q), _ptr(K), _ptr(V), _ptr(S), _ptr(z),
                             _ptr(O), _ptr(ws), _nbytes(ws), _stream(stream)), "la_attention")


def la_block_causal_step(shape: LaShape, Q, K, V, S_carry, z_carry, O, update: int, ws,
                         stream=None) -> None:
    _check(_lib.la_block_causal_step(ctypes.byref(shape), _ptr(Q), _ptr(K), _ptr(V),
                                     _ptr(S_carry), _ptr(z_carry), _ptr(O), int(update),
                                     _ptr(ws), _nbytes(ws), _stream(stream)),
           "la_block_causal_step")


def la_attention_backward(shape: LaShape, Q, K, V, S, z, dO, dQ, dK, dV, dS, dz, ws,
                          stream=None) -> None:
    """Gradients of la_attention; S and z None makes the call reduce the state again."""
    _check(_lib.la_attention_backward(ctypes.byref(shape), _ptr(Q), _ptr(K), _ptr(V), _ptr(S),
                                      _ptr(z), _ptr(dO), _ptr(dQ), _ptr(dK), _ptr(dV), _ptr(dS),
                                      _ptr(dz), _ptr(ws), _nbytes(ws), _stream(stream)),
           "la_attention_backward")


def la_causal_attention(shape: LaShape, Q, K, V, S_carry, z_carry, O, update: int, ws,
                        stream=None) -> None:
    """Token-causal attention; the carry (S_carry, z_carry) may be None when update = 0."""
    _check(_lib.la_causal_attention(ctypes.byref(shape), _ptr(Q), _ptr(K), _ptr(V),
                                    _ptr(S_carry), _ptr(z_carry), _ptr(O), int(update),
                                    _ptr(ws), _nbytes(ws), _stream(stream)),
           "la_causal_attention")


def make_conv_shape(B: int, T: int, Hh: int, W: int, C: int, io_dtype: str = "bf16") -> LaConvShape:
    return LaConvShape(int(B), int(T), int(Hh), int(W), int(C),
                       LA_IO_BF16 if io_dtype == "bf16" else LA_IO_F32)


def la_temporal_conv(shape: LaConvShape, x, w, bias, f_in, f_out, y, stream=None) -> None:
    """Temporal depth-wise conv with shortcut and conv cache (see include/la.h)."""
    _check(_lib.la_temporal_conv(ctypes.byref(shape), _ptr(x), _ptr(w), _ptr(bias), _ptr(f_in),
                                 _ptr(f_out), _ptr(y), _stream(stream)), "la_temporal_conv")


def la_qkv_workspace_bytes(shape: LaShape, C: int) -> int:
    return int(_lib.la_qkv_workspace_bytes(ctypes.byref(shape), int(C)))


def la_qkv_state(shape: LaShape, C: int, X, W, bias, Q, S, z, ws, stream=None) -> None:
    """QKV projection fused with the state reduce (see include/la.h)."""
    _check(_lib.la_qkv_state(ctypes.byref(shape), int(C), _ptr(X), _ptr(W), _ptr(bias), _ptr(Q),
                             _ptr(S), _ptr(z), _ptr(ws), _nbytes(ws), _stream(stream)),
           "la_qkv_state")


def _unfit(*sizes: int) -> ValueError:
    """For numbers that a C int would cut to their low 32 bits. Found by the callers with an or of
    all of them and one shift, which leaves 0, or -1 where one is negative, if all fit."""
    return ValueError(f"{sizes}: a size or place past 32 bits")


def make_gated_shape(B: int, N: int, H: int, D: int = HEAD_DIM, io_dtype: str = "bf16",
                     scale: float = 1.0) -> LaGatedShape:
    io = {"bf16": LA_IO_BF16, "f32": LA_IO_F32, "float32": LA_IO_F32}[io_dtype]
    if (B | N | H | D) >> 31 not in (0, -1):
        raise _unfit(B, N, H, D)
    return LaGatedShape(int(B), int(N), int(H), int(D), io, float(scale))


def la_gated_workspace_bytes(shape: LaGatedShape, backward: bool = False) -> int:
    return int(_lib.la_gated_workspace_bytes(ctypes.byref(shape), int(bool(backward))))


def la_gated_launches(shape: LaGatedShape, backward: bool = False) -> int:
    """Kernel launches of a call; 0 without tokens or for an invalid shape."""
    return int(_lib.la_gated_launches(ctypes.byref(shape), int(bool(backward))))


def la_gated_attention(shape: LaGatedShape, Q, K, V, G, S_in, S_out, O, ws, stream=None) -> None:
    """Gated linear attention; S_in, S_out may be None, S_out may be S_in (see include/la.h)."""
    _check(_lib.la_gated_attention(ctypes.byref(shape), _ptr(Q), _ptr(K), _ptr(V), _ptr(G),
                                   _ptr(S_in), _ptr(S_out), _ptr(O), _ptr(ws), _nbytes(ws),
                                   _stream(stream)), "la_gated_attention")


def la_gated_attention_backward(shape: LaGatedShape, Q, K, V, G, S_in, dO, dS_out, dQ, dK, dV,
                                dG, dS_in, ws, stream=None) -> None:
    """Gradients of la_gated_attention; S_in, dS_out, dS_in may be None."""
    _check(_lib.la_gated_attention_backward(ctypes.byref(shape), _ptr(Q), _ptr(K), _ptr(V),
                                            _ptr(G), _ptr(S_in), _ptr(dO), _ptr(dS_out),
                                            _ptr(dQ), _ptr(dK), _ptr(dV), _ptr(dG), _ptr(dS_in),
                                            _ptr(ws), _nbytes(ws), _stream(stream)),
           "la_gated_attention_backward")


def la_rotary(shape: LaRotaryShape, Q, K, positions, Qo, Ko, stream=None) -> None:
    """Rotary positions of Q and K; K, Ko and positions may be None (see include/la.h)."""
    _check(_lib.la_rotary(ctypes.byref(shape), _ptr(Q), _ptr(K), _ptr(positions), _ptr(Qo), _ptr(Ko),
                          _stream(stream)), "la_rotary")


def make_norm_shape(B: int, N: int, C: int, io_dtype: str = "bf16", norm: str = "layer",
                    eps: float = 1e-6, alpha: float = 1.0) -> LaNormShape:
    io = {"bf16": LA_IO_BF16, "f32": LA_IO_F32, "float32": LA_IO_F32}[io_dtype]
    if (B | N | C) >> 31 not in (0, -1):
        raise _unfit(B, N, C)
    return LaNormShape(int(B), int(N), int(C), io, {"rms": 0, "layer": 1}[norm], float(eps),
                       float(alpha))


def la_gate_residual_norm(shape: LaNormShape, x, f, gate, w_post, w_pre, mod_scale, mod_shift, h, y,
                          stream=None) -> None:
    """Gated residual and norm; all but x may be None (see include/la.h)."""
    _check(_lib.la_gate_residual_norm(ctypes.byref(shape), _ptr(x), _ptr(f), _ptr(gate), _ptr(w_post),
                                      _ptr(w_pre), _ptr(mod_scale), _ptr(mod_shift), _ptr(h), _ptr(y),
                                      _stream(stream)), "la_gate_residual_norm")


def la_norm_workspace_bytes(shape: LaNormShape) -> int:
    return int(_lib.la_norm_workspace_bytes(ctypes.byref(shape)))


def la_gate_residual_norm_backward(shape: LaNormShape, x, f, gate, w_post, w_pre, mod_scale, dh, dy,
                                   dx, df, dgate, dw_post, dw_pre, dmod_scale, dmod_shift, ws,
                                   stream=None) -> None:
    """Gradients of la_gate_residual_norm (see include/la.h for what may be None)."""
    _check(_lib.la_gate_residual_norm_backward(
        ctypes.byref(shape), _ptr(x), _ptr(f), _ptr(gate), _ptr(w_post), _ptr(w_pre),
        _ptr(mod_scale), _ptr(dh), _ptr(dy), _ptr(dx), _ptr(df), _ptr(dgate), _ptr(dw_post),
        _ptr(dw_pre), _ptr(dmod_scale), _ptr(dmod_shift), _ptr(ws), _nbytes(ws), _stream(stream)),
        "la_gate_residual_norm_backward")


def la_state_reset(S, z, B: int, H: int, D: int = HEAD_DIM, stream=None) -> None:
    _check(_lib.la_state_reset(_ptr(S), _ptr(z), int(B), int(H), int(D), _stream(stream)),
           "la_state_reset")


def la_attention_launches(shape: LaShape) -> int:
    """Kernel launches of la_attention / la_block_causal_step (update 0, 1)."""
    return int(_lib.la_attention_launches(ctypes.byref(shape)))


def la_status_string(status: int) -> str:
    return _lib.la_status_string(int(status)).decode()


def la_last_error() -> str:
    return _lib.la_last_error().decode()


def la_wait_selftest(limit_us: int, stream=None) -> None:
    """Launch a warp whose wait nothing satisfies; it gives up after limit_us
    and raises the device error word (see la_device_error)."""
    _check(_lib.la_wait_selftest(int(limit_us), _stream(stream)), "la_wait_selftest")


def la_device_error(reset: bool = False) -> int:
    """The device error word of the current device (0: no kernel gave up a wait)."""
    code = ctypes.c_uint(0)
    _check(_lib.la_device_error(ctypes.byref(code), int(bool(reset))), "la_device_error")
    return int(code.value)


# ---------------------------------------------------------------------------
# Convenience wrappers that allocate outputs with torch (device memory only).

def shape_for(Q, eps: float = 1e-6, rope_grid=None, t_offset: int = 0,
              rope_base: float = 10000.0) -> LaShape:
    """la_shape for a [B, N, H, D] tensor; ``rope_grid`` = (T, Hh, W) turns on RoPE."""
    import torch
    B, N, H, D = Q.shape
    io = "bf16" if Q.dtype == torch.bfloat16 else "f32"
    if rope_grid is None:
        return make_shape(B, N, H, D, io, False, eps=eps)
    T, Hh, W = rope_grid
    return make_shape(B, N, H, D, io, True, T, Hh, W, t_offset, rope_base, eps)


def workspace(shape: LaShape, device="cuda", causal: bool = False):
    """A zero-filled workspace of la_workspace_bytes(shape) bytes
    (la_causal_workspace_bytes(shape) with causal=True)."""
    import torch
    n = la_causal_workspace_bytes(shape) if causal else la_workspace_bytes(shape)
    if n == 0:
        raise LaError(LA_ERR_INVALID_ARG, "la_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def attention(Q, K, V, eps: float = 1e-6, rope_grid=None, t_offset: int = 0,
              rope_base: float = 10000.0, stream=None):
    """O, S, z of non-causal ReLU linear attention for [B, N, H, 32] CUDA tensors."""
    import torch
    shape = shape_for(Q, eps, rope_grid, t_offset, rope_base)
    B, N, H, D = Q.shape
    S = torch.empty((B, H, D, D), dtype=torch.float32, device=Q.device)
    z = torch.empty((B, H, D), dtype=torch.float32, device=Q.device)
    O = torch.empty_like(Q)
    la_attention(shape, Q, K, V, S, z, O, workspace(shape, Q.device), stream)
    return O, S, z


def attention_backward(Q, K, V, dO, S=None, z=None, eps: float = 1e-6, rope_grid=None,
                       t_offset: int = 0, rope_base: float = 10000.0, stream=None):
    """dQ, dK, dV, dS, dz of non-causal ReLU linear attention for [B, N, H, 32] CUDA tensors."""
    import torch
    shape = shape_for(Q, eps, rope_grid, t_offset, rope_base)
    B, N, H, D = Q.shape
    dQ, dK, dV = torch.empty_like(Q), torch.empty_like(K), torch.empty_like(V)
    dS = torch.empty((B, H, D, D), dtype=torch.float32, device=Q.device)
    dz = torch.empty((B, H, D), dtype=torch.float32, device=Q.device)
    la_attention_backward(shape, Q, K, V, S, z, dO, dQ, dK, dV, dS, dz,
                          workspace(shape, Q.device), stream)
    return dQ, dK, dV, dS, dz


def causal_attention(Q, K, V, S_carry=None, z_carry=None, update: int = 0, eps: float = 1e-6,
                     rope_grid=None, t_offset: int = 0, rope_base: float = 10000.0, stream=None):
    """O of token-causal ReLU linear attention for [B, N, H, 32] CUDA tensors."""
    shape = shape_for(Q, eps, rope_grid, t_offset, rope_base)
    import torch
    O = torch.empty_like(Q)
    la_causal_attention(shape, Q, K, V, S_carry, z_carry, O, update,
                        workspace(shape, Q.device, causal=True), stream)
    return O


def temporal_conv(x, w, bias=None, f_in=None, want_cache: bool = False, stream=None):
    """y (and the next conv cache when ``want_cache``) for x [B, T, Hh, W, C] CUDA tensors."""
    import torch
    B, T, Hh, W, C = x.shape
    shape = make_conv_shape(B, T, Hh, W, C, "bf16" if x.dtype == torch.bfloat16 else "f32")
    y = torch.empty_like(x)
    f_out = torch.empty((B, Hh, W, C), dtype=x.dtype, device=x.device) if want_cache else None
    la_temporal_conv(shape, x, w, bias, f_in, f_out, y, stream)
    return (y, f_out) if want_cache else y


def qkv_state(X, W, bias=None, rope_grid=None, t_offset: int = 0, rope_base: float = 10000.0,
              stream=None):
    """Q [B, N, H, 32], S, z of the fused QKV projection + state reduce for
    X [B, N, C] and W [3 H 32, C] bf16 CUDA tensors."""
    import torch
    B, N, C = X.shape
    if W.dim() != 2 or W.shape[1] != C or W.shape[0] % (3 * HEAD_DIM) != 0:
        raise ValueError(f"W must be [3*H*{HEAD_DIM}, C={C}], got {tuple(W.shape)}")
    H = W.shape[0] // (3 * HEAD_DIM)
    if bias is not None and tuple(bias.shape) != (W.shape[0],):
        raise ValueError(f"bias must be [{W.shape[0]}], got {tuple(bias.shape)}")
    if rope_grid is None:
        shape = make_shape(B, N, H, HEAD_DIM, "bf16", False)
    else:
        T, Hh, Wd = rope_grid
        shape = make_shape(B, N, H, HEAD_DIM, "bf16", True, T, Hh, Wd, t_offset, rope_base)
    Q = torch.empty((B, N, H, HEAD_DIM), dtype=torch.bfloat16, device=X.device)
    S = torch.empty((B, H, HEAD_DIM, HEAD_DIM), dtype=torch.float32, device=X.device)
    z = torch.empty((B, H, HEAD_DIM), dtype=torch.float32, device=X.device)
    n = la_qkv_workspace_bytes(shape, C)
    if n == 0:
        raise LaError(LA_ERR_INVALID_ARG, "la_qkv_workspace_bytes")
    ws = torch.empty(n, dtype=torch.uint8, device=X.device)
    la_qkv_state(shape, C, X, W, bias, Q, S, z, ws, stream)
    return Q, S, z


# Gated linear attention, rotary positions, gated residual with norms. These
# wrappers check every tensor, run on the tensors' own device (on its current
# stream unless one is given) and take their workspace from torch's allocator.

_torch = None
_raw_stream = None  # address of a device's current stream without making a Stream object


def _t():
    """torch, imported at the first call that needs it."""
    global _torch, _raw_stream
    if _torch is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _torch = torch
    return _torch


def _io_of(x, name: str) -> int:
    torch = _t()
    if x.dtype is torch.bfloat16:
        return LA_IO_BF16
    if x.dtype is torch.float32:
        return LA_IO_F32
    raise ValueError(f"{name} must be bfloat16 or float32, got {x.dtype}")


def _need(name: str, x, shape, dtype, device: int) -> None:
    """Raise ValueError unless x (None is left to the caller) is a contiguous tensor of this
    shape and type on GPU ``device`` (-1: the CPU)."""
    if x is not None and (x.dtype is not dtype or x.get_device() != device or x.shape != shape
                          or not x.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {tuple(shape)} on GPU {device}, got "
                         f"{x.dtype} {tuple(x.shape)} with strides {x.stride()} on {x.device}")


def _at(x) -> Optional[int]:
    """Address of a tensor that _need has seen."""
    return None if x is None else x.data_ptr()


def _on(stream, x):
    """A context with ``stream`` (a torch stream or an address) as the current one of x's GPU, so
    that outputs and workspaces come from that stream's memory: memory of another stream could
    be handed out again while a kernel here still uses it."""
    torch = _t()
    device = _on_gpu(x)
    if isinstance(stream, int):
        stream = (torch.cuda.ExternalStream(stream, device=device) if stream
                  else torch.cuda.default_stream(device))
    elif stream.device.index != device:
        raise ValueError(f"the stream belongs to {stream.device}, the tensors to GPU {device}")
    return torch.cuda.stream(stream)


def _launch(func, name: str, shape, args, device: int) -> None:
    """Call a C function on the tensors' own GPU and its current stream."""
    cuda = _t().cuda
    stream = cuda.current_stream(device).cuda_stream if _raw_stream is None else _raw_stream(device)
    if device == cuda.current_device():
        status = func(ctypes.byref(shape), *args, stream)
    else:
        with cuda.device(device):
            status = func(ctypes.byref(shape), *args, stream)
    if status != LA_OK:
        raise LaError(status, name)


def _on_gpu(x) -> int:
    if not x.is_cuda:
        raise ValueError("tensor arguments must live on a CUDA device")
    return x.get_device()


def _scratch(nbytes: int, x):
    """A workspace from torch's allocator and its size."""
    torch = _t()
    return torch.empty(nbytes, dtype=torch.uint8, device=x.device), nbytes


def _gated_shape(Q, K, V, G, scale, **states) -> LaGatedShape:
    torch = _t()
    if Q.dim() != 4 or Q.shape[-1] != HEAD_DIM:
        raise ValueError(f"Q must be [B, N, H, {HEAD_DIM}], got {tuple(Q.shape)}")
    io = _io_of(Q, "Q")
    full, device = Q.shape, Q.get_device()
    B, N, H, D = full
    if (B | N | H) >> 31:
        raise _unfit(B, N, H)
    _need("Q", Q, full, Q.dtype, device)
    _need("K", K, full, Q.dtype, device)
    _need("V", V, full, Q.dtype, device)
    _need("G", G, (B, N, H), torch.float32, device)
    for name, x in states.items():
        _need(name, x, (B, H, D, D), torch.float32, device)
    return LaGatedShape(B, N, H, D, io, scale)


def gated_attention(Q, K, V, G, S_in=None, scale: float = 1.0, want_state: bool = False, S_out=None,
                    stream=None):
    """O (and the last state when ``want_state`` or ``S_out`` is given) of gated linear attention:
    S_n = exp(g_n) S_{n-1} + k_n^T v_n, o_n = scale q_n S_n, for [B, N, H, 32] CUDA tensors and
    log gates G [B, N, H] float32. ``S_out`` may be ``S_in``: the state is then updated in place.
    bf16 tensors: the state keeps 24 bits, what only O depends on 17 (see include/la.h)."""
    if stream is not None:
        with _on(stream, Q):
            return gated_attention(Q, K, V, G, S_in, scale, want_state, S_out)
    torch = _t()
    shape = _gated_shape(Q, K, V, G, scale, S_in=S_in, S_out=S_out)
    device = _on_gpu(Q)
    O = torch.empty_like(Q)
    if S_out is None and want_state:
        S_out = G.new_empty((shape.B, shape.H, HEAD_DIM, HEAD_DIM)) if S_in is None else torch.empty_like(S_in)
    n = _lib.la_gated_workspace_bytes(ctypes.byref(shape), 0)
    # 256: what a call that needs none reports
    ws, n = _scratch(n, Q) if n > 256 else (None, 0)
    _launch(_lib.la_gated_attention, "la_gated_attention", shape,
            (Q.data_ptr(), K.data_ptr(), V.data_ptr(), G.data_ptr(), _at(S_in), _at(S_out), O.data_ptr(),
             _at(ws), n), device)
    return O if S_out is None else (O, S_out)


def gated_attention_backward(Q, K, V, G, dO, S_in=None, dS_out=None, scale: float = 1.0,
                             want_state: Optional[bool] = None, stream=None):
    """dQ, dK, dV, dG, dS_in of gated_attention. dS_in is None unless ``want_state`` (by default:
    where an S_in is given); S_in must still hold the state that the forward began with."""
    if stream is not None:
        with _on(stream, Q):
            return gated_attention_backward(Q, K, V, G, dO, S_in, dS_out, scale, want_state)
    torch = _t()
    shape = _gated_shape(Q, K, V, G, scale, S_in=S_in, dS_out=dS_out)
    _need("dO", dO, Q.shape, Q.dtype, Q.get_device())
    device = _on_gpu(Q)
    if want_state is None:
        want_state = S_in is not None
    dQ, dK, dV, dG = (torch.empty_like(x) for x in (Q, K, V, G))
    dS = None
    if want_state:
        dS = torch.empty((shape.B, shape.H, HEAD_DIM, HEAD_DIM), dtype=torch.float32, device=Q.device)
    ws, n = _scratch(_lib.la_gated_workspace_bytes(ctypes.byref(shape), 1), Q)
    _launch(_lib.la_gated_attention_backward, "la_gated_attention_backward", shape,
            (Q.data_ptr(), K.data_ptr(), V.data_ptr(), G.data_ptr(), _at(S_in), dO.data_ptr(), _at(dS_out),
             dQ.data_ptr(), dK.data_ptr(), dV.data_ptr(), dG.data_ptr(), _at(dS), _at(ws), n), device)
    return dQ, dK, dV, dG, dS


_ROTARY_LAYOUTS = {"interleaved": 0, "half": 1}
_ROTARY_SCALINGS = {"linear": 1, "base": 2, "parts": 3}


def make_rotary_shape(B: int, N: int, H: int, Hk: int, D: int, io_dtype: str = "bf16",
                      rot: Optional[int] = None, layout: str = "half", base: float = 10000.0,
                      scaling=None, mscale: float = 1.0, inverse: bool = False,
                      pos_rows: bool = False, offset: int = 0) -> LaRotaryShape:
    """``scaling``: None, ("linear", factor), ("base", factor) or ("parts", factor,
    original_length, slow, fast)."""
    io = {"bf16": LA_IO_BF16, "f32": LA_IO_F32, "float32": LA_IO_F32}[io_dtype]
    kind, factor, length, slow, fast = 0, 1.0, 1.0, 0.0, 1.0
    if scaling is not None:
        kind, factor = _ROTARY_SCALINGS[scaling[0]], scaling[1]
        if len(scaling) != (5 if kind == 3 else 2):
            raise ValueError(f"scaling {scaling!r}: wrong number of values")
        if kind == 3:
            length, slow, fast = scaling[2:]
    rot = D if rot is None else rot
    if (B | N | H | Hk | D | rot | offset) >> 31 not in (0, -1):
        raise _unfit(B, N, H, Hk, D, rot, offset)
    return LaRotaryShape(B, N, H, Hk, D, rot, io, _ROTARY_LAYOUTS[layout], kind,
                         int(inverse), int(pos_rows), offset, base, factor, length, slow, fast, mscale)


def rotary(Q, K=None, positions=None, offset: int = 0, rot: Optional[int] = None,
           layout: str = "half", base: float = 10000.0, scaling=None, mscale: float = 1.0,
           inverse: bool = False, out=None, stream=None):
    """Q [B, N, H, D] and K [B, N, Hk, D] (or None) with rotary positions: returns (Qo, Ko).

    ``positions``: int32 [N] or [B, N], or None for offset + n. ``rot``: dimensions that turn
    (default: all). ``inverse`` turns back, which is the gradient. ``out``: (Qo, Ko), which may be
    (Q, K) to work in place. Frequencies and ``scaling``: see make_rotary_shape and include/la.h."""
    if stream is not None:
        with _on(stream, Q):
            return rotary(Q, K, positions, offset, rot, layout, base, scaling, mscale, inverse, out)
    torch = _t()
    if Q.dim() != 4:
        raise ValueError(f"Q must be [B, N, H, D], got {tuple(Q.shape)}")
    B, N, H, D = Q.shape
    io = "bf16" if _io_of(Q, "Q") == LA_IO_BF16 else "f32"
    device = Q.get_device()
    _need("Q", Q, Q.shape, Q.dtype, device)
    Hk = 0
    if K is not None:
        if K.dim() != 4:
            raise ValueError(f"K must be [B, N, Hk, D], got {tuple(K.shape)}")
        Hk = K.shape[2]
        _need("K", K, (B, N, Hk, D), Q.dtype, device)
    rows = positions is not None and positions.dim() == 2
    _need("positions", positions, (B, N) if rows else (N,), torch.int32, device)
    Qo, Ko = (None, None) if out is None else out
    _need("out[0]", Qo, Q.shape, Q.dtype, device)
    _need("out[1]", Ko, (B, N, Hk, D), Q.dtype, device)
    shape = make_rotary_shape(B, N, H, Hk, D, io, rot, layout, base, scaling, mscale, inverse, rows,
                              offset)
    device = _on_gpu(Q)
    if Qo is None:
        Qo = torch.empty_like(Q)
    if K is None:
        Ko = None
    elif Ko is None:
        Ko = torch.empty_like(K)
    _launch(_lib.la_rotary, "la_rotary", shape,
            (Q.data_ptr(), _at(K), _at(positions), Qo.data_ptr(), _at(Ko)), device)
    return Qo, Ko


_NORMS = {"rms": 0, "layer": 1}


def _norm_shape(x, f, gate, w_post, w_pre, mod_scale, mod_shift, norm, eps, alpha, **like_x):
    torch = _t()
    if x.dim() != 3:
        raise ValueError(f"x must be [B, N, C], got {tuple(x.shape)}")
    io = _io_of(x, "x")
    full, device = x.shape, x.get_device()
    B, N, C = full
    if (B | N | C) >> 31:
        raise _unfit(B, N, C)
    _need("x", x, full, x.dtype, device)
    _need("f", f, full, x.dtype, device)
    for name, t in like_x.items():
        _need(name, t, full, x.dtype, device)
    _need("gate", gate, (B, C), torch.float32, device)
    _need("mod_scale", mod_scale, (B, C), torch.float32, device)
    _need("mod_shift", mod_shift, (B, C), torch.float32, device)
    _need("w_post", w_post, (C,), torch.float32, device)
    _need("w_pre", w_pre, (C,), torch.float32, device)
    return LaNormShape(B, N, C, io, _NORMS[norm], eps, alpha)


def gate_residual_norm(x, f=None, gate=None, w_post=None, w_pre=None, mod_scale=None, mod_shift=None,
                       norm: str = "layer", eps: float = 1e-6, alpha: float = 1.0, out=None,
                       want_h: bool = True, want_y: bool = True, stream=None):
    """h, y of the gated residual and the norms around it, for [B, N, C] CUDA tensors:

    u = f, or RMSNorm(f) w_post;  h = x + alpha gate u;  y = norm(h) w_pre (1 + mod_scale) + mod_shift

    with float32 parameters gate, mod_scale, mod_shift [B, C] and w_post, w_pre [C]. h is None
    without f or with ``want_h=False``, y with ``want_y=False``. ``out``: (h, y), each of which
    may be x or f."""
    if stream is not None:
        with _on(stream, x):
            return gate_residual_norm(x, f, gate, w_post, w_pre, mod_scale, mod_shift, norm, eps, alpha,
                                      out, want_h, want_y)
    torch = _t()
    h, y = (None, None) if out is None else out
    shape = _norm_shape(x, f, gate, w_post, w_pre, mod_scale, mod_shift, norm, eps, alpha, h=h, y=y)
    device = _on_gpu(x)
    if h is None and f is not None and want_h:
        h = torch.empty_like(x)
    if y is None and want_y:
        y = torch.empty_like(x)
    _launch(_lib.la_gate_residual_norm, "la_gate_residual_norm", shape,
            (x.data_ptr(), _at(f), _at(gate), _at(w_post), _at(w_pre), _at(mod_scale), _at(mod_shift),
             _at(h), _at(y)), device)
    return h, y


def gate_residual_norm_backward(x, f, dy, dh, gate=None, w_post=None, w_pre=None, mod_scale=None,
                                mod_shift=None, norm: str = "layer", eps: float = 1e-6,
                                alpha: float = 1.0, stream=None):
    """dx, df, dgate, dw_post, dw_pre, dmod_scale, dmod_shift of gate_residual_norm: None for what
    was not given (dmod_shift with mod_shift). f, and one of dy and dh, may be None."""
    if stream is not None:
        with _on(stream, x):
            return gate_residual_norm_backward(x, f, dy, dh, gate, w_post, w_pre, mod_scale,
                                               mod_shift, norm, eps, alpha)
    torch = _t()
    shape = _norm_shape(x, f, gate, w_post, w_pre, mod_scale, mod_shift, norm, eps, alpha, dy=dy, dh=dh)
    device = _on_gpu(x)
    grads = [None if t is None else torch.empty_like(t)
             for t in (x, f, gate, w_post, w_pre, mod_scale, mod_shift)]
    ws, n = _scratch(_lib.la_norm_workspace_bytes(ctypes.byref(shape)), x)
    _launch(_lib.la_gate_residual_norm_backward, "la_gate_residual_norm_backward", shape,
            (x.data_ptr(), _at(f), _at(gate), _at(w_post), _at(w_pre), _at(mod_scale), _at(dh), _at(dy),
             *(_at(g) for g in grads), _at(ws), n), device)
    return tuple(grads)
