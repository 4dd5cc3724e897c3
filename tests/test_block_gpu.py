"""The block operators in a row, as a causal block runs them: norm and modulation, the QKV
projection, rotary positions, gated attention, the output's gated residual with the next norm.
Forward against the oracles, prompt and single tokens against the whole, and the gradients that
the pieces' backward calls pass along against differences of the chain in float64."""
import numpy as np
import pytest
import torch

import oracle as orc
from tests import parity as P

la = P.la
pytestmark = pytest.mark.gpu
B, H, D = 2, 3, 32
C = H * D


def _weights(seed, io):
    r = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=r)  # noqa: E731
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    return {"w": (n(3 * C, C) / C ** 0.5).to(dt), "scale": 0.2 * n(B, C), "shift": 0.2 * n(B, C),
            "gate": 0.5 + 0.1 * n(B, C), "w_pre": 1 + 0.1 * n(C), "w_post": 1 + 0.1 * n(C)}


def _block(x, g, p, S=None, offset=0, S_out=None):
    """h and y of one block for x [B, N, C], and the state after it."""
    N = x.shape[1]
    _, y = la.gate_residual_norm(x, w_pre=p["w_pre"], mod_scale=p["scale"], mod_shift=p["shift"], norm="rms")
    q, k, v = (t.reshape(B, N, H, D).contiguous() for t in (y @ p["w"].t()).chunk(3, -1))
    q, k = la.rotary(q, k, offset=offset)
    o, S = la.gated_attention(q, k, v, g, S_in=S, scale=D ** -0.5, want_state=True, S_out=S_out)
    h, y = la.gate_residual_norm(x, o.reshape(B, N, C), p["gate"], p["w_post"], p["w_pre"], norm="layer")
    return h, y, S, (q, k, v, o)


def _block64(x, g, p):
    """The same in float64 numpy: h, y, S."""
    N = x.shape[1]
    p = {k: np.asarray(orc.to_f64(t)) for k, t in p.items()}
    _, y = orc.gate_residual_norm(x, w_pre=p["w_pre"], mod_scale=p["scale"], mod_shift=p["shift"], norm="rms")
    q, k, v = (t.reshape(B, N, H, D) for t in np.split(y @ p["w"].T, 3, -1))
    q, k = (orc.rotary(t, np.arange(N), D) for t in (q, k))
    o, S = orc.gated_attention(q, k, v, g, scale=D ** -0.5)
    h, y = orc.gate_residual_norm(x, o.reshape(B, N, C), p["gate"], p["w_post"], p["w_pre"], norm="layer")
    return h, y, S


def _draw(N, io, seed):
    r = torch.Generator().manual_seed(seed)
    x = torch.randn((B, N, C), generator=r).to(torch.bfloat16 if io == "bf16" else torch.float32)
    return x, -0.2 * torch.rand((B, N, H), generator=r)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_block_forward_and_one_token_at_a_time(cuda_device, io):
    """Tolerance: the block rounds six times to its type on the way (y, qkv, q and k turned, o,
    h or y), each a relative 2-norm of at most half a step, and the norm of o carries o's on;
    float32 adds the projection's own sums (torch's, 96 terms)."""
    N, n = 70, 60
    p = _weights(1, io)
    x, g = _draw(N, io, 2)
    dev = {k: t.cuda() for k, t in p.items()}
    xd, gd = x.cuda(), g.cuda()
    h, y, S, _ = _block(xd, gd, dev)
    ref = _block64(orc.to_f64(x), g, p)
    tol = 6 * 2.0 ** -8 if io == "bf16" else 64 * 2.0 ** -24
    for got, want in zip((h, y, S), ref):
        err = np.linalg.norm(orc.to_f64(got.cpu()) - want) / np.linalg.norm(want)
        assert err <= tol, err
    # the same tokens as a prompt of 60 and ten single ones, the state kept in place
    h1, y1, state, _ = _block(xd[:, :n].contiguous(), gd[:, :n].contiguous(), dev)
    parts = [(h1, y1)]
    for i in range(n, N):
        hi, yi, same, _ = _block(xd[:, i:i + 1].contiguous(), gd[:, i:i + 1].contiguous(), dev, S=state, offset=i,
                                 S_out=state)
        assert same is state
        parts.append((hi, yi))
    for j, want in enumerate(ref[:2]):
        got = orc.to_f64(torch.cat([t[j] for t in parts], 1).cpu())
        assert np.linalg.norm(got - want) / np.linalg.norm(want) <= tol
    assert np.linalg.norm(orc.to_f64(state.cpu()) - ref[2]) / np.linalg.norm(ref[2]) <= tol


def test_block_gradients_equal_differences(cuda_device):
    """float32: the backward calls chained by hand give the loss's slope along random ways."""
    N = 40
    p = _weights(3, "f32")
    x, g = _draw(N, "f32", 4)
    r = torch.Generator().manual_seed(5)
    dh, dy = torch.randn((B, N, C), generator=r), torch.randn((B, N, C), generator=r)
    dev = {k: t.cuda() for k, t in p.items()}
    xd, gd = x.cuda(), g.cuda()
    _, y0 = la.gate_residual_norm(xd, w_pre=dev["w_pre"], mod_scale=dev["scale"], mod_shift=dev["shift"],
                                  norm="rms")
    _, _, _, (q, k, v, o) = _block(xd, gd, dev)
    dx, do, dgate, dwo, dwi, _, _ = la.gate_residual_norm_backward(
        xd, o.reshape(B, N, C), dy.cuda(), dh.cuda(), dev["gate"], dev["w_post"], dev["w_pre"], norm="layer")
    dq, dk, dv, dg, _ = la.gated_attention_backward(q, k, v, gd, do.reshape(B, N, H, D), scale=D ** -0.5)
    dq, dk = la.rotary(dq, dk, inverse=True)
    dqkv = torch.cat([t.reshape(B, N, C) for t in (dq, dk, dv)], -1)
    dw = torch.einsum("bno,bnc->oc", dqkv, y0)
    dy0 = (dqkv @ dev["w"]).contiguous()
    dx0, _, _, _, dwi0, dsc, dsh = la.gate_residual_norm_backward(
        xd, None, dy0, None, w_pre=dev["w_pre"], mod_scale=dev["scale"], mod_shift=dev["shift"], norm="rms")
    grads = {"x": dx + dx0, "g": dg, "w": dw, "scale": dsc, "shift": dsh, "gate": dgate, "w_pre": dwi + dwi0,
             "w_post": dwo}

    def loss(xx, gg, pp):
        h, y, _ = _block64(xx, gg, pp)
        return (h * dh.numpy().astype(float)).sum() + (y * dy.numpy().astype(float)).sum()

    base = {"x": orc.to_f64(x), "g": orc.to_f64(g), **{k: orc.to_f64(t) for k, t in p.items()}}
    step = 1e-5
    for name, t in base.items():
        way = np.random.default_rng(7).standard_normal(t.shape)
        ends = []
        for sign in (1, -1):
            moved = dict(base)
            moved[name] = t + sign * step * way
            ends.append(loss(moved["x"], moved["g"], {k: moved[k] for k in p}))
        slope = (ends[0] - ends[1]) / (2 * step)
        got = orc.to_f64(grads[name].cpu())
        # 1e-4 of the sum's size: float32 chains of five operators (2^-20 each) and a central
        # difference with a step of 1e-5 in float64 (1e-9 of the loss / step)
        assert abs((got * way).sum() - slope) <= 1e-4 * np.linalg.norm(got * way) + 1e-4 * abs(slope), name


def test_threads_with_different_sizes(cuda_device):
    """Calls of the same kernels at sizes that need different shared memory, from four threads on
    four streams, as fast as the C functions take them: none is refused, and the numbers are the
    ones that a call gives alone."""
    import ctypes
    import threading
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(11)
    randn = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
    at = lambda *ts: [None if t is None else t.data_ptr() for t in ts]  # noqa: E731

    def gated(N):  # float32 rows of 64 and 128 tokens: two and four warps of one kernel
        q, k, v = (randn(2, N, 4, D) for _ in range(3))
        g, out = -torch.rand((2, N, 4), generator=gen, device=dev), torch.empty_like(q)
        shape = la.make_gated_shape(2, N, 4, io_dtype="f32")
        assert la.la_gated_workspace_bytes(shape) == 256  # one launch without segments
        args = [ctypes.byref(shape), *at(q, k, v, g, None, None, out, None), 0]
        return (q, k, v, g, shape), out, lambda st: la._lib.la_gated_attention(*args, st)

    def norm(width):
        x, f, h, y = (randn(1, 4, width) for _ in range(4))
        shape = la.make_norm_shape(1, 4, width, "f32")
        args = [ctypes.byref(shape), *at(x, f, None, None, None, None, None, h, y)]
        return (x, f, h, shape), y, lambda st: la._lib.la_gate_residual_norm(*args, st)

    def norm_back(width):
        x, f, dh, dy, dx, df = (randn(1, 4, width) for _ in range(6))
        shape = la.make_norm_shape(1, 4, width, "f32")
        n = la.la_norm_workspace_bytes(shape)
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        args = [ctypes.byref(shape), *at(x, f, None, None, None, None, dh, dy, dx, df, *[None] * 5, ws), n]
        return (x, f, dh, dy, df, ws, shape), dx, lambda st: la._lib.la_gate_residual_norm_backward(*args, st)

    for make, sizes in ((gated, (64, 128)), (norm, (4608, 8192)), (norm_back, (1408, 2560)), (norm_back, (2816, 8192))):
        calls = [make(sizes[i % 2]) for i in range(4)]
        want = []
        for _, out, call in calls:
            assert call(torch.cuda.current_stream().cuda_stream) == la.LA_OK
            want.append(out.clone())
        torch.cuda.synchronize()
        refused, wrong, start = [0] * 4, [0] * 4, threading.Barrier(4)

        def work(i):
            _, out, call = calls[i]
            stream = torch.cuda.Stream(dev)
            raw = stream.cuda_stream
            start.wait()
            for _ in range(60):
                for _ in range(200):
                    refused[i] += call(raw) != la.LA_OK
                stream.synchronize()
                wrong[i] += not torch.equal(out, want[i])

        threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert refused == [0] * 4 and wrong == [0] * 4, (make.__name__, sizes, refused, wrong)
