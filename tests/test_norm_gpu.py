"""GPU parity of the gated residual norm against the float64 oracle, element by element.

Tolerances: half a step of the output's type, and 2^-17 of the sum of the absolute values
that an output is made of. The row sums are float32: a thread's up to 72 terms one by one and
then a tree, a relative error of at most 80 x 2^-24 < 2^-17 of their absolute sum; the few
products after them stay below it. Column sums add up to 8 x rows such terms.
"""
import numpy as np
import pytest
import torch

import oracle as orc
from tests import parity as P

la = P.la
pytestmark = pytest.mark.gpu
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
TOL = 2.0 ** -17


def _draw(B, N, C, io, seed, post, mod, f=True):
    r = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=r)  # noqa: E731
    t = {"x": (2 * n(B, N, C) + 0.5).to(DT[io]), "f": (n(B, N, C) + 0.1).to(DT[io]) if f else None,
         "gate": n(B, C) if mod and f else None, "w_post": 1 + 0.3 * n(C) if post and f else None,
         "w_pre": 1 + 0.3 * n(C) if mod or post else None, "mod_scale": 0.5 * n(B, C) if mod else None,
         "mod_shift": 0.5 * n(B, C) if mod else None}
    return t, n(B, N, C).to(DT[io]), n(B, N, C).to(DT[io])


def _dev(t):
    return {k: None if v is None else v.cuda() for k, v in t.items()}


def _near(name, got, ref, size, half):
    got = orc.to_f64(got.cpu())
    err, bound = np.abs(got - ref), half * np.abs(ref) + TOL * size + 1e-30
    assert np.isfinite(got).all() and (err <= bound).all(), f"{name}: {(err / bound).max():.3g} of its bound"


def _sizes(t, norm, eps, alpha):
    """|h|'s terms, n's terms, 1 / std and the post norm's 1 / rms, in float64."""
    f64 = lambda x, d: np.float64(d) if x is None else np.abs(orc.to_f64(x))  # noqa: E731
    wide = lambda x, d: f64(x, d)[:, None] if x is not None else np.float64(d)  # noqa: E731
    h, _ = orc.gate_residual_norm(**t, norm=norm, eps=eps, alpha=alpha)
    xs = f64(t["x"], 0)
    rf = 1.0
    u = f64(t["f"], 0) * np.ones_like(xs)
    if t["w_post"] is not None:
        rf = 1 / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    un = u * rf
    hs = xs + abs(alpha) * wide(t["gate"], 1) * un * f64(t["w_post"], 1)
    a = h - h.mean(-1, keepdims=True) if norm == "layer" else h
    rh = 1 / np.sqrt((a * a).mean(-1, keepdims=True) + eps)
    ns = (hs + hs.mean(-1, keepdims=True)) * rh
    w = f64(t["w_pre"], 1) * (1 + wide(t["mod_scale"], 0))
    return hs, ns, rh, un, rf, w, wide(t["mod_shift"], 0), f64(t["w_post"], 1), abs(alpha) * wide(t["gate"], 1)


def _both(B, N, C, io, norm, post, mod, f=True, eps=1e-5, alpha=0.8, seed=4):
    t, dy, dh = _draw(B, N, C, io, seed, post, mod, f)
    d = _dev(t)
    h, y = la.gate_residual_norm(**d, norm=norm, eps=eps, alpha=alpha)
    h_ref, y_ref = orc.gate_residual_norm(**t, norm=norm, eps=eps, alpha=alpha)
    hs, ns, rh, un, rf, w, shift, wo, gate = _sizes(t, norm, eps, alpha)
    if f:
        _near("h", h, h_ref, hs, HALF[io])
    else:
        assert h is None
    _near("y", y, y_ref, ns * w + shift, HALF[io])
    got = la.gate_residual_norm_backward(d["x"], d["f"], dy.cuda(), dh.cuda(), **{k: d[k] for k in (
        "gate", "w_post", "w_pre", "mod_scale", "mod_shift")}, norm=norm, eps=eps, alpha=alpha)
    ref = orc.gate_residual_norm_backward(t["x"], t["f"], dy, dh, t["gate"], t["w_post"], t["w_pre"],
                                          t["mod_scale"], norm, eps, alpha)
    gy, gh = np.abs(orc.to_f64(dy)), np.abs(orc.to_f64(dh))
    mean = lambda x: x.mean(-1, keepdims=True)  # noqa: E731
    tt = gy * w
    # the projection's own error is that of n (twice) and of the two means
    dxs = gh + 3 * rh * (tt + ns * mean(tt * ns) + mean(tt))
    du = gate * dxs * wo
    dfs = 2 * rf * (du + un * mean(du * un))
    sums = {"x": dxs, "f": dfs, "gate": (abs(alpha) * un * wo * dxs).sum(1), "w_post": (gate * dxs * un).sum((0, 1)),
            "w_pre": (gy * (w / (1 if t["w_pre"] is None else np.abs(orc.to_f64(t["w_pre"])))) * ns).sum((0, 1)),
            "mod_scale": (gy * ns * (1 if t["w_pre"] is None else np.abs(orc.to_f64(t["w_pre"])))).sum(1),
            "mod_shift": gy.sum(1)}
    for name, g in zip(("x", "f", "gate", "w_post", "w_pre", "mod_scale", "mod_shift"), got):
        if t[name] is None:
            assert g is None
        else:
            _near("d" + name, g, ref[name], sums[name], HALF[io] if name in ("x", "f") else HALF["f32"])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("C", [8, 32, 40, 256, 264, 1152, 2240, 2304, 2312, 2560, 2568, 5120, 8192])
def test_widths(cuda_device, io, C):
    _both(2, 5, C, io, "layer" if C % 16 else "rms", True, True)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("post,mod,f", [(True, True, True), (True, False, True), (False, True, True),
                                        (False, False, True), (False, True, False), (False, False, False)])
def test_parts(cuda_device, io, norm, post, mod, f):
    _both(3, 11, 96, io, norm, post, mod, f)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,C", [(1, 1, 64), (1, 1500, 1152), (2, 700, 2240), (300, 1, 32), (1, 3001, 8),
                                   (40, 9, 512), (1, 1300, 768)])
def test_rows(cuda_device, io, B, N, C):
    """Few rows and many: a warp per row and a CTA per row, short and many batch elements."""
    _both(B, N, C, io, "layer", N % 2 == 1, True)


@pytest.mark.parametrize("only", ["h", "y"])
def test_one_side_only(cuda_device, only):
    t, dy, dh = _draw(2, 9, 320, "f32", 5, True, True)
    d = _dev(t)
    both = la.gate_residual_norm(**d)
    h, y = la.gate_residual_norm(**d, want_h=only == "h", want_y=only == "y")
    if only == "h":
        assert y is None and torch.equal(h, both[0])
    else:
        assert h is None and torch.equal(y, both[1])
    par = {k: d[k] for k in ("gate", "w_post", "w_pre", "mod_scale", "mod_shift")}
    zero = torch.zeros_like(dy).cuda()
    a = la.gate_residual_norm_backward(d["x"], d["f"], dy.cuda() if only == "y" else None,
                                       dh.cuda() if only == "h" else None, **par)
    b = la.gate_residual_norm_backward(d["x"], d["f"], dy.cuda() if only == "y" else zero,
                                       dh.cuda() if only == "h" else zero, **par)
    assert all(torch.allclose(p, q, rtol=1e-6, atol=1e-6) for p, q in zip(a, b))


@pytest.mark.parametrize("C", [320, 2240])
def test_in_place(cuda_device, C):
    t, dy, dh = _draw(1, 1300, C, "bf16", 6, True, True)
    d = _dev(t)
    want = la.gate_residual_norm(**d)
    x, f = d["x"].clone(), d["f"].clone()
    la.gate_residual_norm(x, f, *(d[k] for k in ("gate", "w_post", "w_pre", "mod_scale", "mod_shift")), out=(x, f))
    assert torch.equal(x, want[0]) and torch.equal(f, want[1])
    par = [d[k] for k in ("gate", "w_post", "w_pre", "mod_scale")]
    ref = la.gate_residual_norm_backward(d["x"], d["f"], dy.cuda(), dh.cuda(), *par)
    gx, gf = dh.cuda(), dy.cuda()
    shape = la.make_norm_shape(1, 1300, C)
    ws = torch.empty(la.la_norm_workspace_bytes(shape), dtype=torch.uint8, device="cuda")
    la.la_gate_residual_norm_backward(shape, d["x"], d["f"], *par, gx, gf, gx, gf, None, None, None, None, None, ws)
    assert torch.equal(gx, ref[0]) and torch.equal(gf, ref[1])


def test_zero_rows_and_large_means(cuda_device):
    """A row of zeros gives the shift; a row far from zero keeps the digits of its spread."""
    x = torch.zeros((1, 3, 64), device="cuda")
    x[0, 1] = 4096.0 + torch.arange(64, device="cuda") % 2
    shift = torch.randn((1, 64), device="cuda")
    _, y = la.gate_residual_norm(x, mod_shift=shift, eps=1e-6)
    assert torch.equal(y[0, 0], shift[0]) and torch.equal(y[0, 2], shift[0])
    spread = (y[0, 1] - shift[0]).cpu()
    want = torch.tensor([-1.0, 1.0]).repeat(32) * (0.25 / (0.25 + 1e-6)) ** 0.5
    assert torch.allclose(spread, want, rtol=0, atol=2.0 ** -20)


def test_empty_stream_and_graph(cuda_device):
    e = torch.empty((2, 0, 64), device="cuda")
    w, b = torch.ones(64, device="cuda"), torch.ones((2, 64), device="cuda")
    assert la.gate_residual_norm(e, e, b, w, w, b, b)[1].shape == e.shape
    g = la.gate_residual_norm_backward(e, e, e, e, b, w, w, b, b)
    assert all(not t.any() for t in g[2:])
    t, dy, dh = _draw(2, 50, 2240, "bf16", 7, True, True)
    d, dy, dh = _dev(t), dy.cuda(), dh.cuda()
    par = {k: d[k] for k in ("gate", "w_post", "w_pre", "mod_scale", "mod_shift")}
    call = lambda: [*la.gate_residual_norm(**d), *la.gate_residual_norm_backward(  # noqa: E731
        d["x"], d["f"], dy, dh, **par)]
    want = call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = call()
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    d["x"].mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(held, call()))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("C,N", [(96, 40), (264, 1300), (2240, 1300), (2240, 9), (4096, 30)])
def test_rows_are_apart(cuda_device, io, C, N):
    """Rows that are not finite change no other row's bits, forwards or backwards, and no other
    batch element's parameter gradients: a warp and a CTA a row, the next row ahead."""
    t, dy, dh = _draw(3, N, C, io, 8, True, True)
    d, dy, dh = _dev(t), dy.cuda(), dh.cuda()
    par = {k: d[k] for k in ("gate", "w_post", "w_pre", "mod_scale", "mod_shift")}
    call = lambda x, f, a, b: [*la.gate_residual_norm(x, f, **par, norm="layer"),  # noqa: E731
                               *la.gate_residual_norm_backward(x, f, a, b, **par, norm="layer")]
    want = call(d["x"], d["f"], dy, dh)
    x, f, a, b = (y.clone() for y in (d["x"], d["f"], dy, dh))
    rows = [2, N // 2, N - 2]
    x[1, rows[0]], f[1, rows[1], 3], a[1, rows[2]] = float("nan"), float("inf"), float("nan")
    got = call(x, f, a, b)
    keep = torch.ones((3, N), dtype=torch.bool, device="cuda")
    keep[1, rows] = False
    for i in range(4):  # h, y, dx, df
        assert torch.equal(got[i][keep], want[i][keep]), i
    for i in (4, 7, 8):  # dgate, dmod_scale, dmod_shift
        assert torch.equal(got[i][::2], want[i][::2]), i
    assert got[7][1].isnan().all()
