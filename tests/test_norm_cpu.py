"""Gated residual norm without a GPU: the oracle's pins and the refusals."""
import ctypes

import numpy as np
import pytest
import torch

import linear_attention_diffusion_b200 as la
import oracle as orc

FAKE = 0x7f0000000000
MB = 1 << 20


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("post,f_given", [(True, True), (False, True), (False, False)])
def test_oracle_gradients_equal_differences(norm, post, f_given):
    r = np.random.default_rng(2)
    B, N, C = 2, 3, 8
    kw = dict(x=r.standard_normal((B, N, C)), mod_scale=r.standard_normal((B, C)), w_pre=r.standard_normal(C),
              mod_shift=r.standard_normal((B, C)))
    if f_given:
        kw.update(f=r.standard_normal((B, N, C)), gate=r.standard_normal((B, C)))
    if post:
        kw["w_post"] = r.standard_normal(C)
    dy, dh = r.standard_normal((2, B, N, C))
    opt = dict(norm=norm, eps=1e-3, alpha=0.7)

    def loss(k):
        h, y = orc.gate_residual_norm(**k, **opt)
        return (h * dh).sum() + (y * dy).sum()

    g = orc.gate_residual_norm_backward(kw["x"], kw.get("f"), dy, dh, kw.get("gate"), kw.get("w_post"),
                                        kw["w_pre"], kw["mod_scale"], **opt)
    for name, t in kw.items():
        for at in np.ndindex(t.shape):
            hi, lo = dict(kw), dict(kw)
            hi[name], lo[name] = t.copy(), t.copy()
            hi[name][at] += 1e-6
            lo[name][at] -= 1e-6
            assert abs((loss(hi) - loss(lo)) / 2e-6 - g[name][at]) < 1e-6, (name, at)


def test_oracle_norms():
    x = np.random.default_rng(3).standard_normal((1, 4, 64)) + 3
    _, y = orc.gate_residual_norm(x, eps=0.0)
    assert np.allclose(y.mean(-1), 0) and np.allclose((y ** 2).mean(-1), 1)
    _, y = orc.gate_residual_norm(x, norm="rms", eps=0.0)
    assert np.allclose((y ** 2).mean(-1), 1)


def test_shape_struct_and_workspace():
    assert ctypes.sizeof(la.LaNormShape) == 28 and la.LaNormShape.alpha.offset == 24
    n = lambda *a, **k: la.la_norm_workspace_bytes(la.make_norm_shape(*a, **k))  # noqa: E731
    assert n(1, 16384, 2240) % 256 == 0 and n(1, 16384, 2240) < 16384 * 2240
    assert n(0, 5, 64) > 0 and n(5, 0, 64) > 0
    for bad in ((1, 4, 12), (1, 4, 0), (1, 4, 8200), (-1, 4, 64), (1, -4, 64)):
        assert n(*bad) == 0
    assert n(1, 4, 64, eps=-1.0) == 0 and n(1, 4, 64, alpha=float("inf")) == 0


def _call(func, names, shape, **over):
    ptr = {x: FAKE + i * MB for i, x in enumerate(names)}
    ptr.update(over)
    extra = [ptr[x] for x in names]
    if func == "la_gate_residual_norm_backward":
        extra.append(over.get("n", 1 << 20) if "n" in over else 1 << 20)
    return getattr(la._lib, func)(ctypes.byref(shape), *extra, None)


def test_forward_refusals():
    names = ["x", "f", "gate", "w_post", "w_pre", "mod_scale", "mod_shift", "h", "y"]
    s = la.make_norm_shape(2, 8, 64)
    call = lambda **o: _call("la_gate_residual_norm", names, o.pop("shape", s), **o)  # noqa: E731
    inv = la.LA_ERR_INVALID_ARG
    for name in names:
        assert call(**{name: FAKE + 50 * MB + 4}) == inv, name
    assert call(x=None) == inv and call(h=None, y=None) == inv
    assert call(f=None) == inv                                    # gate, w_post and h without f
    assert call(f=None, gate=None, w_post=None) == inv            # h without f
    for out in ("h", "y"):
        for other in names:
            if other != out:
                at = FAKE + names.index(other) * MB
                if other in ("x", "f"):
                    at += 64                                      # a part of it
                assert call(**{out: at}) == inv, (out, other)
    for field, bad in (("norm", 2), ("io_dtype", 3), ("eps", float("nan")), ("alpha", float("nan"))):
        t = la.make_norm_shape(2, 8, 64)
        setattr(t, field, bad)
        assert call(shape=t) == inv, field
    assert call(shape=la.make_norm_shape(2, 8, 60)) == la.LA_ERR_UNSUPPORTED
    assert call(shape=la.make_norm_shape(70000, 8, 64)) == la.LA_ERR_UNSUPPORTED


def test_backward_refusals():
    names = ["x", "f", "gate", "w_post", "w_pre", "mod_scale", "dh", "dy", "dx", "df", "dgate", "dw_post",
             "dw_pre", "dmod_scale", "dmod_shift", "ws"]
    s = la.make_norm_shape(2, 8, 64)

    def call(n=1 << 20, **over):
        ptr = {x: FAKE + i * MB for i, x in enumerate(names)}
        ptr.update(over)
        return la._lib.la_gate_residual_norm_backward(ctypes.byref(s), *[ptr[x] for x in names], n, None)

    inv = la.LA_ERR_INVALID_ARG
    for name in names:
        assert call(**{name: FAKE + 50 * MB + 4}) == inv, name
    assert call(dh=None, dy=None) == inv and call(x=None) == inv and call(dx=None) == inv
    assert call(df=None) == inv and call(f=None) == inv
    assert call(ws=None) == la.LA_ERR_WORKSPACE
    assert call(n=la.la_norm_workspace_bytes(s) - 256) == la.LA_ERR_WORKSPACE
    for out in names[8:]:
        for other in names:
            if other != out:
                at = FAKE + names.index(other) * MB
                if out in ("dx", "df") and other in ("dh", "dy"):
                    at += 64
                assert call(**{out: at}) == inv, (out, other)


def test_binding_refuses_what_does_not_fit():
    x, c, bc = torch.zeros(2, 5, 64), torch.zeros(64), torch.zeros(2, 64)
    with pytest.raises(ValueError):  # not on a GPU
        la.gate_residual_norm(x, x)
    for bad in (dict(f=x.bfloat16()), dict(f=torch.zeros(2, 4, 64)), dict(gate=c), dict(w_pre=bc),
                dict(w_post=c.double()), dict(mod_scale=bc.bfloat16()), dict(mod_shift=bc[:1]),
                dict(f=torch.zeros(2, 64, 5).transpose(1, 2)), dict(out=(None, torch.zeros(2, 5, 32)))):
        with pytest.raises(ValueError):
            la.gate_residual_norm(x, **bad)
    with pytest.raises(ValueError):
        la.gate_residual_norm_backward(x, x, x, torch.zeros(2, 5, 32))
    with pytest.raises(KeyError):
        la.gate_residual_norm(x, norm="batch")
