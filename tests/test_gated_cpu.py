"""Gated linear attention without a GPU: the float64 oracle's pins (quadratic form,
closed forms, finite differences) and the refusals of the C ABI and the binding."""
import ctypes

import numpy as np
import pytest
import torch

import linear_attention_diffusion_b200 as la
import oracle as orc

FAKE = 0x7f0000000000  # aligned, never dereferenced: every call below fails its checks first
MB = 1 << 20


def _draw(B, N, H, D=4, seed=0, stops=()):
    r = np.random.default_rng(seed)
    q, k, v, do = (r.standard_normal((B, N, H, D)) for _ in range(4))
    g = -r.exponential(0.5, (B, N, H))
    for n in stops:
        g[:, n] = -np.inf
    return q, k, v, g, do, r.standard_normal((B, H, D, D)), r.standard_normal((B, H, D, D))


@pytest.mark.parametrize("stops", [(), (0,), (3, 4), (6,)])
def test_oracle_recurrence_equals_quadratic_form(stops):
    q, k, v, g, _, S0, _ = _draw(2, 7, 2, stops=stops)
    for S in (None, S0):
        O, _ = orc.gated_attention(q, k, v, g, S, 0.7)
        assert np.allclose(O, orc.gated_bruteforce(q, k, v, g, S, 0.7), rtol=1e-12, atol=1e-12)


def test_oracle_without_gates_is_a_running_sum():
    q, k, v, g, _, _, _ = _draw(1, 9, 2)
    O, S = orc.gated_attention(q, k, v, np.zeros_like(g))
    run = np.cumsum(np.einsum("bnhd,bnhe->bnhde", k, v), 1)
    assert np.allclose(S, run[:, -1]) and np.allclose(O, np.einsum("bnhd,bnhde->bnhe", q, run))


@pytest.mark.parametrize("stops", [(), (2,)])
def test_oracle_gradients_equal_differences(stops):
    q, k, v, g, do, S0, dS = _draw(1, 6, 1, D=3, seed=3, stops=stops)
    grads = orc.gated_attention_backward(q, k, v, g, do, S0, dS, 0.6)

    def loss(args):
        O, S = orc.gated_attention(*args, 0.6)
        return (O * do).sum() + (S * dS).sum()

    ins = [q, k, v, g, S0]
    h = 1e-6
    for i, x in enumerate(ins):
        for at in np.ndindex(x.shape):
            if not np.isfinite(x[at]):
                assert grads[i][at] == 0.0
                continue
            lo, hi = ([y.copy() for y in ins] for _ in range(2))
            lo[i][at] -= h
            hi[i][at] += h
            assert abs((loss(hi) - loss(lo)) / (2 * h) - grads[i][at]) < 1e-7, (i, at)


def test_shape_struct_matches_header_layout():
    assert ctypes.sizeof(la.LaGatedShape) == 24
    assert la.LaGatedShape.scale.offset == 20


def test_workspace_bytes():
    f, b = (lambda *a: la.la_gated_workspace_bytes(la.make_gated_shape(*a), False),
            lambda *a: la.la_gated_workspace_bytes(la.make_gated_shape(*a), True))
    assert f(1, 1, 70) > 0 and f(0, 5, 3) > 0 and b(0, 5, 3) > 0 and f(2, 0, 3) > 0
    assert f(1, 32760, 70) > 70 * 4096          # states of the segments
    assert f(64, 4096, 70) == 256               # enough heads: no segments
    assert b(1, 16384, 70) >= 70 * 16384 * 4    # a float per token and head
    for bad in ((1, 4, 2, 64), (-1, 4, 2), (1, -4, 2), (1, 4, -2), (1, 4, 70000), (1, (1 << 30) + 1, 1)):
        assert f(*bad) == 0 and b(*bad) == 0
    assert f(1, 4, 2, 32, "bf16", float("inf")) == 0


def _fwd(shape, q=FAKE, k=FAKE + MB, v=FAKE + 2 * MB, g=FAKE + 3 * MB, si=None, so=None,
         o=FAKE + 4 * MB, ws=FAKE + 5 * MB, n=1 << 30):
    return la._lib.la_gated_attention(ctypes.byref(shape) if shape else None, q, k, v, g, si, so, o,
                                      ws, n, None)


def test_forward_refusals():
    s = la.make_gated_shape(1, 640, 2)
    bad = la.make_gated_shape(1, 640, 2)
    bad.io_dtype = 9
    inv, uns, wsp = la.LA_ERR_INVALID_ARG, la.LA_ERR_UNSUPPORTED, la.LA_ERR_WORKSPACE
    assert _fwd(None) == inv
    assert _fwd(bad) == inv
    assert _fwd(la.make_gated_shape(1, 640, 2, 64)) == uns
    assert _fwd(la.make_gated_shape(1, 640, 2, 32, "bf16", float("nan"))) == inv
    for name in ("q", "k", "v", "g", "o"):
        assert _fwd(s, **{name: None}) == inv
        assert _fwd(s, **{name: FAKE + 6 * MB + 8}) == inv and "aligned" in la.la_last_error()
    assert _fwd(s, ws=None) == wsp
    assert _fwd(s, n=la.la_gated_workspace_bytes(s) - 256) == wsp
    assert _fwd(s, o=FAKE) == inv and "overlap" in la.la_last_error()
    assert _fwd(s, o=FAKE + 3 * MB + 64) == inv
    assert _fwd(s, si=FAKE + 6 * MB, so=FAKE + 6 * MB + 4096) == inv   # partly over S_in
    assert _fwd(s, si=FAKE + 4 * MB, so=FAKE + 4 * MB) == inv         # the state inside O
    assert _fwd(s, so=FAKE + 5 * MB) == inv                           # inside the workspace
    assert _fwd(s, si=FAKE + 5 * MB) == inv


def test_backward_refusals():
    s = la.make_gated_shape(1, 100, 2)
    names = ["Q", "K", "V", "G", "S_in", "dO", "dS_out", "dQ", "dK", "dV", "dG", "dS_in"]

    def call(n=1 << 20, shape=s, ws=FAKE + 90 * MB, **over):
        ptr = {x: FAKE + (2 + i) * MB for i, x in enumerate(names)}
        ptr.update(over)
        return la._lib.la_gated_attention_backward(ctypes.byref(shape), *[ptr[x] for x in names],
                                                   ws, n, None)

    for name in names:
        optional = name in ("S_in", "dS_out", "dS_in")
        if not optional:
            assert call(**{name: None}) == la.LA_ERR_INVALID_ARG, name
        assert call(**{name: FAKE + 80 * MB + 4}) == la.LA_ERR_INVALID_ARG, name
    need = la.la_gated_workspace_bytes(s, True)
    assert call(n=need - 256) == la.LA_ERR_WORKSPACE and call(ws=None) == la.LA_ERR_WORKSPACE
    for out in ("dQ", "dK", "dV", "dG", "dS_in"):
        for other in names:
            if other != out:
                at = FAKE + (2 + names.index(other)) * MB
                assert call(**{out: at}) == la.LA_ERR_INVALID_ARG, (out, other)
    assert call(dQ=FAKE + 90 * MB) == la.LA_ERR_INVALID_ARG  # the workspace
    assert call(shape=la.make_gated_shape(1, 100, 2, 16)) == la.LA_ERR_UNSUPPORTED


def test_empty_calls_need_no_pointers():
    for shape in (la.make_gated_shape(0, 7, 2), la.make_gated_shape(3, 7, 0)):
        assert la._lib.la_gated_attention(ctypes.byref(shape), *[None] * 8, 0, None) == la.LA_OK
        assert la._lib.la_gated_attention_backward(ctypes.byref(shape), *[None] * 13, 0, None) == la.LA_OK


def test_binding_refuses_what_does_not_fit():
    def t(*shape, dt=torch.bfloat16):
        return torch.zeros(shape, dtype=dt)

    q, g = t(1, 5, 2, 32), t(1, 5, 2, dt=torch.float32)
    f = torch.float32
    with pytest.raises(ValueError):  # not on a GPU
        la.gated_attention(q, q, q, g)
    for bad in (dict(Q=t(5, 2, 32)), dict(Q=t(1, 5, 2, 64)), dict(K=t(1, 4, 2, 32)), dict(V=t(1, 5, 2, 32, dt=f)),
                dict(G=t(1, 5, 2)), dict(G=t(1, 5, 3, dt=f)), dict(S_in=t(1, 2, 32, 32)),
                dict(S_in=t(2, 32, 32, dt=f)), dict(Q=t(1, 5, 2, 32, dt=torch.float16)),
                dict(K=t(1, 2, 5, 32).transpose(1, 2))):
        args = dict(Q=q, K=q, V=q, G=g)
        args.update(bad)
        with pytest.raises(ValueError):
            la.gated_attention(**args)
    with pytest.raises(ValueError):
        la.gated_attention_backward(q, q, q, g, t(1, 5, 2, 32, dt=f))
    with pytest.raises(ValueError):
        la.gated_attention_backward(q, q, q, g, q, dS_out=t(1, 2, 32, 32))


def test_window_errors_see_what_a_gate_gradient_can_lose():
    """The bound of the GPU's check (2^-15) is far below what zeros, a lost carry between two
    windows of 256 tokens, or a stale one give; the oracle's own numbers in float32 stay below."""
    r = np.random.default_rng(5)
    B, N, H, D = 1, 600, 3, 8
    q, k, v, do = (r.standard_normal((B, N, H, D)) for _ in range(4))
    g = -r.uniform(0.002, 0.5, H) * r.uniform(0.1, 2.1, (B, N, H))
    S, dS = r.standard_normal((2, B, H, D, D))
    dQ, dK, _, dG, _ = orc.gated_attention_backward(q, k, v, g, do, S, dS, 0.4)
    err = lambda x: orc.gated_window_errors(x, dG)  # noqa: E731
    assert err(dG.astype(np.float32)).max() < 2.0 ** -23
    assert (err(np.zeros_like(dG)) == 1.0).all() and err(dG).shape == (1, 3, 3)
    rows = (q * dQ).sum(-1) - (k * dK).sum(-1)
    for lost, at in ((dG[:, 256], slice(0, 256)), (dG[:, 512], slice(256, 512))):
        x = dG.copy()
        x[:, at] -= lost[:, None]                     # the sum of the window's rows alone
        assert np.allclose(x[:, at], rows[:, at][:, ::-1].cumsum(1)[:, ::-1], atol=1e-9)
        assert (err(x).max(1) > 2.0 ** -4).all()
        x[:, at] += dG[:, 100][:, None]               # another place's carry
        assert (err(x).max(1) > 2.0 ** -4).all()


def test_launches_follow_the_cut():
    """One launch for few tokens, a row a CTA or heads that fill the GPU, three where rows are cut;
    backwards two or four."""
    f, b = (lambda *a: la.la_gated_launches(la.make_gated_shape(*a), False),
            lambda *a: la.la_gated_launches(la.make_gated_shape(*a), True))
    assert f(64, 1, 70) == 1 and f(1, 256, 70) == 1 and f(64, 4096, 70) == 1 and f(1, 32760, 70) == 3
    assert b(1, 16384, 70) == 4 and b(64, 4096, 70) == 2 and b(1, 3, 2) == 2
    assert f(2, 0, 3) == 0 and b(0, 9, 3) == 0 and f(1, 4, 2, 64) == 0 and b(-1, 4, 2) == 0



def test_a_stream_of_another_gpu_is_refused():
    """The call would run on the current stream of the tensors' GPU, not on the one given."""
    from types import SimpleNamespace
    x = SimpleNamespace(is_cuda=True, get_device=lambda: 0, device=torch.device("cuda:0"))
    stream = SimpleNamespace(device=torch.device("cuda:1"))
    for call in (lambda: la.gated_attention(x, x, x, x, stream=stream),
                 lambda: la.gated_attention_backward(x, x, x, x, x, stream=stream),
                 lambda: la.rotary(x, stream=stream), lambda: la.gate_residual_norm(x, stream=stream),
                 lambda: la.gate_residual_norm_backward(x, None, x, None, stream=stream)):
        with pytest.raises(ValueError, match="belongs to cuda:1"):
            call()
