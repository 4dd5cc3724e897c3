"""GPU parity of gated linear attention against the float64 oracle, element by element.

Tolerances. Every output is a sum of products; with A the sum of the absolute values of
its terms, |got - ref| <= half a step of the output's type x |ref| + tol x A. For bf16
tensors the computed operands enter the products as two bf16 parts (2^-17 each; a term
meets three: decayed key, state, and on its way the state's own, so 2^-15), for float32
as three (24 bits, sums of up to 32 + 16 terms a product in float32, 2^-18). Each block of
16 tokens a term has crossed adds the error of one decay, 2^-22.
"""
import numpy as np
import pytest
import torch

import oracle as orc
from tests import parity as P

la = P.la
pytestmark = pytest.mark.gpu
D = 32
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _tol(io, N):
    return (2.0 ** -15 if io == "bf16" else 2.0 ** -18) + -(-N // 16) * 2.0 ** -22


def _draw(B, N, H, io, seed, gates="mixed", carry=True):
    r = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    q, k, v, do = (torch.randn((B, N, H, D), generator=r).to(dt) for _ in range(4))
    u = torch.rand((B, N, H), generator=r)
    rate = 0.002 * 250.0 ** torch.rand((H,), generator=r)
    g = -rate * (0.1 + 2 * u)
    if gates == "open":
        g = torch.zeros_like(g)
    elif gates == "strong":
        g = -100.0 * u
    elif gates == "stops":            # single stops, pairs, whole blocks of them
        g = torch.where(u < 0.15, torch.full_like(g, -float("inf")), g)
        g[:, 20:41] = -float("inf")
        g[:, 0] = -1e30
    elif gates == "shut":
        g = torch.full_like(g, -float("inf"))
    S, dS = (torch.randn((B, H, D, D), generator=r) if carry else None for _ in range(2))
    return q, k, v, g, do, S, dS


def _dev(*xs):
    return [None if x is None else x.contiguous().cuda() for x in xs]


def _check(name, got, ref, mag, tol, half):
    got = orc.to_f64(got.cpu())
    err, bound = np.abs(got - ref), half * np.abs(ref) + tol * mag + 1e-36
    worst = (err / bound).max() if err.size else 0.0
    assert np.isfinite(got).all() and (err <= bound).all(), f"{name}: {worst:.3g} of its bound"


def _forward(case, io, gates, carry, seed=5, scale=0.3):
    B, N, H = case
    q, k, v, g, _, S, _ = _draw(B, N, H, io, seed, gates, carry)
    O, So = la.gated_attention(*_dev(q, k, v, g), S_in=_dev(S)[0], scale=scale, want_state=True)
    O_ref, S_ref = orc.gated_attention(q, k, v, g, S, scale)
    A, AS = orc.gated_magnitudes(q, k, v, g, S_in=S, scale=scale)
    tol = _tol(io, N)
    _check("O", O, O_ref, A, tol, HALF[io])
    _check("S", So, S_ref, AS, tol, HALF["f32"])


LENGTHS = [1, 2, 4, 5, 8, 9, 15, 16, 17, 33, 63, 64, 65, 127, 200, 517]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("N", LENGTHS)
def test_forward_lengths(cuda_device, io, N):
    _forward((2, N, 3), io, "mixed", N % 2 == 1)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("gates", ["open", "strong", "stops", "shut"])
@pytest.mark.parametrize("N", [7, 150])
def test_forward_gates(cuda_device, io, gates, N):
    _forward((1, N, 5), io, gates, True)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("case", [(20, 70, 130), (1, 3000, 2), (3, 1, 500), (1, 100, 1), (5, 700, 9), (4, 700, 55),
                                  (6, 270, 46), (3, 1100, 90), (1, 257, 70), (1, 256, 70), (12, 129, 24)], ids=str)
def test_forward_shapes(cuda_device, io, case):
    """One segment per head (more heads than warps fit), many segments, a CTA per row, odd counts."""
    _forward(case, io, "mixed", True)


def _backward(case, io, gates, carry, seed=9, scale=0.4):
    B, N, H = case
    q, k, v, g, do, S, dS = _draw(B, N, H, io, seed, gates, carry)
    dq, dk, dv, dg, dso = _dev(q, k, v, g, do)
    Sd, dSd = _dev(S, dS)
    got = la.gated_attention_backward(dq, dk, dv, dg, dso, S_in=Sd, dS_out=dSd, scale=scale)
    ref = orc.gated_attention_backward(q, k, v, g, do, S, dS, scale)
    mag = orc.gated_magnitudes(q, k, v, g, do, S, dS, scale)
    names = ("dQ", "dK", "dV", "dG", "dS_in")
    for i, name in enumerate(names):
        if got[i] is None:
            assert name == "dS_in" and not carry
            continue
        half = HALF[io] if i < 3 else HALF["f32"]
        _check(name, got[i], ref[i], mag[i], _tol(io, N) * (2 if name == "dG" else 1), half)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("N", LENGTHS)
def test_backward_lengths(cuda_device, io, N):
    _backward((2, N, 3), io, "mixed", N % 2 == 1)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("gates", ["open", "strong", "stops", "shut"])
@pytest.mark.parametrize("N", [7, 150])
def test_backward_gates(cuda_device, io, gates, N):
    _backward((1, N, 5), io, gates, True)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("case", [(20, 70, 130), (1, 3000, 2), (7, 300, 259), (5, 700, 9)], ids=str)
def test_backward_shapes(cuda_device, io, case):
    _backward(case, io, "mixed", case[0] != 5)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_gradients_equal_differences(cuda_device, io):
    """Directional differences of the forward's own outputs, in float32 tensors of the
    same inputs: the loss moves by the gradient's product with the direction. The step
    of 2^-6 leaves a quadratic term, cancelled by the two sides, and a cubic one (the
    gates' exponentials) far below the bound."""
    q, k, v, g, do, S, dS = _draw(2, 90, 3, io, 21)
    dev = _dev(q, k, v, g, do, S, dS)
    grads = la.gated_attention_backward(*dev[:5], S_in=dev[5], dS_out=dev[6])
    r = torch.Generator().manual_seed(3)
    ins = [x.double() for x in (q, k, v, g, S)]

    def loss(xs):
        f = _dev(*[x.float() for x in xs])
        O, So = la.gated_attention(*f[:4], S_in=f[4], want_state=True)
        return float((O.double().cpu() * do.double()).sum() + (So.double().cpu() * dS.double()).sum())

    h = 2.0 ** -6
    for i in range(5):
        way = torch.randn(ins[i].shape, generator=r, dtype=torch.float64)
        lo, hi = list(ins), list(ins)
        lo[i], hi[i] = ins[i] - h * way, ins[i] + h * way
        step = (loss(hi) - loss(lo)) / (2 * h)
        want = float((grads[i].double().cpu() * way).sum())
        size = float((grads[i].double().cpu() * way).norm())
        assert abs(step - want) <= 2e-2 * size + 1e-3, (i, step, want, size)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("cuts", [(300, 1, 1, 5, 40), (8, 9, 330)], ids=str)
def test_pieces_equal_the_whole(cuda_device, io, cuts):
    """Prompt, then single tokens, the state updated in place: the oracle's outputs of
    the whole sequence."""
    B, N, H = 2, sum(cuts), 4
    q, k, v, g, _, S, _ = _draw(B, N, H, io, 33)
    state, outs, n = S.cuda(), [], 0
    for c in cuts:
        part = _dev(*(x[:, n:n + c] for x in (q, k, v, g)))
        O, same = la.gated_attention(*part, S_in=state, S_out=state)
        assert same is state
        outs.append(O)
        n += c
    O_ref, S_ref = orc.gated_attention(q, k, v, g, S)
    A, AS = orc.gated_magnitudes(q, k, v, g, S_in=S)
    _check("O", torch.cat(outs, 1), O_ref, A, _tol(io, N), HALF[io])
    _check("S", state, S_ref, AS, _tol(io, N), HALF["f32"])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("case", [(1, 2000, 3), (2, 1500, 40), (4, 600, 60), (1, 20, 4)], ids=str)
def test_without_the_last_state(cuda_device, io, case):
    q, k, v, g, _, S, _ = _draw(*case, io, 6)
    O = la.gated_attention(*_dev(q, k, v, g), S_in=S.cuda(), scale=0.3)
    ref, _ = orc.gated_attention(q, k, v, g, S, 0.3)
    A, _ = orc.gated_magnitudes(q, k, v, g, S_in=S, scale=0.3)
    _check("O", O, ref, A, _tol(io, case[1]), HALF[io])


@pytest.mark.parametrize("case", [(1, 2000, 3), (4, 600, 60), (2, 3, 4), (1, 20, 4), (16, 50, 90)], ids=str)
def test_state_in_place(cuda_device, case):
    """Segments, a CTA per row, single tokens, one block, a walk per head."""
    q, k, v, g, _, S, _ = _draw(*case, "bf16", 4)
    dev = _dev(q, k, v, g)
    state = S.cuda()
    O1, S1 = la.gated_attention(*dev, S_in=state, want_state=True)
    O2, S2 = la.gated_attention(*dev, S_in=state, S_out=state)
    assert S2 is state and torch.equal(O1, O2) and torch.equal(S1, S2)


def test_empty_sequence_passes_the_state_on(cuda_device):
    e = torch.empty((2, 0, 3, D), dtype=torch.bfloat16, device="cuda")
    g = torch.empty((2, 0, 3), device="cuda")
    S = torch.randn((2, 3, D, D), device="cuda")
    O, So = la.gated_attention(e, e, e, g, S_in=S, want_state=True)
    assert O.shape == e.shape and torch.equal(So, S)
    assert not la.gated_attention(e, e, e, g, want_state=True)[1].any()
    *_, dS = la.gated_attention_backward(e, e, e, g, e, S_in=S, dS_out=S)
    assert torch.equal(dS, S)


def test_same_bits_on_any_stream_and_in_a_graph(cuda_device):
    q, k, v, g, do, S, dS = _dev(*_draw(2, 700, 5, "bf16", 8))
    fwd = lambda: la.gated_attention(q, k, v, g, S_in=S, want_state=True)  # noqa: E731
    bwd = lambda: la.gated_attention_backward(q, k, v, g, do, S_in=S, dS_out=dS)  # noqa: E731
    want = [*fwd(), *bwd()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = [*fwd(), *bwd()]
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = [*fwd(), *bwd()]
    keep = q.clone()
    q.mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(held[0], want[0])
    q.copy_(keep)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, held))


def test_later_tokens_and_other_rows_do_not_reach_earlier_ones(cuda_device):
    q, k, v, g, *_ = _draw(2, 100, 2, "bf16", 12)
    O1 = la.gated_attention(*_dev(q, k, v, g))
    k2, v2, g2 = k.clone(), v.clone(), g.clone()
    k2[:, 51:], v2[:, 51:], g2[:, 51:] = 3.0, -2.0, -0.01
    O2 = la.gated_attention(*_dev(q, k2, v2, g2))
    assert torch.equal(O1[:, :51], O2[:, :51]) and not torch.equal(O1[:, 51:], O2[:, 51:])
    # what follows the last token in memory stays as it was
    B, N, H = 1, 37, 2
    buf = torch.full((B * N * H * D + 4096,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:B * N * H * D].view(B, N, H, D)
    dev = _dev(*(x[:1, :N].contiguous() for x in (q, k, v, g)))
    shape = la.make_gated_shape(B, N, H)
    ws = torch.empty(la.la_gated_workspace_bytes(shape), dtype=torch.uint8, device="cuda")
    la.la_gated_attention(shape, *dev, None, None, out, ws)
    assert torch.equal(out, la.gated_attention(*dev)) and bool((buf[B * N * H * D:] == 7.0).all())


def test_stream_argument(cuda_device):
    """Calls on a stream that is not the current one, its memory its own: many calls whose
    results are dropped at once, and one that is kept."""
    q, k, v, g, do, S, dS = _dev(*_draw(2, 700, 5, "bf16", 8))
    want = [*la.gated_attention(q, k, v, g, S_in=S, want_state=True),
            *la.gated_attention_backward(q, k, v, g, do, S_in=S, dS_out=dS)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        for _ in range(5):
            la.gated_attention_backward(q, k, v, g, do, stream=stream)
            torch.full((1 << 22,), 7.0, device="cuda")  # the current stream's allocations meanwhile
        got = [*la.gated_attention(q, k, v, g, S_in=S, want_state=True, stream=stream),
               *la.gated_attention_backward(q, k, v, g, do, S_in=S, dS_out=dS, stream=stream)]
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.slow
def test_tensors_past_32_bit_offsets(cuda_device):
    """2.2e9 elements a tensor. A stop a few tokens before the end leaves the oracle a short
    sequence; the last heads are the farthest in memory."""
    B, N, H, tail = 1, 67200, 1024, 40
    if torch.cuda.get_device_properties(0).total_memory < 100 << 30:
        pytest.skip("needs 60 GB")
    r = torch.Generator(device="cuda").manual_seed(5)
    q, k, v, do = (torch.randn((B, N, H, D), generator=r, device="cuda", dtype=torch.bfloat16) for _ in range(4))
    g = -0.1 * torch.rand((B, N, H), generator=r, device="cuda")
    g[:, N - tail] = -float("inf")
    cut = [x[:, N - tail:, H - 3:].contiguous().cpu() for x in (q, k, v, g, do)]
    O, S = la.gated_attention(q, k, v, g, scale=0.3, want_state=True)
    ref, S_ref = orc.gated_attention(*cut[:4], scale=0.3)
    A, AS = orc.gated_magnitudes(*cut[:4], scale=0.3)
    _check("O", O[:, N - tail:, H - 3:], ref, A, _tol("bf16", tail), HALF["bf16"])
    _check("S", S[:, H - 3:], S_ref, AS, _tol("bf16", tail), HALF["f32"])
    del O, S
    grads = la.gated_attention_backward(q, k, v, g, do, scale=0.3)
    refs = orc.gated_attention_backward(*cut, scale=0.3)
    mags = orc.gated_magnitudes(*cut, scale=0.3)
    for i, name in enumerate(("dQ", "dK", "dV", "dG")):
        _check(name, grads[i][:, N - tail:, H - 3:], refs[i], mags[i], 2 * _tol("bf16", tail),
               HALF["bf16" if i < 3 else "f32"])
    del grads, v, do, g
    Qo, Ko = la.rotary(q, k, out=(q, k))
    for x, src in ((Qo, cut[0]), (Ko, cut[1])):
        want = orc.rotary(src, np.arange(N - tail, N), D)
        err = np.abs(orc.to_f64(x[:, N - tail:, H - 3:].cpu()) - want)
        assert (err <= HALF["bf16"] * np.abs(want) + 2.0 ** -20 * 8).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("N,bad,stop", [(3000, 700, 740), (200, 5, 40), (300, 0, 64)])
def test_a_stop_ends_what_is_not_finite(cuda_device, io, N, bad, stop):
    """NaN and infinity in one sequence reach neither the tokens before their block nor, 32
    tokens after the next one's start, the sequence packed behind it, whichever way the row
    is cut into segments."""
    q, k, v, g, do, _, _ = _draw(1, N, 3, io, 17, carry=False)
    g[:, stop] = -float("inf")
    v[:, bad, 1] = float("nan")
    k[:, bad, 2] = float("inf")
    O, S = la.gated_attention(*_dev(q, k, v, g), want_state=True)
    tail = [x[:, stop:] for x in (q, k, v, g)]
    ref, S_ref = orc.gated_attention(*tail)
    A, AS = orc.gated_magnitudes(*tail)
    _check("O", O[:, stop + 32:], ref[:, 32:], A[:, 32:], _tol(io, N), HALF[io])
    _check("S", S, S_ref, AS, _tol(io, N), HALF["f32"])
    first = bad // 16 * 16
    ref, _ = orc.gated_attention(*(x[:, :first] for x in (q, k, v, g)))
    A, _ = orc.gated_magnitudes(*(x[:, :first] for x in (q, k, v, g)))
    _check("O before", O[:, :first], ref, A, _tol(io, N), HALF[io])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("N,bad,stop", [(3000, 705, 710), (200, 33, 36), (100, 70, 72), (24, 17, 18), (3000, 710, 705),
                                        (200, 36, 33), (100, 72, 72), (24, 9, 3)])
def test_a_stop_holds_inside_a_step(cuda_device, io, N, bad, stop):
    """What is not finite (k, v or a gate, one head each) and a stop within 16 tokens of each
    other: neither it nor what it spoils passes the stop, forwards or backwards, in the
    outputs, the states or the gradients. Long rows in segments, a CTA per row, one walk."""
    q, k, v, g, do, S0, dS = _draw(1, N, 4, io, 19)
    clean = [x.clone() for x in (q, k, v, g, do)]
    g[:, stop] = clean[3][:, stop] = -float("inf")
    if bad != stop:
        g[:, bad, 0] = float("nan")
    v[:, bad, 1] = float("nan")
    k[:, bad, 2] = float("inf")
    do[:, bad, 3] = float("nan")
    tol = _tol(io, N)
    after = bad < stop
    part = slice(stop, N) if after else slice(0, stop)
    cut = [x[:, part] for x in clean]
    first, last = (None, dS) if after else (S0, None)
    ref, S_ref = orc.gated_attention(*cut[:4], first)
    A, AS = orc.gated_magnitudes(*cut[:4], S_in=first)
    dev = _dev(q, k, v, g)
    O, S = la.gated_attention(*dev, S_in=S0.cuda(), want_state=True)
    _check("O", O[:, part], ref, A, tol, HALF[io])
    _check("O alone", la.gated_attention(*dev, S_in=S0.cuda())[:, part], ref, A, tol, HALF[io])
    if after:
        _check("S", S, S_ref, AS, tol, HALF["f32"])
    grads = la.gated_attention_backward(*dev, do.cuda(), S_in=S0.cuda(), dS_out=dS.cuda())
    refs = orc.gated_attention_backward(*cut, first, last)
    mags = orc.gated_magnitudes(*cut, first, last)
    for i, name in enumerate(("dQ", "dK", "dV", "dG")):
        _check(name, grads[i][:, part], refs[i], mags[i], 2 * tol, HALF[io] if i < 3 else HALF["f32"])
    if not after:
        _check("dS_in", grads[4], refs[4], mags[4], tol, HALF["f32"])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("gates", ["mixed", "packed"])
@pytest.mark.parametrize("B,N,H", [(1, 3000, 6), (1, 600, 920), (2, 700, 5)], ids=str)
def test_gate_gradients_window_by_window(cuda_device, io, gates, B, N, H):
    """dG in the 2-norm of every head's windows of 256 tokens: the sums between two anchors, their
    carry from one segment to the next, stops between them. B H = 920 rows are not cut, so a
    segment holds two inner anchors. Bound 2^-15: a row product carries 2^-19 of its terms (two
    chains of some 16 float32 sums), and the up to 256 of them in a gate's gradient add up like
    independent errors, 2^4 of that; gradient and row products are of one size in this draw.
    All zeros, or a window whose carry is lost, are off by more than 2^-4 (test_gated_cpu.py)."""
    q, k, v, g, do, S, dS = _draw(B, N, H, io, 23)
    if gates == "packed":
        g[torch.rand((B, N), generator=torch.Generator().manual_seed(2)) < 0.01] = -float("inf")
    dG = la.gated_attention_backward(*_dev(q, k, v, g, do), S_in=S.cuda(), dS_out=dS.cuda(), scale=0.4)[3]
    some = [0, H // 2, H - 1]  # heads are independent
    cut = [x[:, :, some] for x in (q, k, v, g, do)] + [x[:, some] for x in (S, dS)]
    ref = orc.gated_attention_backward(*cut, 0.4)[3]
    err = orc.gated_window_errors(dG[:, :, some].cpu(), ref)
    assert err.max() <= 2.0 ** -15, err.max()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,H,seed", [(1, 61, 3, 1), (2, 333, 5, 2), (3, 1000, 2, 3), (1, 40, 900, 4), (1, 700, 70, 5)])
def test_packed_sequences_are_apart(cuda_device, io, B, N, H, seed):
    """Rows packed from sequences of 1 to some 40 tokens, with numbers that are not finite strewn
    over them: every sequence without one, and the states at its ends, is what it would be alone."""
    q, k, v, g, do, S0, dS = _draw(B, N, H, io, seed)
    r = torch.Generator().manual_seed(seed + 100)
    stop = torch.rand((B, N, H), generator=r) < 0.08
    bad = torch.rand((B, N, H), generator=r) < 0.02
    kind = torch.randint(0, 5, (B, N, H), generator=r)
    g[stop] = -float("inf")
    clean = [x.clone() for x in (q, k, v, g, do)]
    for i, x in enumerate((q, k, v, do)):
        x[..., i][bad & (kind == i)] = float("nan") if seed % 2 else float("inf")
        clean[i if i < 3 else 4][bad & (kind == i)] = 0
    g[bad & (kind == 4) & ~stop] = float("nan")
    number = stop.long().cumsum(1)                              # of each token's sequence in its row
    spoiled = torch.zeros((B, N + 1, H), dtype=torch.long).scatter_add_(1, number, bad.long()) > 0
    fine = ~spoiled.gather(1, number)
    assert 0.2 < fine.float().mean() < 0.95
    first, last = ~spoiled[:, 0], fine[:, -1]                   # the states' sequences, [B, H]
    tol = _tol(io, N)

    def check(name, got, ref, mag, tol, half, ok):
        got, ok = orc.to_f64(got.cpu()), ok.numpy()
        err, bound = np.abs(got - ref)[ok], (half * np.abs(ref) + tol * mag + 1e-36)[ok]
        assert np.isfinite(got[ok]).all() and (err <= bound).all(), name

    dev = _dev(q, k, v, g)
    O, S = la.gated_attention(*dev, S_in=S0.cuda(), want_state=True)
    ref, S_ref = orc.gated_attention(*clean[:4], S0)
    A, AS = orc.gated_magnitudes(*clean[:4], S_in=S0)
    check("O", O, ref, A, tol, HALF[io], fine)
    check("S", S, S_ref, AS, tol, HALF["f32"], last)
    check("O alone", la.gated_attention(*dev, S_in=S0.cuda()), ref, A, tol, HALF[io], fine)
    got = la.gated_attention_backward(*dev, do.cuda(), S_in=S0.cuda(), dS_out=dS.cuda())
    refs = orc.gated_attention_backward(*clean, S0, dS)
    mags = orc.gated_magnitudes(*clean, S0, dS)
    for i, name in enumerate(("dQ", "dK", "dV", "dG")):
        check(name, got[i], refs[i], mags[i], 2 * tol, HALF[io] if i < 3 else HALF["f32"], fine)
    check("dS_in", got[4], refs[4], mags[4], tol, HALF["f32"], first)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 3, 9, 16])
def test_what_passes_strong_gates_keeps_its_bits(cuda_device, io, N):
    """Without keys the state is a product of decays times the one before. Bound 2^-20 relative: an
    exponential of 2^-22 and a few float32 roundings, for each of up to three tokens of their own or
    for a block of 16; a rounded exponent of 2^7 alone would be off by 2^-18. It holds for normal
    numbers: below 2^-126 a step of float32 is 2^-149, whatever the number. Backwards the same for
    the gradient of the first state."""
    r = torch.Generator().manual_seed(4)
    B, H = 4, 60
    q, do = (torch.randn((B, N, H, D), generator=r).to(torch.bfloat16 if io == "bf16" else torch.float32) for _ in range(2))
    zero = torch.zeros_like(q)
    g = -80 * torch.rand((B, N, H), generator=r) / max(1, N / 2)
    S, dS = (torch.randn((B, H, D, D), generator=r) for _ in range(2))
    decay = np.exp(orc.to_f64(g).sum(1))[..., None, None]
    got = la.gated_attention(*_dev(q, zero, zero, g), S_in=S.cuda(), want_state=True)[1]
    want = decay * orc.to_f64(S)
    normal = np.abs(want) > 2.0 ** -122
    assert normal.mean() > 0.4 and (np.abs(orc.to_f64(got.cpu()) - want)[normal] <= 2.0 ** -20 * np.abs(want)[normal]).all()
    got = la.gated_attention_backward(*_dev(zero, zero, zero, g, do), S_in=S.cuda(), dS_out=dS.cuda())[4]
    want = decay * orc.to_f64(dS)
    normal = np.abs(want) > 2.0 ** -122
    assert normal.mean() > 0.4 and (np.abs(orc.to_f64(got.cpu()) - want)[normal] <= 2.0 ** -20 * np.abs(want)[normal]).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,H", [(2, 3, 3), (2, 40, 3), (1, 200, 60), (1, 1000, 2), (1, 60, 900)], ids=str)
def test_states_that_are_not_finite_end_at_a_stop(cuda_device, io, B, N, H):
    """A first state of NaN reaches no token from a stop on; backwards, the gradient of a last
    state reaches none before it. Single tokens, a walk, a CTA per row, segments, uncut rows."""
    q, k, v, g, do, S0, dS = _draw(B, N, H, io, 29)
    stop = N // 2
    g[:, stop] = -float("inf")
    nan = torch.full_like(S0, float("nan"))
    dev = _dev(q, k, v, g)
    late = [x[:, stop:] for x in (q, k, v, g, do)]
    O, S = la.gated_attention(*dev, S_in=nan.cuda(), want_state=True)
    ref, S_ref = orc.gated_attention(*late[:4])
    A, AS = orc.gated_magnitudes(*late[:4])
    tol = _tol(io, N)
    _check("O", O[:, stop:], ref, A, tol, HALF[io])
    _check("S", S, S_ref, AS, tol, HALF["f32"])
    for states, part in ((dict(S_in=nan, dS_out=dS), slice(stop, N)), (dict(S_in=S0, dS_out=nan), slice(0, stop))):
        got = la.gated_attention_backward(*dev, do.cuda(), **{n: x.cuda() for n, x in states.items()})
        cut = [x[:, part] for x in (q, k, v, g, do)]
        ends = (None, dS) if part.start else (S0, None)
        refs, mags = orc.gated_attention_backward(*cut, *ends), orc.gated_magnitudes(*cut, *ends)
        for i, name in enumerate(("dQ", "dK", "dV", "dG")):
            _check(name, got[i][:, part], refs[i], mags[i], 2 * tol, HALF[io] if i < 3 else HALF["f32"])
        if not part.start:
            _check("dS_in", got[4], refs[4], mags[4], tol, HALF["f32"])
