"""GPU parity of rotary positions against the float64 oracle.

Tolerance per number: half a step of the output's type, and 2^-22 (float32 cosine, sine and
two products) plus |position| 2^-51 (the angle is a float64) of m (|a| + |b|), the two numbers
of the pair. Passed dimensions keep their bits.
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


def _check(got, x, positions, rot, layout, io, mscale=1.0, **kw):
    ref = orc.rotary(x, positions, rot, layout, mscale=mscale, **kw)
    assert torch.equal(got[..., rot:].cpu(), x[..., rot:])
    k = np.arange(rot // 2)
    i, j = (2 * k, 2 * k + 1) if layout == "interleaved" else (k, k + rot // 2)
    a = np.abs(orc.to_f64(x))
    size = np.zeros_like(a)
    size[..., i] = size[..., j] = a[..., i] + a[..., j]
    pos = np.abs(np.asarray(positions, dtype=np.float64))
    pos = pos[..., None, None] if pos.ndim == 2 else pos[None, :, None, None]
    err = np.abs(orc.to_f64(got.cpu()) - ref)
    bound = HALF[io] * np.abs(ref) + (2.0 ** -22 + pos * 2.0 ** -51) * abs(mscale) * size
    assert (err <= bound).all(), (err / np.maximum(bound, 1e-30)).max()


def _draw(shape, io, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(DT[io])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot", [(32, 32), (32, 20), (32, 2), (8, 8), (8, 6), (64, 48), (128, 96), (256, 256),
                                   (40, 32), (32, 0)])
def test_layouts_and_widths(cuda_device, io, layout, D, rot):
    q, k = _draw((2, 9, 3, D), io, 1), _draw((2, 9, 2, D), io, 2)
    pos = torch.randint(0, 50000, (2, 9), dtype=torch.int32)
    Qo, Ko = la.rotary(q.cuda(), k.cuda(), positions=pos.cuda(), rot=rot, layout=layout)
    _check(Qo, q, pos.numpy(), rot, layout, io)
    _check(Ko, k, pos.numpy(), rot, layout, io)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("scaling", [("linear", 4.0), ("base", 8.0), ("parts", 16.0, 4096, 1.0, 32.0)], ids=str)
def test_scalings_far_positions_and_inverse(cuda_device, layout, scaling):
    q = _draw((1, 6, 2, 64), "f32", 3)
    pos = torch.tensor([0, 1, 131071, 10 ** 6, 2 ** 31 - 1, -5], dtype=torch.int32)
    for inverse in (False, True):
        Qo, none = la.rotary(q.cuda(), positions=pos.cuda(), layout=layout, scaling=scaling, mscale=1.25,
                             inverse=inverse)
        assert none is None
        _check(Qo, q, pos.numpy(), 64, layout, "f32", mscale=1.25, scaling=scaling, inverse=inverse)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,H,Hk", [(1, 1, 1, 0), (1, 1, 70, 1), (64, 1, 16, 16), (1, 2049, 5, 5), (3, 700, 70, 1),
                                      (2, 1, 3, 0)])
def test_shapes_without_positions(cuda_device, io, B, N, H, Hk):
    q, k = _draw((B, N, H, 32), io, 5), _draw((B, N, Hk, 32), io, 6) if Hk else None
    Qo, Ko = la.rotary(q.cuda(), None if k is None else k.cuda(), offset=77)
    pos = 77 + np.arange(N)
    _check(Qo, q, pos, 32, "half", io)
    if Hk:
        _check(Ko, k, pos, 32, "half", io)


@pytest.mark.parametrize("layout,rot", [("half", 32), ("half", 12), ("interleaved", 22)])
def test_in_place_and_neighbours(cuda_device, layout, rot):
    q, k = _draw((2, 33, 3, 32), "bf16", 7).cuda(), _draw((2, 33, 1, 32), "bf16", 8).cuda()
    want = la.rotary(q, k, rot=rot, layout=layout)
    buf = torch.full((q.numel() + 512,), 3.0, dtype=torch.bfloat16, device="cuda")
    mine = buf[256:256 + q.numel()].view(q.shape)
    mine.copy_(q)
    got = la.rotary(mine, k, rot=rot, layout=layout, out=(mine, k))
    assert got[0] is mine and got[1] is k
    assert torch.equal(mine, want[0]) and torch.equal(k, want[1])
    assert bool((buf[:256] == 3).all()) and bool((buf[256 + q.numel():] == 3).all())


def test_inverse_is_the_gradient(cuda_device):
    """<R x, y> = <x, R^T y>: sums of 2 x 9216 float32 numbers whose own errors are 2^-22."""
    x, y = _draw((1, 96, 3, 32), "f32", 9).cuda(), _draw((1, 96, 3, 32), "f32", 10).cuda()
    for layout, rot in (("half", 32), ("interleaved", 18), ("half", 22)):
        kw = dict(rot=rot, layout=layout, mscale=0.7)
        a = (la.rotary(x, **kw)[0].double() * y.double()).sum()
        b = (x.double() * la.rotary(y, inverse=True, **kw)[0].double()).sum()
        size = (x.double().norm() * y.double().norm()).item()
        assert abs((a - b).item()) <= 2.0 ** -21 * size


def test_empty_and_special_numbers(cuda_device):
    e = torch.empty((2, 0, 3, 32), device="cuda")
    assert la.rotary(e)[0].shape == e.shape
    x = torch.zeros((1, 2, 1, 32), device="cuda")
    x[..., 24:] = float("inf")          # passed dimensions keep infinities as they are
    x[..., 25] = float("nan")
    for layout in ("half", "interleaved"):
        y, _ = la.rotary(x, rot=24, layout=layout, offset=3)
        assert not y[..., :24].any() and bool(y[..., 24].isinf().all()) and bool(y[..., 25].isnan().all())
    x = torch.zeros((1, 2, 1, 32), device="cuda")
    x[..., 22:] = float("inf")          # 22 is inside a 16-byte piece
    y, _ = la.rotary(x, rot=22, layout="interleaved", offset=3)
    assert not y[..., :22].any() and bool(y[..., 22:].isinf().all())


def test_in_a_graph_and_on_another_stream(cuda_device):
    q, k = _draw((1, 40, 3, 32), "bf16", 11).cuda(), _draw((1, 40, 2, 32), "bf16", 12).cuda()
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    want = la.rotary(q, k, positions=pos)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = la.rotary(q, k, positions=pos)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = la.rotary(q, k, positions=pos)
    pos += 1000
    graph.replay()
    torch.cuda.synchronize()
    want = la.rotary(q, k, positions=pos)
    assert all(torch.equal(a, b) for a, b in zip(held, want))


@pytest.mark.parametrize("layout,rot", [("interleaved", 22), ("interleaved", 2), ("interleaved", 24), ("half", 22),
                                        ("half", 16)])
def test_passed_dimensions_keep_their_bits(cuda_device, layout, rot):
    """Every 16-bit pattern, the many NaNs among them, in the dimensions that pass; `rot` = 22 and
    2 end inside a 16-byte piece."""
    bits = torch.arange(-2 ** 15, 2 ** 15, dtype=torch.int32).to(torch.int16)
    x = bits.reshape(1, -1, 1, 1).expand(1, -1, 2, 32).contiguous().view(torch.bfloat16).cuda()
    x[..., :rot] = 1.0
    y, _ = la.rotary(x, rot=rot, layout=layout)
    assert torch.equal(y.view(torch.int16)[..., rot:], x.view(torch.int16)[..., rot:])
