"""Rotary positions without a GPU: the oracle's pins and the refusals."""
import ctypes
import math

import numpy as np
import pytest
import torch

import linear_attention_diffusion_b200 as la
import oracle as orc

FAKE = 0x7f0000000000
MB = 1 << 20


def test_oracle_keeps_norms_and_relative_positions():
    r = np.random.default_rng(1)
    q, k = r.standard_normal((2, 1, 9, 2, 16))
    for layout in ("half", "interleaved"):
        turn = lambda x, p: orc.rotary(x, p, 16, layout)  # noqa: E731
        p = np.arange(9)
        assert np.allclose((turn(q, p) ** 2).sum(-1), (q ** 2).sum(-1))
        a = np.einsum("bnhd,bmhd->bhnm", turn(q, p), turn(k, p))
        b = np.einsum("bnhd,bmhd->bhnm", turn(q, p + 77), turn(k, p + 77))
        assert np.allclose(a, b)  # only differences of positions count
        back = orc.rotary(turn(q, p), p, 16, layout, inverse=True)
        assert np.allclose(back, q)


def test_oracle_rates():
    assert np.allclose(orc.rotary_rates(8), [1, 0.1, 0.01, 0.001])
    assert np.allclose(orc.rotary_rates(8, scaling=("linear", 4.0)), orc.rotary_rates(8) / 4)
    # the base is raised so that the slowest pair turns exactly `factor` times slower
    assert np.allclose(orc.rotary_rates(8, scaling=("base", 4.0))[[0, 3]], [1, 0.001 / 4])
    parts = orc.rotary_rates(64, scaling=("parts", 8.0, 4096, 1.0, 32.0))
    plain = orc.rotary_rates(64)
    turns = 4096 * plain / (2 * math.pi)
    assert np.allclose(parts[turns > 32], plain[turns > 32])
    assert np.allclose(parts[turns < 1], plain[turns < 1] / 8)
    assert ((parts <= plain) & (parts >= plain / 8)).all()


def test_shape_struct_matches_header_layout():
    assert ctypes.sizeof(la.LaRotaryShape) == 96 and la.LaRotaryShape.base.offset == 48


def _call(q=FAKE, k=FAKE + MB, pos=FAKE + 2 * MB, qo=FAKE + 3 * MB, ko=FAKE + 4 * MB, shape=None, **set_):
    s = shape if shape is not None else la.make_rotary_shape(2, 5, 4, 2, 32)
    for name, x in set_.items():
        setattr(s, name, x)
    return la._lib.la_rotary(ctypes.byref(s), q, k, pos, qo, ko, None)


def test_refusals():
    inv, uns = la.LA_ERR_INVALID_ARG, la.LA_ERR_UNSUPPORTED
    for bad in (dict(B=-1), dict(Hk=-2), dict(rot=7), dict(rot=34), dict(rot=-2), dict(io_dtype=5), dict(half=2),
                dict(inverse=3), dict(pos_rows=-1), dict(scaling=4), dict(pos_offset=-1),
                dict(pos_offset=0x7fffffff), dict(base=1.0), dict(base=float("inf")),
                dict(mscale=float("nan")), dict(scaling=1, factor=0.5), dict(scaling=3, fast=0.0),
                dict(scaling=3, original_length=0.0), dict(scaling=2, factor=float("nan"))):
        assert _call(**bad) == inv, bad
    for bad in (dict(D=36, rot=8), dict(D=264), dict(D=0, rot=0), dict(H=1 << 20), dict(B=1 << 20, N=1 << 14)):
        assert _call(**bad) == uns, bad
    for name in ("q", "k", "qo", "ko"):
        assert _call(**{name: None}) == inv and _call(**{name: FAKE + 9 * MB + 8}) == inv
    assert _call(pos=FAKE + 2) == inv
    assert _call(qo=FAKE + 64) == inv                # partly over Q
    assert _call(qo=FAKE + MB) == inv                # over K
    assert _call(qo=FAKE, ko=FAKE) == inv            # over each other
    assert _call(qo=FAKE + 2 * MB) == inv            # over the positions


def test_binding_refuses_what_does_not_fit():
    q = torch.zeros(1, 5, 2, 32)
    with pytest.raises(ValueError):  # not on a GPU
        la.rotary(q)
    for bad in (dict(K=torch.zeros(1, 4, 2, 32)), dict(K=torch.zeros(1, 5, 2, 32).bfloat16()),
                dict(positions=torch.arange(5)), dict(positions=torch.arange(4, dtype=torch.int32)),
                dict(positions=torch.zeros(2, 5, dtype=torch.int32)), dict(scaling=("parts", 2.0)),
                dict(out=(torch.zeros(1, 5, 3, 32), None))):
        with pytest.raises(ValueError):
            la.rotary(q, **bad)
    for bad in (dict(layout="third"), dict(scaling=("cubic", 2.0))):
        with pytest.raises(KeyError):
            la.rotary(q, **bad)


def test_sizes_past_32_bits_are_refused():
    """A C int would keep their low 32 bits: 2^32 + 5 tokens would be 5."""
    big = 2 ** 32 + 5
    for bad in (dict(offset=big), dict(rot=2 ** 32 + 32), dict(offset=-big)):
        with pytest.raises(ValueError, match="32 bits"):
            la.make_rotary_shape(1, 4, 2, 2, 32, **bad)
    for make, args in ((la.make_rotary_shape, (1, big, 2, 2, 32)), (la.make_gated_shape, (1, big, 2)),
                       (la.make_gated_shape, (big, 1, 2)), (la.make_norm_shape, (1, big, 64)),
                       (la.make_norm_shape, (1, 1, big))):
        with pytest.raises(ValueError, match="32 bits"):
            make(*args)
    f, e = torch.float32, torch.empty
    with pytest.raises(ValueError, match="32 bits"):
        la.gated_attention(*[e((1, big, 0, 32), dtype=f)] * 3, e((1, big, 0), dtype=f))
    with pytest.raises(ValueError, match="32 bits"):
        la.rotary(e((1, big, 0, 32), dtype=f))
    with pytest.raises(ValueError, match="32 bits"):
        la.rotary(e((1, 2, 2, 32), dtype=f), offset=big)
    with pytest.raises(ValueError, match="32 bits"):
        la.gate_residual_norm(e((0, big, 64), dtype=f))
