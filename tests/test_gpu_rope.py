"""tm_rope against its definition in 64 bits (angles as exact fractions of a turn).

Tolerance: sine and cosine are off by at most 2.1e-7 (the argument's rounding
pi 2^-25, one place of sincospif, the gain's rounding), the two products and the
sum add 2^-23 of |a| + |b|: 1.5 * 2^-22 of |gain| (|a| + |b|), and one rounding.
"""
import numpy as np
import pytest
import torch

import block_ref as ref
from masking_tm_affine_gb300 import tm

pytestmark = pytest.mark.gpu


def dev_turns(t):
    return torch.from_numpy(np.ctypeslib.as_array(t).view(np.int64).copy()).cuda()


def bound(x, rot, gain, inter):
    a = np.abs(x).copy()
    if rot:
        i0, i1 = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if inter else (np.arange(rot // 2), np.arange(rot // 2, rot))
        s = (a[..., i0] + a[..., i1]) * abs(gain) * 1.5 * 2.0 ** -22
        a[:] = 0
        a[..., i0] = s
        a[..., i1] = s
    else:
        a[:] = 0
    return a


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,H,D,rot", [(1, 1, 2, 2), (1, 40, 128, 128), (5, 3, 80, 40), (70, 2, 96, 24), (3, 7, 10, 6),
                                       (9, 5, 64, 0), (2500, 3, 64, 64), (700, 40, 128, 64), (2, 1, 1000, 998)])
def test_rope(cuda, kind, inter, T, H, D, rot):
    t = ref.TYPES[kind]
    rng = np.random.default_rng(T + D + rot)
    turns = tm.tm_rope_turns(rot, 10000.0) if rot else tm.tm_rope_turns(2, 10000.0)
    pos = rng.integers(-(1 << 20), 1 << 40, T)
    pos[0] = 0
    x = torch.from_numpy(rng.standard_normal((T, H, D))).to(t).cuda()
    P, TU = torch.from_numpy(pos).cuda(), dev_turns(turns)
    want = ref.rope(ref.f64(x), pos, turns, rot, 1.25, inter)
    y = torch.full_like(x, 9.0)
    flags = tm.TM_ROPE_INTERLEAVED if inter else 0
    tm.tm_rope(x, H * D, D, y, H * D, D, P, TU, T, H, D, rot, 1.25, ref.CODE[kind], flags)
    tm.tm_check()
    r, a = ref.half_step(t)
    lim = bound(ref.f64(x), rot, 1.25, inter) + r * np.abs(want) * (1 + 1e-5) + a
    assert np.all(np.abs(ref.f64(y) - want) <= lim)
    # in place, and back
    z = x.clone()
    tm.tm_rope(z, H * D, D, z, H * D, D, P, TU, T, H, D, rot, 1.25, ref.CODE[kind], flags)
    assert torch.equal(z, y)
    back = torch.empty_like(x)
    tm.tm_rope(x, H * D, D, back, H * D, D, P, TU, T, H, D, rot, 1.25, ref.CODE[kind], flags | tm.TM_ROPE_INVERSE)
    tm.tm_check()
    want = ref.rope(ref.f64(x), pos, turns, rot, 1.25, inter, True)
    assert np.all(np.abs(ref.f64(back) - want) <= bound(ref.f64(x), rot, 1.25, inter) + r * np.abs(want) * (1 + 1e-5) + a)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_gradient_against_differences(cuda, inter):
    # <rope(x), g> is linear in x: its gradient is the inverse call on g, its differences exact up to rounding
    rng = np.random.default_rng(3)
    T, H, D, rot = 4, 2, 16, 12
    turns = tm.tm_rope_turns(rot, 500000.0)
    pos = np.array([0, 1, 777, 100000])
    g = torch.from_numpy(rng.standard_normal((T, H, D))).float().cuda()
    dx = torch.empty_like(g)
    tm.tm_rope(g, H * D, D, dx, H * D, D, torch.from_numpy(pos).cuda(), dev_turns(turns), T, H, D, rot, 0.75, tm.TM_F32,
               (tm.TM_ROPE_INTERLEAVED if inter else 0) | tm.TM_ROPE_INVERSE)
    tm.tm_check()
    f = lambda x: (ref.rope(x, pos, turns, rot, 0.75, inter) * ref.f64(g)).sum()  # noqa: E731
    x = rng.standard_normal((T, H, D))
    for i in range(0, x.size, 5):
        e = np.zeros(x.size)
        e[i] = 1.0
        e = e.reshape(x.shape)
        assert abs((f(x + e) - f(x - e)) / 2 - ref.f64(dx).reshape(-1)[i]) < 1e-5


@pytest.mark.parametrize("shift", [0, 1])
def test_rope_strides_and_gaps(cuda, shift):
    # the queries and keys of a fused projection, rotated in place; values and gaps untouched
    T, Hq, Hkv, D, rot, ld = 65, 6, 2, 64, 32, 10 * 64 + 8
    rng = np.random.default_rng(4)
    buf = torch.from_numpy(rng.standard_normal(T * ld + 64)).to(torch.bfloat16).cuda()
    ref0 = buf.clone()
    x = buf[shift:][:T * ld].view(T, ld)
    turns = tm.tm_rope_turns(rot, 10000.0)
    pos = np.arange(T) + 100
    before = x[:, :8 * D].reshape(T, 8, D).clone()
    tm.tm_rope(x, ld, D, x, ld, D, torch.from_numpy(pos).cuda(), dev_turns(turns), T, Hq + Hkv, D, rot, 1.0, tm.TM_BF16)
    tm.tm_check()
    want = ref.rope(ref.f64(before), pos, turns, rot)
    got = ref.f64(x[:, :8 * D].reshape(T, 8, D))
    assert np.all(np.abs(got - want) <= bound(ref.f64(before), rot, 1.0, False) + 2.0 ** -8 * np.abs(want) * 1.001 + 1e-38)
    x[:, :8 * D] = ref0[shift:][:T * ld].view(T, ld)[:, :8 * D]
    assert torch.equal(buf, ref0)
