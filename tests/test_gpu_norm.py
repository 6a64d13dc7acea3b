"""tm_rmsnorm and tm_rmsnorm_bwd against their definitions in 64 bits.

Tolerances.  A row's sum of squares is added in fp32 by lanes of at most 64
terms and then along a tree and at most 32 warps: below 112 roundings of 2^-24,
halved by the root; rsqrtf is good to 2 places, the two products and the
addition add three roundings: y is within 64 * 2^-24 of itself, and one rounding
to its type.  An e4m3 code is one more rounding: 2^-4 of the value, or half the
smallest step (2^-10 in units of the scale).  The gradient's row mean has the
same 112 roundings of the sum of magnitudes; a weight's gradient is a sum over
the rows, at most one rounding each and 128 along the joins.
"""
import numpy as np
import pytest
import torch

import block_ref as ref
from masking_tm_affine_gb300 import tm

pytestmark = pytest.mark.gpu
U = ref.U
EPS = 1e-5


def rows(rng, M, ld, t, scale=1.0, fill=float("nan")):
    """[M, ld] on the device; what lies past N in a row is the caller's business."""
    return torch.from_numpy(rng.standard_normal((M, ld)) * scale).to(t).cuda()


def close(got, want, rel, t, extra=0.0):
    r, a = ref.half_step(t)
    bound = (rel + r * (1 + 2 * rel)) * np.abs(want) + a + extra
    bad = ~(np.abs(ref.f64(got) - want) <= bound)
    assert not bad.any(), (np.argwhere(bad)[:4], ref.f64(got)[bad][:4], want[bad][:4])


def check_e4m3(codes, scales, want, group):
    M, N = want.shape
    g = group or N
    code = ref.f64(codes.view(torch.float8_e4m3fn).float())
    for j0 in range(0, N, g):
        y = want[:, j0:j0 + g]
        top = np.abs(y).max(1)
        s = np.where(top > 0, top / 448, 1.0)
        got = ref.f64(scales)[:, j0 // g]
        assert np.all(np.abs(got - s) <= 70 * U * s)
        z = y / s[:, None]
        assert np.all(np.abs(code[:, j0:j0 + g] - z) <= np.maximum(np.abs(z) / 16, 2.0 ** -10) * (1 + 1e-4) + 140 * U * np.abs(z))


SHAPES = [(1, 1), (1, 4096), (3, 7), (5, 64), (2, 80), (33, 96), (4, 1000), (3, 1001), (2, 4097), (7, 8192), (2, 16384),
          (1, 20000), (1, 32768), (1, 32767), (700, 512), (310, 1024), (311, 4096)]


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm(cuda, kind, shape, residual):
    t, (M, N) = ref.TYPES[kind], shape
    rng = np.random.default_rng(M * 7 + N)
    x, r = rows(rng, M, N, t), rows(rng, M, N, t, 3.0) if residual else None
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(N)).to(t).cuda()
    y, h = torch.full_like(x, 7.0), torch.full_like(x, 7.0) if residual else None
    rstd = torch.zeros(M, device="cuda")
    tm.tm_rmsnorm(x, N, r, N, h, N, w, M, N, EPS, y, N, None, rstd, ref.CODE[kind], ref.CODE[kind], ref.CODE[kind])
    tm.tm_check()
    hw, sw, yw = ref.rmsnorm(ref.f64(x), ref.f64(r) if residual else None, ref.f64(w), EPS)
    close(y, yw, 64 * U, t)
    close(rstd, sw, 62 * U, torch.float32)
    if residual:
        close(h, hw, U, t)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("shape", [(1, 1), (2, 32), (3, 40), (5, 100), (4, 1000), (3, 1001), (2, 4100), (400, 2048),
                                   (2, 8192), (1, 16384), (1, 32768), (2, 9001)])
def test_norm_e4m3(cuda, kind, group, shape):
    t, (M, N) = ref.TYPES[kind], shape
    rng = np.random.default_rng(M + N + group)
    x, r = rows(rng, M, N, t), rows(rng, M, N, t)
    if M > 1:
        x[1], r[1] = 0.0, 0.0   # a row of zeros: codes 0, scale 1
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(N)).float().cuda()
    ng = -(-N // group) if group else 1
    y = torch.full((M, N), 0x55, dtype=torch.uint8, device="cuda")
    sc = torch.full((M, ng), -1.0, device="cuda")
    tm.tm_rmsnorm(x, N, r, N, None, N, w, M, N, EPS, y, N, sc, None, ref.CODE[kind], tm.TM_F32, tm.TM_E4M3, group)
    tm.tm_check()
    check_e4m3(y, sc, ref.rmsnorm(ref.f64(x), ref.f64(r), ref.f64(w), EPS)[2], group)
    if M > 1:
        assert not (y[1] & 0x7F).any() and bool((sc[1] == 1).all())   # zeros of either sign


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_norm_strides_gaps_and_in_place(cuda, kind):
    t, M, N, ld = ref.TYPES[kind], 37, 120, 136
    rng = np.random.default_rng(5)
    for shift in (0, 1):                       # vector path, and single elements
        base = torch.full((M * ld + 64,), 300.0, dtype=t, device="cuda")
        res = base.clone()
        x, r = base[shift:][:M * ld].view(M, ld), res[shift:][:M * ld].view(M, ld)
        x[:, :N], r[:, :N] = rows(rng, M, N, t), rows(rng, M, N, t)
        x0, r0 = x[:, :N].clone(), r[:, :N].clone()
        w = rows(rng, 1, N, t)
        hw, _, yw = ref.rmsnorm(ref.f64(x0), ref.f64(r0), ref.f64(w), EPS)
        # h in place of r, y in place of x
        tm.tm_rmsnorm(x, ld, r, ld, r, ld, w, M, N, EPS, x, ld, None, None, ref.CODE[kind], ref.CODE[kind], ref.CODE[kind])
        tm.tm_check()
        close(r[:, :N], hw, U, t)
        close(x[:, :N], yw, 64 * U, t)
        for buf, v in ((base, x), (res, r)):   # the gaps and the ends are untouched
            v[:, :N] = 300.0
            assert bool((buf == 300.0).all())


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm_gradient(cuda, kind, shape, residual):
    t, (M, N) = ref.TYPES[kind], shape
    rng = np.random.default_rng(M * 3 + N)
    h, dy = rows(rng, M, N, t, 2.0), rows(rng, M, N, t)
    dr = rows(rng, M, N, t) if residual else None
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(N)).to(t).cuda()
    rstd64 = 1 / np.sqrt((ref.f64(h) ** 2).mean(1) + EPS)
    rstd = torch.from_numpy(rstd64).float().cuda()
    dx, dw = torch.full_like(h, 7.0), torch.full((N,), 7.0, dtype=t, device="cuda")
    ws = tm.tm_rmsnorm_bwd_workspace_bytes(M, N)
    scratch = torch.full((ws // 4,), float("nan"), device="cuda")
    tm.tm_rmsnorm_bwd(dy, N, h, N, w, rstd, dr, N, dx, N, dw, M, N, ref.CODE[kind], ref.CODE[kind], scratch, ws)
    tm.tm_check()
    s, h64, dy64, w64 = ref.f64(rstd), ref.f64(h), ref.f64(dy), ref.f64(w)
    dr64 = ref.f64(dr) if residual else None
    dxw, dww = ref.rmsnorm_bwd(dy64, h64, w64, s, dr64)
    n = np.abs(h64) * s[:, None]
    gn = np.abs(dy64 * w64) * n
    mean = gn.mean(1, keepdims=True)
    extra = U * (8 * (s[:, None] * (np.abs(dy64 * w64) + n * mean) + (np.abs(dr64) if residual else 0)) + 112 * s[:, None] * n * mean)
    close(dx, dxw, 0.0, t, extra)
    close(dw, dww, 0.0, t, U * (M + 128) * (np.abs(dy64) * n).sum(0))


# Rows enough for every block of the GPU to walk some (the form that copies rows ahead), with an odd
# count, a gap between rows, short rows (several to a block) and long ones.
MANY = [(4901, 1000, 1008), (2501, 4096, 4096), (1301, 8192, 8200), (641, 16384, 16384), (10001, 520, 520)]


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", MANY)
@pytest.mark.parametrize("residual", [False, True])
def test_norm_of_many_rows(cuda, kind, shape, residual):
    t, (M, N, ld) = ref.TYPES[kind], shape
    rng = np.random.default_rng(M + N)
    gen = torch.Generator(device="cuda").manual_seed(M)
    make = lambda s: (torch.randn(M, ld, generator=gen, device="cuda") * s).to(t)  # noqa: E731
    x, r, dy = make(1.0), make(3.0) if residual else None, make(1.0)
    wkind = "f32" if residual else kind            # weights of another type too
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(N)).to(ref.TYPES[wkind]).cuda()
    y, h = torch.full_like(x, 7.0), torch.full_like(x, 7.0) if residual else None
    rstd = torch.zeros(M, device="cuda")
    code = ref.CODE[kind]
    tm.tm_rmsnorm(x, ld, r, ld, h, ld, w, M, N, EPS, y, ld, None, rstd, code, ref.CODE[wkind], code)
    codes, sc = torch.zeros(M, ld, dtype=torch.uint8, device="cuda"), torch.zeros(M, -(-N // 64), device="cuda")
    tm.tm_rmsnorm(x, ld, r, ld, None, ld, w, M, N, EPS, codes, ld, sc, None, code, ref.CODE[wkind], tm.TM_E4M3, 64)
    codes1, sc1 = torch.zeros(M, ld, dtype=torch.uint8, device="cuda"), torch.zeros(M, 1, device="cuda")
    tm.tm_rmsnorm(x, ld, r, ld, None, ld, w, M, N, EPS, codes1, ld, sc1, None, code, ref.CODE[wkind], tm.TM_E4M3, 0)
    dx, dw = torch.full_like(x, 7.0), torch.zeros(N, dtype=ref.TYPES[wkind], device="cuda")
    ws = tm.tm_rmsnorm_bwd_workspace_bytes(M, N)
    scratch = torch.full((ws // 4,), float("nan"), device="cuda")
    stream = h if residual else x
    dr = r if residual else None
    tm.tm_rmsnorm_bwd(dy, ld, stream, ld, w, rstd, dr, ld, dx, ld, dw, M, N, code, ref.CODE[wkind], scratch, ws)
    tm.tm_check()
    hw, sw, yw = ref.rmsnorm(ref.f64(x[:, :N]), ref.f64(r[:, :N]) if residual else None, ref.f64(w), EPS)
    close(y[:, :N], yw, 64 * U, t)
    close(rstd, sw, 62 * U, torch.float32)
    if residual:
        close(h[:, :N], hw, U, t)
        assert bool((h[:, N:] == 7.0).all())
    assert bool((y[:, N:] == 7.0).all()) and bool((dx[:, N:] == 7.0).all()) and not codes[:, N:].any()
    check_e4m3(codes[:, :N].contiguous(), sc, yw, 64)
    check_e4m3(codes1[:, :N].contiguous(), sc1, yw, 0)
    s, h64, dy64, w64 = ref.f64(rstd), ref.f64(stream[:, :N]), ref.f64(dy[:, :N]), ref.f64(w)
    dr64 = ref.f64(dr[:, :N]) if residual else None
    dxw, dww = ref.rmsnorm_bwd(dy64, h64, w64, s, dr64)
    n = np.abs(h64) * s[:, None]
    gn = np.abs(dy64 * w64) * n
    mean = gn.mean(1, keepdims=True)
    extra = U * (8 * (s[:, None] * (np.abs(dy64 * w64) + n * mean) + (np.abs(dr64) if residual else 0)) + 112 * s[:, None] * n * mean)
    close(dx[:, :N], dxw, 0.0, t, extra)
    close(dw, dww, 0.0, ref.TYPES[wkind], U * (M + 128) * (np.abs(dy64) * n).sum(0))


def test_norm_gradient_against_differences(cuda):
    # d/dx of sum(y * dy), by central differences of the forward definition in 64 bits
    rng = np.random.default_rng(2)
    M, N, eps = 3, 40, 1e-5
    x, dy, w = rows(rng, M, N, torch.float32), rows(rng, M, N, torch.float32), rows(rng, 1, N, torch.float32)[0]
    y, rstd = torch.empty_like(x), torch.empty(M, device="cuda")
    tm.tm_rmsnorm(x, N, None, 0, None, 0, w, M, N, eps, y, N, None, rstd)
    dx, dw = torch.empty_like(x), torch.empty(N, device="cuda")
    scratch = torch.empty(M * N, device="cuda")
    tm.tm_rmsnorm_bwd(dy, N, x, N, w, rstd, None, 0, dx, N, dw, M, N, 0, 0, scratch, M * N * 4)
    tm.tm_check()
    x64, w64, dy64 = ref.f64(x), ref.f64(w), ref.f64(dy)
    f = lambda a, b: (ref.rmsnorm(a, None, b, eps)[2] * dy64).sum()  # noqa: E731
    d = 1e-5   # differences are good to about d^2 * 10 and 1e-16 * 100 / d
    for i in range(M):
        for j in range(0, N, 7):
            e = np.zeros_like(x64)
            e[i, j] = d
            assert abs((f(x64 + e, w64) - f(x64 - e, w64)) / (2 * d) - ref.f64(dx)[i, j]) < 2e-5
    for j in range(0, N, 7):
        e = np.zeros_like(w64)
        e[j] = d
        assert abs((f(x64, w64 + e) - f(x64, w64 - e)) / (2 * d) - ref.f64(dw)[j]) < 2e-5


def test_norm_special_rows(cuda):
    x = torch.randn(4, 256, device="cuda")
    x[1, 3] = float("nan")
    x[2] = 0.0
    x[3] *= 1e-20                                     # eps decides
    y, rstd = torch.empty_like(x), torch.empty(4, device="cuda")
    tm.tm_rmsnorm(x, 256, None, 0, None, 0, None, 4, 256, EPS, y, 256, None, rstd)
    tm.tm_check()
    assert bool(torch.isfinite(y[0]).all()) and bool(torch.isnan(y[1]).all())
    assert not y[2].any() and abs(rstd[2].item() * EPS ** 0.5 - 1) < 1e-6
    assert bool(torch.isfinite(y[3]).all())


def test_norm_empty(cuda):
    x = torch.zeros(16, device="cuda")
    tm.tm_rmsnorm(x, 4, None, 0, None, 0, None, 0, 4, EPS, x, 4)
    dw = torch.full((4,), 5.0, device="cuda")
    tm.tm_rmsnorm_bwd(x, 4, x, 4, None, None, None, 0, x, 4, dw, 0, 4)
    tm.tm_check()
    assert not dw.any()                               # the sum over no rows


def test_norm_overlapped_chain(cuda):
    # independent norms of one resident tensor, each overlapped on the one before
    rng = np.random.default_rng(9)
    x = rows(rng, 4100, 1000, torch.bfloat16)
    outs = [torch.empty_like(x) for _ in range(4)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        for o in outs:
            tm.tm_rmsnorm(x, 1000, None, 0, None, 0, None, 4100, 1000, EPS, o, 1000, None, None, 2, 2, 2, 0, tm.TM_PDL)
    tm.tm_check(st)
    yw = ref.rmsnorm(ref.f64(x), None, None, EPS)[2]
    for o in outs:
        close(o, yw, 64 * U, torch.bfloat16)
