"""tm_rmsnorm's 8-bit output where a group's values are next to nothing, against its
definition in 64 bits with the tolerances of test_gpu_norm.py.  Below fp32's normal
range a rounding is off by up to 2^-150: two of them in a scale, one in a product of
h and w (448 / max|h w| times that in a code)."""
import numpy as np
import pytest
import torch

import block_ref as ref
from masking_tm_affine_gb300 import tm

pytestmark = pytest.mark.gpu
U, EPS = ref.U, 1e-5


# Few rows, single elements (odd widths), and rows enough for the copies ahead.
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("M,N", [(6, 256), (5, 8192), (6, 333), (700, 2048), (1300, 8192)])
def test_groups_next_to_nothing(cuda, kind, group, M, N):
    t = ref.TYPES[kind]
    rng = np.random.default_rng(M + N + group)
    # x w of size 1; in row 0 all of it about 2^-122; in the other rows the first 128 columns about 2^-122 2^-i
    # (fp16 has no such values: its weights have)
    small = 2.0 ** -122
    x, w = rng.standard_normal((M, N)), 1.0 + 0.3 * rng.standard_normal(N)
    if kind == "f16":
        w[:128] *= small
        x[1:, :128] *= 2.0 ** -(np.arange(1, M) % 4)[:, None]
    else:
        x[0] *= small
        x[1:, :128] *= small * 2.0 ** -(np.arange(1, M) % 4)[:, None]
    x[:, 3::7] = 0.0
    X, W = torch.from_numpy(x).to(t).cuda(), torch.from_numpy(w).float().cuda()
    g = group or N
    y = torch.full((M, N), 0x55, dtype=torch.uint8, device="cuda")
    sc = torch.full((M, -(-N // g)), -1.0, device="cuda")
    tm.tm_rmsnorm(X, N, None, 0, None, 0, W, M, N, EPS, y, N, sc, None, ref.CODE[kind], tm.TM_F32, tm.TM_E4M3, group)
    tm.tm_check()
    _, rstd, want = ref.rmsnorm(ref.f64(X), None, ref.f64(W), EPS)
    code = ref.f64(y.view(torch.float8_e4m3fn).float())
    assert np.isfinite(code).all()
    tiny = 2.0 ** -150
    for j0 in range(0, N, g):
        v = want[:, j0:j0 + g]
        top = np.abs(v).max(1)
        s = np.where(top > 0, top / 448, 1.0)
        assert np.all(np.abs(ref.f64(sc)[:, j0 // g] - s) <= 70 * U * s + 2 * tiny)
        z = v / s[:, None]
        lost = np.where(top > 0, 448 * tiny * rstd / np.where(top > 0, top, 1.0), 0.0)[:, None]
        lim = np.maximum(np.abs(z) / 16, 2.0 ** -10) * (1 + 1e-4) + 140 * U * np.abs(z) + 2 * lost
        assert np.all(np.abs(code[:, j0:j0 + g] - z) <= lim)
        assert not code[:, j0:j0 + g][v == 0].any()
