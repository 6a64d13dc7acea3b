"""Long sums of one sign to 16-bit outputs.  Additions in the tensor cores lose towards zero, so such a sum shows how many of
them there are: every output stays within (512 + K / 512 + 9) 2^-23 of the sum, whatever its length, and one rounding.

Sums lie just above a power of two, where half a step of the output's type is the largest part of a value that it gets; among
some thousands of them there are roundings of every size and direction."""
import numpy as np
import pytest
import torch

import products_ref as ref
from masking_tm_affine_gb300 import tm

pytestmark = pytest.mark.gpu
TYPES, CODE = ref.TYPES, ref.CODE
LONG = 131072


def operands(outer_a, outer_b, n, kind, seed=0):
    """[outer_a, n] and [outer_b, n] in their type: positive, rows' products of about 1.01 * 2^10."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    a, b = (0.5 + 0.5 * torch.rand(o, n, generator=g, device="cuda") for o in (outer_a, outer_b))
    return a.to(TYPES[kind]), (b * (1.01 * 2 ** 10 / (0.5625 * n))).to(TYPES[kind])


def check(got, a, b, n, kind):
    want = (a.double() @ b.double().T).cpu().numpy()
    ref.check(got, want, want, ref.sum_bound(n, torch.float32), TYPES[kind])


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("T,N", [(20, 264), (300, 136), (300, 1700)])      # small tiles, larger, and pairs of SMs
def test_products(cuda, kind, T, N):
    x, w = operands(T, N, LONG, kind)
    y = torch.empty(T, N, dtype=TYPES[kind], device="cuda")
    tm.tm_gemm_experts(x, LONG, w, LONG, y, N, None, 1, T, N, LONG, CODE[kind], CODE[kind])
    tm.tm_check()
    check(y, x, w, LONG, kind)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("T,K", [(20, 264), (300, 136), (300, 1704)])
def test_gradient_of_the_rows(cuda, kind, T, K):
    dy, wt = operands(T, K, LONG, kind, seed=1)
    w, dx = wt.T.contiguous(), torch.empty(T, K, dtype=TYPES[kind], device="cuda")
    tm.tm_gemm_experts_bwd(dy, LONG, None, K, w, K, dx, K, None, K, None, 1, T, LONG, K, CODE[kind], CODE[kind])
    tm.tm_check()
    check(dx, dy, wt, LONG, kind)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("N,K", [(136, 264), (1040, 2104)])                # sums shared by pairs of SMs, and not
def test_gradient_of_the_weights(cuda, kind, N, K):
    dyt, xt = operands(N, K, LONG, kind, seed=2)
    rest = 700                                                             # of a second expert
    g = torch.Generator(device="cuda").manual_seed(3)
    dy, x = (torch.cat([t.T, torch.randn(rest, t.shape[0], generator=g, device="cuda").to(t.dtype)]) for t in (dyt, xt))
    dw = torch.empty(2, N, K, dtype=TYPES[kind], device="cuda")
    tm.tm_gemm_experts_bwd(dy, N, x, K, None, K, None, K, dw, K, ref.starts_of([LONG, rest]), 2, LONG + rest, N, K, CODE[kind],
                           CODE[kind])
    tm.tm_check()
    check(dw[0], dyt, xt, LONG, kind)
    a, b = dy[LONG:].double(), x[LONG:].double()
    ref.check(dw[1], (a.T @ b).cpu().numpy(), (a.abs().T @ b.abs()).cpu().numpy(), ref.sum_bound(rest, torch.float32), TYPES[kind])
