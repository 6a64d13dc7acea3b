"""Plain 64-bit definitions of the products on operands of 8 and 16 bits, of the 8-bit
quantisation and of gradient clipping, and the tolerances of their tests.

Sums.  Products of two 16-bit (or two e4m3) values are exact in fp32.  The tensor
cores' additions are taken as fp32 with truncation, 2^-23 of the partial sum each, and
a partial sum is at most S = sum |a b|: K of them for 16 bits (to fp32 outputs 512 a
run, and one rounding a run), at most 128 a block for e4m3, whose blocks then take one
rounding of the scales' product, one of the addition (2^-24 each), and up to 8 parts of a
split sum one more each.
"""
import numpy as np
import torch

import block_ref as ref

TYPES, CODE = ref.TYPES, ref.CODE
E4M3 = torch.float8_e4m3fn
ULP = 2.0 ** -23


def starts_of(counts, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def padded(n, e, gap=0):
    return -(-n * e // 16) * 16 // e + gap * 16 // e


def rows(x, ld, fill=float("nan")):
    """x [R, n] (CPU) of its type on the device with row stride ld; the gaps hold `fill`."""
    out = torch.full((x.shape[0], ld), 0.0, dtype=torch.float32).fill_(fill).to(x.dtype)
    out[:, :x.shape[1]] = x
    return out.cuda()


def sum_bound(K, out):
    return ((K if out != torch.float32 else min(K, 512) + -(-K // 512)) + 9) * ULP


def block_bound(K):
    return (128 + -(-K // 128) + 9) * ULP


def check(got, want, size, rel, t, what=""):
    """|got - want| within rel * size and one rounding to type t."""
    r, a = ref.half_step(t)
    got = ref.f64(got) if isinstance(got, torch.Tensor) else got
    err = np.abs(got - want)
    bound = rel * size * (1 + r) + r * np.abs(want) + a
    bad = ~(err <= bound)
    assert not bad.any(), (what, np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], bad.sum())


def forward(x, w, starts):
    """y and sum |x w|: x [T, K], w [E, N, K] in 64 bits."""
    y, s = np.zeros((x.shape[0], w.shape[1])), np.zeros((x.shape[0], w.shape[1]))
    for e in range(w.shape[0]):
        at = slice(starts[e], starts[e + 1])
        y[at], s[at] = x[at] @ w[e].T, np.abs(x[at]) @ np.abs(w[e]).T
    return y, s


def backward(dy, x, w, starts):
    """dx, dw and their sums of magnitudes."""
    E, N, K = w.shape
    dx, sx, dw, sw = np.zeros((x.shape[0], K)), np.zeros((x.shape[0], K)), np.zeros((E, N, K)), np.zeros((E, N, K))
    for e in range(E):
        at = slice(starts[e], starts[e + 1])
        dx[at], sx[at] = dy[at] @ w[e], np.abs(dy[at]) @ np.abs(w[e])
        dw[e], sw[e] = dy[at].T @ x[at], np.abs(dy[at]).T @ np.abs(x[at])
    return dx, sx, dw, sw


def stretched(s, rows_, cols, block):
    """Scales [.., R, C] over an [.., rows, cols] matrix, `block` rows each (1: a row's own)."""
    return np.repeat(np.repeat(s, block, -2)[..., :rows_, :], 128, -1)[..., :cols]


def nearest_code(v):
    """Nearest e4m3 value to v (|v| <= 448), ties to the even code."""
    e = np.maximum(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -9))), -6)
    e = np.where(2.0 ** (e + 1) <= np.abs(v), e + 1, np.where((2.0 ** e > np.abs(v)) & (e > -6), e - 1, e))
    step = 2.0 ** (e - 3)
    return np.rint(v / step) * step


def quantise(x, rows_):
    """Code values and scales of x [M, N] in 64 bits."""
    M, N = x.shape
    p = np.zeros((-(-M // rows_) * rows_, -(-N // 128) * 128))
    p[:M, :N] = x
    b = np.abs(p).reshape(-1, rows_, p.shape[1] // 128, 128).max((1, 3))
    top = stretched(b, M, N, rows_)
    return nearest_code(np.where(top > 0, x * 448 / np.where(top > 0, top, 1), 0.0)), np.where(b > 0, b / 448, 1.0)
