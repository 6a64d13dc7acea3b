"""tm_gemm_experts and tm_gemm_experts_bwd against their definitions in 64 bits.  Integer-valued operands make every sum
exact in fp32, so those results must be equal; others stay within the bound of products_ref."""
import numpy as np
import pytest
import torch

import products_ref as ref
from masking_tm_affine_gb300 import tm

pytestmark = pytest.mark.gpu
TYPES, CODE = ref.TYPES, ref.CODE


class Case:
    """One layer: rows of each expert (in order), idle rows before and behind them, row strides with gaps of NaN."""

    def __init__(self, counts, N, K, kind="bf16", seed=0, before=0, behind=0, gap=0, ints=False, poison=True, starts=True):
        g = np.random.default_rng(seed)
        self.E, self.N, self.K, self.kind, self.t = len(counts), N, K, kind, TYPES[kind]
        self.T = before + sum(counts) + behind
        self.starts = [before + sum(counts[:e]) for e in range(self.E + 1)]
        self.d_starts = ref.starts_of(counts, before) if starts else None
        make = (lambda *s: g.integers(-4, 5, s).astype(np.float64)) if ints else (lambda *s: g.standard_normal(s))
        to = lambda a: torch.from_numpy(a).to(self.t)  # noqa: E731
        x, w, dy = to(make(self.T, K)), to(make(self.E * N, K)), to(make(self.T, N))
        self.x64, self.w64, self.dy64 = (a.double().numpy() for a in (x, w, dy))
        self.w64 = self.w64.reshape(self.E, N, K)
        if poison:   # rows of nobody, and matrices of experts without rows
            for a in (x, dy):
                a[:before], a[self.T - behind:] = float("nan"), float("nan")
            for e, n in enumerate(counts):
                if n == 0:
                    w[e * N:(e + 1) * N] = float("inf")
        self.ldk, self.ldn = ref.padded(K, 2, gap), ref.padded(N, 2, gap)
        self.x, self.w, self.dy = ref.rows(x, self.ldk), ref.rows(w, self.ldk), ref.rows(dy, self.ldn)
        self.mine = np.zeros(self.T, dtype=bool)
        self.mine[before:self.T - behind] = True
        self.ints = ints

    def forward(self, ytype=None, ldy=None, flags=0, stream=None):
        ytype = ytype or self.kind
        ldy = ldy or self.N
        y = torch.full((self.T, ldy), 7.0, dtype=TYPES[ytype], device="cuda")
        tm.tm_gemm_experts(self.x, self.ldk, self.w, self.ldk, y, ldy, self.d_starts, self.E, self.T, self.N, self.K,
                           CODE[self.kind], CODE[ytype], flags, stream)
        return y

    def backward(self, wtype=None, lddx=None, lddw=None, rows=True, weights=True, flags=0, stream=None):
        wtype = wtype or self.kind
        lddx, lddw = lddx or self.K, lddw or self.K
        dx = torch.full((self.T, lddx), 7.0, dtype=self.t, device="cuda") if rows else None
        dw = torch.full((self.E * self.N, lddw), 7.0, dtype=TYPES[wtype], device="cuda") if weights else None
        tm.tm_gemm_experts_bwd(self.dy, self.ldn, self.x, self.ldk, self.w, self.ldk, dx, lddx, dw, lddw, self.d_starts,
                               self.E, self.T, self.N, self.K, CODE[self.kind], CODE[wtype], flags, stream)
        return dx, dw

    def check_forward(self, y, ytype):
        want, size = ref.forward(self.x64, self.w64, self.starts)
        got = y.double().cpu().numpy()
        assert np.all(got[~self.mine] == 7.0) and np.all(got[:, self.N:] == 7.0)
        ref.check(got[self.mine, :self.N], want[self.mine], size[self.mine], 0 if self.ints else ref.sum_bound(self.K, TYPES[ytype]),
                  TYPES[ytype], "y")

    def check_backward(self, dx, dw, wtype):
        wx, sx, ww, sw = ref.backward(self.dy64, self.x64, self.w64, self.starts)
        if dx is not None:
            got = dx.double().cpu().numpy()
            assert np.all(got[~self.mine] == 7.0) and np.all(got[:, self.K:] == 7.0)
            ref.check(got[self.mine, :self.K], wx[self.mine], sx[self.mine], 0 if self.ints else ref.sum_bound(self.N, self.t), self.t, "dx")
        if dw is not None:
            got = dw.double().cpu().numpy()
            assert np.all(got[:, self.K:] == 7.0)
            got = got[:, :self.K].reshape(self.E, self.N, self.K)
            ref.check(got, ww, sw, 0 if self.ints else ref.sum_bound(max(1, self.T), TYPES[wtype]), TYPES[wtype], "dw")

    def check_all(self, out="f32", **kw):
        y = self.forward(out, **kw)
        dx, dw = self.backward(out, **kw)
        tm.tm_check()
        self.check_forward(y, out)
        self.check_backward(dx, dw, out)


# counts, N, K: single rows, rows at the borders of 16, 32, 64, 128 and 256, experts without rows, few rows an expert and
# many, extents that end inside every tile
SHAPES = [([1], 8, 8), ([1], 1, 1), ([3], 64, 64), ([16], 128, 128), ([17], 130, 72), ([0, 1, 0, 2], 40, 200),
          ([32, 31, 33], 256, 520), ([64, 65, 1, 127], 96, 1000), ([128], 512, 256), ([129], 520, 136), ([200, 0, 56], 264, 320),
          ([256], 256, 64), ([257], 300, 300), ([1000], 72, 40), ([300, 301, 5, 0], 250, 333), ([1500, 700], 1000, 520),
          ([5] * 40, 129, 257), ([0, 0, 0], 64, 64), ([2049], 1024, 768)]


@pytest.mark.parametrize("counts,N,K", SHAPES)
def test_integers_are_exact(cuda, counts, N, K):
    Case(counts, N, K, "bf16", seed=N + K, ints=True).check_all("f32")


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("out", ["same", "f32"])
@pytest.mark.parametrize("counts,N,K", [([5, 0, 40], 200, 264), ([300, 77, 150], 384, 260), ([700], 520, 1000)])
def test_values(cuda, counts, N, K, kind, out):
    c = Case(counts, N, K, kind, seed=K)
    c.check_all(kind if out == "same" else "f32")


@pytest.mark.parametrize("counts,N,K", [([20], 136, 6000), ([600], 72, 5000), ([5000, 3000], 200, 136)])
def test_long_sums_to_32_bits(cuda, counts, N, K):
    Case(counts, N, K, "bf16", seed=K).check_all("f32")


@pytest.mark.parametrize("counts", [[3, 0, 30], [290, 0, 300, 45]])
def test_rows_of_nobody_and_gaps(cuda, counts):
    N, K = 200, 264
    c = Case(counts, N, K, "bf16", seed=3, before=5, behind=70, gap=3, ints=True)
    y, (dx, dw) = c.forward("f32", ldy=N + 3), c.backward("f32", lddx=K + 1, lddw=K + 5)
    tm.tm_check()
    c.check_forward(y, "f32")
    c.check_backward(dx, dw, "f32")


@pytest.mark.parametrize("n", list(range(0, 36)) + [47, 48, 49, 63, 64, 65, 79, 80, 127, 128, 129, 191, 255, 256, 257])
def test_sums_over_any_number_of_rows(cuda, n):
    # what lies behind an expert's rows is NaN: none of it may reach the weights' gradient
    Case([n], 72, 136, "f16", seed=n, ints=True, behind=64, before=3).check_all("f32")


# few tiles with long sums: forward (long K), rows' gradient (long N), weights' gradient (many rows, shared by pairs of SMs)
@pytest.mark.parametrize("counts,N,K", [([600], 264, 2000), ([600], 264, 4100), ([700, 40], 130, 3333), ([600], 3400, 264),
                                        ([4000], 264, 130), ([9001], 72, 520), ([3000, 0, 1700], 130, 136), ([513], 72, 6000),
                                        ([3500], 1000, 1000), ([0, 6003], 257, 300)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_few_long_sums(cuda, counts, N, K, out):
    Case(counts, N, K, "bf16", seed=N, ints=True, behind=3).check_all(out)
    c = Case(counts, N, K, "bf16", seed=N)
    c.check_all(out)
    y, (dx, dw) = c.forward(out), c.backward(out)
    again, (dx2, dw2) = c.forward(out), c.backward(out)
    tm.tm_check()
    assert torch.equal(y, again) and torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_one_matrix_without_borders(cuda):
    for T in (9, 600):
        Case([T], 192, 320, "bf16", ints=True, starts=False).check_all("f32")


@pytest.mark.parametrize("T", [4, 900])
def test_infinities_and_nans_stay_in_their_rows(cuda, T):
    c = Case([T // 2, T - T // 2], 136, 200, "bf16", seed=1, ints=True)
    bad = {0: float("inf"), T - 1: float("nan")}
    for r, v in bad.items():
        c.x[r, 3], c.dy[r, 5] = v, v
    y, (dx, _) = c.forward("f32"), c.backward("f32", weights=False)
    tm.tm_check()
    for got, (want, _) in ((y, ref.forward(c.x64, c.w64, c.starts)), (dx, ref.backward(c.dy64, c.x64, c.w64, c.starts)[:2])):
        got = got.double().cpu().numpy()
        keep = [r for r in range(T) if r not in bad]
        assert not np.isfinite(got[list(bad)]).any(1).all()
        assert np.isnan(got[T - 1]).all()
        ref.check(got[keep], want[keep], np.abs(want[keep]), 0, torch.float32 if got.shape[1] == 136 else c.t)


def test_one_gradient_alone(cuda):
    c = Case([40, 300], 72, 136, "bf16", ints=True)
    dx, _ = c.backward("f32", weights=False)
    _, dw = c.backward("f32", rows=False)
    tm.tm_check()
    c.check_backward(dx, dw, "f32")


def test_empty_extents(cuda):
    # a sum over nothing is zero; nothing to write is nothing done
    for counts in ([3, 4], [400, 300]):
        T = sum(counts)
        st, y = ref.starts_of(counts), torch.full((T, 40), 7.0, device="cuda")
        tm.tm_gemm_experts(None, 0, None, 0, y, 40, st, 2, T, 40, 0, tm.TM_BF16, tm.TM_F32)
        dx, dw = torch.full((T, 40), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((80, 24), 7.0, device="cuda")
        tm.tm_gemm_experts_bwd(None, 0, None, 0, None, 40, dx, 40, None, 0, st, 2, T, 0, 40)
        tm.tm_gemm_experts_bwd(None, 40, None, 24, None, 24, None, 0, dw, 24, ref.starts_of([0, 0]), 2, 0, 40, 24, 2, 0)
        one = torch.full((80, 24), 7.0, dtype=torch.bfloat16, device="cuda")
        tm.tm_gemm_experts_bwd(None, 80, None, 24, None, 24, None, 0, one, 24, None, 1, 0, 80, 24)
        tm.tm_check()
        assert not y.any() and not dx.any() and not dw.any() and not one.any()


def test_borders_out_of_range(cuda):
    # an expert whose borders leave the rows, fall, or lie before an earlier one has none; the others are computed
    c = Case([10, 20, 30], 40, 64, "bf16", ints=True, poison=False)
    for bad in ([0, 10, 30, 61], [0, 10, 30, 1 << 30], [0, 10, 30, -5], [-1, 10, 30, 60], [0, 40, 30, 60]):
        c.d_starts = torch.tensor(bad, dtype=torch.int32, device="cuda")
        y, (dx, dw) = c.forward("f32"), c.backward("f32")
        with pytest.raises(tm.TmError) as e:
            tm.tm_check()
        assert e.value.status == tm.TM_ERR_INDEX
        mine = {(0, 10): [10, 20, 0], (-1, 10): [0, 20, 30], (0, 40): [40, 0, 0]}[tuple(bad[:2])]
        lo, want = [max(bad[e], 0) if n else 0 for e, n in enumerate(mine)], np.full((60, 40), 7.0)
        for e, n in enumerate(mine):
            at = slice(lo[e], lo[e] + n)
            want[at] = c.x64[at] @ c.w64[e].T
            assert np.array_equal(dw.double().cpu().numpy().reshape(3, 40, 64)[e], c.dy64[at].T @ c.x64[at])
        assert np.array_equal(y.double().cpu().numpy(), want)
    torch.cuda.synchronize()


def test_gradients_against_differences(cuda):
    # d/dx and d/dw of sum(y * dy): the loss is linear in each, so a difference of any size is exact up to rounding
    c = Case([7, 0, 12], 24, 40, "f16", seed=5)
    dx, dw = c.backward("f32")
    tm.tm_check()
    f = lambda x, w: (ref.forward(x, w, c.starts)[0] * c.dy64).sum()  # noqa: E731
    g = np.random.default_rng(0)
    for _ in range(5):
        ux, uw = g.standard_normal(c.x64.shape), g.standard_normal(c.w64.shape)
        sx = (ux * dx.double().cpu().numpy()).sum()
        sw = (uw * dw.double().cpu().numpy().reshape(c.w64.shape)).sum()
        # dx is rounded to fp16: half a step of each of its terms
        slack = 2.0 ** -11 * (np.abs(ux) * np.abs(dx.double().cpu().numpy())).sum()
        assert abs(f(c.x64 + ux, c.w64) - f(c.x64 - ux, c.w64) - 2 * sx) <= 2 * slack + 1e-6
        assert abs(f(c.x64, c.w64 + uw) - f(c.x64, c.w64 - uw) - 2 * sw) <= 1e-3


@pytest.mark.parametrize("counts", [[9, 0, 50], [400, 500]])
def test_the_same_bits_every_time_and_from_a_graph(cuda, counts):
    c = Case(counts, 200, 1000, "bf16", seed=9)
    y, (dx, dw) = c.forward(), c.backward("f32")
    tm.tm_check()
    again = c.forward(), *c.backward("f32")
    outs = [torch.full_like(a, 3.0) for a in (y, dx, dw)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            tm.tm_gemm_experts(c.x, c.ldk, c.w, c.ldk, outs[0], c.N, c.d_starts, c.E, c.T, c.N, c.K)
            tm.tm_gemm_experts_bwd(c.dy, c.ldn, c.x, c.ldk, c.w, c.ldk, outs[1], c.K, outs[2], c.K, c.d_starts, c.E, c.T, c.N,
                                   c.K, 2, 0)
    torch.cuda.synchronize()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    tm.tm_check()
    for a, b, d in zip((y, dx, dw), again, outs):
        assert torch.equal(a, b) and torch.equal(a, d)
    # the borders live on the device: a graph follows them
    c.d_starts.copy_(torch.tensor([0] * (c.E + 1), dtype=torch.int32))
    outs[0].fill_(3.0)
    graph.replay()
    torch.cuda.synchronize()
    assert bool((outs[0] == 3.0).all()) and not outs[2].any()


@pytest.mark.parametrize("T", [4, 900])
def test_rows_that_hold_an_infinity_or_a_nan(cuda, T):
    # an infinity times a weight, or times 0; the rest of such a row's sum is finite
    c = Case([T // 2, T - T // 2], 136, 200, "bf16", seed=1, ints=True)
    c.x[0, 3], c.dy[0, 5], c.x[T - 1, 3], c.dy[T - 1, 5] = float("inf"), float("-inf"), float("nan"), float("nan")
    y, (dx, _) = c.forward("f32"), c.backward("f32", weights=False)
    tm.tm_check()
    for got, sign, w in ((y, 1.0, c.w64[0, :, 3]), (dx, -1.0, c.w64[0, 5])):
        got = got.double().cpu().numpy()
        assert (w == 0).any() and (w != 0).any()
        assert np.isnan(got[0][w == 0]).all()
        assert np.array_equal(got[0][w != 0], sign * np.sign(w[w != 0]) * np.inf)
        assert np.isnan(got[T - 1]).all()
