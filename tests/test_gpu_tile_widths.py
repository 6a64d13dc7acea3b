"""The products by expert at sizes that take tiles of each width (64, 128 and 256 along the narrow extent; in 8 bits also
of 128 by 128), among them calls with more tiles than SMs hold at once and tiles that end after one row or one column."""
import numpy as np
import pytest
import torch

from masking_tm_affine_gb300 import tm
from test_gpu_e4m3 import TYPES, Case as Case8, check_quant, quant
from test_gpu_experts import Case

pytestmark = pytest.mark.gpu

# rows of each expert, N, K
SHAPES = [([900, 800, 333, 5, 0, 700], 1000, 330), ([900, 800, 333, 5, 0, 700], 500, 330), ([129] * 50, 200, 72), ([65] * 60, 256, 136),
          ([33] * 70, 130, 264), ([257] * 48, 100, 200), ([64, 65, 63, 1, 129, 128, 127], 257, 129), ([3000], 264, 1000),
          ([1025], 1025, 512), ([255, 257, 513], 72, 1032), ([2000, 1, 2000], 260, 64), ([127, 0, 0, 300, 40, 1], 1000, 136),
          ([100] * 20, 1100, 200), ([34, 128, 0, 129, 1], 136, 1160)]


@pytest.mark.parametrize("counts,N,K", SHAPES)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_16_bits(cuda, counts, N, K, out):
    Case(counts, N, K, "bf16", seed=N + K, ints=True, behind=3, gap=1).check_all(out)
    Case(counts, N, K, "bf16", seed=N + K).check_all(out)


@pytest.mark.parametrize("counts,N,K", SHAPES)
@pytest.mark.parametrize("out,group", [("bf16", 128), ("f32", 0)])
def test_8_bits(cuda, counts, N, K, out, group):
    for ints in (True, False):
        c = Case8(counts, N, K, group, seed=N, ints=ints, behind=3)
        for ldc in (N, N + 3):
            y = c.run(out, ldc)
            tm.tm_check()
            c.check(y, out)


@pytest.mark.parametrize("counts", [[700], [300, 400], [150] * 4])
@pytest.mark.parametrize("K", [2040, 2048, 2200])
def test_sums_on_both_sides_of_a_rule(cuda, counts, K):
    # long sums over few tiles go to the kernel that cuts them: the results are the definition's either way
    Case(counts, 256, K, "f16", seed=K, ints=True).check_all("f32")
    c = Case8(counts, 256, K, 128, seed=K, ints=True)
    y, again = c.run("f32"), c.run("f32")
    tm.tm_check()
    c.check(y, "f32")
    assert torch.equal(y, again)


# the kernel and its tiles are chosen from T and E alone: any borders must do, also where they move between a graph's replays
SPREADS = [[100, 100, 100, 100, 100, 100], [600, 0, 0, 0, 0, 0], [0, 0, 0, 0, 1, 599], [1, 2, 4, 8, 16, 569], [0, 300, 0, 300, 0, 0]]


@pytest.mark.parametrize("N,K", [(1000, 264), (136, 1032)])
def test_borders_move_under_a_graph(cuda, N, K):
    c, c8 = Case(SPREADS[0], N, K, "bf16", seed=1, ints=True), Case8(SPREADS[0], N, K, 128, seed=2, ints=True)
    # scales of one, so that no expert's own enter the oracle's operands wrongly when rows change hands
    c8.sa.fill_(1.0), c8.sb.fill_(1.0)
    plain = lambda t, ld: t.view(torch.float8_e4m3fn).float().double().cpu().numpy().reshape(-1, ld)[:, :K]  # noqa: E731
    c8.a64, c8.b64 = plain(c8.a, c8.ld), plain(c8.b, c8.ld).reshape(6, N, K)
    st = torch.cuda.Stream()
    out = [torch.empty(600, N, device="cuda"), torch.empty(600, N, device="cuda"), torch.empty(600, K, device="cuda").bfloat16(),
           torch.empty(6 * N, K, device="cuda")]
    torch.cuda.synchronize()
    s = st.cuda_stream

    def run(flags):
        tm.tm_gemm_experts(c.x, c.ldk, c.w, c.ldk, out[0], N, c.d_starts, 6, 600, N, K, 2, 0, flags, s)
        tm.tm_gemm_e4m3(c8.a, c8.ld, c8.sa, 128, c8.b, c8.ld, c8.sb, out[1], N, c.d_starts, 6, 600, N, K, 0, flags, s)
        tm.tm_gemm_experts_bwd(c.dy, c.ldn, c.x, c.ldk, c.w, c.ldk, out[2], K, out[3], K, c.d_starts, 6, 600, N, K, 2, 0, flags, s)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        with torch.cuda.graph(graph, stream=st):
            run(0)
            run(tm.TM_PDL)
    for spread in SPREADS:
        starts = np.concatenate([[0], np.cumsum(spread)])
        c.starts = c8.starts = [int(v) for v in starts]
        with torch.cuda.stream(st):
            c.d_starts.copy_(torch.tensor(starts, dtype=torch.int32))
            for o in out:
                o.fill_(float("nan"))
            graph.replay()
        st.synchronize()
        tm.tm_check(st)
        c.check_forward(out[0], "f32")
        c8.check(out[1])
        c.check_backward(out[2], out[3], "f32")


@pytest.mark.parametrize("counts,N,K", [([100] * 20, 1100, 200), ([257] * 48, 100, 200), ([700], 256, 2200)])
def test_overlapped_calls(cuda, counts, N, K):
    c, c8, st = Case(counts, N, K, "bf16", seed=4), Case8(counts, N, K, 128, seed=5), torch.cuda.Stream()
    torch.cuda.synchronize()
    runs = []
    with torch.cuda.stream(st):
        first = c.forward("f32", stream=st), c8.run("f32", stream=st), *c.backward("f32", stream=st)
        for _ in range(4):
            runs.append((c.forward("f32", flags=tm.TM_PDL, stream=st), c8.run("f32", flags=tm.TM_PDL, stream=st),
                         *c.backward("f32", flags=tm.TM_PDL, stream=st)))
    tm.tm_check(st)
    for r in runs:
        assert all(torch.equal(a, b) for a, b in zip(first, r))


@pytest.mark.parametrize("kind", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("N,ldx,ldy,x0,y0", [(260, 260, 260, 0, 0), (260, 264, 268, 4, 4), (264, 264, 264, 4, 0), (264, 268, 264, 0, 0),
                                             (264, 264, 264, 0, 4), (264, 264, 265, 0, 0), (262, 264, 264, 0, 0), (262, 262, 262, 2, 6),
                                             (264, 264, 264, 2, 2), (2, 2, 2, 0, 0), (4, 4, 4, 0, 0)])
def test_quantisation_in_vectors_of_each_width(cuda, kind, rows, N, ldx, ldy, x0, y0):
    g = torch.Generator().manual_seed(N + ldx)
    flat = torch.full((131 * ldx + x0,), float("nan")).to(TYPES[kind])
    x = flat[x0:].view(131, ldx)
    x[:, :N] = torch.randn(131, N, generator=g).to(TYPES[kind])
    x = flat.cuda()[x0:].view(131, ldx)[:, :N]
    check_quant(x, *quant(x, kind, rows, ldy, y0), rows)
