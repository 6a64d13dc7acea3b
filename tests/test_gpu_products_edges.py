"""The products by expert, quantisation and clipping where they can go wrong: overlapped launches, several host threads,
other streams, many experts, bad borders, offsets past 2^31 and 2^32, strides far beyond the rows."""
import numpy as np
import pytest
import torch

import products_ref as ref
from masking_tm_affine_gb300 import tm
from test_gpu_clip import Clip, tensors
from test_gpu_e4m3 import Case as Case8
from test_gpu_experts import Case
from test_gpu_threads import at_once

pytestmark = pytest.mark.gpu
E4M3, P = ref.E4M3, tm.TM_PDL


class Work:
    """One call of each operator, few and many rows an expert."""

    def __init__(self, seed=0):
        self.few, self.many = Case([5, 0, 40], 200, 1000, seed=seed), Case([300, 77, 500], 264, 520, seed=seed + 1)
        self.few8, self.many8 = Case8([9, 0, 50], 200, 2000, seed=seed), Case8([400, 500], 264, 700, seed=seed + 1)
        self.x = torch.randn(300, 1000, device="cuda").bfloat16()
        self.clip = Clip(tensors([70000, 5, 300001], ["bf16", "f32"], seed=seed), "new")
        torch.cuda.synchronize()

    def outputs(self):
        full = lambda *s, t=torch.float32: torch.full(s, 9.0, device="cuda").to(t)  # noqa: E731
        out = [full(c.T, c.N) for c in (self.few, self.many, self.few8, self.many8)]
        for c in (self.few, self.many):
            out += [full(c.T, c.K, t=c.t), full(c.E * c.N, c.K)]
        return out + [full(300, 1000, t=torch.uint8), full(3, 8), full(300, 8)]

    def run(self, o, flags, s):
        s = getattr(s, "cuda_stream", s)
        for i, c in enumerate((self.few, self.many)):
            tm.tm_gemm_experts(c.x, c.ldk, c.w, c.ldk, o[i], c.N, c.d_starts, c.E, c.T, c.N, c.K, 2, 0, flags, s)
            tm.tm_gemm_experts_bwd(c.dy, c.ldn, c.x, c.ldk, c.w, c.ldk, o[4 + 2 * i], c.K, o[5 + 2 * i], c.K, c.d_starts, c.E,
                                   c.T, c.N, c.K, 2, 0, flags, s)
        for i, c in enumerate((self.few8, self.many8)):
            tm.tm_gemm_e4m3(c.a, c.ld, c.sa, 128, c.b, c.ld, c.sb, o[2 + i], c.N, c.d_starts, c.E, c.T, c.N, c.K, 0, flags, s)
        tm.tm_quant_e4m3(self.x, 1000, 300, 1000, o[8], 1000, o[9], 128, 2, flags, s)
        tm.tm_quant_e4m3(self.x, 1000, 300, 1000, o[8], 1000, o[10], 1, 2, flags, s)
        self.clip.run(3.0, flags=flags, stream=s)


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_overlapped_calls_give_the_same_bits(cuda):
    w, st = Work(), torch.cuda.Stream()
    plain = w.outputs()
    torch.cuda.synchronize()
    w.run(plain, 0, st)
    tm.tm_check(st)
    norm, outs = w.clip.norm.clone(), [o.clone() for o in w.clip.outs]
    runs = [w.outputs() for _ in range(6)]
    torch.cuda.synchronize()
    for o in runs:                                  # back to back: each call overlaps the one before
        w.run(o, P, st)
    tm.tm_check(st)
    assert all(same(o, plain) for o in runs)
    assert torch.equal(norm, w.clip.norm) and all(torch.equal(a, b) for a, b in zip(outs, w.clip.outs))


@pytest.mark.parametrize("counts", [[9, 30], [300, 400]])
def test_a_store_waits_for_the_call_before_it(cuda, counts):
    # a second call, overlapped, overwrites what the first one reads
    N = K = 264
    a, b = Case(counts, N, K, seed=1), Case(counts, N, K, seed=2)
    st = torch.cuda.Stream()
    x0 = a.x.clone()
    want = torch.empty(a.T, N, device="cuda")
    torch.cuda.synchronize()
    tm.tm_gemm_experts(a.x, a.ldk, a.w, a.ldk, want, N, a.d_starts, 2, a.T, N, K, 2, 0, 0, st)
    tm.tm_check(st)
    for _ in range(8):
        a.x.copy_(x0)
        got = torch.empty_like(want)
        torch.cuda.synchronize()
        tm.tm_gemm_experts(a.x, a.ldk, a.w, a.ldk, got, N, a.d_starts, 2, a.T, N, K, 2, 0, 0, st)
        tm.tm_gemm_experts(b.x, b.ldk, b.w, b.ldk, a.x, a.ldk, b.d_starts, 2, b.T, N, K, 2, 2, P, st)
        tm.tm_check(st)
        assert torch.equal(got, want) and not torch.equal(a.x, x0)


def test_several_host_threads(cuda):
    works = [Work(seed=10 * i) for i in range(4)]
    want = []
    for w in works:
        o = w.outputs()
        torch.cuda.synchronize()
        w.run(o, 0, torch.cuda.current_stream())
        torch.cuda.synchronize()
        want.append((o, w.clip.norm.clone()))
    streams = [torch.cuda.Stream() for _ in works]
    got = [[w.outputs() for _ in range(5)] for w in works]
    torch.cuda.synchronize()

    def go(i):
        def run():
            for o in got[i]:
                works[i].run(o, 0, streams[i])
        return run
    at_once([go(i) for i in range(4)])
    torch.cuda.synchronize()
    tm.tm_check()
    for i, (o, norm) in enumerate(want):
        assert all(same(g, o) for g in got[i]) and torch.equal(norm, works[i].clip.norm)


def test_two_graphs_of_one_expert_list_at_once(cuda):
    w = Work()
    plain = w.outputs()
    torch.cuda.synchronize()
    w.run(plain, 0, torch.cuda.current_stream())
    torch.cuda.synchronize()
    c, outs, graphs, streams = w.many, [], [], [torch.cuda.Stream() for _ in range(2)]
    for st in streams:
        o = w.outputs()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            for _ in range(4):
                tm.tm_gemm_experts(c.x, c.ldk, c.w, c.ldk, o[1], c.N, c.d_starts, c.E, c.T, c.N, c.K, 2, 0)
                tm.tm_gemm_experts_bwd(c.dy, c.ldn, c.x, c.ldk, c.w, c.ldk, o[6], c.K, o[7], c.K, c.d_starts, c.E, c.T, c.N, c.K,
                                       2, 0)
        outs.append(o)
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(5):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    tm.tm_check()
    for o in outs:
        assert all(torch.equal(o[i], plain[i]) for i in (1, 6, 7))


FIRST = """
import sys, torch
sys.path.insert(0, %r)
from masking_tm_affine_gb300 import tm
T, N, K, E = %d, 136, 264, 2
x, w = torch.randint(-3, 4, (T, K)).bfloat16().cuda(), torch.randint(-3, 4, (E, N, K)).bfloat16().cuda()
y, dx = torch.zeros(T, N, device="cuda"), torch.zeros(T, K, device="cuda").bfloat16()
dw, q, sc = torch.zeros(E, N, K, device="cuda"), torch.zeros(T, 272, dtype=torch.uint8, device="cuda"), torch.zeros(T, 3, device="cuda")
b, sb, z = torch.full((N, 272), 0x38, dtype=torch.uint8, device="cuda"), torch.ones(2, 3, device="cuda"), torch.zeros(T, N, device="cuda")
st = torch.tensor([0, T // 3, T], dtype=torch.int32, device="cuda")
norm, ws = torch.zeros(1, device="cuda"), torch.zeros(tm.tm_clip_workspace_bytes(), dtype=torch.uint8, device="cuda")
plan = tm.tm_clip_plan([x], None, [T * K], [2]).cuda()
torch.cuda.synchronize()
g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
with torch.cuda.graph(g, stream=s):
    tm.tm_gemm_experts(x, K, w, K, y, N, st, E, T, N, K, 2, 0)
    tm.tm_gemm_experts_bwd(x, K, x, K, w.view(E, K, N), N, dx, N, None, 0, st, E, T, K, N)
    tm.tm_gemm_experts_bwd(w.view(-1)[:T * N], N, x, K, None, 0, None, 0, dw, K, st, E, T, N, K, 2, 0)
    tm.tm_quant_e4m3(x, K, T, K, q, 272, sc, 1, 2)
    tm.tm_gemm_e4m3(q, 272, sc, 128, b, 272, sb, z, N, None, 1, T, N, K)
    tm.tm_clip_grads(plan, tm.tm_clip_chunks([T * K]), 1.0, 0.0, norm, ws, ws.numel())
g.replay()
tm.tm_check(s)
torch.cuda.synchronize()
for e, at in ((0, slice(0, T // 3)), (1, slice(T // 3, T))):
    assert torch.equal(y[at].double(), x[at].double() @ w[e].double().T)
v = q[:, :K].view(torch.float8_e4m3fn).double() * sc.double().repeat_interleave(128, 1)[:, :K]
assert float((z.double() - v.sum(1, keepdim=True)).abs().max()) <= 2.0 ** -10 * float(v.abs().sum(1).max())
assert abs(float(norm) - float(x.double().norm())) <= 2.0 ** -19 * float(norm) and dx.any() and dw.any()
print("captured first")
"""


@pytest.mark.parametrize("T", [40, 900])
def test_a_process_whose_first_calls_are_captured(cuda, T):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    # (w has room for the T rows of the weights' gradient: E * N * K elements)
    r = subprocess.run([sys.executable, "-c", FIRST % (root, min(T, 2 * 264))], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


# ------------------------------------------------------------------ experts
@pytest.mark.parametrize("E,per", [(1024, 1), (1000, 3), (300, 70), (257, 40)])
def test_many_experts(cuda, E, per):
    g = np.random.default_rng(E)
    counts = g.integers(0, 2 * per + 1, E).tolist()
    Case(counts, 24, 40, seed=E, ints=True, behind=7).check_all("f32")
    c = Case8(counts, 24, 40, seed=E, ints=True, behind=7)
    got = c.run()
    tm.tm_check()
    c.check(got)


@pytest.mark.parametrize("bad,mine", [([0, 500, 900, 1501], [500, 400, 0]), ([0, 500, 900, -1], [500, 400, 0]),
                                      ([0, 700, 600, 1500], [700, 0, 0]), ([-3, 500, 900, 1500], [0, 400, 600]),
                                      ([0, 1 << 30, 900, 1500], [0, 0, 0])])
def test_bad_borders_of_many_rows(cuda, bad, mine):
    c, c8 = Case([500, 400, 600], 264, 136, ints=True, poison=False), Case8([500, 400, 600], 264, 136, ints=True)
    c.d_starts = c8.d_starts = torch.tensor(bad, dtype=torch.int32, device="cuda")
    y, (dx, dw), y8 = c.forward("f32"), c.backward("f32"), c8.run()
    with pytest.raises(tm.TmError) as e:
        tm.tm_check()
    assert e.value.status == tm.TM_ERR_INDEX
    want, want8, wx = np.full((1500, 264), 7.0), np.full((1500, 264), 7.0), np.full((1500, 136), 7.0)
    for i, n in enumerate(mine):
        at = slice(max(bad[i], 0), max(bad[i], 0) + n) if n else slice(0, 0)
        want[at], want8[at], wx[at] = c.x64[at] @ c.w64[i].T, c8.a64[at] @ c8.b64[i].T, c.dy64[at] @ c.w64[i]
        assert np.array_equal(dw.double().cpu().numpy().reshape(3, 264, 136)[i], c.dy64[at].T @ c.x64[at])
    assert np.array_equal(y.double().cpu().numpy(), want) and np.array_equal(y8.double().cpu().numpy(), want8)
    ref.check(dx, wx, np.abs(wx), 0, torch.bfloat16)


# ------------------------------------------------------------------ large
def free_memory(gb):
    if torch.cuda.mem_get_info()[0] < gb * 2 ** 30:
        pytest.skip("needs %d GB of device memory" % gb)


def ints(shape, t, g, hi=3):
    return torch.randint(-hi, hi + 1, shape, generator=g, device="cuda", dtype=torch.int8).to(t)


def test_weights_past_2_to_32_elements(cuda):
    free_memory(60)
    E, N, K, g = 66, 8192, 8200, torch.Generator(device="cuda").manual_seed(1)      # 4.4e9 elements
    w = torch.empty(E, N, K, dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        w[e] = ints((N, K), torch.bfloat16, g)
    for counts in ([0] * 60 + [3, 0, 1, 9, 0, 2], [0] * 60 + [300, 0, 40, 300, 0, 100]):
        T, st = sum(counts), ref.starts_of(counts)
        x, dy = ints((T, K), torch.bfloat16, g), ints((T, N), torch.bfloat16, g)
        y, dx = torch.empty(T, N, device="cuda"), torch.empty_like(x)
        tm.tm_gemm_experts(x, K, w, K, y, N, st, E, T, N, K, 2, 0)
        tm.tm_gemm_experts_bwd(dy, N, x, K, w, K, dx, K, None, 0, st, E, T, N, K)
        tm.tm_check()
        first = np.concatenate([[0], np.cumsum(counts)])
        for e in range(60, E):
            at = slice(first[e], first[e + 1])
            assert torch.equal(y[at].double(), x[at].double() @ w[e].double().T)
            assert torch.equal(dx[at], (dy[at].double() @ w[e].double()).to(torch.bfloat16))
    dw, counts = w, [2] + [0] * 63 + [5, 40]
    T, st = 47, ref.starts_of(counts)
    tm.tm_gemm_experts_bwd(dy, N, x, K, None, 0, None, 0, dw, K, st, E, T, N, K)
    tm.tm_check()
    for e, at in ((0, slice(0, 2)), (64, slice(2, 7)), (65, slice(7, 47))):
        assert torch.equal(dw[e], (dy[at].double().T @ x[at].double()).to(torch.bfloat16))
    assert not dw[1:64].any()


def test_outputs_past_2_to_31_elements(cuda):
    free_memory(40)
    T, N, K, g = 70001, 32776, 16, torch.Generator(device="cuda").manual_seed(2)
    x, w = ints((T, K), torch.float16, g), ints((N, K), torch.float16, g)
    y = torch.empty(T, N, dtype=torch.float16, device="cuda")
    tm.tm_gemm_experts(x, K, w, K, y, N, None, 1, T, N, K, 1, 1)
    tm.tm_check()
    for r in (0, 1, 65531, 65537, T - 1):
        assert torch.equal(y[r].double(), x[r].double() @ w.double().T)
    a, b = x.to(E4M3).view(torch.uint8), w.to(E4M3).view(torch.uint8)
    sa, sb = torch.full((T, 1), 2.0, device="cuda"), torch.full((-(-N // 128), 1), 0.5, device="cuda")
    y.fill_(7.0)
    tm.tm_gemm_e4m3(a, K, sa, 128, b, K, sb, y, N, None, 1, T, N, K, 1)
    tm.tm_check()
    for r in (0, 1, 65531, 65537, T - 1):
        assert torch.equal(y[r].double(), x[r].double() @ w.double().T)


def test_far_strides(cuda):
    # rows 2^21 elements apart: offsets past 2^31 from a few thousand rows
    free_memory(40)
    T, N, K, ld, g = 2100, 72, 40, 1 << 21, torch.Generator(device="cuda").manual_seed(3)
    pool = torch.zeros(T * ld, dtype=torch.bfloat16, device="cuda").view(T, ld)
    pool[:, :K] = ints((T, K), torch.bfloat16, g)
    pool[:, 1024:1024 + N] = ints((T, N), torch.bfloat16, g)
    x, dy, w = pool[:, :K], pool[:, 1024:1024 + N], ints((2 * N, K), torch.bfloat16, g)
    counts = [700, 1400]
    st, y = ref.starts_of(counts), pool[:, 2048:2048 + N]
    tm.tm_gemm_experts(x, ld, w, K, y, ld, st, 2, T, N, K)
    dx, dw = pool[:, 4096:4096 + K], torch.empty(2 * N, K, device="cuda")
    tm.tm_gemm_experts_bwd(dy, ld, x, ld, w, K, dx, ld, dw, K, st, 2, T, N, K, 2, 0)
    tm.tm_check()
    for e, at in ((0, slice(0, 700)), (1, slice(700, 2100))):
        we = w[e * N:(e + 1) * N].double()
        assert torch.equal(y[at], (x[at].double() @ we.T).to(torch.bfloat16))
        assert torch.equal(dx[at], (dy[at].double() @ we).to(torch.bfloat16))
        assert torch.equal(dw[e * N:(e + 1) * N].double(), dy[at].double().T @ x[at].double())
    assert not pool[:, 8192:8300].any()


@pytest.mark.parametrize("rows", [1, 128])
def test_quantisation_past_2_to_31_elements(cuda, rows):
    free_memory(20)
    M, N = 70001, 32776
    x = torch.empty(M, N, dtype=torch.bfloat16, device="cuda").normal_()
    y, sc = torch.empty(M, N, dtype=torch.uint8, device="cuda"), torch.empty(-(-M // rows), 257, device="cuda")
    tm.tm_quant_e4m3(x, N, M, N, y, N, sc, rows, 2)
    tm.tm_check()
    for b in (0, 65536 // rows, (M - 1) // rows):
        at = slice(b * rows, min(M, (b + 1) * rows))
        want, scale = ref.quantise(x[at].double().cpu().numpy(), rows)
        assert np.array_equal(y[at].view(E4M3).double().cpu().numpy(), want)
        assert np.all(np.abs(sc[b].double().cpu().numpy() - scale[0]) <= 2.0 ** -24 * scale[0])


def test_clipping_past_2_to_31_elements(cuda):
    free_memory(20)
    n = (1 << 31) + 100003
    t = torch.full((n,), 2.0 ** -10, dtype=torch.bfloat16, device="cuda")
    t[-1] = 3.0
    plan = tm.tm_clip_plan([t], [t], [n], [2]).cuda()
    norm, ws = torch.empty(1, device="cuda"), torch.empty(tm.tm_clip_workspace_bytes(), dtype=torch.uint8, device="cuda")
    tm.tm_clip_grads(plan, tm.tm_clip_chunks([n]), 1.0, 0.0, norm, ws, ws.numel())
    tm.tm_check()
    want = ((n - 1) * 2.0 ** -20 + 9.0) ** 0.5
    assert abs(float(norm) - want) <= 18 * 2.0 ** -24 * want
    for i in (0, 1 << 31, n - 1):
        assert abs(float(t[i]) - (3.0 if i == n - 1 else 2.0 ** -10) / want) <= 2.0 ** -8 * 3.0 / want


def test_as_many_tiles_as_are_allowed(cuda):
    # few rows an expert, and more than 2^28 tiles of 128 columns: 2^30 is the limit
    E, N = 16, 2_040_000_000
    if torch.cuda.mem_get_info()[0] < 80e9:
        pytest.skip("64 GB of outputs")
    y = torch.empty(E, N, dtype=torch.bfloat16, device="cuda")
    y[0].fill_(7.0)
    y[1:, ::4_000_000] = 7.0
    starts = torch.tensor([0] * E + [1], dtype=torch.int32, device="cuda")     # one row, the last expert's
    tm.tm_gemm_experts(None, 0, None, 0, y, N, starts, E, E, N, 0)             # the sum of nothing
    tm.tm_check()
    assert not y[0].any() and bool((y[1:, ::4_000_000] == 7.0).all())
