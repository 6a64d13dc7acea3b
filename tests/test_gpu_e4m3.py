"""tm_quant_e4m3 and tm_gemm_e4m3 against their definitions in 64 bits.

Codes are those of the exact quotient, so they must be equal; a scale is one division (2^-24).  Products with integer
codes and scales that are powers of two are exact in fp32 and must be equal; others stay within products_ref's bound."""
import numpy as np
import pytest
import torch

import products_ref as ref
from masking_tm_affine_gb300 import tm

pytestmark = pytest.mark.gpu
TYPES, CODE, E4M3 = ref.TYPES, ref.CODE, ref.E4M3


# ------------------------------------------------------------------ quantisation
def quant(x, kind, rows, ldy=None, shift=0):
    M, N = x.shape
    ldy = ldy or N
    y = torch.full((M * ldy + 16,), 0x55, dtype=torch.uint8, device="cuda")
    sc = torch.full((-(-M // rows) * -(-N // 128) + 1,), -3.0, device="cuda")
    tm.tm_quant_e4m3(x, x.stride(0), M, N, y[shift:], ldy, sc, rows, CODE[kind])
    tm.tm_check()
    assert float(sc[-1]) == -3.0
    out = y[shift:shift + M * ldy].view(M, ldy)
    assert bool((out[:, N:] == 0x55).all()) and bool((y[:shift] == 0x55).all()) and bool((y[shift + M * ldy:] == 0x55).all())
    return out[:, :N], sc[:-1].view(-(-M // rows), -(-N // 128))


def check_quant(x, codes, sc, rows):
    x64 = x.double().cpu().numpy()
    want, scale = ref.quantise(x64, rows)
    got = codes.contiguous().view(E4M3).double().cpu().numpy()
    assert np.array_equal(got, want), (np.argwhere(got != want)[:4], got[got != want][:4], want[got != want][:4])
    s = sc.double().cpu().numpy()
    assert np.all(np.abs(s - scale) <= 2.0 ** -24 * scale + 2.0 ** -150)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("M,N", [(1, 1), (1, 128), (3, 7), (5, 130), (128, 128), (129, 260), (200, 1000), (33, 1001), (300, 4096)])
def test_quantisation(cuda, kind, rows, M, N):
    g = torch.Generator().manual_seed(M * N)
    x = (torch.randn(M, N, generator=g) * torch.exp(torch.randn(M, 1, generator=g))).to(TYPES[kind])
    if M > 2:
        x[1] = 0.0                                      # zeros: scale 1 where a whole block is
    x = x.cuda()
    check_quant(x, *quant(x, kind, rows), rows)
    wide = torch.full((M, N + 9), float("nan"), dtype=x.dtype, device="cuda")   # odd strides and starts
    wide[:, 1:N + 1] = x
    check_quant(x, *quant(wide[:, 1:N + 1], kind, rows, N + 3, 1), rows)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows", [1, 128])
def test_quotients_on_a_border(cuda, kind, rows):
    # every border between two codes, its neighbours in the type, and tops for which 448 / top is not exact
    codes = torch.arange(0, 127, dtype=torch.uint8).view(E4M3).double()
    borders = (codes[1:] + codes[:-1]) / 2
    out = []
    for top in (448.0, 7.0, 133 / 64, 147 / 128, 1.75 * 2 ** -6, 189 / 128, 1.0, 245.0):
        v = (borders * top / 448).to(TYPES[kind])
        v = torch.nn.functional.pad(v, (0, 127 - v.numel()))
        out.append(torch.cat([v, torch.tensor([top]).to(v.dtype)]))
        f = v.float()
        for step in (1, -1):
            whole = torch.int32 if kind == "f32" else torch.int16
            n = (v.view(whole) + step * (v != 0).to(whole)).view(v.dtype)
            out.append(torch.cat([n, torch.tensor([top]).to(v.dtype)]))
    x = torch.stack(out)
    x = torch.cat([x, -x]).cuda()
    check_quant(x, *quant(x, kind, rows), rows)


@pytest.mark.parametrize("rows", [1, 128])
def test_far_ends_of_the_range(cuda, rows):
    g = torch.Generator().manual_seed(0)
    x = torch.randn(128, 128 * 6, generator=g)
    for j, s in enumerate((2.0 ** -148, 2.0 ** -126, 2.0 ** -70, 2.0 ** -20, 2.0 ** 100, 2.0 ** 125)):
        x[:, 128 * j:128 * j + 128] *= s
    x = x.cuda()
    check_quant(x, *quant(x, "f32", rows), rows)


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_blocks_that_are_not_finite(cuda, rows, bad):
    x = torch.randn(128, 384, device="cuda")
    x[5, 130] = bad
    codes, sc = quant(x, "f32", rows)
    block = slice(5, 6) if rows == 1 else slice(0, 128)
    assert bool((codes[block, 128:256] == 0x7F).all()) and bool(torch.isnan(sc[block.start // rows, 1]))
    keep = x.clone()
    keep[block, 128:256] = 0.0
    codes, sc = codes.clone(), sc.clone()
    codes[block, 128:256], sc[block.start // rows, 1] = 0, 1.0
    check_quant(keep, codes, sc, rows)


# ------------------------------------------------------------------ products
class Case:
    def __init__(self, counts, N, K, group=128, seed=0, behind=0, ints=False, gap=0, starts=True):
        g = np.random.default_rng(seed)
        self.E, self.N, self.K, self.group, self.T, self.ints = len(counts), N, K, group, sum(counts) + behind, ints
        self.starts = [sum(counts[:e]) for e in range(self.E + 1)]
        self.d_starts = ref.starts_of(counts) if starts else None
        KB, NB = -(-K // 128), -(-N // 128)
        if ints:
            a, b = g.integers(-8, 9, (self.T, K)), g.integers(-8, 9, (self.E * N, K))
            sa = 2.0 ** g.integers(-1, 2, (self.T, KB if group else 1))
            sb = 2.0 ** g.integers(-1, 2, (self.E, NB, KB))
        else:
            a, b = g.standard_normal((self.T, K)) * 100, g.standard_normal((self.E * N, K)) * 100
            sa = np.exp(g.standard_normal((self.T, KB if group else 1)))
            sb = np.exp(g.standard_normal((self.E, NB, KB)))
        code = lambda v: torch.from_numpy(v).float().clamp(-448, 448).to(E4M3)  # noqa: E731
        a, b = code(a), code(b)
        sa, sb = torch.from_numpy(sa).float(), torch.from_numpy(sb).float()
        self.a64 = a.float().double().numpy() * (np.repeat(sa.double().numpy(), 128, 1)[:, :K] if group else sa.double().numpy())
        self.b64 = b.float().double().numpy().reshape(self.E, N, K) * ref.stretched(sb.double().numpy(), N, K, 128)
        a[self.T - behind:] = float("nan")
        if behind:
            sa[self.T - behind:] = float("nan")
        self.ld = ref.padded(K, 1, gap)
        put = lambda v: torch.nn.functional.pad(v.view(torch.uint8), (0, self.ld - K), value=0x7F).cuda()  # noqa: E731
        self.a, self.b, self.sa, self.sb = put(a), put(b), sa.cuda(), sb.cuda()

    def run(self, out="f32", ldc=None, flags=0, stream=None):
        ldc = ldc or self.N
        c = torch.full((self.T, ldc), 7.0, dtype=TYPES[out], device="cuda")
        tm.tm_gemm_e4m3(self.a, self.ld, self.sa, self.group, self.b, self.ld, self.sb, c, ldc, self.d_starts, self.E, self.T,
                        self.N, self.K, CODE[out], flags, stream)
        return c

    def check(self, c, out="f32"):
        want, size = ref.forward(self.a64, self.b64, self.starts)
        got = c.double().cpu().numpy()
        end = self.starts[-1]
        assert np.all(got[end:] == 7.0) and np.all(got[:, self.N:] == 7.0)
        ref.check(got[:end, :self.N], want[:end], size[:end], 0 if self.ints else ref.block_bound(self.K), TYPES[out])


SHAPES = [([1], 1, 1), ([1], 8, 16), ([3], 64, 64), ([16], 128, 128), ([17], 130, 129), ([0, 1, 0, 2], 40, 200),
          ([32, 31, 33], 256, 520), ([64, 65, 1, 127], 96, 1000), ([128], 512, 256), ([129], 520, 136), ([257], 300, 300),
          ([300, 301, 5, 0], 250, 333), ([1500, 700], 1000, 520), ([5] * 40, 129, 257), ([1000], 72, 40), ([0, 0, 0], 64, 64),
          ([2049], 1024, 768), ([20], 384, 4100), ([500, 20, 0, 300], 640, 2100)]


@pytest.mark.parametrize("counts,N,K", SHAPES)
@pytest.mark.parametrize("group", [0, 128])
def test_integers_are_exact(cuda, counts, N, K, group):
    c = Case(counts, N, K, group, seed=N + K, ints=True, behind=K % 3 * 11)
    got = c.run()
    tm.tm_check()
    c.check(got)


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("counts,N,K", [([5, 0, 40], 200, 2000), ([300, 77, 150], 384, 260), ([700], 520, 1000)])
def test_values(cuda, counts, N, K, out, group):
    c = Case(counts, N, K, group, seed=K, behind=9, gap=2)
    if out == "f16":                       # within fp16's range
        c.sa *= 2.0 ** -12
        c.a64 *= 2.0 ** -12
    got = c.run(out, ldc=N + 5)
    tm.tm_check()
    c.check(got, out)


# few tiles with long sums
@pytest.mark.parametrize("counts,N,K", [([300], 264, 4100), ([300], 264, 2000), ([700, 240], 130, 3333), ([513], 72, 8000), ([250, 0, 300], 1000, 4100)])
@pytest.mark.parametrize("out,group", [("bf16", 128), ("f32", 0)])
def test_few_long_sums(cuda, counts, N, K, out, group):
    c = Case(counts, N, K, group, seed=N, ints=True, behind=3)
    got = c.run("f32")
    tm.tm_check()
    c.check(got)
    c = Case(counts, N, K, group, seed=N)
    got, again = c.run(out, ldc=N + 8), c.run(out, ldc=N + 8)
    tm.tm_check()
    c.check(got, out)
    assert torch.equal(got, again)


def test_one_matrix_without_borders(cuda):
    for T in (9, 600):
        c = Case([T], 192, 320, ints=True, starts=False)
        got = c.run()
        tm.tm_check()
        c.check(got)


@pytest.mark.parametrize("T", [4, 900])
def test_infinities_and_nans_stay_in_their_rows(cuda, T):
    c = Case([T // 2, T - T // 2], 136, 520, seed=1, ints=True)
    c.a[0, 3], c.sa[T - 1, 2] = 0x7F, float("inf")
    got = c.run()
    tm.tm_check()
    want, _ = ref.forward(c.a64, c.b64, c.starts)
    got = got.double().cpu().numpy()
    assert np.isnan(got[0]).all() and not np.isfinite(got[T - 1]).any()
    assert np.array_equal(got[1:T - 1], want[1:T - 1])


def test_empty_sum(cuda):
    for T in (5, 700):
        c = torch.full((T, 40), 7.0, device="cuda")
        tm.tm_gemm_e4m3(None, 0, None, 128, None, 0, None, c, 40, None, 1, T, 40, 0)
        tm.tm_check()
        assert not c.any()


@pytest.mark.parametrize("counts", [[9, 0, 50], [400, 500]])
def test_the_same_bits_every_time_and_from_a_graph(cuda, counts):
    c = Case(counts, 200, 2000, seed=9)
    y = c.run("bf16")
    tm.tm_check()
    again, out = c.run("bf16"), torch.full_like(y, 3.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            tm.tm_gemm_e4m3(c.a, c.ld, c.sa, 128, c.b, c.ld, c.sb, out, c.N, c.d_starts, c.E, c.T, c.N, c.K, tm.TM_BF16)
    torch.cuda.synchronize()
    for _ in range(3):
        graph.replay()
    tm.tm_check()
    torch.cuda.synchronize()
    assert torch.equal(y, again) and torch.equal(y, out)


def test_norm_quantise_multiply(cuda):
    # the 8-bit path as a block has it: norm to codes, product, quantise its output, product
    M, H, F = 70, 512, 640
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(M, H, generator=g, device="cuda").bfloat16()
    w1, w2 = (torch.randn(a, b, generator=g, device="cuda").bfloat16() / b ** 0.5 for a, b in ((F, H), (H, F)))
    u8 = lambda *s: torch.empty(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    f32 = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    q1, s1, q2, s2 = u8(F, H), f32(5, 4), u8(H, F), f32(4, 5)
    tm.tm_quant_e4m3(w1, H, F, H, q1, H, s1, 128, tm.TM_BF16)
    tm.tm_quant_e4m3(w2, F, H, F, q2, F, s2, 128, tm.TM_BF16)
    a, sa, h = u8(M, H), f32(M, 4), torch.empty(M, F, dtype=torch.bfloat16, device="cuda")
    tm.tm_rmsnorm(x, H, None, 0, None, 0, None, M, H, 1e-5, a, H, sa, None, tm.TM_BF16, tm.TM_BF16, tm.TM_E4M3, 128)
    tm.tm_gemm_e4m3(a, H, sa, 128, q1, H, s1, h, F, None, 1, M, F, H, tm.TM_BF16)
    b, sb, y = u8(M, F), f32(M, 5), f32(M, H)
    tm.tm_quant_e4m3(h, F, M, F, b, F, sb, 1, tm.TM_BF16)
    tm.tm_gemm_e4m3(b, F, sb, 128, q2, F, s2, y, H, None, 1, M, H, F)
    tm.tm_check()
    val = lambda q, s, r: q.view(E4M3).double().cpu().numpy() * ref.stretched(s.double().cpu().numpy(), *q.shape, r)  # noqa: E731
    w = val(q1, s1, 128)
    ref.check(h, val(a, sa, 1) @ w.T, np.abs(val(a, sa, 1)) @ np.abs(w).T, ref.block_bound(H), torch.bfloat16)
    v = val(q2, s2, 128)
    ref.check(y, val(b, sb, 1) @ v.T, np.abs(val(b, sb, 1)) @ np.abs(v).T, ref.block_bound(F), torch.float32)
    # and the whole of it against no quantisation at all: four roundings of 2^-4 of values, averaged over the sums
    n = x.double() / (x.double().pow(2).mean(1, keepdim=True) + 1e-5).sqrt()
    full = n @ w1.double().T @ w2.double().T
    assert float((y.double() - full).norm() / full.norm()) < 4 * 2.0 ** -4


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("shape", [(128, 768), (40, 767), (130, 770)])
def test_small_blocks_of_bf16(cuda, rows, shape):
    # tops below 2^-100, where 448 / top nears or passes fp32's range, down to bf16's least value
    g = torch.Generator().manual_seed(0)
    x = torch.randn(*shape, generator=g)
    for j, s in enumerate((2.0 ** -133, 2.0 ** -126, 2.0 ** -119, 2.0 ** -110, 2.0 ** -102, 2.0 ** -99)):
        x[:, 128 * j:128 * j + 128] *= s
    x = x.bfloat16().cuda()
    check_quant(x, *quant(x, "bf16", rows), rows)


@pytest.mark.parametrize("counts,N,K", [([5, 0, 9], 264, 200), ([300, 77, 150], 384, 260), ([200], 130, 1000)])
def test_gradient_of_the_rows(cuda, counts, N, K):
    # y = x W^T in 8 bits has dx = dy W: the same product with the transposed codes and scales of W
    E, T = len(counts), sum(counts)
    g = torch.Generator(device="cuda").manual_seed(N)
    w, dy = (torch.randn(*s, generator=g, device="cuda").bfloat16() for s in ((E, N, K), (T, N)))
    KB, NB, ldk, ldn = -(-K // 128), -(-N // 128), ref.padded(K, 1), ref.padded(N, 1)
    q, sb = torch.zeros(E, N, ldk, dtype=torch.uint8, device="cuda"), torch.empty(E, NB, KB, device="cuda")
    for e in range(E):
        tm.tm_quant_e4m3(w[e], K, N, K, q[e], ldk, sb[e], 128, tm.TM_BF16)
    qt = torch.zeros(E, K, ldn, dtype=torch.uint8, device="cuda")
    qt[..., :N] = q[..., :K].transpose(1, 2)
    st = sb.transpose(1, 2).contiguous()
    a, sa = torch.zeros(T, ldn, dtype=torch.uint8, device="cuda"), torch.empty(T, NB, device="cuda")
    tm.tm_quant_e4m3(dy, N, T, N, a, ldn, sa, 1, tm.TM_BF16)
    dx, starts = torch.full((T, K), 7.0, device="cuda"), [sum(counts[:e]) for e in range(E + 1)]
    tm.tm_gemm_e4m3(a, ldn, sa, 128, qt, ldn, st, dx, K, ref.starts_of(counts), E, T, K, N)
    tm.tm_check()
    value = lambda c, s, n, b: c[..., :n].contiguous().view(E4M3).double().cpu().numpy() * ref.stretched(  # noqa: E731
        s.double().cpu().numpy(), c.shape[-2], n, b)
    wv, dv = value(q, sb, K, 128), value(a, sa, N, 1)
    want, size = ref.forward(dv, wv.transpose(0, 2, 1), starts)
    ref.check(dx, want, size, ref.block_bound(N), torch.float32)
    # codes are within 2^-4 of their values, or 2^-10 of a code where they are smallest: x 2^-4 + top / 448 2^-10
    err = lambda v, t: np.abs(v) * 2.0 ** -4 + t * 2.0 ** -10 / 448  # noqa: E731
    w64, d64 = w.double().cpu().numpy(), dy.double().cpu().numpy()
    top_w = ref.stretched(sb.double().cpu().numpy(), N, K, 128) * 448
    top_d = ref.stretched(sa.double().cpu().numpy(), T, N, 1) * 448
    assert np.all(np.abs(wv - w64) <= err(w64, top_w) * (1 + 1e-6)) and np.all(np.abs(dv - d64) <= err(d64, top_d) * (1 + 1e-6))
    full, _ = ref.forward(d64, w64.transpose(0, 2, 1), starts)
    sizes, _ = ref.forward(np.abs(d64) + err(d64, top_d), (np.abs(w64) + err(w64, top_w)).transpose(0, 2, 1), starts)
    plain, _ = ref.forward(np.abs(d64), np.abs(w64).transpose(0, 2, 1), starts)
    got = dx.double().cpu().numpy()
    assert np.all(np.abs(got - full) <= sizes - plain + ref.block_bound(N) * sizes + 2.0 ** -24 * np.abs(full))
