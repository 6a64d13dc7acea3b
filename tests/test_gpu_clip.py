"""tm_clip_plan and tm_clip_grads against their definition in 64 bits.

A thread's part of at most 32 squares is added in fp32 (32 roundings of 2^-24, all terms positive) and joins the rest in 64
bits, so the norm is within 16 * 2^-24 + one rounding of itself; a gradient is the product with the factor (its own
rounding, the norm's error, one of the product) and one rounding to its type."""
import math

import numpy as np
import pytest
import torch

import block_ref as ref
from masking_tm_affine_gb300 import tm

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


class Clip:
    def __init__(self, tensors, outs="new", shift=0):
        """tensors: device tensors; outs: new, in place, none, or mixed."""
        self.g = tensors
        self.kinds = [next(k for k in ref.TYPES if ref.TYPES[k] == t.dtype) for t in tensors]
        self.sizes = [t.numel() for t in tensors]
        self.before = [t.clone() for t in tensors]
        mode = lambda i: outs if outs != "mixed" else ("new", "place", "none")[i % 3]  # noqa: E731
        self.outs = [torch.full((n + 8,), 5.0, dtype=t.dtype, device="cuda")[shift:] if mode(i) == "new" else
                     t if mode(i) == "place" else None for i, (t, n) in enumerate(zip(tensors, self.sizes))]
        self.plan = tm.tm_clip_plan(tensors, self.outs, self.sizes, [ref.CODE[k] for k in self.kinds]).cuda()
        self.chunks = tm.tm_clip_chunks(self.sizes)
        self.need = tm.tm_clip_workspace_bytes()
        self.ws = torch.full((self.need // 8,), float("nan"), dtype=torch.float64, device="cuda")
        self.norm = torch.full((1,), -1.0, device="cuda")

    def run(self, max_norm, eps=1e-6, flags=0, stream=None):
        tm.tm_clip_grads(self.plan, self.chunks, max_norm, eps, self.norm, self.ws, self.need, flags, stream)

    def check(self, max_norm, eps=1e-6):
        g64 = [t.double().cpu().numpy() for t in self.before]
        norm = math.sqrt(sum(float((a * a).sum()) for a in g64))
        got = float(self.norm)
        assert abs(got - norm) <= 18 * U * norm + 2.0 ** -150, (got, norm)
        f = min(1.0, float(np.float32(max_norm)) / (norm + float(np.float32(eps)))) if math.isfinite(max_norm) else 1.0
        for a, o, t, n in zip(g64, self.outs, self.g, self.sizes):
            if o is None:
                assert np.array_equal(t.double().cpu().numpy(), a)
                continue
            r, small = ref.half_step(o.dtype)
            err = np.abs(o[:n].double().cpu().numpy() - a * f)
            assert np.all(err <= (r + 20 * U) * np.abs(a * f) + small)
            if o is not t:
                assert bool((o[n:] == 5.0).all())


def tensors(sizes, kinds, scale=1.0, seed=0, shift=0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n + shift, generator=g) * scale).to(ref.TYPES[kinds[i % len(kinds)]]).cuda()[shift:]
            for i, n in enumerate(sizes)]


SIZES = [[1], [7, 1, 3], [16384, 16383, 16385], [1000, 0, 70000, 5, 128], [3] * 300, [500000, 2, 300001]]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("kinds", [["f32"], ["bf16"], ["f16"], ["bf16", "f32", "f16"]])
@pytest.mark.parametrize("outs", ["new", "place", "mixed"])
def test_norm_and_clipping(cuda, sizes, kinds, outs):
    for max_norm in (0.25 * math.sqrt(sum(sizes)), 1e6):
        c = Clip(tensors(sizes, kinds, seed=len(sizes)), outs)
        c.run(max_norm)
        tm.tm_check()
        c.check(max_norm)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_odd_addresses(cuda, kind):
    for gs, os in ((1, 0), (0, 1), (1, 1)):
        c = Clip(tensors([1000, 33000], [kind], shift=gs), "new", os)
        c.run(3.0)
        tm.tm_check()
        c.check(3.0)


@pytest.mark.parametrize("scale", [2.0 ** -130, 2.0 ** -100, 2.0 ** -63, 2.0 ** -41, 2.0 ** 49, 2.0 ** 63, 2.0 ** 100, 2.0 ** 115])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_squares_beyond_the_range(cuda, scale, kind):
    c = Clip(tensors([5000, 40001], [kind], scale), "new")
    c.run(scale, 0.0)
    tm.tm_check()
    c.check(scale, 0.0)


def test_large_beside_small(cuda):
    t = tensors([70000, 70000], ["f32"])
    t[0] *= 2.0 ** 70
    t[1] *= 2.0 ** -60
    c = Clip(t)
    c.run(1.0)
    tm.tm_check()
    c.check(1.0)


def test_nothing_and_zeros(cuda):
    c = Clip(tensors([0, 0], ["f32"]))
    c.run(1.0)
    tm.tm_check()
    assert float(c.norm) == 0.0
    c = Clip([torch.zeros(5000, device="cuda")])
    c.run(1.0, 0.0)     # max_norm / 0: no clipping
    tm.tm_check()
    assert float(c.norm) == 0.0 and not c.outs[0][:5000].any()
    c = Clip([torch.zeros(70, device="cuda")])
    c.run(0.0, 0.0)     # 0 / 0
    tm.tm_check()
    assert float(c.norm) == 0.0 and not c.outs[0][:70].any()
    c = Clip(tensors([5000], ["f32"]))
    c.run(0.0)
    tm.tm_check()
    assert not c.outs[0][:5000].any()


def test_not_finite(cuda):
    for bad, want in ((float("nan"), "nan"), (float("inf"), "inf")):
        t = tensors([40000, 300], ["f32"])
        t[1][7] = bad
        c = Clip(t)
        c.run(1.0)
        tm.tm_check()
        assert str(float(c.norm)) == want
        o = torch.cat([x[:n] for x, n in zip(c.outs, c.sizes)])
        if want == "nan":
            assert bool(torch.isnan(o).all())
        else:       # times 0: zeros, and NaN where the infinity was
            assert int(torch.isnan(o).sum()) == 1 and not torch.nan_to_num(o, nan=0.0).any()
    t = tensors([100], ["f32"])
    c = Clip(t, "place")
    c.run(float("inf"))
    tm.tm_check()
    assert torch.equal(t[0], c.before[0])


def test_many_tensors_the_same_bits_and_a_graph(cuda):
    # more chunks than blocks, so that blocks walk several
    c = Clip(tensors([1 << 21] * 12 + [77] * 9, ["bf16", "f32"]), "new")
    c.run(2.0)
    tm.tm_check()
    c.check(2.0)
    norm, outs = c.norm.clone(), [o.clone() for o in c.outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            c.run(2.0)
            c.run(2.0, flags=tm.TM_PDL)       # overlapped on the first, through the same workspace
    for _ in range(3):
        c.norm.fill_(-1.0)
        for o in c.outs:
            o.fill_(9.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.norm, norm) and all(torch.equal(a[:n], b[:n]) for a, b, n in zip(c.outs, outs, c.sizes))


@pytest.mark.parametrize("outs", ["new", "place"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_no_clipping_whatever_the_norm_is(cuda, outs, bad):
    # an infinite max_norm comes first: the gradients stay as they are, and the norm tells what they hold
    t = tensors([40000, 300], ["f32", "bf16"])
    t[1][7] = bad
    c = Clip(t, outs)
    c.run(float("inf"))
    tm.tm_check()
    assert str(float(c.norm)) == str(bad)
    for o, b, n in zip(c.outs, c.before, c.sizes):
        kept = torch.isnan(b) if math.isnan(bad) else torch.zeros_like(b, dtype=torch.bool)
        assert bool((torch.isnan(o[:n]) == torch.isnan(b)).all()) and torch.equal(o[:n][~kept], b[~kept])
