"""A feed-forward layer whose tokens are routed to experts, served in 8 bits and trained in 16.

serve()  -- residual addition + RMS norm to 8-bit codes, the two best experts of each token, its codes
            sorted by expert, the experts' first product in 8 bits, the activation, its output
            quantised, the second product, and the experts' answers added with their weights; run as
            it is and from a CUDA graph, whose replays follow the tokens' routes.
train()  -- the same layer in 16 bits under torch's autograd: the gradients of the rows and of all
            matrices from the library, clipped together by their norm in place.

Routing (scores, sorting, gathering) is torch's part.  Weights and inputs are random.

    python examples/expert_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from masking_tm_affine_gb300 import tm  # noqa: E402

EPS = 1e-5
TYPE, CODE = torch.bfloat16, tm.TM_BF16


def route(scores, k):
    """scores [T, E] -> the rows' order by expert, their tokens, weights, and the experts' borders, all on the device."""
    T, E = scores.shape
    best, expert = scores.softmax(-1).topk(k, -1)
    expert, order = expert.reshape(-1).sort(stable=True)
    starts = torch.searchsorted(expert, torch.arange(E + 1, device=scores.device)).to(torch.int32)
    return order // k, (best / best.sum(-1, keepdim=True)).reshape(-1)[order], starts


def codes_of(rows, n, dev):
    """Room for rows of n codes, their stride a multiple of 16 as the products want it, and for their scales."""
    return torch.empty(rows, -(-n // 16) * 16, dtype=torch.uint8, device=dev), torch.empty(rows, -(-n // 128), device=dev)


def act(h):
    return torch.nn.functional.silu(h)


# ------------------------------------------------------------------ served in 8 bits
class Matrices8:
    """The experts' matrices [E, N, K] as codes with a scale for each 128 by 128."""

    def __init__(self, w):
        E, N, K = w.shape
        self.shape = w.shape
        self.ld = -(-K // 16) * 16
        self.codes = torch.empty(E, N, self.ld, dtype=torch.uint8, device=w.device)
        self.scales = torch.empty(E, -(-N // 128), -(-K // 128), device=w.device)
        for e in range(E):  # blocks start anew with each expert
            tm.tm_quant_e4m3(w[e], K, N, K, self.codes[e], self.ld, self.scales[e], 128, CODE)

    def __call__(self, a, sa, starts):
        (E, N, K), T = self.shape, a.shape[0]
        y = torch.empty(T, N, dtype=TYPE, device=a.device)
        tm.tm_gemm_e4m3(a, self.ld, sa, 128, self.codes, self.ld, self.scales, y, N, starts, E, T, N, K, CODE)
        return y


def layer8(x, h, norm, gate, up, down, k):
    """x [T, H] joins the residual stream h in place; returns the layer's addition to it."""
    T, H = x.shape
    a, sa = codes_of(T, H, x.device)
    tm.tm_rmsnorm(x, H, h, H, h, H, norm, T, H, EPS, a, a.shape[1], sa, None, CODE, CODE, tm.TM_E4M3, 128)
    token, weight, starts = route(h.float() @ gate, k)
    y = act(up(a[token], sa[token], starts))
    R, F = y.shape
    b, sb = codes_of(R, F, x.device)
    tm.tm_quant_e4m3(y, F, R, F, b, b.shape[1], sb, 1, CODE)
    z = down(b, sb, starts)
    return torch.zeros(T, H, device=x.device).index_add_(0, token, z.float() * weight[:, None])


def parameters(H, F, E, seed, dev):
    g = torch.Generator(device=dev).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    return ((1.0 + 0.1 * rand(H)).to(TYPE), rand(H, E) / H**0.5, (rand(E, F, H) / H**0.5).to(TYPE),
            (rand(E, H, F) / F**0.5).to(TYPE))


def serve(T=24, H=512, F=640, E=8, k=2, steps=3, seed=0, dev="cuda"):
    """Returns for each step the outputs from the graph, from direct calls, and of the layer without quantisation."""
    norm, gate, w1, w2 = parameters(H, F, E, seed, dev)
    up, down = Matrices8(w1), Matrices8(w2)
    g = torch.Generator(device=dev).manual_seed(seed + 1)
    x, h = torch.empty(T, H, dtype=TYPE, device=dev), torch.empty(T, H, dtype=TYPE, device=dev)
    inputs = [(torch.randn(T, H, generator=g, device=dev).to(TYPE), torch.randn(T, H, generator=g, device=dev).to(TYPE))
              for _ in range(steps)]

    def load(i):
        x.copy_(inputs[i][0])
        h.copy_(inputs[i][1])

    load(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # once as it is: a capture wants everything loaded
        layer8(x, h, norm, gate, up, down, k)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer8(x, h, norm, gate, up, down, k)
    results = []
    for i in range(steps):
        load(i)
        graph.replay()
        replayed = out.clone()
        load(i)
        direct = layer8(x, h, norm, gate, up, down, k)
        s = inputs[i][0].double() + inputs[i][1].double()
        n = s / (s.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * norm.double()
        token, weight, starts = route(h.float() @ gate, k)
        z = torch.cat([act(n[token[a:b]] @ w1[e].double().T) @ w2[e].double().T
                       for e, (a, b) in enumerate(zip(starts.tolist(), starts.tolist()[1:]))])
        results.append((replayed, direct, torch.zeros(T, H, device=dev).double().index_add_(0, token, z * weight[:, None])))
    tm.tm_check()
    return results


# ------------------------------------------------------------------ trained in 16 bits
def first_derivatives(backward):
    """A backward pass that cannot be differentiated itself, and so refuses to be part of a graph (create_graph=True).
    Marked once_differentiable it would be cut off without an error where torch.autograd.grad is given its inputs."""
    def run(ctx, *grads):
        if torch.is_grad_enabled():
            raise RuntimeError("only first derivatives: call it without create_graph")
        return backward(ctx, *grads)
    return run


class Experts(torch.autograd.Function):
    """rows [T, K], matrices [E, N, K], borders -> [T, N]"""

    @staticmethod
    def forward(ctx, x, w, starts):
        ctx.save_for_backward(x, w, starts)
        (E, N, K), T = w.shape, x.shape[0]
        y = torch.empty(T, N, dtype=x.dtype, device=x.device)
        tm.tm_gemm_experts(x, K, w, K, y, N, starts, E, T, N, K, CODE, CODE)
        return y

    @staticmethod
    @first_derivatives
    def backward(ctx, dy):
        x, w, starts = ctx.saved_tensors
        (E, N, K), T = w.shape, x.shape[0]
        dy = dy.contiguous()
        dx, dw = (torch.empty_like(t) if need else None for t, need in zip((x, w), ctx.needs_input_grad))
        tm.tm_gemm_experts_bwd(dy, N, x, K, w, K, dx, K, dw, K, starts, E, T, N, K, CODE, CODE)
        return dx, dw, None


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w):
        T, H = x.shape
        y, rstd = torch.empty_like(x), torch.empty(T, device=x.device)
        tm.tm_rmsnorm(x, H, None, 0, None, 0, w, T, H, EPS, y, H, None, rstd, CODE, CODE, CODE)
        ctx.save_for_backward(x, w, rstd)
        return y

    @staticmethod
    @first_derivatives
    def backward(ctx, dy):
        x, w, rstd = ctx.saved_tensors
        T, H = x.shape
        dy, dx, dw = dy.contiguous(), torch.empty_like(x), torch.empty_like(w) if ctx.needs_input_grad[1] else None
        need = tm.tm_rmsnorm_bwd_workspace_bytes(T, H)
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device=x.device)
        tm.tm_rmsnorm_bwd(dy, H, x, H, w, rstd, None, 0, dx, H, dw, T, H, CODE, CODE, ws, need)
        return dx if ctx.needs_input_grad[0] else None, dw


class Clip:
    """The gradients of some tensors, clipped together in place: the plan is laid out once, for the tensors it was given."""

    def __init__(self, grads, max_norm):
        sizes = [g.numel() for g in grads]
        kinds = {torch.float32: tm.TM_F32, torch.float16: tm.TM_F16, torch.bfloat16: tm.TM_BF16}
        dev = grads[0].device
        self.plan = tm.tm_clip_plan(grads, grads, sizes, [kinds[g.dtype] for g in grads]).to(dev)
        self.chunks, self.max_norm = tm.tm_clip_chunks(sizes), max_norm
        self.norm = torch.empty(1, device=dev)
        self.need = tm.tm_clip_workspace_bytes()
        self.ws = torch.empty(self.need, dtype=torch.uint8, device=dev)

    def __call__(self):
        tm.tm_clip_grads(self.plan, self.chunks, self.max_norm, 1e-6, self.norm, self.ws, self.need)
        return self.norm


def layer16(x, norm, gate, w1, w2, k, experts=Experts.apply, normed=Norm.apply):
    token, weight, starts = route(x.detach().float() @ gate, k)
    z = experts(act(experts(normed(x, norm)[token], w1, starts)), w2, starts)
    return torch.zeros(x.shape, dtype=torch.float32 if z.dtype != torch.float64 else z.dtype,
                       device=x.device).index_add(0, token, z.to(weight.dtype if z.dtype != torch.float64 else z.dtype) * weight[:, None])


def plain_experts(x, w, starts):
    s = starts.tolist()
    return torch.cat([x[a:b] @ w[e].T for e, (a, b) in enumerate(zip(s, s[1:]))])


def plain_norm(x, w):
    return x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * w


def train(T=150, H=256, F=384, E=6, k=2, seed=0, max_norm=0.5, dev="cuda"):
    """One step's gradients: clipped, their norm before, and the same layer's in 64 bits (unclipped)."""
    norm, gate, w1, w2 = parameters(H, F, E, seed, dev)
    g = torch.Generator(device=dev).manual_seed(seed + 1)
    x, c = (torch.randn(T, H, generator=g, device=dev) for _ in range(2))
    leaves = [t.to(TYPE).requires_grad_() for t in (x, norm, w1, w2)]
    wide = [t.detach().double().requires_grad_() for t in leaves]
    (layer16(leaves[0], leaves[1], gate, leaves[2], leaves[3], k) * c).sum().backward()
    (layer16(wide[0], wide[1], gate, wide[2], wide[3], k, plain_experts, plain_norm) * c).sum().backward()
    total = Clip([t.grad for t in leaves], max_norm)().clone()
    tm.tm_check()
    return [t.grad for t in leaves], total, [t.grad for t in wide]


if __name__ == "__main__":
    for replayed, direct, exact in serve():
        print(f"served: graph and direct calls differ by {float((replayed - direct).abs().max()):.1e}; quantisation changes "
              f"the output by {float((direct - exact).norm() / exact.norm()):.3f} of it")
    grads, total, wide = train()
    print(f"trained: norm {float(total):.4f} (64 bits {float(torch.stack([w.norm() for w in wide]).norm()):.4f}), "
          f"clipped to {float(torch.stack([t.double().norm() for t in grads]).norm()):.4f}")
