"""The attention half of a decoder block, served and differentiated.

serve()  -- ragged prompts in one call, then single tokens through a CUDA graph:
            residual addition + RMS norm, the q/k/v product, rotation of q and k and the
            append to a paged 4-bit cache, attention over it, the output product.  The
            tokens the graph produced are then run again as one prompt, which takes the
            attention's other forms over the same cache format; both must agree.
train()  -- the norm, the query product and the rotation, with the gradient back through
            all three, beside a difference quotient of the loss.

Weights and inputs are random; everything is fp32, the type of the library's gemm.

    python examples/decoder_block.py
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from masking_tm_affine_gb300 import tm  # noqa: E402

EPS = 1e-5


def gemm(A, B):
    """A [M, K] times B [K, N], both contiguous."""
    (M, K), N = A.shape, B.shape[1]
    C = torch.empty(M, N, device=A.device)
    raw = torch.empty(tm.tm_gemm_workspace_bytes(M, N, K) + 1024, dtype=torch.uint8, device=A.device)
    at = -raw.data_ptr() % 1024  # the workspace starts on a 1024-byte boundary
    tm.tm_gemm(A, K, B, N, C, N, M, N, K, 1.0, 0.0, raw[at:], raw.numel() - at)
    return C


def turns_of(rot, base, dev):
    t = tm.tm_rope_turns(rot, base)
    return torch.from_numpy(np.ctypeslib.as_array(t).view("int64").copy()).to(dev)


class Block:
    """One block's attention half and its cache: `pages` pages of `page` tokens."""

    def __init__(self, E, Hq, Hkv, D, page, pages, seed, dev):
        self.E, self.Hq, self.Hkv, self.D, self.page, self.pages = E, Hq, Hkv, D, page, pages
        g = torch.Generator(device=dev).manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
        self.norm = 1.0 + 0.1 * rand(E)
        self.qkv = rand(E, (Hq + 2 * Hkv) * D) / E**0.5
        self.out = rand(Hq * D, E) / (Hq * D) ** 0.5
        self.turns = turns_of(D, 10000.0, dev)
        self.pool = torch.zeros(pages * tm.tm_kv4_page_bytes(Hkv, D, page), dtype=torch.uint8, device=dev)

    def __call__(self, x, h, pos, slots, table, lens, qstart, max_q, max_len):
        """x [T, E] joins the residual stream h [T, E] in place; returns the block's addition to it."""
        T, (Hq, Hkv, D) = x.shape[0], (self.Hq, self.Hkv, self.D)
        dev, B, W = x.device, lens.numel(), (Hq + 2 * Hkv) * D
        y = torch.empty_like(x)
        tm.tm_rmsnorm(x, self.E, h, self.E, h, self.E, self.norm, T, self.E, EPS, y, self.E)
        p = gemm(y, self.qkv)
        q, k, v = p, p[:, Hq * D:], p[:, (Hq + Hkv) * D:]  # heads at stride D, tokens at stride W
        tm.tm_kv4_append(q, W, D, q, W, D, Hq, k, W, D, v, W, D, pos, self.turns, slots, self.pool, self.pages,
                         self.page, T, Hkv, D, D)
        o = torch.empty(T, Hq * D, device=dev)
        need = tm.tm_kv4_attention_workspace_bytes(B, T, max_q, max_len, Hq, Hkv, D)
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
        tm.tm_kv4_attention(q, W, D, o, Hq * D, D, None, self.pool, self.pages, self.page, table, table.shape[1], lens,
                            qstart, B, T, max_q, max_len, Hq, Hkv, D, D**-0.5, workspace=ws, ws_bytes=need)
        return gemm(o, self.out)


def slots_of(table, page, seq, pos):
    return table[seq, pos // page].long() * page + pos % page


def serve(prompts=(5, 130, 1, 64), steps=6, E=256, Hq=8, Hkv=2, D=64, page=32, seed=0, dev="cuda"):
    """Returns the last step's outputs [B, E] from the graph and from one prompt of the same tokens."""
    B, total = len(prompts), [n + steps for n in prompts]
    per = -(-max(total) // page)
    # pages in no particular order, as an allocator would hand them out
    order = torch.randperm(B * per, generator=torch.Generator().manual_seed(seed))
    table = order.reshape(B, per).to(torch.int32).to(dev)
    g = torch.Generator(device=dev).manual_seed(seed + 1)
    x = [torch.randn(n, E, generator=g, device=dev) for n in total]

    def prompt(block, counts):
        """The first counts[b] tokens of every sequence."""
        seq = torch.cat([torch.full((n,), b) for b, n in enumerate(counts)]).to(dev)
        pos = torch.cat([torch.arange(n) for n in counts]).to(dev)
        qstart = torch.tensor([0, *np.cumsum(counts)], dtype=torch.int32, device=dev)
        lens = torch.tensor(counts, dtype=torch.int32, device=dev)
        xs = torch.cat([t[:n] for t, n in zip(x, counts)])
        h = torch.zeros_like(xs)
        return block(xs, h, pos, slots_of(table, page, seq, pos), table, lens, qstart, max(counts), max(counts)), qstart

    block = Block(E, Hq, Hkv, D, page, B * per, seed + 2, dev)
    prompt(block, prompts)
    # a step: the cache grows by a token a sequence; everything it reads lives at fixed addresses
    xs, h = torch.empty(B, E, device=dev), torch.empty(B, E, device=dev)
    pos, seq = torch.tensor(prompts, device=dev), torch.arange(B, device=dev)
    lens = pos.to(torch.int32)

    def step():
        h.zero_()
        lens.add_(1)
        y = block(xs, h, pos, slots_of(table, page, seq, pos), table, lens, None, 1, max(total))
        pos.add_(1)
        return y

    def load(i):
        xs.copy_(torch.stack([t[n + i] for t, n in zip(x, prompts)]))

    load(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # the first step as it is: a capture wants everything loaded
        y = step()
    torch.cuda.current_stream().wait_stream(side)
    if steps > 1:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = step()
        for i in range(1, steps):
            load(i)
            graph.replay()
    again, qstart = prompt(Block(E, Hq, Hkv, D, page, B * per, seed + 2, dev), total)
    tm.tm_check()
    return y, again[qstart[1:].long() - 1]


def train(T=37, E=256, H=4, D=64, seed=0, dev="cuda"):
    """Returns the loss's derivative along a random direction of x and of the norm's weights: from the gradient,
    and from a difference quotient."""
    g = torch.Generator(device=dev).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    x, w, wq, c = rand(T, E), 1.0 + 0.1 * rand(E), rand(E, H * D) / E**0.5, rand(T, H * D)
    pos, turns = torch.arange(T, device=dev), turns_of(D, 10000.0, dev)

    def forward(x, w):
        y, rstd = torch.empty_like(x), torch.empty(T, device=dev)
        tm.tm_rmsnorm(x, E, None, 0, None, 0, w, T, E, EPS, y, E, rstd=rstd)
        q = gemm(y, wq)
        tm.tm_rope(q, H * D, D, q, H * D, D, pos, turns, T, H, D, D)
        return q, rstd

    def loss(x, w):
        return float((forward(x, w)[0].double() * c.double()).sum())

    _, rstd = forward(x, w)
    dq = torch.empty_like(c)  # the rotation's gradient is the rotation back
    tm.tm_rope(c, H * D, D, dq, H * D, D, pos, turns, T, H, D, D, flags=tm.TM_ROPE_INVERSE)
    dy = gemm(dq, wq.t().contiguous())
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    need = tm.tm_rmsnorm_bwd_workspace_bytes(T, E)
    tm.tm_rmsnorm_bwd(dy, E, x, E, w, rstd, None, 0, dx, E, dw, T, E,
                      workspace=torch.empty(max(need, 16), dtype=torch.uint8, device=dev), ws_bytes=need)
    ux, uw, e = rand(T, E), rand(E), 2.0**-7
    slope = float((dx.double() * ux.double()).sum() + (dw.double() * uw.double()).sum())
    quotient = (loss(x + e * ux, w + e * uw) - loss(x - e * ux, w - e * uw)) / (2 * e)
    tm.tm_check()
    return slope, quotient


if __name__ == "__main__":
    graph, whole = serve()
    print(f"served: {graph.shape[0]} sequences, largest difference of the two ways {float((graph - whole).abs().max()):.2e} "
          f"of {float(whole.abs().max()):.2f}")
    slope, quotient = train()
    print(f"trained: derivative {slope:.5f}, difference quotient {quotient:.5f}")
