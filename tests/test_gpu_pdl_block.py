"""Overlapped launches (TM_PDL) of the transformer-block operators: the same bits as
without, with workspaces shared by neighbouring calls, and no store ahead of an
earlier kernel's read.  Inputs are written long before (the flag's condition)."""
import numpy as np
import pytest
import torch

from masking_tm_affine_gb300 import tm
from test_gpu_attention import Case

pytestmark = pytest.mark.gpu
P, BF16 = tm.TM_PDL, tm.TM_BF16


class Work:
    """One call of each operator on inputs of its own; outputs of a run are a list of tensors."""

    def __init__(self, qn):
        self.c = Case("bf16", [700, 150, 64], qn, 8, 2, 128, 16)
        c = self.c
        c.run()                                    # brings its device arrays
        self.T, self.H, self.D = 500, 10, 128
        g = torch.Generator(device="cuda").manual_seed(7)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
        self.x, self.pos = rand(self.T, self.H, self.D), torch.arange(self.T, device="cuda") * 77
        self.turns = torch.from_numpy(np.ctypeslib.as_array(tm.tm_rope_turns(128, 10000.0)).view("int64").copy()).cuda()
        self.slots = torch.randperm(c.pages * 16, generator=g, device="cuda")[:self.T].contiguous()
        self.norm = {}
        for M, N in ((40, 1000), (1300, 4096)):    # a block a row; rows copied ahead
            h, dy = rand(M, N), rand(M, N)
            rstd = 1 / h.float().pow(2).mean(1).add(1e-5).sqrt()
            need = tm.tm_rmsnorm_bwd_workspace_bytes(M, N)
            self.norm[M, N] = h, dy, rand(N), rstd, torch.empty(need, dtype=torch.uint8, device="cuda"), need
        torch.cuda.synchronize()

    def outputs(self):
        c, n = self.c, self.slots.numel()
        new = lambda *s, t=torch.bfloat16: torch.full(s, 9.0, dtype=t, device="cuda")  # noqa: E731
        out = [new(c.Tq, c.row), new(c.Tq, c.Hq, t=torch.float32), torch.empty_like(self.x), new(n, 2, 128), new(n, 2, 128)]
        for M, N in self.norm:
            out += [new(M, N), new(N)]
        return out

    def run(self, out, flags, stream):
        c, n = self.c, self.slots.numel()
        s = stream.cuda_stream
        o, lse, y, k, v = out[:5]
        tm.tm_kv4_attention(c.q, c.row, c.D, o, c.row, c.D, lse, c.dpool, c.pages, c.page, c.keep[0], c.table.shape[1],
                            c.keep[1], c.keep[2], 3, c.Tq, c.max_q, 700, c.Hq, c.Hkv, c.D, c.scale, 0, BF16, c.ws,
                            c.ws.numel() * 4, flags, s)
        tm.tm_rope(self.x, self.H * 128, 128, y, self.H * 128, 128, self.pos, self.turns, self.T, self.H, 128, 128, 1.0, BF16,
                   flags, s)
        tm.tm_kv4_gather(c.dpool, c.pages, c.page, self.slots, k, 256, 128, v, 256, 128, n, 2, 128, BF16, flags, s)
        for i, ((M, N), (h, dy, w, rstd, ws, need)) in enumerate(self.norm.items()):
            tm.tm_rmsnorm_bwd(dy, N, h, N, w, rstd, None, 0, out[5 + 2 * i], N, out[6 + 2 * i], M, N, BF16, BF16, ws, need,
                              flags, s)


@pytest.mark.parametrize("qn", [[1, 1, 1], [70, 64, 64]])   # single queries; chunks
def test_overlapped_calls_give_the_same_bits(cuda, qn):
    w, st = Work(qn), torch.cuda.Stream()
    plain = w.outputs()
    w.run(plain, 0, st)
    tm.tm_check(st)
    runs = [w.outputs() for _ in range(6)]
    torch.cuda.synchronize()
    for out in runs:                               # back to back: each call overlaps the one before
        w.run(out, P, st)
    tm.tm_check(st)
    for out in runs:
        assert all(torch.equal(a, b) for a, b in zip(out, plain))


@pytest.mark.parametrize("qn", [[1, 1, 1], [70, 64, 64]])
def test_a_store_waits_for_the_attention_before_it(cuda, qn):
    # the queries, the cache's pages and the output of an attention are overwritten by overlapped calls behind it
    w, st = Work(qn), torch.cuda.Stream()
    c = w.c
    plain = w.outputs()
    w.run(plain, 0, st)
    tm.tm_check(st)
    q0, pool0, Hq = c.q.clone(), c.dpool.clone(), c.Hq
    src = torch.randn(c.Tq, c.Hq, c.D, device="cuda").bfloat16()
    pos = torch.arange(c.Tq, device="cuda")
    kv = torch.randn(c.pages * 16, 2, 128, device="cuda").bfloat16()
    slots, kpos = torch.arange(c.pages * 16, device="cuda"), torch.zeros(c.pages * 16, dtype=torch.int64, device="cuda")
    for _ in range(8):
        c.q.copy_(q0)
        c.dpool.copy_(pool0)
        out = w.outputs()
        torch.cuda.synchronize()
        o, lse = out[:2]
        s = st.cuda_stream
        tm.tm_kv4_attention(c.q, c.row, c.D, o, c.row, c.D, lse, c.dpool, c.pages, c.page, c.keep[0], c.table.shape[1],
                            c.keep[1], c.keep[2], 3, c.Tq, c.max_q, 700, c.Hq, c.Hkv, c.D, c.scale, 0, BF16, c.ws,
                            c.ws.numel() * 4, 0, s)
        tm.tm_rope(src, Hq * 128, 128, c.q, c.row, 128, pos, w.turns, c.Tq, Hq, 128, 128, 1.0, BF16, P, s)
        tm.tm_kv4_append(None, 0, 0, None, 0, 0, 0, kv, 256, 128, kv, 256, 128, kpos, w.turns, slots, c.dpool, c.pages, c.page,
                         c.pages * 16, 2, 128, 128, 1.0, BF16, P, s)
        tm.tm_check(st)
        assert torch.equal(o, plain[0]) and torch.equal(lse, plain[1])
        assert not torch.equal(c.q, q0) and not torch.equal(c.dpool, pool0)
