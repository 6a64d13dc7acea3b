"""Calls of several host threads: each on a stream of its own, none may depend on
what another asks for (the binding releases the interpreter's lock in a call)."""
import threading

import numpy as np
import pytest
import torch

import block_ref as ref
from masking_tm_affine_gb300 import tm

pytestmark = pytest.mark.gpu
U, EPS, BF16 = ref.U, 1e-5, 2


def at_once(works):
    """Every work on a thread of its own, started together; the first exception is raised here."""
    start, failed = threading.Barrier(len(works)), []

    def go(w):
        try:
            start.wait()
            w()
        except BaseException as e:  # noqa: B902
            failed.append(e)
    threads = [threading.Thread(target=go, args=(w,)) for w in works]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if failed:
        raise failed[0]


# Widths that one kernel instance serves with different amounts of shared memory: many rows (rows copied
# ahead), and the gradient of a few long ones.
@pytest.mark.parametrize("M,widths", [(304, (5120, 8192)), (8, (20000, 32768))])
def test_norm_of_two_widths(cuda, M, widths):
    calls = []
    for N in widths:
        g = torch.Generator(device="cuda").manual_seed(N)
        x, r, dy = (torch.randn(M, N, generator=g, device="cuda").bfloat16() for _ in range(3))
        w = torch.ones(N, device="cuda").bfloat16()
        h, y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)
        rstd, need = torch.empty(M, device="cuda"), tm.tm_rmsnorm_bwd_workspace_bytes(M, N)
        calls.append((N, torch.cuda.Stream(), x, r, h, w, y, rstd, dy, dx, dw, torch.empty(need, dtype=torch.uint8, device="cuda"), need))
    torch.cuda.synchronize()

    def work(N, st, x, r, h, w, y, rstd, dy, dx, dw, ws, need):
        # straight to the library, so that the threads spend their time in it, with short queues
        lib, p = tm.load(), lambda t: t.data_ptr()  # noqa: E731
        fwd = (p(x), N, p(r), N, p(h), N, p(w), M, N, EPS, p(y), N, None, p(rstd), BF16, BF16, BF16, 0, 0, st.cuda_stream)
        bwd = (p(dy), N, p(h), N, p(w), p(rstd), None, 0, p(dx), N, p(dw), M, N, BF16, BF16, p(ws), need, 0, st.cuda_stream)
        for i in range(20000):
            assert lib.tm_rmsnorm(*fwd) == tm.TM_OK, (N, i)
            assert lib.tm_rmsnorm_bwd(*bwd) == tm.TM_OK, (N, i)
            if i % 100 == 99:
                st.synchronize()
    at_once([lambda c=c: work(*c) for c in calls])
    tm.tm_check()
    torch.cuda.synchronize()
    half, _ = ref.half_step(torch.bfloat16)
    for N, _, x, r, h, w, y, rstd, dy, dx, dw, *_ in calls:
        hw, sw, yw = ref.rmsnorm(ref.f64(x), ref.f64(r), None, EPS)
        assert np.all(np.abs(ref.f64(y) - yw) <= (64 * U + half * (1 + 128 * U)) * np.abs(yw))
        h64, dy64 = ref.f64(h), ref.f64(dy)
        dxw, dww = ref.rmsnorm_bwd(dy64, h64, None, ref.f64(rstd), None)
        n = np.abs(h64) * ref.f64(rstd)[:, None]
        mean = (np.abs(dy64) * n).mean(1, keepdims=True)
        lim = U * ref.f64(rstd)[:, None] * (8 * np.abs(dy64) + 120 * n * mean)   # the norm tests' terms
        assert np.all(np.abs(ref.f64(dx) - dxw) <= lim + half * (np.abs(dxw) + lim))
        lim = U * (M + 128) * (np.abs(dy64) * n).sum(0)
        assert np.all(np.abs(ref.f64(dw) - dww) <= lim + half * (np.abs(dww) + lim))
