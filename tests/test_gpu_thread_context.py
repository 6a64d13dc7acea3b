"""A host thread's first call of the library may be one that builds tensor maps (the driver wants a context of the thread)."""
import threading

import pytest
import torch

from masking_tm_affine_gb300 import tm

pytestmark = pytest.mark.gpu


def test_gemm_as_a_threads_first_call(cuda):
    M, N, K = 130, 70, 40
    a, b = torch.randint(-4, 5, (M, K), device="cuda").float(), torch.randint(-4, 5, (K, N), device="cuda").float()
    c = torch.empty(M, N, device="cuda")
    need = tm.tm_gemm_workspace_bytes(M, N, K)
    raw = torch.empty(need + 1024, dtype=torch.uint8, device="cuda")
    ws = raw.data_ptr() + -raw.data_ptr() % 1024
    stream = torch.cuda.Stream().cuda_stream
    tm.tm_gemm(a, K, b, N, c, N, M, N, K, 1.0, 0.0, ws, need, stream=stream)   # the kernel and its limits are known
    torch.cuda.synchronize()
    c.fill_(float("nan"))
    torch.cuda.synchronize()
    failed = []

    def go():
        try:
            tm.tm_gemm(a, K, b, N, c, N, M, N, K, 1.0, 0.0, ws, need, stream=stream)
        except tm.TmError as e:
            failed.append(e)
    t = threading.Thread(target=go)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not failed and torch.equal(c, a @ b)
