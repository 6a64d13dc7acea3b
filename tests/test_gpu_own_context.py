"""A thread that works in a driver context of its own keeps it: calls that build tensor maps run in it and leave it current."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# A process of its own, without torch: whose only context is the one it makes.
CHILD = """
import ctypes
import numpy as np
from masking_tm_affine_gb300 import tm

cu = ctypes.CDLL("libcuda.so.1")
def ok(status):
    assert status == 0, status
own, now, dev = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_int()
ok(cu.cuInit(0))
ok(cu.cuDeviceGet(ctypes.byref(dev), 0))
ok(cu.cuCtxCreate_v2(ctypes.byref(own), 0, dev))

def buffer(a):
    p = ctypes.c_uint64()
    ok(cu.cuMemAlloc_v2(ctypes.byref(p), ctypes.c_size_t(a.nbytes)))
    ok(cu.cuMemcpyHtoD_v2(p, ctypes.c_void_p(a.ctypes.data), ctypes.c_size_t(a.nbytes)))
    return p.value

def back(p, a):
    out = np.empty_like(a)
    ok(cu.cuMemcpyDtoH_v2(ctypes.c_void_p(out.ctypes.data), ctypes.c_uint64(p), ctypes.c_size_t(a.nbytes)))
    return out

def kept():
    ok(cu.cuCtxGetCurrent(ctypes.byref(now)))
    assert now.value == own.value, "the thread's context was replaced"

g = np.random.default_rng(0)
ints = lambda *s: g.integers(-4, 5, s).astype(np.float32)

M, N, K = 130, 72, 40
a, b, c = ints(M, K), ints(K, N), np.zeros((M, N), np.float32)
need = tm.tm_gemm_workspace_bytes(M, N, K)
raw = buffer(np.zeros(need + 1024, np.uint8))
pc = buffer(c)
tm.tm_gemm(buffer(a), K, buffer(b), N, pc, N, M, N, K, 1.0, 0.0, raw + -raw % 1024, need)
kept()
tm.tm_check()
assert np.array_equal(back(pc, c), a @ b)

for T in (20, 700):                       # small tiles; pairs of SMs
    N, K = 520, 264
    x, w, y = ints(T, K).astype(np.float16), ints(N, K).astype(np.float16), np.zeros((T, N), np.float32)
    py = buffer(y)
    tm.tm_gemm_experts(buffer(x), K, buffer(w), K, py, N, None, 1, T, N, K, tm.TM_F16, tm.TM_F32)
    kept()
    tm.tm_check()
    assert np.array_equal(back(py, y), x.astype(np.float32) @ w.astype(np.float32).T)

M, N = 4096, 2048                         # staged column sums
x, s = ints(M, N), np.zeros(N, np.float32)
ps = buffer(s)
need = tm.tm_colsum_workspace_bytes(M, N, 32, 128, tm.TM_VAR_STAGED)
tm.tm_colsum(buffer(x), N, M, N, ps, buffer(np.zeros(max(need, 16), np.uint8)), need, 32, 128, tm.TM_VAR_STAGED)
kept()
tm.tm_check()
assert np.array_equal(back(ps, s), x.sum(0))
kept()
print("kept")
"""


def test_a_context_of_the_threads_own_stays_current(cuda):
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "kept", r.stdout + r.stderr
