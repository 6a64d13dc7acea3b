"""Host-side checks of the quantisation, the 8- and 16-bit products and the gradients' clipping: every refusal below is
decided before any CUDA call (no GPU needed)."""
import ctypes
import math

import pytest
import torch

from masking_tm_affine_gb300 import tm

A, B, C, W, S, X, Z = (0x7F0000000000 + (i << 36) for i in range(7))   # fake, far apart, aligned
INVALID, TILE, MIS, WS, OK = (tm.TM_ERR_INVALID_ARG, tm.TM_ERR_UNSUPPORTED_TILE, tm.TM_ERR_MISALIGNED, tm.TM_ERR_WORKSPACE,
                              tm.TM_OK)


@pytest.fixture(scope="module", autouse=True)
def lib():
    from masking_tm_affine_gb300 import build
    if torch.cuda.is_available():
        pytest.skip("fake-address host checks run only on a machine without a GPU")
    build.build()
    return tm.load()


def quant(x=A, ldx=64, M=8, N=64, y=B, ldy=64, sc=C, rows=1, t=2, flags=0):
    return tm.load().tm_quant_e4m3(x, ldx, M, N, y, ldy, sc, rows, t, flags, None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(t=3)), (INVALID, dict(t=-1)), (INVALID, dict(flags=1)), (INVALID, dict(x=None)), (INVALID, dict(y=None)),
    (INVALID, dict(sc=None)), (INVALID, dict(M=-1)), (INVALID, dict(N=-1)), (INVALID, dict(ldx=63)), (INVALID, dict(ldy=63)),
    (TILE, dict(rows=0)), (TILE, dict(rows=64)), (MIS, dict(x=A + 1)), (MIS, dict(t=0, x=A + 2)), (MIS, dict(sc=C + 2)),
    (INVALID, dict(y=A + 1023)), (INVALID, dict(sc=A)), (INVALID, dict(sc=B + 4)), (INVALID, dict(M=1 << 60, ldx=1 << 30)),
    (OK, dict(M=0)), (OK, dict(N=0, x=None, y=None, sc=None))])
def test_quantisation_refusals(want, kw):
    assert quant(**kw) == want


def e4m3(a=A, lda=64, sa=S, group=128, b=B, ldb=64, sb=X, c=C, ldc=40, starts=W, E=2, M=8, N=40, K=64, t=2, flags=0):
    return tm.load().tm_gemm_e4m3(a, lda, sa, group, b, ldb, sb, c, ldc, starts, E, M, N, K, t, flags, None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(t=3)), (INVALID, dict(flags=2)), (INVALID, dict(E=0)), (INVALID, dict(starts=None)), (TILE, dict(E=1025)),
    (INVALID, dict(M=-1)), (INVALID, dict(N=-1)), (INVALID, dict(K=-1)), (TILE, dict(M=1 << 31)), (TILE, dict(N=1 << 31)),
    (TILE, dict(K=1 << 31)), (TILE, dict(group=64)), (INVALID, dict(lda=63)), (INVALID, dict(ldb=48)), (INVALID, dict(ldc=39)),
    (INVALID, dict(a=None)), (INVALID, dict(b=None)), (INVALID, dict(c=None)), (INVALID, dict(sa=None)), (INVALID, dict(sb=None)),
    (MIS, dict(a=A + 8)), (MIS, dict(lda=72)), (MIS, dict(b=B + 1)), (MIS, dict(ldb=65)), (MIS, dict(c=C + 1)), (MIS, dict(sa=S + 1)),
    (MIS, dict(sb=X + 2)), (MIS, dict(starts=W + 2)), (INVALID, dict(c=A)), (INVALID, dict(c=B + 64)), (INVALID, dict(c=S)),
    (INVALID, dict(c=X)), (INVALID, dict(c=W)), (INVALID, dict(lda=1 << 40)), (OK, dict(M=0)), (OK, dict(N=0, b=None, sb=None))])
def test_e4m3_refusals(want, kw):
    assert e4m3(**kw) == want


def fwd(x=A, ldx=64, w=B, ldw=64, y=C, ldy=40, starts=W, E=2, T=8, N=40, K=64, xt=2, yt=2, flags=0):
    return tm.load().tm_gemm_experts(x, ldx, w, ldw, y, ldy, starts, E, T, N, K, xt, yt, flags, None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(xt=0, yt=0)), (INVALID, dict(xt=3)), (INVALID, dict(yt=1)), (INVALID, dict(flags=4)), (INVALID, dict(E=0)),
    (INVALID, dict(starts=None)), (TILE, dict(E=2000)), (INVALID, dict(T=-1)), (TILE, dict(T=(1 << 31) - 1)), (INVALID, dict(ldx=63)),
    (INVALID, dict(ldw=63)), (INVALID, dict(ldy=39)), (INVALID, dict(x=None)), (INVALID, dict(w=None)), (INVALID, dict(y=None)),
    (MIS, dict(x=A + 2)), (MIS, dict(ldx=68)), (MIS, dict(w=B + 8)), (MIS, dict(ldw=67)), (MIS, dict(y=C + 1)),
    (MIS, dict(yt=0, y=C + 2)), (INVALID, dict(y=A)), (INVALID, dict(y=B)), (INVALID, dict(y=W)), (OK, dict(T=0)),
    # columns of the rows' own tensor: beside them, or over their ends
    (INVALID, dict(ldx=128, y=A + 126, ldy=128)), (INVALID, dict(ldx=128, y=A + 178, ldy=128)), (INVALID, dict(ldx=128, y=A + 128, ldy=120)),
    (INVALID, dict(ldx=128, y=A - 78, ldy=128)), (OK, dict(N=0, w=None))])
def test_forward_refusals(want, kw):
    assert fwd(**kw) == want


def bwd(dy=A, lddy=40, x=B, ldx=64, w=C, ldw=64, dx=S, lddx=64, dw=X, lddw=64, starts=W, E=2, T=8, N=40, K=64, xt=2, wt=2, flags=0):
    return tm.load().tm_gemm_experts_bwd(dy, lddy, x, ldx, w, ldw, dx, lddx, dw, lddw, starts, E, T, N, K, xt, wt, flags, None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(xt=0, wt=0)), (INVALID, dict(wt=1)), (INVALID, dict(flags=1)), (INVALID, dict(E=0)), (INVALID, dict(starts=None)),
    (INVALID, dict(dy=None)), (INVALID, dict(x=None)), (INVALID, dict(w=None)), (INVALID, dict(lddy=39)), (INVALID, dict(lddx=63)),
    (INVALID, dict(lddw=63)), (INVALID, dict(ldx=63)), (INVALID, dict(ldw=63)), (MIS, dict(dy=A + 2)), (MIS, dict(lddy=44)),
    (MIS, dict(x=B + 4)), (MIS, dict(w=C + 2)), (MIS, dict(dx=S + 1)), (MIS, dict(wt=0, dw=X + 2)), (INVALID, dict(dx=A)),
    (INVALID, dict(dw=B)), (INVALID, dict(dx=C)), (INVALID, dict(dw=W)), (INVALID, dict(dx=X)), (OK, dict(dx=None, dw=None)),
    (OK, dict(T=0, dw=None)), (OK, dict(dx=None, N=0)), (OK, dict(dx=None, dw=None, x=None, w=None)), (OK, dict(K=0))])
def test_backward_refusals(want, kw):
    assert bwd(**kw) == want


def test_clip_plan():
    sizes, types = [0, 1, 16384, 16385, 70000], [0, 2, 1, 0, 2]
    grads, outs = [None, A, B, C, W], [None, None, B, S, X]
    assert tm.tm_clip_chunks([]) == tm.tm_clip_chunks([0, 0]) == 0 and tm.tm_clip_chunks([-1]) == -1 and tm.tm_clip_chunks([1]) == 1
    rows = tm.tm_clip_plan(grads, outs, sizes, types).view(torch.int64).view(-1, 4).tolist()
    assert len(rows) == tm.tm_clip_chunks(sizes)
    rows = [(r[0], r[1], r[2] & 0xFFFFFFFF, r[2] >> 32) for r in rows]
    for g, o, n, t in zip(grads, outs, sizes, types):      # each tensor's chunks follow one another and cover it
        e, at = (4, 2, 2)[t], 0
        while at < n:
            src, dst, count, kind = rows.pop(0)
            assert (src, dst, kind) == (g + at * e, 0 if o is None else o + at * e, t) and 0 < count <= n - at
            assert at % 8 == 0                             # whole 16-byte vectors from the tensor's start
            at += count
    assert not rows
    assert tm.tm_clip_plan([A], None, [5], [0]).view(torch.int64).tolist()[1] == 0


@pytest.mark.parametrize("want,args", [
    (INVALID, ([A], [B], [5], [3])), (INVALID, ([None], [B], [5], [0])), (MIS, ([A + 2], [B], [5], [0])), (MIS, ([A], [B + 1], [5], [2])),
    (INVALID, ([A], [A + 8], [5], [0])), (INVALID, ([A], [B], [-5], [0])), (INVALID, ([A, B], None, [5], [0]))])
def test_clip_plan_refusals(want, args):
    with pytest.raises(tm.TmError) as e:
        tm.tm_clip_plan(*args)
    assert e.value.status == want


def clip(plan=A, chunks=3, max_norm=1.0, eps=1e-6, norm=B, ws=C, wsb=32768, flags=0):
    return tm.load().tm_clip_grads(plan, chunks, max_norm, eps, norm, ws, wsb, flags, None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(plan=None)), (INVALID, dict(chunks=-1)), (INVALID, dict(norm=None)), (INVALID, dict(max_norm=-1.0)),
    (INVALID, dict(max_norm=math.nan)), (INVALID, dict(eps=-1.0)), (INVALID, dict(eps=math.nan)), (INVALID, dict(flags=1)),
    (MIS, dict(plan=A + 8)), (MIS, dict(norm=B + 2)), (WS, dict(ws=None)), (WS, dict(wsb=32767)), (WS, dict(ws=C + 8)),
    (INVALID, dict(ws=A)), (INVALID, dict(norm=A + 4)), (INVALID, dict(norm=C + 8))])
def test_clip_refusals(want, kw):
    assert tm.tm_clip_workspace_bytes() == 32768
    assert clip(**kw) == want


def test_the_c_plan_refuses_missing_tables():
    f = tm.load().tm_clip_plan
    one = (ctypes.c_int64 * 1)(5)
    assert f(None, None, None, None, None, 0) == OK
    assert f(None, None, None, ctypes.cast(one, ctypes.c_void_p), None, 1) == INVALID
