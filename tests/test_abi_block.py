"""Host-side checks of the transformer-block entry points: every refusal below is
decided before any CUDA call (no GPU needed)."""
import math

import numpy as np
import pytest
import torch

import block_ref as ref
from masking_tm_affine_gb300 import tm

A, B, C, W, S, X = (0x7F0000000000 + (i << 36) for i in range(6))   # fake, far apart, aligned
INVALID, TILE, MIS, WS, OK = (tm.TM_ERR_INVALID_ARG, tm.TM_ERR_UNSUPPORTED_TILE, tm.TM_ERR_MISALIGNED, tm.TM_ERR_WORKSPACE,
                              tm.TM_OK)


@pytest.fixture(scope="module", autouse=True)
def lib():
    from masking_tm_affine_gb300 import build
    if torch.cuda.is_available():
        pytest.skip("fake-address host checks run only on a machine without a GPU")
    build.build()
    return tm.load()


def norm(X_=A, ldx=64, R=B, ldr=64, H=B, ldh=64, w=W, M=8, N=64, eps=1e-5, Y=C, ldy=64, sc=None, rstd=None, xt=2, wt=2,
         yt=2, group=0, flags=0):
    return tm.load().tm_rmsnorm(X_, ldx, R, ldr, H, ldh, w, M, N, eps, Y, ldy, sc, rstd, xt, wt, yt, group, flags, None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(xt=3, wt=3, yt=3)), (INVALID, dict(xt=9)), (INVALID, dict(wt=1)), (INVALID, dict(yt=0)),
    (INVALID, dict(flags=1)), (INVALID, dict(eps=-1.0)), (INVALID, dict(eps=math.nan)), (INVALID, dict(M=-1)),
    (INVALID, dict(ldx=63)), (INVALID, dict(ldy=63)), (INVALID, dict(ldr=63)), (INVALID, dict(ldh=63)),
    (INVALID, dict(X_=None)), (INVALID, dict(Y=None)), (INVALID, dict(sc=S)), (INVALID, dict(yt=3)),
    (TILE, dict(group=32)), (TILE, dict(yt=3, sc=S, group=48)), (TILE, dict(N=32769, ldx=32769, ldr=32769, ldh=32769, ldy=32769)),
    (MIS, dict(X_=A + 1)), (MIS, dict(w=W + 1)), (MIS, dict(yt=3, sc=S + 2)), (MIS, dict(rstd=S + 1)),
    (INVALID, dict(Y=A + 2)), (INVALID, dict(H=A + 128)), (INVALID, dict(Y=B)), (INVALID, dict(H=None, Y=B, ldy=72)),
    (INVALID, dict(yt=3, sc=S, Y=A)), (INVALID, dict(rstd=A)), (INVALID, dict(Y=W)), (INVALID, dict(yt=3, sc=C)),
    (OK, dict(M=0)), (OK, dict(N=0, X_=None, Y=None, R=None, H=None))])
def test_norm_refusals(want, kw):
    assert norm(**kw) == want


def bwd(DY=A, lddy=64, H=B, ldh=64, w=W, rstd=S, DR=None, lddr=64, DX=C, lddx=64, DW=X, M=8, N=64, xt=2, wt=2,
        ws=X + (1 << 30), wsb=8 * 64 * 4, flags=0):
    return tm.load().tm_rmsnorm_bwd(DY, lddy, H, ldh, w, rstd, DR, lddr, DX, lddx, DW, M, N, xt, wt, ws, wsb, flags, None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(xt=3)), (INVALID, dict(wt=1)), (INVALID, dict(flags=2)), (INVALID, dict(lddy=60)), (INVALID, dict(rstd=None)),
    (INVALID, dict(DY=None)), (INVALID, dict(DX=None)), (TILE, dict(N=40000, lddy=40000, ldh=40000, lddx=40000)),
    (MIS, dict(H=B + 1)), (MIS, dict(DW=X + 1)), (WS, dict(ws=None)), (WS, dict(wsb=8 * 64 * 4 - 1)), (WS, dict(ws=X + 4)),
    (INVALID, dict(DX=A + 2)), (INVALID, dict(DX=A, lddx=72)), (INVALID, dict(DW=A)), (INVALID, dict(DX=W)),
    (INVALID, dict(ws=C)), (INVALID, dict(DW=X + (1 << 30))), (INVALID, dict(DX=S)), (OK, dict(N=0)), (OK, dict(M=0, DW=None))])
def test_norm_gradient_refusals(want, kw):
    assert bwd(**kw) == want


def test_norm_workspace():
    f = tm.tm_rmsnorm_bwd_workspace_bytes
    assert f(8, 64) == 8 * 64 * 4 and f(10 ** 6, 100) == 608 * 100 * 4
    assert f(0, 64) == f(8, 0) == f(-1, 8) == f(8, 32769) == 0


def rope(X_=A, xt=64, xh=64, Y=C, yt=64, yh=64, pos=B, turns=W, T=8, H=1, D=64, rot=64, gain=1.0, e=2, flags=0):
    return tm.load().tm_rope(X_, xt, xh, Y, yt, yh, pos, turns, T, H, D, rot, gain, e, flags, None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(e=3)), (INVALID, dict(flags=1)), (INVALID, dict(rot=63)), (INVALID, dict(rot=66)), (INVALID, dict(rot=-2)),
    (INVALID, dict(T=-1)), (INVALID, dict(xt=-64)), (INVALID, dict(pos=None)), (INVALID, dict(turns=None)),
    (INVALID, dict(X_=None)), (INVALID, dict(Y=None)), (TILE, dict(D=1026, rot=2)), (MIS, dict(X_=A + 1)), (MIS, dict(pos=B + 4)),
    (INVALID, dict(Y=A + 2)), (INVALID, dict(Y=A, yt=128)), (INVALID, dict(Y=B)), (INVALID, dict(Y=W)), (OK, dict(T=0)),
    (OK, dict(H=0)), (OK, dict(D=0, rot=0))])
def test_rope_refusals(want, kw):
    assert rope(**kw) == want


@pytest.mark.parametrize("args", [(3, 1e4), (0, 1e4), (64, 1.0), (64, math.nan), (64, 1e4, 9), (64, 1e4, -1), (64, 1e4, 1, 0.5),
                                  (2, 1e4, 2, 4.0), (64, 1e4, 3, 4.0, 1.0, 4.0, 0), (64, 1e4, 3, 4.0, 4.0, 1.0, 8192),
                                  (64, 1e4, 4, 4.0, 0.0, 4.0, 8192), (64, math.inf)])
def test_turns_refusals(args):
    with pytest.raises(tm.TmError) as e:
        tm.tm_rope_turns(*args)
    assert e.value.status == INVALID


def test_turns_follow_their_definitions():
    rot, base, orig, factor = 64, 10000.0, 8192, 8.0
    f = base ** (-np.arange(0, rot, 2) / rot)
    n = orig * f / (2 * np.pi)
    got = lambda *a: np.ctypeslib.as_array(tm.tm_rope_turns(rot, base, *a)).astype(np.float64) / 2.0 ** 64 * 2 * np.pi  # noqa: E731
    close = lambda x, y: np.allclose(x, y, rtol=1e-12, atol=0)  # noqa: E731
    assert close(got(), f)
    assert close(got(tm.TM_ROPE_LINEAR, factor), f / factor)
    assert close(got(tm.TM_ROPE_BASE, factor), (base * factor ** (rot / (rot - 2))) ** (-np.arange(0, rot, 2) / rot))
    keep = np.clip((n - 1.0) / (4.0 - 1.0), 0, 1)
    assert close(got(tm.TM_ROPE_BY_TURNS, factor, 1.0, 4.0, orig), keep * f + (1 - keep) * f / factor)
    at = lambda x: rot * np.log(orig / (x * 2 * np.pi)) / (2 * np.log(base))  # noqa: E731
    d0, d1 = np.floor(at(32.0)), np.ceil(at(1.0))
    keep = 1 - np.clip((np.arange(rot // 2) - d0) / (d1 - d0), 0, 1)
    assert close(got(tm.TM_ROPE_BY_DIM, factor, 1.0, 32.0, orig), keep * f + (1 - keep) * f / factor)
    # 2^-64 turns: the angle at a far position keeps its fraction
    p, t = 10 ** 6 + 3, tm.tm_rope_turns(rot, base)
    assert abs(ref.angles([p], t)[0, 0] - math.remainder(p, 2 * math.pi)) < 1e-9


def append(Q=A, qt=512, qh=64, QO=C, qot=256, qoh=64, Hq=4, K=A + 512, kt=512, kh=64, V=A + 768, vt=512, vh=64, pos=B, turns=W,
           slots=S, pool=X, pages=4, page=16, T=8, Hkv=2, D=64, rot=64, gain=1.0, e=2, flags=0):
    return tm.load().tm_kv4_append(Q, qt, qh, QO, qot, qoh, Hq, K, kt, kh, V, vt, vh, pos, turns, slots, pool, pages, page, T,
                                   Hkv, D, rot, gain, e, flags, None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(e=4)), (INVALID, dict(flags=tm.TM_ROPE_INVERSE)), (INVALID, dict(T=-1)), (INVALID, dict(Hq=-1)),
    (INVALID, dict(pages=-1)), (INVALID, dict(rot=80)), (TILE, dict(D=96)), (TILE, dict(rot=24)), (TILE, dict(page=8)),
    (TILE, dict(page=0)), (INVALID, dict(Q=None)), (INVALID, dict(QO=None)), (INVALID, dict(K=None)), (INVALID, dict(V=None)),
    (INVALID, dict(slots=None)), (INVALID, dict(pos=None)), (INVALID, dict(pool=None)), (MIS, dict(pool=X + 8)),
    (MIS, dict(slots=S + 4)), (MIS, dict(K=A + 513)), (INVALID, dict(QO=A + 2, qot=512)), (INVALID, dict(QO=A + 512, qot=512)),
    (INVALID, dict(QO=S)), (INVALID, dict(pool=A)), (INVALID, dict(pool=C)), (OK, dict(T=0)), (OK, dict(Hq=0, Hkv=0, Q=None))])
def test_append_refusals(want, kw):
    assert append(**kw) == want


def gather(pool=X, pages=4, page=16, slots=S, K=A, kt=128, kh=64, V=B, vt=128, vh=64, T=8, Hkv=2, D=64, e=2, flags=0):
    return tm.load().tm_kv4_gather(pool, pages, page, slots, K, kt, kh, V, vt, vh, T, Hkv, D, e, flags, None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(e=3)), (INVALID, dict(flags=1)), (INVALID, dict(T=-1)), (TILE, dict(D=32)), (TILE, dict(page=24)),
    (INVALID, dict(pool=None)), (INVALID, dict(slots=None)), (MIS, dict(K=A + 1)), (MIS, dict(pool=X + 4)),
    (INVALID, dict(V=A + 2)), (INVALID, dict(K=X)), (INVALID, dict(V=S)), (OK, dict(T=0)), (OK, dict(K=None, V=None))])
def test_gather_refusals(want, kw):
    assert gather(**kw) == want


def attn(Q=A, qt=256, qh=64, O=C, ot=256, oh=64, lse=None, pool=X, pages=64, page=16, table=B, ldt=8, lens=S, qstart=None, b=2,
         Tq=2, max_q=1, max_len=128, Hq=4, Hkv=2, D=64, scale=0.125, window=0, e=2, ws=W, wsb=1 << 30, flags=0):
    return tm.load().tm_kv4_attention(Q, qt, qh, O, ot, oh, lse, pool, pages, page, table, ldt, lens, qstart, b, Tq, max_q,
                                      max_len, Hq, Hkv, D, scale, window, e, ws, wsb, flags, None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(e=3)), (INVALID, dict(flags=1)), (INVALID, dict(b=-1)), (INVALID, dict(Hq=3)), (INVALID, dict(Hkv=0)),
    (INVALID, dict(window=-1)), (INVALID, dict(window=5, flags=tm.TM_ATTN_FULL)), (TILE, dict(D=80)), (TILE, dict(page=20)),
    (INVALID, dict(Q=None)), (INVALID, dict(O=None)), (INVALID, dict(pool=None)), (INVALID, dict(table=None)),
    (INVALID, dict(lens=None)), (INVALID, dict(Tq=3)), (INVALID, dict(max_q=0)), (INVALID, dict(ldt=7)), (INVALID, dict(pages=0)),
    (INVALID, dict(max_len=-1)), (MIS, dict(Q=A + 1)), (MIS, dict(pool=X + 8)), (MIS, dict(lens=S + 2)), (MIS, dict(lse=C + (1 << 30) + 2)),
    (INVALID, dict(O=A)), (INVALID, dict(O=B)), (INVALID, dict(lse=C)), (INVALID, dict(lse=X)),
    (WS, dict(max_len=8192, ldt=512, ws=None)), (WS, dict(max_len=8192, ldt=512, wsb=100)), (WS, dict(max_len=8192, ldt=512, ws=W + 4)),
    (INVALID, dict(max_len=8192, ldt=512, ws=A)), (OK, dict(b=0, Tq=0)), (OK, dict(Tq=0))])
def test_attention_refusals(want, kw):
    assert attn(**kw) == want


def test_sizes():
    assert tm.tm_kv4_page_bytes(8, 128, 64) == 8 * 4 * 16 * 136
    assert tm.tm_kv4_page_bytes(8, 96, 64) == tm.tm_kv4_page_bytes(0, 64, 16) == tm.tm_kv4_page_bytes(1, 64, 8) == 0
    f = tm.tm_kv4_attention_workspace_bytes
    assert f(64, 64, 1, 100, 32, 8, 128) == 0                       # one split: nothing to join
    assert 0 < f(1, 1, 1, 131072, 64, 8, 128) < 32 << 20             # a slot or two a block, whatever the length
    assert f(0, 0, 1, 100, 4, 2, 64) == f(1, 1, 1, 100, 4, 3, 64) == f(1, 1, 1, 100, 4, 2, 80) == 0
