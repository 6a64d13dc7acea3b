"""Thin ctypes binding of ``libtm.so`` (declared in ``include/tm.h``).

Argument marshalling only: every entry point keeps its C name and argument
order; pointers may be given as integers or as objects with ``data_ptr()``
(torch tensors); ``stream=None`` means torch's current CUDA stream when torch
is loaded, else the legacy default stream.  A non-OK status raises
``TmError`` (its ``.status`` holds the code).  There is no fallback: if the
library was not built this module raises on first use.
"""
from __future__ import annotations

import ctypes
import os
import sys
import threading

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libtm.so")

# status codes (tm_status)
TM_OK = 0
TM_ERR_INVALID_ARG = 1
TM_ERR_UNSUPPORTED_TILE = 2
TM_ERR_MISALIGNED = 3
TM_ERR_BROKEN_PROMISE = 4
TM_ERR_CUDA = 5
TM_ERR_WORKSPACE = 6
TM_ERR_TIMEOUT = 7
TM_ERR_INDEX = 8

# flags
TM_ALIGNED = 0x1
TM_PATH_SCALAR = 0x10
TM_PATH_VEC = 0x20
TM_PATH_TMA = 0x40
TM_PDL = 0x200  # overlapped launch; tm_affine takes it OR-ed into the variant

# tm_variant
TM_VAR_AUTO = 0
TM_VAR_SCALAR = 1
TM_VAR_VEC_UNALIGNED = 2
TM_VAR_VEC4 = 3
TM_VAR_VEC8 = 4
TM_VAR_NAIVE = 5
TM_VAR_STAGED = 6
TM_VAR_REGDIRECT = 7
TM_VAR_CLUSTER = 8

# tm_fill
TM_FILL_NEG_INF = 0
TM_FILL_ZERO = 1

# Every function include/tm.h declares, with its ctypes signature.
_i64, _i32, _u32, _f32, _vp, _sz = (ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32, ctypes.c_float,
                                    ctypes.c_void_p, ctypes.c_size_t)
_st = ctypes.c_int
SIGNATURES = {
    "tm_status_string": (ctypes.c_char_p, [_st]),
    "tm_version": (ctypes.c_int, []),
    "tm_affine": (_st, [_vp, _vp, _i64, _st, _vp]),
    "tm_scale2d": (_st, [_vp, _i64, _vp, _i64, _i64, _i64, _f32, _i32, _i32, _u32, _vp]),
    "tm_copy2d": (_st, [_vp, _i64, _vp, _i64, _i64, _i64, _i32, _i32, _u32, _vp]),
    "tm_channel_affine": (_st, [_vp, _i64, _i64, _i64, _vp, _vp, _i64, _i32, _vp, _i64, _i32, _i32, _u32, _vp]),
    "tm_padded_extent": (_i64, [_i64, _vp, _i32]),
    "tm_row_stride": (_i64, [_i64, _i32]),
    "tm_pad2d": (_st, [_vp, _i64, _i64, _i64, _vp, _i64, _i64, _i64, _vp]),
    "tm_rowsum": (_st, [_vp, _i64, _i64, _i64, _vp, _i32, _i32, _u32, _vp]),
    "tm_colsum_workspace_bytes": (_sz, [_i64, _i64, _i32, _i32, _st]),
    "tm_colsum": (_st, [_vp, _i64, _i64, _i64, _vp, _vp, _sz, _i32, _i32, _st, _u32, _vp]),
    "tm_rowmax_masked": (_st, [_vp, _i64, _i64, _i64, _vp, _i32, _i32, _st, _u32, _vp]),
    "tm_softmax_rowstats": (_st, [_vp, _i64, _i64, _i64, _vp, _vp, _i32, _i32, _st, _u32, _vp]),
    "tm_colsum_noalloc": (_st, [_vp, _i64, _i64, _i64, _vp, _i32, _i32, _st, _u32, _vp]),
    "tm_gemm_workspace_bytes": (_sz, [_i64, _i64, _i64, _i32]),
    "tm_gemm": (_st, [_vp, _i64, _vp, _i64, _vp, _i64, _i64, _i64, _i64, _f32, _f32, _i32, _i32, _i32, _u32,
                      _vp, _sz, _vp]),
    "tm_rmsnorm": (_st, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i64, _f32, _vp, _i64, _vp, _vp, _i32, _i32, _i32,
                         _i32, _u32, _vp]),
    "tm_rmsnorm_bwd_workspace_bytes": (_sz, [_i64, _i64]),
    "tm_rmsnorm_bwd": (_st, [_vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _vp, _i64, _vp, _i64, _i64, _i32, _i32, _vp, _sz,
                             _u32, _vp]),
    "tm_rope_turns": (_st, [_vp, _i32, _f32, _i32, _f32, _f32, _f32, _i64]),
    "tm_rope": (_st, [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _i32, _i32, _i32, _f32, _i32, _u32, _vp]),
    "tm_kv4_page_bytes": (_sz, [_i32, _i32, _i32]),
    "tm_kv4_append": (_st, [_vp, _i64, _i64, _vp, _i64, _i64, _i32, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _vp, _vp,
                            _i64, _i32, _i64, _i32, _i32, _i32, _f32, _i32, _u32, _vp]),
    "tm_kv4_gather": (_st, [_vp, _i64, _i32, _vp, _vp, _i64, _i64, _vp, _i64, _i64, _i64, _i32, _i32, _i32, _u32, _vp]),
    "tm_kv4_attention_workspace_bytes": (_sz, [_i32, _i64, _i32, _i64, _i32, _i32, _i32]),
    "tm_kv4_attention": (_st, [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _i32, _vp, _i64, _vp, _vp, _i32, _i64,
                               _i32, _i64, _i32, _i32, _i32, _f32, _i32, _i32, _vp, _sz, _u32, _vp]),
    "tm_quant_e4m3": (_st, [_vp, _i64, _i64, _i64, _vp, _i64, _vp, _i32, _i32, _u32, _vp]),
    "tm_gemm_e4m3": (_st, [_vp, _i64, _vp, _i32, _vp, _i64, _vp, _vp, _i64, _vp, _i32, _i64, _i64, _i64, _i32, _u32, _vp]),
    "tm_gemm_experts": (_st, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i32, _i64, _i64, _i64, _i32, _i32, _u32, _vp]),
    "tm_gemm_experts_bwd": (_st, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i32, _i64, _i64, _i64,
                                  _i32, _i32, _u32, _vp]),
    "tm_clip_chunks": (_i64, [_vp, _i32]),
    "tm_clip_plan": (_st, [_vp, _vp, _vp, _vp, _vp, _i32]),
    "tm_clip_workspace_bytes": (_sz, []),
    "tm_clip_grads": (_st, [_vp, _i64, _f32, _f32, _vp, _vp, _sz, _u32, _vp]),
    "tm_check": (_st, [_vp]),
    "tm_tile_walk_probe": (_st, [_i64, _i32, _vp, _vp]),
    "tm_scale2d_unchecked": (_st, [_vp, _i64, _vp, _i64, _i64, _i64, _f32, _i32, _i32, _vp]),
    "tm_wait_timeout_probe": (_st, [_vp]),
    "tm_read_probe_blocks": (_i64, [_i64, _i32]),
    "tm_read_probe": (_st, [_vp, _i64, _vp, _i32, _vp]),
    "tm_read_probe_fixed_share": (_i64, [_i64, _i32]),
    "tm_read_probe_fixed": (_st, [_vp, _i64, _vp, _i32, _vp]),
}

_lib = None
_lock = threading.Lock()


class TmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s" % (where, status_string(status)))


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libtm.so (once) and attach the signatures; raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError("libtm.so is not built (%s); run "
                                   "`python -m masking_tm_affine_gb300.build`" % path)
            lib = ctypes.CDLL(path)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
        return _lib


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(s) -> int | None:
    if s is None:
        torch = sys.modules.get("torch")
        if torch is not None and torch.cuda.is_initialized():
            # what torch.cuda.current_stream().cuda_stream reads, without building a Stream object (3.8 us a
            # call); those two are not torch's public functions, so a version may lack them
            raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
            if raw is None or device is None:
                return torch.cuda.current_stream().cuda_stream
            return raw(device())
        return None
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _ok(st: int, where: str) -> None:
    if st != TM_OK:
        raise TmError(st, where)


def status_string(st: int) -> str:
    return load().tm_status_string(st).decode()


def tm_version() -> int:
    return load().tm_version()


def tm_affine(a, out, n: int, variant: int = TM_VAR_AUTO, stream=None) -> None:
    _ok(load().tm_affine(_ptr(a), _ptr(out), n, variant, _stream(stream)), "tm_affine")


def tm_scale2d(X, ldx: int, Y, ldy: int, M: int, N: int, alpha: float, TM: int, TN: int,
               flags: int = 0, stream=None) -> None:
    _ok(load().tm_scale2d(_ptr(X), ldx, _ptr(Y), ldy, M, N, alpha, TM, TN, flags, _stream(stream)),
        "tm_scale2d")


def tm_copy2d(A, lda: int, B, ldb: int, M: int, N: int, TM: int, TN: int, flags: int = 0,
              stream=None) -> None:
    _ok(load().tm_copy2d(_ptr(A), lda, _ptr(B), ldb, M, N, TM, TN, flags, _stream(stream)), "tm_copy2d")


TM_CHANNELS_LAST = 0
TM_CHANNELS_FIRST = 1


def tm_channel_affine(X, ldx: int, R: int, K: int, scale, bias, C: int, layout: int, Y, ldy: int,
                      TM: int = 32, TN: int = 128, flags: int = 0, stream=None) -> None:
    _ok(load().tm_channel_affine(_ptr(X), ldx, R, K, _ptr(scale), _ptr(bias), C, layout, _ptr(Y), ldy, TM, TN,
                                 flags, _stream(stream)), "tm_channel_affine")


def tm_padded_extent(extent: int, tiles) -> int:
    arr = (ctypes.c_int32 * len(tiles))(*tiles)
    return int(load().tm_padded_extent(extent, ctypes.cast(arr, ctypes.c_void_p), len(tiles)))


def tm_row_stride(N: int, align_bytes: int = 16) -> int:
    return int(load().tm_row_stride(N, align_bytes))


def tm_pad2d(A, lda: int, M: int, N: int, B, ldb: int, Mp: int, Np: int, stream=None) -> None:
    _ok(load().tm_pad2d(_ptr(A), lda, M, N, _ptr(B), ldb, Mp, Np, _stream(stream)), "tm_pad2d")


def tm_rowsum(X, ldx: int, M: int, N: int, r, TM: int = 8, TN: int = 512, flags: int = 0,
              stream=None) -> None:
    _ok(load().tm_rowsum(_ptr(X), ldx, M, N, _ptr(r), TM, TN, flags, _stream(stream)), "tm_rowsum")


def tm_colsum_workspace_bytes(M: int, N: int, TM: int = 32, TN: int = 128,
                              variant: int = TM_VAR_AUTO) -> int:
    return int(load().tm_colsum_workspace_bytes(M, N, TM, TN, variant))


def tm_colsum(X, ldx: int, M: int, N: int, c, workspace, ws_bytes: int, TM: int = 32, TN: int = 128,
              variant: int = TM_VAR_AUTO, flags: int = 0, stream=None) -> None:
    _ok(load().tm_colsum(_ptr(X), ldx, M, N, _ptr(c), _ptr(workspace), ws_bytes, TM, TN, variant, flags,
                         _stream(stream)), "tm_colsum")


TM_NOALLOC_SCRATCH_BYTES = 8 << 20  # include/tm.h


def tm_colsum_noalloc(X, ldx: int, M: int, N: int, c, TM: int = 32, TN: int = 128,
                      variant: int = TM_VAR_AUTO, flags: int = 0, stream=None) -> None:
    """tm_colsum without a workspace, for callers that cannot allocate device
    memory; see include/tm.h for the scratch limit and the concurrency rule."""
    _ok(load().tm_colsum_noalloc(_ptr(X), ldx, M, N, _ptr(c), TM, TN, variant, flags, _stream(stream)),
        "tm_colsum_noalloc")


def tm_rowmax_masked(S, lds: int, M: int, N: int, m, BR: int = 8, BC: int = 64,
                     fill: int = TM_FILL_NEG_INF, flags: int = 0, stream=None) -> None:
    _ok(load().tm_rowmax_masked(_ptr(S), lds, M, N, _ptr(m), BR, BC, fill, flags, _stream(stream)),
        "tm_rowmax_masked")


def tm_softmax_rowstats(S, lds: int, M: int, N: int, m, l, BR: int = 8, BC: int = 64,
                        fill: int = TM_FILL_NEG_INF, flags: int = 0, stream=None) -> None:
    _ok(load().tm_softmax_rowstats(_ptr(S), lds, M, N, _ptr(m), _ptr(l), BR, BC, fill, flags, _stream(stream)),
        "tm_softmax_rowstats")


TM_GEMM_TF32 = 0x100  # include/tm.h


def tm_gemm_workspace_bytes(M: int, N: int, K: int, TN: int = 256) -> int:
    return load().tm_gemm_workspace_bytes(M, N, K, TN)


def tm_gemm(A, lda: int, B, ldb: int, C, ldc: int, M: int, N: int, K: int, alpha: float, beta: float,
            workspace, ws_bytes: int, TM: int = 256, TN: int = 256, TK: int = 32, flags: int = 0,
            stream=None) -> None:
    """C = alpha * (A B) + beta * C on the tensor cores (3xTF32 unless TM_GEMM_TF32).
    TM = 256 runs CTA pairs (the default, fastest); TM = 128 single CTAs."""
    _ok(load().tm_gemm(_ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc, M, N, K, alpha, beta, TM, TN, TK, flags,
                       _ptr(workspace), ws_bytes, _stream(stream)), "tm_gemm")


# Operators of a transformer block: element types, layouts and flags (include/tm.h)
TM_F32 = 0
TM_F16 = 1
TM_BF16 = 2
TM_E4M3 = 3
TM_ROPE_PLAIN = 0
TM_ROPE_LINEAR = 1
TM_ROPE_BASE = 2
TM_ROPE_BY_TURNS = 3
TM_ROPE_BY_DIM = 4
TM_ROPE_INTERLEAVED = 0x400
TM_ROPE_INVERSE = 0x800
TM_ATTN_FULL = 0x1000


def tm_rmsnorm(X, ldx: int, R, ldr: int, H, ldh: int, W, M: int, N: int, eps: float, Y, ldy: int, scales=None,
               rstd=None, xtype: int = TM_F32, wtype: int = TM_F32, ytype: int = TM_F32, group: int = 0,
               flags: int = 0, stream=None) -> None:
    """y = (x + r) * w / rms(x + r); with ytype TM_E4M3 in 8 bits, a scale a row or a group of columns."""
    _ok(load().tm_rmsnorm(_ptr(X), ldx, _ptr(R), ldr, _ptr(H), ldh, _ptr(W), M, N, eps, _ptr(Y), ldy, _ptr(scales),
                          _ptr(rstd), xtype, wtype, ytype, group, flags, _stream(stream)), "tm_rmsnorm")


def tm_rmsnorm_bwd_workspace_bytes(M: int, N: int) -> int:
    return int(load().tm_rmsnorm_bwd_workspace_bytes(M, N))


def tm_rmsnorm_bwd(DY, lddy: int, H, ldh: int, W, rstd, DR, lddr: int, DX, lddx: int, DW, M: int, N: int,
                   xtype: int = TM_F32, wtype: int = TM_F32, workspace=None, ws_bytes: int = 0, flags: int = 0,
                   stream=None) -> None:
    _ok(load().tm_rmsnorm_bwd(_ptr(DY), lddy, _ptr(H), ldh, _ptr(W), _ptr(rstd), _ptr(DR), lddr, _ptr(DX), lddx,
                              _ptr(DW), M, N, xtype, wtype, _ptr(workspace), ws_bytes, flags, _stream(stream)),
        "tm_rmsnorm_bwd")


def tm_rope_turns(rot: int, base: float, scaling: int = TM_ROPE_PLAIN, factor: float = 1.0, low: float = 0.0,
                  high: float = 0.0, orig: int = 0):
    """The rot/2 frequencies tm_rope and tm_kv4_append take, as a host ctypes array of unsigned 64-bit values
    (``numpy.ctypeslib.as_array(t).view("int64")`` makes it an array to copy to the device)."""
    arr = (ctypes.c_uint64 * max(rot // 2, 1))()
    _ok(load().tm_rope_turns(ctypes.cast(arr, ctypes.c_void_p), rot, base, scaling, factor, low, high, orig),
        "tm_rope_turns")
    return arr


def tm_rope(X, xs_tok: int, xs_head: int, Y, ys_tok: int, ys_head: int, pos, turns, T: int, H: int, D: int, rot: int,
            gain: float = 1.0, xtype: int = TM_F32, flags: int = 0, stream=None) -> None:
    _ok(load().tm_rope(_ptr(X), xs_tok, xs_head, _ptr(Y), ys_tok, ys_head, _ptr(pos), _ptr(turns), T, H, D, rot, gain,
                       xtype, flags, _stream(stream)), "tm_rope")


def tm_kv4_page_bytes(Hkv: int, D: int, page: int) -> int:
    return int(load().tm_kv4_page_bytes(Hkv, D, page))


def tm_kv4_append(Q, qs_tok: int, qs_head: int, QO, qos_tok: int, qos_head: int, Hq: int, K, ks_tok: int, ks_head: int,
                  V, vs_tok: int, vs_head: int, pos, turns, slots, pool, pages: int, page: int, T: int, Hkv: int,
                  D: int, rot: int, gain: float = 1.0, xtype: int = TM_F32, flags: int = 0, stream=None) -> None:
    """Rotate q into QO and k into the 4-bit cache, v as it is, in one launch."""
    _ok(load().tm_kv4_append(_ptr(Q), qs_tok, qs_head, _ptr(QO), qos_tok, qos_head, Hq, _ptr(K), ks_tok, ks_head,
                             _ptr(V), vs_tok, vs_head, _ptr(pos), _ptr(turns), _ptr(slots), _ptr(pool), pages, page, T,
                             Hkv, D, rot, gain, xtype, flags, _stream(stream)), "tm_kv4_append")


def tm_kv4_gather(pool, pages: int, page: int, slots, K, ks_tok: int, ks_head: int, V, vs_tok: int, vs_head: int,
                  T: int, Hkv: int, D: int, xtype: int = TM_F32, flags: int = 0, stream=None) -> None:
    _ok(load().tm_kv4_gather(_ptr(pool), pages, page, _ptr(slots), _ptr(K), ks_tok, ks_head, _ptr(V), vs_tok, vs_head,
                             T, Hkv, D, xtype, flags, _stream(stream)), "tm_kv4_gather")


def tm_kv4_attention_workspace_bytes(B: int, Tq: int, max_q: int, max_len: int, Hq: int, Hkv: int, D: int) -> int:
    return int(load().tm_kv4_attention_workspace_bytes(B, Tq, max_q, max_len, Hq, Hkv, D))


def tm_kv4_attention(Q, qs_tok: int, qs_head: int, O, os_tok: int, os_head: int, lse, pool, pages: int, page: int,
                     table, ldt: int, lens, qstart, B: int, Tq: int, max_q: int, max_len: int, Hq: int, Hkv: int,
                     D: int, scale: float, window: int = 0, xtype: int = TM_F32, workspace=None, ws_bytes: int = 0,
                     flags: int = 0, stream=None) -> None:
    """Attention of each sequence's newest queries over its pages of the 4-bit cache."""
    _ok(load().tm_kv4_attention(_ptr(Q), qs_tok, qs_head, _ptr(O), os_tok, os_head, _ptr(lse), _ptr(pool), pages, page,
                                _ptr(table), ldt, _ptr(lens), _ptr(qstart), B, Tq, max_q, max_len, Hq, Hkv, D, scale,
                                window, xtype, _ptr(workspace), ws_bytes, flags, _stream(stream)), "tm_kv4_attention")


def tm_quant_e4m3(X, ldx: int, M: int, N: int, Y, ldy: int, scales, rows: int = 1, xtype: int = TM_F32, flags: int = 0,
                  stream=None) -> None:
    """Codes of x in 8 bits, with a scale for each run of 128 columns of 1 or 128 rows."""
    _ok(load().tm_quant_e4m3(_ptr(X), ldx, M, N, _ptr(Y), ldy, _ptr(scales), rows, xtype, flags, _stream(stream)),
        "tm_quant_e4m3")


def tm_gemm_e4m3(A, lda: int, sa, group: int, B, ldb: int, sb, C, ldc: int, starts, E: int, M: int, N: int, K: int,
                 ctype: int = TM_F32, flags: int = 0, stream=None) -> None:
    """C = A B^T of 8-bit operands with their scales, each row with its expert's matrix."""
    _ok(load().tm_gemm_e4m3(_ptr(A), lda, _ptr(sa), group, _ptr(B), ldb, _ptr(sb), _ptr(C), ldc, _ptr(starts), E, M, N, K,
                            ctype, flags, _stream(stream)), "tm_gemm_e4m3")


def tm_gemm_experts(X, ldx: int, W, ldw: int, Y, ldy: int, starts, E: int, T: int, N: int, K: int, xtype: int = TM_BF16,
                    ytype: int = TM_BF16, flags: int = 0, stream=None) -> None:
    """Y[t] = W_e X[t] for the rows t of each expert e."""
    _ok(load().tm_gemm_experts(_ptr(X), ldx, _ptr(W), ldw, _ptr(Y), ldy, _ptr(starts), E, T, N, K, xtype, ytype, flags,
                               _stream(stream)), "tm_gemm_experts")


def tm_gemm_experts_bwd(DY, lddy: int, X, ldx: int, W, ldw: int, DX, lddx: int, DW, lddw: int, starts, E: int, T: int,
                        N: int, K: int, xtype: int = TM_BF16, wtype: int = TM_BF16, flags: int = 0, stream=None) -> None:
    """DX[t] = W_e^T DY[t] and DW_e = sum over e's rows of DY[t] X[t]^T; either may be None."""
    _ok(load().tm_gemm_experts_bwd(_ptr(DY), lddy, _ptr(X), ldx, _ptr(W), ldw, _ptr(DX), lddx, _ptr(DW), lddw,
                                   _ptr(starts), E, T, N, K, xtype, wtype, flags, _stream(stream)), "tm_gemm_experts_bwd")


TM_CLIP_CHUNK_BYTES = 32  # include/tm.h


def tm_clip_chunks(sizes) -> int:
    return int(load().tm_clip_chunks(ctypes.cast((_i64 * max(len(sizes), 1))(*sizes), _vp), len(sizes)))


def tm_clip_plan(grads, outs, sizes, types):
    """The table tm_clip_grads takes, as a torch byte tensor on the host, to be copied to the device.  ``outs`` may be
    None (only the norm), and so may any of its entries; an entry that is its gradient is clipped in place."""
    import torch
    n = len(sizes)
    if len(grads) != n or len(types) != n or (outs is not None and len(outs) != n):
        raise TmError(TM_ERR_INVALID_ARG, "tm_clip_plan")
    plan = torch.empty(max(tm_clip_chunks(sizes), 1) * TM_CLIP_CHUNK_BYTES, dtype=torch.uint8)
    table = lambda t, v: ctypes.cast((t * max(n, 1))(*v), _vp)  # noqa: E731
    _ok(load().tm_clip_plan(plan.data_ptr(), table(_vp, [_ptr(g) for g in grads]),
                            None if outs is None else table(_vp, [_ptr(o) for o in outs]), table(_i64, sizes),
                            table(_i32, types), n), "tm_clip_plan")
    return plan


def tm_clip_workspace_bytes() -> int:
    return int(load().tm_clip_workspace_bytes())


def tm_clip_grads(plan, chunks: int, max_norm: float, eps: float, norm, workspace, ws_bytes: int, flags: int = 0,
                  stream=None) -> None:
    """The norm of all gradients of the plan, and the gradients times min(1, max_norm / (norm + eps))."""
    _ok(load().tm_clip_grads(_ptr(plan), chunks, max_norm, eps, _ptr(norm), _ptr(workspace), ws_bytes, flags,
                             _stream(stream)), "tm_clip_grads")


def tm_check(stream=None) -> None:
    _ok(load().tm_check(_stream(stream)), "tm_check")


def tm_tile_walk_probe(K: int, T: int, out4, stream=None) -> None:
    _ok(load().tm_tile_walk_probe(K, T, _ptr(out4), _stream(stream)), "tm_tile_walk_probe")


def tm_read_probe_blocks(n: int, per_thread: int = 4) -> int:
    return int(load().tm_read_probe_blocks(n, per_thread))


def tm_read_probe(x, n: int, out, per_thread: int = 4, stream=None) -> None:
    """The plain streaming read of n floats (one fp32 sum per 1024*per_thread elements)."""
    _ok(load().tm_read_probe(_ptr(x), n, _ptr(out), per_thread, _stream(stream)), "tm_read_probe")


def tm_read_probe_fixed_share(n: int, blocks: int) -> int:
    return int(load().tm_read_probe_fixed_share(n, blocks))


def tm_read_probe_fixed(x, n: int, out, blocks: int, stream=None) -> None:
    """The same read with exactly `blocks` blocks, each summing its own fixed contiguous share."""
    _ok(load().tm_read_probe_fixed(_ptr(x), n, _ptr(out), blocks, _stream(stream)), "tm_read_probe_fixed")


def tm_wait_timeout_probe(stream=None) -> None:
    """A bounded wait that runs out (~1 s): the next tm_check raises TM_ERR_TIMEOUT."""
    _ok(load().tm_wait_timeout_probe(_stream(stream)), "tm_wait_timeout_probe")


def tm_scale2d_unchecked(X, ldx: int, Y, ldy: int, M: int, N: int, alpha: float, TM: int, TN: int,
                         stream=None) -> None:
    _ok(load().tm_scale2d_unchecked(_ptr(X), ldx, _ptr(Y), ldy, M, N, alpha, TM, TN, _stream(stream)),
        "tm_scale2d_unchecked")
