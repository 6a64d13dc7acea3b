"""Plain 64-bit definitions of the transformer-block operators, and the byte
layout of the 4-bit cache (include/tm.h), for the tests.  numpy only."""
import math

import numpy as np
import torch

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
CODE = {"f32": 0, "f16": 1, "bf16": 2}
U = 2.0 ** -24


def half_step(t):
    """Largest relative error of one rounding to type t, and the absolute one below its normal range."""
    f = torch.finfo(t)
    return f.eps / 2, f.tiny * f.eps / 2


def f64(x):
    return x.detach().to(torch.float64).cpu().numpy()


# ------------------------------------------------------------------ norm
def rmsnorm(x, r, w, eps):
    h = x if r is None else x + r
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h, rstd, h * rstd[:, None] * (1.0 if w is None else w)


def rmsnorm_bwd(dy, h, w, rstd, dr):
    n = h * rstd[:, None]
    g = dy * (1.0 if w is None else w)
    c = (g * n).mean(1, keepdims=True)
    dx = rstd[:, None] * (g - n * c)
    return dx if dr is None else dx + dr, (dy * n).sum(0)


# ------------------------------------------------------------------ rotation
def angles(pos, turns):
    """Radians of pos * turns * 2^-64 turns, the fraction exact."""
    pos, turns = [int(p) for p in pos], [int(t) for t in turns]
    f = [[((p * t + (1 << 63)) % (1 << 64) - (1 << 63)) / 2.0 ** 63 * math.pi for t in turns] for p in pos]
    return np.array(f, dtype=np.float64).reshape(len(pos), len(turns))


def rope(x, pos, turns, rot, gain=1.0, inter=False, inverse=False):
    """x [T, H, D] in 64 bits."""
    y = x.copy()
    if rot == 0:
        return y
    a = angles(pos, turns)[:, None, :]
    c, s = np.cos(a) * gain, np.sin(a) * gain * (-1.0 if inverse else 1.0)
    i0, i1 = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if inter else (np.arange(rot // 2), np.arange(rot // 2, rot))
    y[..., i0], y[..., i1] = x[..., i0] * c - x[..., i1] * s, x[..., i0] * s + x[..., i1] * c
    return y


# ------------------------------------------------------------------ the 4-bit cache
def half_by_float(x):
    with np.errstate(over="ignore"):
        return np.clip(x.astype(np.float32), -65504, 65504).astype(np.float16)


def hold(x):
    """Codes and (step, low) fp16 of vectors [..., D] in 64 bits."""
    bad = ~np.isfinite(x).all(-1, keepdims=True)
    z = np.where(bad, 0.0, x)
    lo, hi = z.min(-1, keepdims=True), z.max(-1, keepdims=True)
    step, low = half_by_float((hi - lo) / 15), half_by_float(lo)
    d = step.astype(np.float64)
    t = (z - low.astype(np.float64)) / np.where(d > 0, d, 1.0)
    c = np.where(d > 0, np.clip(np.rint(t), 0, 15), 0).astype(np.uint8)
    p = np.concatenate([step, low], -1)
    p = np.where(bad, np.float16(np.nan), p)
    return np.where(bad, np.uint8(0), c), p


def stands_for(codes, params):
    p = params.astype(np.float64)
    return p[..., 1:] + codes * p[..., :1]


def block_bytes(D):
    return 16 * (D + 8)


def empty_pool(pages, Hkv, page, D, fill=0xA5):
    return np.full((pages, Hkv, page // 16, block_bytes(D)), fill, dtype=np.uint8)


def put(pool, slot, page, head, which, codes, params):
    """Write one vector (which: 'k' or 'v') of one slot and head."""
    D = codes.size
    b = pool[slot // page, head, slot % page // 16]
    r = slot % 16
    packed = codes[0::2] | (codes[1::2] << 4)
    if which == "k":
        b[r * D // 2:(r + 1) * D // 2] = packed
        off = 16 * D + 4 * r
    else:
        for s in range(8):
            at = 8 * D + (r // 2) * D + s * (D // 8) + (r % 2) * (D // 16)
            b[at:at + D // 16] = packed[s * (D // 16):(s + 1) * (D // 16)]
        off = 16 * D + 64 + 4 * r
    b[off:off + 4] = params.view(np.uint8)


def append(pool, slots, page, k, v):
    """Hold k, v [T, Hkv, D] (64 bits, rotated) at their slots."""
    kc, kp = hold(k)
    vc, vp = hold(v)
    for t, s in enumerate(slots):
        if s < 0:
            continue
        for h in range(k.shape[1]):
            put(pool, s, page, h, "k", kc[t, h], kp[t, h])
            put(pool, s, page, h, "v", vc[t, h], vp[t, h])
    return stands_for(kc, kp), stands_for(vc, vp)


def random_cache(rng, pages, Hkv, page, D, shift=0.5):
    """A pool with every slot filled, and the values [pages * page, Hkv, D] it stands for."""
    n = pages * page
    k = rng.standard_normal((n, Hkv, D)) + shift * rng.standard_normal((1, Hkv, D))
    v = rng.standard_normal((n, Hkv, D))
    pool = empty_pool(pages, Hkv, page, D)
    kk, vv = append(pool, range(n), page, k, v)
    return pool, kk, vv


def attention(q, kk, vv, table, lens, qstart, page, scale, window=0, full=False):
    """q [Tq, Hq, D]; kk, vv [slots, Hkv, D].  Returns o, lse and, for tolerances, for each (query, head) the largest
    sum_d |q_d k_jd| * scale, the largest |v|, and how many keys it sees."""
    Tq, Hq, D = q.shape
    G = Hq // kk.shape[1]
    o, lse = np.zeros((Tq, Hq, D)), np.full((Tq, Hq), -np.inf)
    size, vmax, seen = np.zeros((Tq, Hq)), np.zeros((Tq, Hq)), np.zeros((Tq, Hq))
    for b in range(len(lens)):
        n = qstart[b + 1] - qstart[b]
        for i in range(n):
            p = lens[b] - n + i
            hi = lens[b] if full else min(lens[b], p + 1)
            lo = max(0, p + 1 - window) if window else 0
            if hi <= lo:
                continue
            j = np.arange(lo, hi)
            at = np.asarray(table[b])[j // page] * page + j % page
            for h in range(Hq):
                t = qstart[b] + i
                k, v = kk[at, h // G], vv[at, h // G]
                s = k @ q[t, h] * scale
                m = s.max()
                e = np.exp(s - m)
                lse[t, h] = m + np.log(e.sum())
                o[t, h] = (e / e.sum()) @ v
                size[t, h] = (np.abs(k) @ np.abs(q[t, h])).max() * scale
                vmax[t, h] = np.abs(v).max()
                seen[t, h] = hi - lo
    return o, lse, size, vmax, seen
