"""The 4-bit paged cache: tm_kv4_append byte for byte against its definition in
64 bits (codes, steps and lows are whole decisions, so there is no tolerance),
and tm_kv4_gather within its roundings (one fp32 multiply-add, one to the type).
"""
import numpy as np
import pytest
import torch

import block_ref as ref
from masking_tm_affine_gb300 import tm

pytestmark = pytest.mark.gpu


def dev_turns(t):
    return torch.from_numpy(np.ctypeslib.as_array(t).view(np.int64).copy()).cuda()


def run_append(rng, kind, T, Hq, Hkv, D, rot, page, pages, slots, inter, values=None, shift=0, gain=1.0):
    t = ref.TYPES[kind]
    H = Hq + 2 * Hkv
    x = rng.standard_normal((T, H, D)) if values is None else values
    buf = torch.zeros(T * H * D + 16, dtype=t, device="cuda")
    qkv = buf[shift:][:T * H * D].view(T, H, D)
    qkv.copy_(torch.from_numpy(x).to(t))
    pos = rng.integers(0, 1 << 30, T)
    turns = tm.tm_rope_turns(max(rot, 2), 500000.0)
    pool = torch.from_numpy(ref.empty_pool(pages + 1, Hkv, page, D)).cuda()  # the last page is not the call's
    qo = torch.full((T, max(Hq, 1), D), 9.0, dtype=t, device="cuda")
    S = torch.from_numpy(np.asarray(slots, dtype=np.int64)).cuda()
    tm.tm_kv4_append(qkv, H * D, D, qo, max(Hq, 1) * D, D, Hq, qkv[:, Hq:], H * D, D, qkv[:, Hq + Hkv:], H * D, D,
                     torch.from_numpy(pos).cuda(), dev_turns(turns), S, pool, pages, page, T, Hkv, D, rot, gain,
                     ref.CODE[kind], tm.TM_ROPE_INTERLEAVED if inter else 0)
    x64 = ref.f64(qkv)
    qk = ref.rope(x64[:, :Hq + Hkv], pos, turns, rot, float(np.float32(gain)), inter)
    want = ref.empty_pool(pages + 1, Hkv, page, D)
    held = [s if 0 <= s < pages * page else -1 for s in slots]
    kk, vv = ref.append(want, held, page, qk[:, Hq:], x64[:, Hq + Hkv:])
    return pool, want, qo, qk[:, :Hq], x64[:, :Hq], S, kk, vv


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,page,shift", [
    (1, 1, 1, 64, 64, 16, 0), (1, 32, 8, 128, 128, 16, 0), (37, 4, 2, 128, 64, 48, 0), (20, 0, 3, 256, 256, 32, 0),
    (33, 3, 1, 64, 0, 16, 0), (9, 2, 2, 256, 16, 128, 0), (40, 8, 8, 128, 128, 64, 1), (200, 2, 4, 64, 32, 16, 0)])
def test_append_and_gather(cuda, kind, inter, T, Hq, Hkv, D, rot, page, shift):
    rng = np.random.default_rng(T + D + rot + page)
    pages = -(-T // page) + 3
    slots = rng.permutation(pages * page)[:T].tolist()
    if T > 4:
        slots[3] = -1
    pool, want, qo, qw, q64, S, kk, vv = run_append(rng, kind, T, Hq, Hkv, D, rot, page, pages, slots, inter, shift=shift)
    tm.tm_check()
    assert np.array_equal(pool.cpu().numpy(), want)
    t = ref.TYPES[kind]
    r, a = ref.half_step(t)
    if Hq:
        err = np.abs(q64) + np.abs(q64).max(-1, keepdims=True)      # at least |a| + |b|
        assert np.all(np.abs(ref.f64(qo) - qw) <= 1.5 * 2.0 ** -22 * err + r * np.abs(qw) * (1 + 1e-5) + a)
    k, v = torch.full((T, Hkv, D), 9.0, dtype=t, device="cuda"), torch.full((T, Hkv, D), 9.0, dtype=t, device="cuda")
    tm.tm_kv4_gather(pool, pages, page, S, k, Hkv * D, D, v, Hkv * D, D, T, Hkv, D, ref.CODE[kind])
    both = torch.full((T, Hkv, 2, D), 9.0, dtype=t, device="cuda")  # K and V interleaved by heads
    tm.tm_kv4_gather(pool, pages, page, S, both, 2 * Hkv * D, 2 * D, both[:, :, 1], 2 * Hkv * D, 2 * D, T, Hkv, D,
                     ref.CODE[kind])
    tm.tm_check()
    live = np.array(slots) >= 0
    for got, w in ((k, kk), (v, vv)):
        g = ref.f64(got)
        assert np.all(np.abs(g - w)[live] <= (2.0 ** -24 + r) * (1 + 1e-6) * np.abs(w)[live] + a)
        assert not g[~live].any()
    assert torch.equal(both[:, :, 0], k) and torch.equal(both[:, :, 1], v)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_append_hard_roundings(cuda, kind):
    # vectors where fp32 cannot decide: offsets far above the spread, exact ties, constants, tiny and huge values
    rng = np.random.default_rng(11)
    T, Hkv, D = 64, 2, 128
    x = np.zeros((T, 2 * Hkv, D))
    x[0:8] = 100.0 + rng.standard_normal((8, 4, D)) * 1e-2
    x[8:16] = rng.integers(0, 16, (8, 4, D))            # codes at whole steps
    x[16:24] = rng.integers(0, 31, (8, 4, D)) / 2.0     # and halfway between them
    x[24:28] = rng.standard_normal((4, 4, 1))           # constant vectors: step 0
    x[28:32] = rng.standard_normal((4, 4, D)) * 1e-6    # steps among fp16's subnormal numbers
    x[32:36] = rng.standard_normal((4, 4, D)) * 1e5     # steps or lows beyond fp16: clamped
    x[36:40] = rng.standard_normal((4, 4, D)) * 1e30
    x[40:44] = np.sign(rng.standard_normal((4, 4, D)))  # two values only
    x[44:] = rng.standard_normal((20, 4, D))
    for rot in (0, 128):
        pool, want, *_ = run_append(rng, kind, T, 0, Hkv, D, rot, 16, 4, list(range(T)), False, values=x)
        tm.tm_check()
        assert np.array_equal(pool.cpu().numpy(), want), rot


def test_append_many_values_exactly(cuda):
    # four million rotated values: some thousands lie where fp32 alone would decide wrongly or not at all
    rng = np.random.default_rng(12)
    T, Hkv, D = 4096, 8, 128
    x = torch.from_numpy(rng.standard_normal((T, 2 * Hkv, D))).float().cuda()
    pos = rng.integers(0, 1 << 20, T)
    turns = tm.tm_rope_turns(D, 500000.0)
    pool = torch.zeros(T // 16 * tm.tm_kv4_page_bytes(Hkv, D, 16), dtype=torch.uint8, device="cuda")
    tm.tm_kv4_append(None, 0, 0, None, 0, 0, 0, x, 2 * Hkv * D, D, x[:, Hkv:], 2 * Hkv * D, D, torch.from_numpy(pos).cuda(),
                     dev_turns(turns), torch.arange(T, device="cuda"), pool, T // 16, 16, T, Hkv, D, D)
    tm.tm_check()
    f = ((pos[:, None] * np.ctypeslib.as_array(turns).astype(object)[None]) % (1 << 64)).astype(np.uint64)
    ang = f.view(np.int64).astype(np.float64) * 2.0 ** -63 * np.pi
    x64 = ref.f64(x)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    a, b = x64[:, :Hkv, :64], x64[:, :Hkv, 64:]
    kc, kp = ref.hold(np.concatenate([a * c - b * s, a * s + b * c], -1))
    vc, vp = ref.hold(x64[:, Hkv:])
    P = pool.cpu().numpy().reshape(T // 16, Hkv, ref.block_bytes(D))
    kb = (kc[..., 0::2] | (kc[..., 1::2] << 4)).reshape(T // 16, 16, Hkv, 64).transpose(0, 2, 1, 3)
    assert np.array_equal(P[..., :1024].reshape(kb.shape), kb)
    vb = (vc[..., 0::2] | (vc[..., 1::2] << 4)).reshape(T // 16, 8, 2, Hkv, 8, 8).transpose(0, 3, 1, 4, 2, 5)
    assert np.array_equal(P[..., 1024:2048].reshape(vb.shape), vb)
    for off, p in ((2048, kp), (2112, vp)):
        w = p.view(np.uint16).reshape(T // 16, 16, Hkv, 2).transpose(0, 2, 1, 3)
        assert np.array_equal(np.ascontiguousarray(P[..., off:off + 64]).view(np.uint16).reshape(w.shape), w)


def test_append_not_finite(cuda):
    rng = np.random.default_rng(13)
    x = rng.standard_normal((8, 2, 64))
    x[1, 0, 5], x[2, 1, 6], x[3, 0, 7] = np.nan, np.inf, -np.inf
    pool, want, _, _, _, S, kk, vv = run_append(rng, "f32", 8, 0, 1, 64, 0, 16, 1, list(range(8)), False, values=x)
    k, v = torch.empty(8, 1, 64, device="cuda"), torch.empty(8, 1, 64, device="cuda")
    tm.tm_kv4_gather(pool, 1, 16, S, k, 64, 64, v, 64, 64, 8, 1, 64)
    tm.tm_check()
    for t in range(8):
        assert bool(torch.isnan(k[t]).all()) == (t in (1, 3)) and bool(torch.isnan(v[t]).all()) == (t == 2)
    ok = np.isfinite(kk).all(-1)
    assert np.all(np.abs(ref.f64(k) - kk)[ok] <= 1.1 * 2.0 ** -23 * np.abs(kk)[ok])


def test_slots_outside_the_pool(cuda):
    rng = np.random.default_rng(14)
    slots = [0, 64, 5, -1, -2, 1 << 60, 7, 63]       # the pool's 4 pages hold slots 0 .. 63
    pool, want, *_ , S, kk, vv = run_append(rng, "f32", 8, 1, 1, 64, 64, 16, 4, slots, False)
    with pytest.raises(tm.TmError) as e:
        tm.tm_check()
    assert e.value.status == tm.TM_ERR_INDEX
    assert np.array_equal(pool.cpu().numpy(), want)  # the others are written, nothing else is
    k = torch.full((8, 1, 64), 9.0, device="cuda")
    tm.tm_kv4_gather(pool, 4, 16, S, k, 64, 64, None, 0, 0, 8, 1, 64)
    with pytest.raises(tm.TmError) as e:
        tm.tm_check()
    assert e.value.status == tm.TM_ERR_INDEX
    assert not k[[1, 3, 4, 5]].any() and k[0].any()
    tm.tm_check()


def test_append_in_place_queries_on_a_stream(cuda):
    # q rotated inside the fused projection, on a stream of its own, overlapped
    rng = np.random.default_rng(15)
    T, Hq, Hkv, D = 50, 4, 2, 128
    x = torch.from_numpy(rng.standard_normal((T, Hq + 2 * Hkv, D))).to(torch.float16).cuda()
    x64, pos = ref.f64(x), np.arange(T) * 1000
    turns = tm.tm_rope_turns(D, 10000.0)
    pool = torch.zeros(4 * tm.tm_kv4_page_bytes(Hkv, D, 16), dtype=torch.uint8, device="cuda")
    P, TU, S = torch.from_numpy(pos).cuda(), dev_turns(turns), torch.arange(T, device="cuda")
    ld = (Hq + 2 * Hkv) * D
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    tm.tm_kv4_append(x, ld, D, x, ld, D, Hq, x[:, Hq:], ld, D, x[:, Hq + Hkv:], ld, D, P, TU, S, pool, 4, 16, T, Hkv, D, D,
                     1.0, tm.TM_F16, tm.TM_PDL, st)
    tm.tm_check(st)
    want = ref.empty_pool(4, Hkv, 16, D, 0)
    ref.append(want, range(T), 16, ref.rope(x64[:, Hq:Hq + Hkv], pos, turns, D), x64[:, Hq + Hkv:])
    assert np.array_equal(pool.cpu().numpy().reshape(want.shape), want)
    qw = ref.rope(x64[:, :Hq], pos, turns, D)
    assert np.all(np.abs(ref.f64(x)[:, :Hq] - qw) <= 2.0 ** -11 * np.abs(qw) * 1.001 + 1e-5)
    assert np.array_equal(ref.f64(x)[:, Hq:], x64[:, Hq:])
