"""tm_kv4_attention where one row, one size or one window could spoil others: the
definition in 64 bits and the tolerances of test_gpu_attention.py."""
import numpy as np
import pytest
import torch

import block_ref as ref
from masking_tm_affine_gb300 import tm
from test_gpu_attention import KINDS, Case

pytestmark = pytest.mark.gpu


def check_rows(c, keep, window=0):
    """Rows (query, head) where keep is true against the definition."""
    q = c.q64()
    q[~keep] = 0.0
    o, l, size, vmax, seen = ref.attention(q, c.kk, c.vv, c.table, c.lens, c.qstart, c.page, c.scale, window)
    delta = (c.D + 16) * 2.0 ** -23 * 3 * size
    prob = 2.0 ** -11 if c.kind != "f32" else 2.0 ** -22
    tol = ((2 * delta + 2.0 ** -21 + 2 * prob + seen / 16 * 2.0 ** -23) * vmax)[..., None]
    r, a = ref.half_step(c.t)
    got, lse = ref.f64(c.o)[:, :c.Hq * c.D].reshape(o.shape), ref.f64(c.lse)
    err = np.abs(got - o) / (tol + r * (np.abs(o) + tol) + a)
    assert np.all(err[keep] <= 1), err[keep].max()
    live = keep & (seen > 0)
    assert np.all(np.abs(lse[live] - l[live]) <= delta[live] + 2.0 ** -21 + 2.0 ** -22 * np.abs(l[live]))
    return got


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv,qn", [(4, 1, [1, 1]), (8, 1, [2, 1]), (12, 2, [3, 2])])
def test_an_infinite_query_spoils_its_own_row_only(cuda, kind, D, Hq, Hkv, qn):
    c = Case(kind, [70, 300], qn, Hq, Hkv, D, 16)
    keep = np.ones((c.Tq, Hq), dtype=bool)
    for t, h, x in ((0, 1, np.inf), (c.Tq - 1, Hq - 1, -np.inf), (c.Tq - 1, 0, np.nan)):
        c.q[t, h * D + 7] = float(x)
        keep[t, h] = False
    c.run()
    tm.tm_check()
    got = check_rows(c, keep)
    assert np.isnan(got[~keep]).all()


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,qn,Hq,Hkv", [([400], [150], 2, 1), ([700, 90], [70, 64], 8, 2)])
def test_an_infinite_query_spoils_its_own_row_only_in_chunks(cuda, kind, D, lens, qn, Hq, Hkv):
    c = Case(kind, lens, qn, Hq, Hkv, D, 32)
    keep = np.ones((c.Tq, Hq), dtype=bool)
    for t, h, x in ((0, 0, np.inf), (c.Tq - 1, Hq - 1, -np.inf), (40, 1, np.nan)):
        c.q[t, h * D + 7] = float(x)
        keep[t, h] = False
    c.run()
    tm.tm_check()
    got = check_rows(c, keep)
    assert np.isnan(got[~keep]).all()


# A row far above the others (its own softmax is one key's, and not looked at here).
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("qn,Hq,D", [([1], 4, 128), ([3], 8, 64), ([160], 2, 128)])
def test_a_huge_query_takes_nothing_from_other_rows(cuda, kind, qn, Hq, D):
    c = Case(kind, [260], qn, Hq, 1, D, 16)
    keep = np.ones((c.Tq, Hq), dtype=bool)
    c.q[0, D:2 * D] *= 2.0 ** 60
    keep[0, 1] = False
    c.run()
    tm.tm_check()
    check_rows(c, keep)


# Windows that hide nothing, up to the largest an int32 holds, are no window: the same bits.  Long sequences (split
# over blocks), fewer keys than queries, an empty sequence; both forms.
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("lens,qn,Hq,Hkv,D", [
    ([5000, 1, 1281], [1, 1, 1], 8, 2, 128), ([130, 40, 3, 64, 0], [40, 5, 7, 0, 2], 6, 2, 64), ([7], [12], 4, 2, 128),
    ([300, 20, 129], [133, 90, 5], 4, 1, 128), ([1500, 900], [600, 900], 2, 1, 64)])
def test_a_window_that_hides_nothing(cuda, kind, lens, qn, Hq, Hkv, D):
    c = Case(kind, lens, qn, Hq, Hkv, D, 16)
    c.run()
    tm.tm_check()
    o, lse = c.o.clone(), c.lse.clone()
    c.check()
    for window in (2 ** 31 - 1, 2 ** 31 - 40, 2 ** 31 - 300, 2 ** 30, max(lens) + 1, max(lens)):
        c.o.fill_(9.0)
        c.lse.fill_(9.0)
        c.run(window=window)
        tm.tm_check()
        assert torch.equal(lse, c.lse) and torch.equal(o, c.o), window


# One key far above all others, and its value zero: the output is what the others leave, each a probability of about
# 2^-bits.  (Keys' and queries' parts of the tolerance are taken key by key.)  A probability is off by fp16's half step, or
# below fp16's range by 2^-32 (chunks: 2^-25 behind a reference 2^7 down) of the value.
def faint(c, bits, seed=0):
    rng = np.random.default_rng(seed)
    n, page, D = c.pages * c.page, c.page, c.D
    q = 1.0 + 0.01 * rng.standard_normal((c.Tq, c.Hq * D))
    c.q.copy_(torch.from_numpy(q).to(c.t))
    k = 0.01 * rng.standard_normal((n, 1, D))
    v = 1.0 + 0.1 * rng.random((n, 1, D))
    v[:, :, 0] = -1.0                                   # lows far from the values: the codes carry them
    first = int(c.table[0][0]) * page
    k[first], v[first] = bits * np.log(2.0) / D ** 0.5, 0.0
    c.pool = ref.empty_pool(c.pages, 1, page, D)
    c.kk, c.vv = ref.append(c.pool, range(n), page, k, v)


def check_faint(c, rel, absolute, rows, lossy):
    """Row t sees rows[t] keys.  `absolute`: what a key's share may lose whatever its size, as a share of the largest |v|,
    and of how many keys."""
    at = np.concatenate([p * c.page + np.arange(c.page) for p in c.table[0]])
    q, got = c.q64(), ref.f64(c.o).reshape(c.Tq, c.Hq, c.D)
    half, a = ref.half_step(c.t)
    for t, n in rows.items():
        k, v = c.kk[at[:n], 0], c.vv[at[:n], 0]
        for h in range(c.Hq):
            s = k @ q[t, h] * c.scale
            size = np.abs(k) @ np.abs(q[t, h]) * c.scale
            p = np.exp(s - s.max())
            p /= p.sum()
            delta = (c.D + 16) * 2.0 ** -23 * 3 * (size + size[0]) + 2.0 ** -20
            want, vmax = p @ v, np.abs(v).max()
            assert np.abs(want).max() > 0
            lim = (p * (delta + 2 * rel + n / 16 * 2.0 ** -23)) @ np.abs(v) + min(n, lossy) * absolute * vmax
            lim += half * (np.abs(want) + lim) + a
            err = np.abs(got[t, h] - want) / lim
            assert np.all(err <= 1), (t, h, err.max(), got[t, h, 1], want[1])
            assert lim[1] < 0.5 * want[1]               # the check would see them vanish


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bits", [16, 26])
def test_faint_keys_of_a_chunk(cuda, kind, D, bits):
    c = Case(kind, [6000], [130], 1, 1, D, 16)
    faint(c, bits)
    c.run()
    tm.tm_check()
    check_faint(c, 2.0 ** -11, 2.0 ** -32, {t: 6000 - 130 + t + 1 for t in range(130)}, 6000)


# Single queries.  p * step goes in with the largest step at 2^4 to 2^7 (fp32: in two parts, behind a reference 2^6 down): a
# key may lose half of fp16's smallest number there, 2^-29 (2^-35) of the largest step, times at most eight steps of
# 2 |v| / 15 each: 2^-28 and 2^-34 of |v|.  Only keys of the strong key's own warp can: more sequences than blocks, so that
# a block has most of one, and a quarter of the keys (in tiles of 32) are that warp's.
@pytest.mark.parametrize("kind,bits", [("bf16", 22), ("f16", 22), ("f32", 22), ("f32", 31)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_faint_keys_of_single_queries(cuda, kind, bits, D):
    n, B = 1500, 700
    c = Case(kind, [n], [B], 1, 1, D, 16)
    faint(c, bits)
    c.lens, c.max_q, c.qstart = [n] * B, 1, list(range(B + 1))     # B sequences of one query over the same pages
    c.table = np.repeat(c.table, B, axis=0)
    c.run()
    tm.tm_check()
    bound = (2.0 ** -22, 2.0 ** -34) if kind == "f32" else (2.0 ** -11, 2.0 ** -28)
    check_faint(c, *bound, {t: n for t in range(0, B, 5)}, n // 4 + 64)


# Any real scale: negative, zero.
@pytest.mark.parametrize("kind,qn,D", [("f32", [1, 3], 128), ("bf16", [1, 3], 64), ("f16", [90, 70], 128), ("bf16", [130, 5], 64)])
@pytest.mark.parametrize("scale", [-0.125, 0.0, -0.0])
def test_scales_of_either_sign(cuda, kind, qn, D, scale):
    c = Case(kind, [300, 70], qn, 4, 2, D, 16)
    c.scale = scale
    c.run()
    tm.tm_check()
    o, l, size, vmax, seen = ref.attention(c.q64(), c.kk, c.vv, c.table, c.lens, c.qstart, c.page, scale)
    delta = (D + 16) * 2.0 ** -23 * 3 * np.abs(size)
    prob = 2.0 ** -11 if kind != "f32" else 2.0 ** -22
    tol = ((2 * delta + 2.0 ** -21 + 2 * prob + seen / 16 * 2.0 ** -23) * vmax)[..., None]
    r, a = ref.half_step(c.t)
    got = ref.f64(c.o)[:, :c.Hq * D].reshape(o.shape)
    assert np.all(np.abs(got - o) <= tol + r * (np.abs(o) + tol) + a)
    assert np.all(np.abs(ref.f64(c.lse) - l)[seen > 0] <= (delta + 2.0 ** -21 + 2.0 ** -22 * np.abs(l))[seen > 0])


# Tokens that a row does not see, their values as large as the cache holds: beyond the window of every row, and in chunks
# ahead of a row too.  (Tolerances are by the values that the row sees.)
def giants(c, tokens):
    at = [int(c.table[0][j // c.page]) * c.page + j % c.page for j in tokens]
    rng = np.random.default_rng(5)
    big = 1e30 * np.sign(rng.standard_normal((len(at), c.vv.shape[1], c.D)))
    c.kk[at], c.vv[at] = ref.append(c.pool, at, c.page, c.kk[at], big)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [100, 250])
def test_giants_outside_the_window(cuda, kind, D, window):
    c = Case(kind, [419], [1], 4, 2, D, 16)
    giants(c, [419 - window - 1, 419 - window - 3])
    c.run(window=window)
    tm.tm_check()
    got = check_rows(c, np.ones((1, 4), dtype=bool), window)
    assert np.abs(got).max() < 10
    # in the 2-norm, as test_gpu_attention.py has it: errors of different keys are independent
    o = ref.attention(c.q64(), c.kk, c.vv, c.table, c.lens, c.qstart, c.page, c.scale, window)[0]
    assert np.linalg.norm(got - o) <= {"f32": 1e-5, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[kind] * np.linalg.norm(o)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 180])
def test_giants_that_a_row_of_a_chunk_does_not_see(cuda, kind, D, window):
    c = Case(kind, [500], [150], 2, 1, D, 16)
    giants(c, [490, 495] + ([150] if window else []))            # the first of them is seen from query 140 on
    c.run(window=window)
    tm.tm_check()
    keep = np.zeros((150, 2), dtype=bool)
    keep[:140] = True                                            # 150 is before each of their windows (350 - 180 + 1)
    got = check_rows(c, keep, window)
    assert np.abs(got[keep]).max() < 10
