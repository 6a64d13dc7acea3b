"""tm_kv4_attention against its definition in 64 bits.

Tolerance.  A logit is a sum of D products of exact factors (fp16 and bf16
queries are held whole, fp32 ones to 2^-22) accumulated in fp32 by the tensor
cores, taken as losing 2^-23 of the sum of magnitudes at each of D additions:
delta = (D + 16) 2^-23 max_j scale sum_d |q_d| |k_jd|-like magnitudes (codes and
lows separately: at most 3 times that sum here).  A probability is then off by
2 delta + 2^-21, the output by that share of the largest |v|, plus the rounding
of p * step to fp16 (2^-11 of at most 15 steps <= 2 max|v|; 2^-22 with fp32) and
the additions over n keys (n / 16 of 2^-23 each).
"""
import numpy as np
import pytest
import torch

import block_ref as ref
from masking_tm_affine_gb300 import tm

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, kind, lens, qn, Hq, Hkv, D, page, seed=0, ld_gap=0, shift=0, extra_pages=2):
        rng = np.random.default_rng(seed + D + page + sum(lens))
        self.kind, self.t = kind, ref.TYPES[kind]
        self.lens, self.Hq, self.Hkv, self.D, self.page = list(lens), Hq, Hkv, D, page
        self.qstart = [0] + list(np.cumsum(qn))
        self.Tq, self.max_q = int(self.qstart[-1]), max(qn)
        per = max(1, -(-max(lens) // page))
        self.pages = len(lens) * per + extra_pages
        self.table = rng.permutation(self.pages)[:len(lens) * per].reshape(len(lens), per)
        self.pool, self.kk, self.vv = ref.random_cache(rng, self.pages, Hkv, page, D)
        self.row = Hq * D + ld_gap
        buf = torch.from_numpy(rng.standard_normal(self.Tq * self.row + 16)).to(self.t).cuda()
        self.q = buf[shift:][:self.Tq * self.row].view(self.Tq, self.row)
        self.obuf = torch.full((self.Tq * self.row + 16,), 9.0, dtype=self.t, device="cuda")
        self.o = self.obuf[shift:][:self.Tq * self.row].view(self.Tq, self.row)
        self.lse = torch.full((self.Tq, Hq), 9.0, device="cuda")
        self.scale = float(np.float32(D ** -0.5))

    def q64(self):
        return ref.f64(self.q)[:, :self.Hq * self.D].reshape(self.Tq, self.Hq, self.D)

    def run(self, window=0, flags=0, max_len=None, qstart=True, lens=None, table=None, stream=None, pages=None, lse=True):
        dev = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()  # noqa: E731
        B = len(self.lens)
        max_len = max(self.lens) if max_len is None else max_len
        ws = tm.tm_kv4_attention_workspace_bytes(B, self.Tq, self.max_q, max_len, self.Hq, self.Hkv, self.D)
        self.ws = torch.full((max(ws // 4, 1),), float("nan"), device="cuda")
        self.dpool = torch.from_numpy(self.pool).cuda()
        self.keep = (dev(self.table if table is None else table), dev(self.lens if lens is None else lens), dev(self.qstart))
        if stream is not None:
            torch.cuda.synchronize()
        tm.tm_kv4_attention(self.q, self.row, self.D, self.o, self.row, self.D, self.lse if lse else None, self.dpool,
                            self.pages if pages is None else pages, self.page, self.keep[0], self.table.shape[1],
                            self.keep[1], self.keep[2] if qstart else None, B, self.Tq, self.max_q, max_len, self.Hq,
                            self.Hkv, self.D, self.scale, window, ref.CODE[self.kind], self.ws, ws, flags, stream)

    def check(self, window=0, full=False, lens=None, lse=True):
        o, l, size, vmax, seen = ref.attention(self.q64(), self.kk, self.vv, self.table, self.lens if lens is None else lens,
                                               self.qstart, self.page, self.scale, window, full)
        delta = (self.D + 16) * 2.0 ** -23 * 3 * size
        prob = 2.0 ** -11 if self.kind != "f32" else 2.0 ** -22
        tol = (2 * delta + 2.0 ** -21 + 2 * prob + seen / 16 * 2.0 ** -23) * vmax
        r, a = ref.half_step(self.t)
        got = ref.f64(self.o)[:, :self.Hq * self.D].reshape(o.shape)
        lim = tol[..., None] + r * (np.abs(o) + tol[..., None]) + a
        assert np.all(np.abs(got - o) <= lim), np.max(np.abs(got - o) / lim)
        # the errors of different terms are independent: in the 2-norm they stay near the type's own rounding
        live = seen > 0
        if live.any():
            rel = np.linalg.norm(got[live] - o[live]) / np.linalg.norm(o[live])
            assert rel <= {"f32": 1e-5, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[self.kind], rel
        assert not got[~live].any()
        if lse:
            gl = ref.f64(self.lse)
            assert np.array_equal(np.isneginf(gl), ~live)
            assert np.all(np.abs(gl[live] - l[live]) <= delta[live] + 2.0 ** -21 + 2.0 ** -22 * np.abs(l[live]))


KINDS = ["f32", "bf16", "f16"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 100, 127, 128, 129, 257, 1000])
def test_one_token(cuda, kind, D, n):
    c = Case(kind, [n], [1], 4, 2, D, 16)
    c.run()
    tm.tm_check()
    c.check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (8, 1), (16, 2), (24, 2), (20, 1)])
@pytest.mark.parametrize("page", [16, 32, 48, 128])
def test_groups_and_pages(cuda, kind, Hq, Hkv, page):
    c = Case(kind, [300, 77, 0, 129], [1, 1, 1, 1], Hq, Hkv, 128, page)
    c.run(qstart=False)
    tm.tm_check()
    c.check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 1, 20, 64])
def test_several_queries(cuda, kind, D, window):
    # chunks, one longer than its cache (its first queries see nothing), a sequence without queries, an empty one
    c = Case(kind, [130, 40, 3, 64, 0], [40, 5, 7, 0, 2], 6, 2, D, 32)
    c.run(window=window)
    tm.tm_check()
    c.check(window=window)


# 128 query rows a KV head and more: the form for chunks of a prompt.
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,qn,Hq,Hkv,page", [
    ([130], [128], 1, 1, 16), ([128], [128], 1, 1, 128), ([70], [32], 4, 1, 32), ([40], [40], 8, 2, 48),
    ([300, 0, 129], [33, 5, 129], 4, 1, 16), ([1000, 260, 64], [70, 64, 64], 12, 3, 64), ([20, 500], [90, 1], 4, 2, 16)])
def test_chunks(cuda, kind, D, lens, qn, Hq, Hkv, page):
    c = Case(kind, lens, qn, Hq, Hkv, D, page)
    c.run()
    tm.tm_check()
    c.check()


# Whole prompts and late chunks of several row tiles, which see more and more: every tile step (256 / heads
# of a group, and a group that does not divide it), sequences beside them of one tile, of none, of fewer keys than
# queries, and more queries than any sequence has tokens.
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("lens,qn,Hq,Hkv,D,max_len", [
    ([700], [700], 2, 2, 64, 700), ([700, 20, 0], [700, 20, 3], 2, 1, 64, 704), ([600, 257], [600, 130], 4, 1, 128, 600),
    ([520, 0, 300], [300, 0, 300], 8, 1, 128, 520), ([129, 400, 1], [129, 65, 1], 16, 1, 64, 400),
    ([300, 290], [300, 150], 6, 2, 128, 300), ([500, 9], [300, 400], 4, 2, 64, 500), ([260], [400], 4, 2, 64, 260),
    ([257], [257], 1, 1, 128, 257), ([256, 255], [256, 255], 4, 1, 64, 256), ([1100], [1100], 2, 2, 64, 1100),
    ([1500, 20, 0, 1030], [1500, 20, 3, 300], 4, 1, 128, 1504), ([1200, 1217], [400, 1200], 8, 1, 64, 1217),
    ([1100], [1100], 16, 1, 64, 1100), ([2000, 700], [600, 700], 6, 2, 128, 2000), ([1056, 3], [1056, 40], 4, 4, 64, 1056),
    ([1300, 1], [1300, 300], 2, 1, 128, 1312)])
def test_chunks_of_several_row_tiles(cuda, kind, lens, qn, Hq, Hkv, D, max_len):
    c = Case(kind, lens, qn, Hq, Hkv, D, 32)
    c.run(max_len=max_len)
    tm.tm_check()
    c.check()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [1, 50, 200])
def test_chunks_with_a_window(cuda, D, window):
    c = Case("bf16", [700, 150], [80, 150], 4, 2, D, 32)
    c.run(window=window)
    tm.tm_check()
    c.check(window=window)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_chunks_every_key_split_over_blocks(cuda, kind):
    c = Case(kind, [5000], [64], 4, 1, 128, 64)
    c.run(flags=tm.TM_ATTN_FULL)
    tm.tm_check()
    c.check(full=True)


@pytest.mark.parametrize("shift", [0, 1])
def test_chunks_strides_and_gaps(cuda, shift):
    c = Case("bf16", [260, 90], [80, 50], 6, 2, 64, 16, ld_gap=24, shift=shift)
    c.run(lse=False)
    tm.tm_check()
    c.check(lse=False)
    c.o[:, :c.Hq * c.D] = 9.0
    assert bool((c.obuf == 9.0).all())


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_chunks_scales_of_very_different_size(cuda, kind):
    c = Case(kind, [900], [140], 2, 1, 128, 16)
    rng = np.random.default_rng(3)
    grow = 2.0 ** rng.integers(-8, 5, (c.pages * 16, 1, 1)).astype(np.float64)
    v = rng.standard_normal((c.pages * 16, 1, 128)) * grow
    c.pool = ref.empty_pool(c.pages, 1, 16, 128)
    c.kk, c.vv = ref.append(c.pool, range(c.pages * 16), 16, c.kk, v)
    c.q *= torch.from_numpy(2.0 ** rng.integers(-8, 3, (c.Tq, c.row))).to(c.t).cuda()
    c.run()
    tm.tm_check()
    c.check()


def test_chunks_not_finite_where_masked_and_where_seen(cuda):
    c = Case("bf16", [200], [150], 2, 1, 64, 16, extra_pages=0)
    order = [int(c.table[0][j // 16]) * 16 + j % 16 for j in range(208)]
    nan = np.full((1, 64), np.nan)
    kk, vv = c.kk.copy(), c.vv.copy()
    for which in ("k", "v"):
        for j in (190, 201, 207):     # seen by the last ten queries; past the end
            at = order[j]
            ref.append(c.pool, [at], 16, (nan if which == "k" else kk[at])[None], (nan if which == "v" else vv[at])[None])
        c.run()
        tm.tm_check()
        o, l = ref.f64(c.o).reshape(150, 2, 64), ref.f64(c.lse)
        w, lw, *_ = ref.attention(c.q64()[:140], kk, vv, c.table, [190], [0, 140], 16, c.scale)
        assert np.isnan(o[140:]).all() and np.isnan(l[140:]).all() == (which == "k")
        assert np.abs(o[:140] - w).max() < 0.05 and np.abs(l[:140] - lw).max() < 1e-3
        ref.append(c.pool, [order[190]], 16, kk[order[190]][None], vv[order[190]][None])


def test_chunks_bad_pages_and_lengths(cuda):
    c = Case("bf16", [300, 280], [130, 130], 1, 1, 64, 16)
    good = c.table.copy()
    for at, page in ((3, c.pages), (0, -1)):
        bad = good.copy()
        bad[1, at] = page
        c.run(table=bad)
        with pytest.raises(tm.TmError) as e:
            tm.tm_check()
        assert e.value.status == tm.TM_ERR_INDEX
    c.run(lens=[300, 301])
    with pytest.raises(tm.TmError) as e:
        tm.tm_check()
    assert e.value.status == tm.TM_ERR_INDEX
    c.run()
    first, l = c.o.clone(), c.lse.clone()
    c.run()
    tm.tm_check()
    c.check()
    assert torch.equal(first, c.o) and torch.equal(l, c.lse)


@pytest.mark.parametrize("kind", KINDS)
def test_every_key(cuda, kind):
    c = Case(kind, [50, 33], [3, 40], 4, 4, 64, 16)
    c.run(flags=tm.TM_ATTN_FULL)
    tm.tm_check()
    c.check(full=True)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [0, 700])
def test_splits(cuda, kind, window):
    # few sequences and long ones: the tokens are split over blocks and joined
    c = Case(kind, [5000, 1, 1281], [1, 1, 1], 8, 2, 128, 64)
    c.run(window=window)
    tm.tm_check()
    c.check(window=window)
    loose = c.o.clone()
    c.run(window=window, max_len=c.table.shape[1] * 64)   # another bound: another split, the same result within rounding
    tm.tm_check()
    c.check(window=window)
    assert torch.allclose(loose.float(), c.o.float(), atol=0.05)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [0, 1])
def test_strides_and_gaps(cuda, kind, shift):
    c = Case(kind, [200, 31], [2, 3], 4, 2, 64, 16, ld_gap=24, shift=shift)
    c.run(lse=False)
    tm.tm_check()
    c.check(lse=False)
    c.o[:, :c.Hq * c.D] = 9.0
    assert bool((c.obuf == 9.0).all())


@pytest.mark.parametrize("kind", KINDS)
def test_scales_of_very_different_size(cuda, kind):
    # values whose steps differ by 2^12 between tokens, rows of q by 2^10: the running exponents move
    c = Case(kind, [400], [2], 8, 1, 128, 16)
    rng = np.random.default_rng(3)
    grow = 2.0 ** rng.integers(-8, 5, (c.pages * 16, 1, 1)).astype(np.float64)
    v = rng.standard_normal((c.pages * 16, 1, 128)) * grow
    c.pool = ref.empty_pool(c.pages, 1, 16, 128)
    c.kk, c.vv = ref.append(c.pool, range(c.pages * 16), 16, c.kk, v)
    c.q *= torch.from_numpy(2.0 ** rng.integers(-8, 3, (c.Tq, c.row))).to(c.t).cuda()
    c.run()
    tm.tm_check()
    c.check()


@pytest.mark.parametrize("kind", KINDS)
def test_large_logits(cuda, kind):
    # a softmax that is all but one-hot
    c = Case(kind, [600], [1], 4, 1, 64, 16)
    c.q *= 64
    c.run()
    tm.tm_check()
    c.check()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_not_finite_where_masked_and_where_seen(cuda, kind):
    # tokens held as NaN: past the end, ahead of a query, and seen by the last query only
    c = Case(kind, [70], [3], 2, 1, 64, 16, extra_pages=0)
    nan = np.full((1, 64), np.nan)
    order = [int(c.table[0][j // 16]) * 16 + j % 16 for j in range(80)]
    clean_k, clean_v = c.kk.copy(), c.vv.copy()
    for which in ("k", "v"):
        c.kk, c.vv = clean_k.copy(), clean_v.copy()
        for j in (69, 70, 71, 79):
            pair = (nan, c.vv[order[j]]) if which == "k" else (c.kk[order[j]], nan)
            ref.append(c.pool, [order[j]], 16, pair[0][None], pair[1][None])
        c.run()
        tm.tm_check()
        o = ref.f64(c.o).reshape(3, 2, 64)
        assert np.isnan(o[2]).all() and np.isfinite(o[:2]).all()
        assert np.isfinite(ref.f64(c.lse)[:2]).all() and np.isnan(ref.f64(c.lse)[2]).all() == (which == "k")
        w, *_ = ref.attention(c.q64(), c.kk, c.vv, c.table, [69], [0, 2], 16, c.scale)
        assert np.abs(o[:2] - w[:2]).max() < (1e-4 if kind == "f32" else 0.05)
        ref.append(c.pool, [order[69]], 16, clean_k[order[69]][None], clean_v[order[69]][None])


def test_infinite_and_nan_queries(cuda):
    c = Case("f32", [40, 40], [1, 1], 2, 1, 64, 16)
    c.q[0, 3], c.q[1, 70] = float("nan"), float("inf")
    c.run()
    tm.tm_check()
    o = ref.f64(c.o).reshape(2, 2, 64)
    assert np.isnan(o[0, 0]).all() and np.isnan(o[1, 1]).all()


def test_bad_pages_lengths_and_counts(cuda):
    c = Case("bf16", [100, 90], [1, 1], 2, 1, 64, 16)
    good = c.table.copy()
    for at, page in ((3, c.pages), (0, -1), (6, 1 << 30)):
        bad = good.copy()
        bad[0, at] = page
        c.run(table=bad)
        with pytest.raises(tm.TmError) as e:
            tm.tm_check()
        assert e.value.status == tm.TM_ERR_INDEX, (at, page)
    c.run(lens=[100, 101])        # longer than max_len
    with pytest.raises(tm.TmError) as e:
        tm.tm_check()
    assert e.value.status == tm.TM_ERR_INDEX
    c.run(lens=[100, -5])
    with pytest.raises(tm.TmError):
        tm.tm_check()
    keep = c.qstart
    for q in ([0, 2, 2], [0, 1, 3], [1, 0, 2], [0, 1, -1]):   # more than max_q, past Tq, not rising
        c.qstart = q
        c.run()
        with pytest.raises(tm.TmError) as e:
            tm.tm_check()
        assert e.value.status == tm.TM_ERR_INDEX, q
    c.qstart = keep
    c.run()
    tm.tm_check()
    c.check()


def test_captured_in_a_graph_on_a_stream(cuda):
    # a decode step captured once and replayed with other lengths
    c = Case("bf16", [900, 500], [1, 1], 8, 2, 128, 32)
    st = torch.cuda.Stream()
    c.run(stream=st)
    tm.tm_check(st)
    g = torch.cuda.CUDAGraph()
    args = (c.q, c.row, c.D, c.o, c.row, c.D, c.lse, c.dpool, c.pages, c.page, c.keep[0], c.table.shape[1], c.keep[1],
            c.keep[2], 2, c.Tq, c.max_q, 900, c.Hq, c.Hkv, c.D, c.scale, 0, 2, c.ws, c.ws.numel() * 4, 0)
    with torch.cuda.graph(g, stream=st):
        tm.tm_kv4_attention(*args, torch.cuda.current_stream())
    for lens in ([900, 500], [1, 0], [64, 899]):
        c.keep[1].copy_(torch.tensor(lens, dtype=torch.int32))
        c.o.fill_(9.0)
        g.replay()
        tm.tm_check()
        c.check(lens=lens)


def test_twice_the_same_bits(cuda):
    c = Case("bf16", [3000, 2999], [1, 1], 8, 2, 128, 16)
    c.run()
    first, l = c.o.clone(), c.lse.clone()
    for _ in range(3):
        c.run()
        assert torch.equal(first, c.o) and torch.equal(l, c.lse)
    tm.tm_check()


def test_offsets_past_32_bits(cuda):
    # a pool of 4.6 GB: the pages in use lie at its end
    Hkv, D, page = 8, 128, 64
    per = tm.tm_kv4_page_bytes(Hkv, D, page)
    pages = (1 << 32) // per + 400
    c = Case("bf16", [200], [1], 16, Hkv, D, page, extra_pages=0)
    big = torch.zeros(pages * per, dtype=torch.uint8, device="cuda").view(pages, per)
    small = torch.from_numpy(c.pool).cuda().view(-1, per)
    first = pages - small.shape[0]
    big[first:] = small
    table = torch.from_numpy((c.table + first).astype(np.int32)).cuda()
    lens = torch.tensor([200], dtype=torch.int32, device="cuda")
    tm.tm_kv4_attention(c.q, c.row, D, c.o, c.row, D, c.lse, big, pages, page, table, c.table.shape[1], lens, None, 1, 1, 1,
                        200, 16, Hkv, D, c.scale, 0, 2, None, 0)
    tm.tm_check()
    c.check()
