// tm_kv4_attn.cuh -- what the two attention kernels over the 4-bit cache share:
// the codes' fp16 forms, the call's arguments, and how the work is cut and found.
#pragma once

#include "tm_host.h"

#include "tm_elem.cuh"
#include "tm_kv4.cuh"

namespace libtm {

constexpr int kTile = 32;    // tokens: first tokens of a row tile are rounded down to it
// p goes up to 2^kSlack, p stepV 2^E up to 2^kSlack 2^(kStepBits + 3) <= 2^15
constexpr int kSlack = 8, kStepBits = 4;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2eF = 1.4426950408889634f;

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float2 half2_at(const uint8_t *p)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(p));
}

// The codes of two nibbles 16 bits apart as an fp16 pair, from the low nibble
// position (even dims of a word) or the next one (odd dims).
// Plain: the bits as they are, subnormal fp16: c 2^-24, or c 2^-20.
__device__ __forceinline__ uint32_t plain_even(uint32_t x) { return x & 0x000f000fu; }
__device__ __forceinline__ uint32_t plain_odd(uint32_t x) { return x & 0x00f000f0u; }

// Centred: c - 8, or 16 (c - 8), normal numbers: the nibble joins the low bits of
// 1024 and the subtraction is exact.  `bias` holds 1024 twice and comes from the
// launch's arguments: as a constant it would share the one immediate an instruction
// has with the mask, and cost an instruction more for each pair.
__device__ __forceinline__ uint32_t centred(uint32_t x, uint16_t middle)
{
    const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&x), __halves2half2(__ushort_as_half(middle), __ushort_as_half(middle)));
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t centred_even(uint32_t x, uint32_t bias) { return centred((x & 0x000f000fu) | bias, 0x6408); }  // 1032
__device__ __forceinline__ uint32_t centred_odd(uint32_t x, uint32_t bias) { return centred((x & 0x00f000f0u) | bias, 0x6480); }   // 1152

constexpr int kUnitShift = 8, kUnit = 1 << kUnitShift;             // tokens of a unit of work
constexpr int kChunkRows = 256;        // the chunk kernel's row tile
static_assert(kChunkRows <= kUnit, "a tile's step is at most a unit");
constexpr int kMostBlocks = 608;       // 152 SMs x 4: what the workspace is sized for

// The window the kernels take: 0 for one that hides nothing from any query.  A window
// below max_len (at most 2^30) keeps their sums of lengths and windows within 32 bits.
__host__ __device__ constexpr int window_of(int window, int64_t max_len) { return window >= max_len ? 0 : window; }

struct AttnArgs {
    const void *Q;
    void *O;
    float *lse;
    const uint8_t *pool;
    const int32_t *table, *lens, *qstart;
    float *part;      // [2 gridDim.x] slots of [ROWS][D] outputs and [ROWS][2] (maximum, sum)
    int2 *job;        // [B][Hkv][row_tiles]: the first block an item lies in, and how many; or NULL
    int64_t qs_tok, qs_head, os_tok, os_head, pages, page_bytes, ldt, Tq, max_len;
    int B, Hq, Hkv, G, window, full, vec, max_q, blocks_per_page, row_tiles;
    int grid;       // blocks of the attention's launch, the bound of a job's blocks
    int tile_step;  // chunk kernel, in log2: tokens a row tile sees more than the one before (-1: all count alike)
    uint32_t bias;  // 1024 in both halves of an fp16 pair
    float scale;
    FastDiv by_page, by_group;  // cache blocks of a page, heads of a group
    unsigned *status;
};

// What a sequence's queries are: their first row of Q, their count and the
// cache's length, checked against the call's bounds.
struct Seq {
    int q0, n, len;
};

__device__ __forceinline__ Seq sequence(const AttnArgs &a, int b, bool report)
{
    Seq s;
    int q1;
    if (a.qstart) {
        s.q0 = a.qstart[b];
        q1 = a.qstart[b + 1];
    } else {
        s.q0 = b;
        q1 = b + 1;
    }
    s.len = a.lens[b];
    if (s.q0 < 0 || q1 < s.q0 || q1 > a.Tq || q1 - s.q0 > a.max_q || s.len < 0 || s.len > a.max_len) {
        if (report) atomicOr(a.status, kStatusIndex);
        s.n = 0;
        s.len = 0;
        return s;
    }
    s.n = q1 - s.q0;
    return s;
}

// Keys a query at place t of its sequence sees: [lower, upper).
__device__ __forceinline__ int upper(const AttnArgs &a, const Seq &s, int t)
{
    return a.full ? s.len : min(s.len, max(0, s.len - s.n + t + 1));
}
__device__ __forceinline__ int lower(const AttnArgs &a, const Seq &s, int t)
{
    return a.window > 0 ? max(0, s.len - s.n + t + 1 - a.window) : 0;
}

// Row tiles of a sequence, and the units each of its items counts (one at
// least: an item that sees nothing still has its zeros to write).  With a
// window every row tile counts as many units as the widest could need.  In the
// chunk kernel, where the queries are a large part of the tokens, a causal item counts
// what its last row sees, end + tile 2^step tokens, and one unit for its own start and
// end: a prompt's first row tiles see next to nothing.
struct Load {
    int tiles, units, end, step, head;  // units: of every item, where step < 0; head: of a KV head's items
    __device__ __forceinline__ int total(int Hkv) const { return head * Hkv; }  // the host bounds the sum
    // Units of the first t row tiles, sum over k < t of 1 + ceil((end + k 2^step) / kUnit):
    // with x = (end - 1) >> step and 2^r = kUnit / 2^step, a term is ((x + k) >> r) + 2.
    __device__ __forceinline__ int before(int t) const
    {
        if (step < 0) return t * units;
        const int r = kUnitShift - step, x = end - 1 >> step;
        return (int)(below(x + t, r) - below(x, r)) + 2 * t;
    }
    // Sum over i < x of i >> r.
    static __device__ __forceinline__ int64_t below(int64_t x, int r)
    {
        const int64_t m = x >> r;
        return (m * (m - 1) / 2 << r) + m * (x - (m << r));
    }
};

__device__ __forceinline__ Load load_of(const AttnArgs &a, const Seq &s, int rows_of_tile)
{
    Load l;
    const bool chunk = rows_of_tile == kChunkRows;
    l.tiles = (s.n * a.G + rows_of_tile - 1) / rows_of_tile;
    l.step = chunk ? a.tile_step : -1;
    l.end = l.step < 0 ? 1 : max(1, min(s.len, s.len - s.n + (1 << l.step)));
    int range = s.len;
    if (a.window > 0) range = min(range, a.window + rows_of_tile / a.G + 1 + kTile);
    l.units = max(1, (range + kUnit - 1) / kUnit);
    l.head = l.before(l.tiles);
    return l;
}

// A block's run of units, [pos, stop) of all items' one after another; pos lies in
// sequence b, whose units start at base.  `share` units a block.
struct Run {
    int pos, stop, share, base, b;
    Seq seq;
    Load load;
};

// Called by whole warps, each for itself: sequences are added up 32 at a time.
// False if the block has nothing to do.
__device__ __forceinline__ bool find_run(const AttnArgs &a, int rows_of_tile, bool report, Run &r)
{
    const int lane = threadIdx.x & 31;
    auto lane_load = [&](int i, bool say, Seq &q) {
        q = {0, 0, 0};
        if (i < a.B) q = sequence(a, i, say);
        return load_of(a, q, rows_of_tile).total(a.Hkv);
    };
    int all = 0, mine = 0;
    Seq q;
    for (int b0 = 0; b0 < a.B; b0 += 32) all += mine = lane_load(b0 + lane, report && blockIdx.x == 0, q);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    r.share = (all + (int)gridDim.x - 1) / (int)gridDim.x;
    r.pos = min(r.share * (int)blockIdx.x, all);
    r.stop = min(all, r.pos + r.share);
    if (r.pos >= r.stop) return false;
    int before = 0;
    for (r.b = 0;; r.b += 32) {
        if (a.B > 32) mine = lane_load(r.b + lane, false, q);
        int inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += x;
        }
        const int sum = __shfl_sync(0xffffffffu, inc, 31);
        if (r.pos < before + sum) {
            const int at = __ffs(__ballot_sync(0xffffffffu, r.pos < before + inc)) - 1;
            r.b += at;
            r.base = before + __shfl_sync(0xffffffffu, inc - mine, at);
            r.seq.q0 = __shfl_sync(0xffffffffu, q.q0, at);
            r.seq.n = __shfl_sync(0xffffffffu, q.n, at);
            r.seq.len = __shfl_sync(0xffffffffu, q.len, at);
            break;
        }
        before += sum;
    }
    r.load = load_of(a, r.seq, rows_of_tile);
    return true;
}

// A segment of the run: units [unit0, unit0 + count) of an item, its tokens [c0, c1).
struct Segment {
    int unit0, count, kvh, tile, rows, begin, end, c0, c1;
    bool whole, last;  // the whole item; its last unit among them
};

__device__ __forceinline__ Segment next_segment(const AttnArgs &a, int rows_of_tile, Run &r)
{
    while (r.pos >= r.base + r.load.total(a.Hkv)) {
        r.base += r.load.total(a.Hkv);
        r.seq = sequence(a, ++r.b, false);
        r.load = load_of(a, r.seq, rows_of_tile);
    }
    Segment s;
    int units = r.load.units;
    s.kvh = (r.pos - r.base) / r.load.head;
    s.unit0 = r.pos - r.base - s.kvh * r.load.head;
    if (r.load.step < 0) {
        s.tile = s.unit0 / units;
        s.unit0 -= s.tile * units;
    } else {
        int lo = 0, hi = r.load.tiles;  // before(lo) <= unit0 < before(hi)
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            (r.load.before(mid) <= s.unit0 ? lo : hi) = mid;
        }
        s.tile = lo;
        const int first = r.load.before(lo);
        units = r.load.before(lo + 1) - first;
        s.unit0 -= first;
    }
    s.count = min(units - s.unit0, r.stop - r.pos);
    s.whole = s.count == units;
    s.last = s.unit0 + s.count == units;
    s.rows = min(rows_of_tile, r.seq.n * a.G - s.tile * rows_of_tile);
    const int first = s.tile * rows_of_tile;
    s.begin = lower(a, r.seq, (int)fdiv(first, a.by_group)) / kTile * kTile;
    s.end = upper(a, r.seq, (int)fdiv(first + s.rows - 1, a.by_group));
    s.c0 = min(s.end, s.begin + s.unit0 * kUnit);
    s.c1 = s.last ? s.end : min(s.end, s.c0 + s.count * kUnit);
    return s;
}

// The blocks an item lies in, noted for the join by the block that ends it (call it
// before the run moves on).
__device__ __forceinline__ void note_job(const AttnArgs &a, const Run &r, const Segment &s)
{
    const int c0 = (r.pos - s.unit0) / r.share;
    a.job[((int64_t)r.b * a.Hkv + s.kvh) * a.row_tiles + s.tile] = make_int2(c0, (int)blockIdx.x - c0 + 1);
}

// Whether a job names blocks of the launch.  A block that gave up on a wait has noted
// nothing for the items after it: their jobs are whatever the workspace held.
__host__ __device__ constexpr bool job_in_grid(int first, int count, int grid)
{
    return first >= 0 && count >= 1 && count <= grid && first <= grid - count;
}

// The kernel for many query rows (tm_kv4_chunk.cu).
tm_status launch_chunk_attn(int D, int32_t xtype, AttnArgs &a, int device, int sms, bool join, cudaStream_t s, bool pdl);
bool chunk_attn_fits(int32_t xtype, int64_t rows, int D);
size_t chunk_attn_slots_bytes(int D);

// The join of its partial outputs (tm_kv4_attn.cu).
tm_status launch_chunk_join(int D, int32_t xtype, AttnArgs &a, int sms, cudaStream_t s);

}  // namespace libtm
