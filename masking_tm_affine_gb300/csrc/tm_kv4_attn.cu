// tm_kv4_attn.cu -- attention over the 4-bit paged cache.
//
//   s_tj = scale q_t . k_j,  o_t = sum_j softmax(s_t)_j v_j,   k_j = lowK_j + stepK_j ck_j,  v_j = lowV_j + stepV_j cv_j
//
// The codes are never turned into values: with integer codes c in 0 .. 15,
//   s_tj = scale (stepK_j (q_t . ck_j) + lowK_j sum(q_t))
//   o_t  = sum_j (p_tj stepV_j) cv_j + sum_j p_tj lowV_j
// so the products run on codes and the scales meet one value per (query, token).
//
// Decode is bound by HBM (D + 8 bytes a token and KV head against 4 D flops for
// each of its query heads); what it must not do is spend more than about three
// instructions a code.  A K nibble becomes half of an fp16 pair by one AND: the
// bits 0x000c read as fp16 are the subnormal c 2^-24, 0x00c0 is c 2^-20, both
// exact.  Eight codes of a 32-bit word are four pairs for four ANDs and a shift;
// the factor 16 between even and odd nibbles is folded into q (K) and into the
// output (V).  V's codes (and K's with fp32 tensors) take one subtraction a pair
// more and go in as c - 8: a sum of positive codes over many tokens is 10 to 1000
// times what is left of it in the output, and the tensor cores, which align a
// step's products to the largest exponent (a subnormal counting as 2^-14) and cut
// what lies below fp32's last place, would leave that many times their own error.
//
// Products are mma.sync m16n8k16 with tokens (or dims) as the 16 rows and up to
// NT x 8 query rows (queries x the heads that share a KV head) as columns, so
// one query token's group of 8 heads fills a tile and the accumulators are small:
//   S^T [16 tokens, 8 rows] += K codes [16 tokens, 16 dims] . Q^T [16 dims, 8 rows]
//   O^T [16 dims, 8 rows]   += V codes^T [16 dims, 16 tokens] . P^T [16 tokens, 8 rows]
// A lane's K operand for all D/16 steps is D/8 contiguous bytes of two tokens;
// V is laid out in token pairs so that two byte permutes pair the tokens; P^T is
// the first product's accumulator, transposed by movmatrix in registers.
//
// Work.  An item is a (sequence, KV head, row tile); its tokens are cut into units of
// 256.  The launch has as many blocks as the GPU holds at once, and each takes an
// equal run of the concatenated units of all items, whatever the lengths: lengths
// live on the device, so every block adds them up itself (one load and a scan).  A
// block's run is a few segments of items; a segment that is a whole item writes its
// output, the others write partial outputs that a second launch joins in order.
// Each of a block's four warps streams its own tiles of 32 tokens through a private
// ring of bulk copies (a cache block is contiguous: one or two copies a tile), so no
// barrier is in the loop; each keeps its own running maximum, sum and output, joined
// in shared memory at a segment's end.
//
// P stepV is rounded to fp16 for the second product, scaled by a 2^E that keeps the
// largest of them in range: off by at most 2^-11 of itself, errors that the sum over
// tokens averages below the output's own rounding, or, for probabilities below 2^-18 of the
// largest that the same warp meets, by 2^-29 of that (times the largest step: half of fp16's
// smallest number).  With fp32 tensors q and P stepV go in as two fp16 parts each: 22 bits, those
// of P stepV down to 2^-12 of the largest, and 2^-35 of it below that.
//
// Measured with the join, D 128, 8 KV heads: 64 sequences of 1000 to 8192 tokens, 32
// heads, bf16, 78 us (321 MB, 60% of the copy rate); one of 131071, 64 heads, fp16, 43 us
// (143 MB, 49%; longer ones approach 77%).  Issue slots are 54 to 58% busy: a tile's chain of
// copy, products and softmax bounds it, and a fixed 10 us of start and join.
#include <atomic>

#include "tm_kv4_attn.cuh"

namespace libtm {
namespace {

constexpr int kWarps = 4;              // a warp takes tiles of kTile tokens
static_assert(kUnit % (kWarps * kTile) == 0, "a unit is whole tiles of every warp");

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

template <int D>
__host__ __device__ constexpr int stage_bytes()
{
    return 2 * kv4_block_bytes(D);
}

// Stages of the copy ring: enough bytes in flight (about 16 KB a warp), and four
// blocks of four warps in an SM's 227 KB.
template <int D>
__host__ __device__ constexpr int ring_stages()
{
    return D == 64 ? 5 : D == 128 ? 3 : 2;
}

template <int D>
__host__ __device__ constexpr int attn_smem()
{
    return kWarps * ring_stages<D>() * stage_bytes<D>() + 128;
}

// Blocks an SM holds, by registers (the instances with 16 column rows or two fp16
// parts need more) and shared memory.
template <typename T, int D, int NT>
__host__ __device__ constexpr int blocks_per_sm()
{
    return NT > 1 ? 2 : sizeof(T) == 4 ? (D == 64 ? 4 : D == 128 ? 3 : 2) : D == 256 ? 3 : 4;
}

// T: element type.  NT: column tiles of 8 query rows.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, blocks_per_sm<T, D, NT>())
    kv4_attn_kernel(const __grid_constant__ AttnArgs a)
{
    constexpr bool SPLIT = sizeof(T) == 4;     // two fp16 parts
    constexpr int PARTS = SPLIT ? 2 : 1;
    // The reference lies 2^LEAD below the maximum that set it: what P stepV keeps of faint keys
    // against how often a new maximum moves the state.  0 / 2 / 4 / 6 in fp32: 64 sequences 97.9 / 98.1 /
    // 98.7 / 99.2 us, one of 131071 tokens 52.3 / 52.4 / 52.7 / 53.5.
    constexpr int LEAD = SPLIT ? 6 : 0;
    constexpr int KS = D / 16;                 // steps of the first product = row tiles of the second
    constexpr int LD = D / 4;                  // dims of a row that a lane holds for the first product
    constexpr int STAGES = ring_stages<D>();
    constexpr int SB = stage_bytes<D>(), BB = kv4_block_bytes(D);
    constexpr int ROWS = 8 * NT;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t bars[kWarps][STAGES];
    __shared__ float4 cols[kWarps][NT][4];  // factors of d and of K's low for two rows

    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, j = lane & 3;
    uint8_t *ring = smem + warp * (STAGES * SB);
    const uint32_t ring_s = smem_u32(ring), bar_s = smem_u32(&bars[warp][0]);
    if (lane == 0) {
#pragma unroll
        for (int s = 0; s < STAGES; ++s)
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar_s + 8 * s) : "memory");
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncwarp();  // every lane copies and waits on these barriers

    Run run;
    if (!find_run(a, ROWS, warp == 0, run)) {
        pdl_wait();
        return;
    }
    const uint64_t policy = l2_evict_first_policy();
    const uint32_t bias = a.bias;
    int stage = 0;       // of the next tile to read, in this warp's ring
    uint32_t phase = 0;  // and its parity
    int fill = 0;        // stage of the next tile to copy
    bool alive = true;

    while (run.pos < run.stop) {
        const Segment seg = next_segment(a, ROWS, run);
        const Seq seq = run.seq;
        const int kvh = seg.kvh, tile = seg.tile, rows = seg.rows, end = seg.end, c0 = seg.c0, b = run.b;
        if (a.job && seg.last && tid == 0) {
            pdl_wait();
            note_job(a, run, seg);
        }
        run.pos += seg.count;
        // Where every row of the tile sees every token: [safe0, safe1).
        const int safe0 = lower(a, seq, (int)fdiv(tile * ROWS + rows - 1, a.by_group));
        const int safe1 = upper(a, seq, (int)fdiv(tile * ROWS, a.by_group));
        const int first = lower(a, seq, (int)fdiv(tile * ROWS, a.by_group));  // nothing before it is seen

        // ---- this lane's queries, asked for before the copies' page numbers
        Vec<T, 8> raw[NT][LD / 8];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = tile * ROWS + nt * 8 + g, t = (int)fdiv(row, a.by_group), hh = row - t * a.G;
            const T *p = reinterpret_cast<const T *>(a.Q) + (int64_t)(seq.q0 + t) * a.qs_tok +
                         (int64_t)(kvh * a.G + hh) * a.qs_head + j * LD;
#pragma unroll
            for (int w = 0; w < LD / 8; ++w) {
                if (nt * 8 + g >= rows) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) raw[nt][w].v[e] = from_f<T>(0.0f);
                } else if (a.vec) {
                    load_vec(p + 8 * w, raw[nt][w]);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) raw[nt][w].v[e] = p[8 * w + e];
                }
            }
        }

        // ---- the copies: this warp's tiles are warp, warp + 4, ... of the segment.  Of each
        // 32 tiles a lane works out one's source (two blocks, which can lie in two
        // pages) and copies it when its turn comes.
        const int tiles = (seg.c1 - c0 + kTile - 1) / kTile;
        const int mine = tiles > warp ? (tiles - warp + kWarps - 1) / kWarps : 0;
        const int32_t *trow = a.table + (int64_t)b * a.ldt;
        const uint8_t *src0 = nullptr, *src1 = nullptr;
        int blocks = 0;  // of this lane's tile: 1, 2, or 3 for two that are adjacent
        auto find = [&](int i) {
            if (i < mine) {
                const int blk = (c0 + (warp + i * kWarps) * kTile) / kBlockTokens;
                const int e0 = (int)fdiv(blk, a.by_page), in0 = blk - e0 * a.blocks_per_page;
                const bool two = (blk + 1) * kBlockTokens < end, next = in0 + 1 == a.blocks_per_page;
                int p0 = trow[e0], p1 = two && next ? trow[e0 + 1] : p0;
                if (p0 < 0 || p0 >= a.pages || p1 < 0 || p1 >= a.pages) {
                    atomicOr(a.status, kStatusIndex);
                    p0 = p0 < 0 || p0 >= a.pages ? 0 : p0;
                    p1 = p1 < 0 || p1 >= a.pages ? 0 : p1;
                }
                const uint8_t *head = a.pool + (int64_t)kvh * a.blocks_per_page * BB;
                src0 = head + p0 * a.page_bytes + (int64_t)in0 * BB;
                src1 = next ? head + p1 * a.page_bytes : src0 + BB;
                blocks = !two ? 1 : next ? 2 : 3;
            }
        };
        auto issue = [&](int i) {
            if ((i & 31) == 0) find(i + lane);
            if (lane == (i & 31)) {
                const uint32_t dst = ring_s + fill * SB, bar = bar_s + 8 * fill;
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar),
                             "r"(blocks == 1 ? BB : 2 * BB)
                             : "memory");
                asm volatile(
                    "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, "
                    "[%3], %4;" ::"r"(dst), "l"(src0), "r"(blocks == 3 ? 2 * BB : BB), "r"(bar), "l"(policy)
                    : "memory");
                if (blocks == 2)
                    asm volatile(
                        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], "
                        "%2, [%3], %4;" ::"r"(dst + BB), "l"(src1), "r"(BB), "r"(bar), "l"(policy)
                        : "memory");
            }
            fill = fill + 1 == STAGES ? 0 : fill + 1;
        };
        int issued = 0;
        for (; issued < STAGES && issued < mine; ++issued) issue(issued);

    // ---- queries: lane (g, j) holds dims j D/4 .. of row g of each column tile, as the
    // second operand of the first product.  Each row is scaled by a power of two of its
    // own, so that its largest lies in [2^14, 2^15): bf16's eight bits, and fp16's
    // eleven down to 2^-28 of the largest, are kept whole, and a row with an infinity or
    // far larger than the others takes nothing from them.
    uint32_t qf[PARTS][NT][KS][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float top = 0.0f, sum = 0.0f;
#pragma unroll
        for (int w = 0; w < LD / 8; ++w)
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(to_f(raw[nt][w].v[e])));
        top = lanes_max(top, 4);
        // 2^qe: exponent of the largest, kept where 2^(14 - qe) and its inverse are normal
        const int qe = max(-100, min((int)(__float_as_uint(top) >> 23) - 127, 127));
        const float up = ldexpf(1.0f, 14 - qe);
#pragma unroll
        for (int w = 0; w < LD / 8; ++w) {
            float f[8];
            widen(raw[nt][w], f);
            // word w of a lane's codes: pairs (0,4), (1,5)/16 in step 2w and (2,6), (3,7)/16 in step 2w + 1
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                f[e] *= up;
                sum += f[e];
                if (e & 1) f[e] *= 0.0625f;
            }
#pragma unroll
            for (int pr = 0; pr < 4; ++pr) {
                const uint32_t hi = pack_half2(f[pr], f[pr + 4]);
                qf[0][nt][2 * w + (pr >> 1)][pr & 1] = hi;
                if constexpr (SPLIT) {
                    const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                    qf[PARTS - 1][nt][2 * w + (pr >> 1)][pr & 1] =
                        pack_half2((f[pr] - h.x) * 2048.0f, (f[pr + 4] - h.y) * 2048.0f);
                }
            }
        }
        // logits in base 2 are (acc stepK + lowK qsum) * unit, acc in units of 2^-24 where codes are subnormal
        const float unit = a.scale * kLog2eF * ldexpf(1.0f, qe - 14), qsum = lanes_sum(sum, 4) * unit;
        // of rows 2j and 2j + 1, this lane's accumulator columns (kept in shared memory: registers are
        // what the loop lacks)
        const float ku = SPLIT ? unit : unit * 0x1p24f;
        const float4 col = make_float4(__shfl_sync(0xffffffffu, ku, 8 * j), __shfl_sync(0xffffffffu, ku, 8 * j + 4),
                                       __shfl_sync(0xffffffffu, qsum, 8 * j), __shfl_sync(0xffffffffu, qsum, 8 * j + 4));
        if (g == 0) cols[warp][nt][j] = col;
    }
    __syncwarp();

    // ---- running state: per column (2j, 2j + 1 of each tile); the maximum is the
    // warp's, the sums are this lane's share (its tokens)
    float o[KS][NT][4], m[NT][2], l[NT][2], lowsum[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[k][nt][e] = 0.0f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            m[nt][c] = -INFINITY;
            l[nt][c] = lowsum[nt][c] = 0.0f;
        }
    }
    float vcap = 0.0f, vscale = 1.0f;  // largest stepV is below vcap; vscale = 2^E
    int vexp = 0;
    for (int i = 0; i < mine; ++i) {
        const int tok0 = c0 + (warp + i * kWarps) * kTile;
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar_s + 8 * stage, phase))) {  // a warp gives up together
            alive = false;
            break;
        }
        const uint8_t *st = ring + stage * SB;
        const bool masked = tok0 < safe0 || tok0 + kTile > safe1;
        float y[2][NT][4];
        float2 vp[2][2];
        // first product, both blocks at once, the dims in two chains: four independent
        // accumulators hide the latency of a chain
        {
            float acc[2][PARTS][NT][2][4];
            uint32_t k0[2][LD / 8], k1[2][LD / 8];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
#pragma unroll
                for (int p = 0; p < PARTS; ++p)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[q][p][nt][0][e] = acc[q][p][nt][1][e] = 0.0f;
                const uint8_t *kr = st + q * BB + g * (D / 2) + j * (D / 8);
                if constexpr (D == 64) {
                    *reinterpret_cast<uint2 *>(k0[q]) = *reinterpret_cast<const uint2 *>(kr);
                    *reinterpret_cast<uint2 *>(k1[q]) = *reinterpret_cast<const uint2 *>(kr + 8 * (D / 2));
                } else {
#pragma unroll
                    for (int x = 0; x < LD / 32; ++x) {
                        reinterpret_cast<uint4 *>(k0[q])[x] = reinterpret_cast<const uint4 *>(kr)[x];
                        reinterpret_cast<uint4 *>(k1[q])[x] = reinterpret_cast<const uint4 *>(kr + 8 * (D / 2))[x];
                    }
                }
            }
#pragma unroll
            for (int w = 0; w < LD / 8; ++w)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const uint32_t x0 = hf ? k0[q][w] >> 8 : k0[q][w], x1 = hf ? k1[q][w] >> 8 : k1[q][w];
                        const uint32_t a0 = SPLIT ? centred_even(x0, bias) : plain_even(x0);
                        const uint32_t a1 = SPLIT ? centred_even(x1, bias) : plain_even(x1);
                        const uint32_t a2 = SPLIT ? centred_odd(x0, bias) : plain_odd(x0);
                        const uint32_t a3 = SPLIT ? centred_odd(x1, bias) : plain_odd(x1);
#pragma unroll
                        for (int p = 0; p < PARTS; ++p)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16816(acc[q][p][nt][hf], a0, a1, a2, a3, qf[p][nt][2 * w + hf][0],
                                         qf[p][nt][2 * w + hf][1]);
                    }
            // logits: this lane's tokens g and g + 8
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const uint8_t *blk = st + q * BB;
                float2 kp0 = half2_at(blk + kv4_ks_off(D) + 4 * g), kp1 = half2_at(blk + kv4_ks_off(D) + 4 * (g + 8));
                vp[q][0] = half2_at(blk + kv4_vs_off(D) + 4 * g);
                vp[q][1] = half2_at(blk + kv4_vs_off(D) + 4 * (g + 8));
                // centred codes count from low + 8 step
                if constexpr (SPLIT) {
                    kp0.y = fmaf(8.0f, kp0.x, kp0.y);
                    kp1.y = fmaf(8.0f, kp1.x, kp1.y);
                }
                vp[q][0].y = fmaf(8.0f, vp[q][0].x, vp[q][0].y);
                vp[q][1].y = fmaf(8.0f, vp[q][1].x, vp[q][1].y);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float4 col = cols[warp][nt][j];
                    const float ku[2] = {col.x, col.y}, qs[2] = {col.z, col.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float d = acc[q][0][nt][0][e] + acc[q][0][nt][1][e];
                        if constexpr (SPLIT)
                            d = fmaf(acc[q][PARTS - 1][nt][0][e] + acc[q][PARTS - 1][nt][1][e], 1.0f / 2048.0f, d);
                        y[q][nt][e] = fmaf(d, (e < 2 ? kp0.x : kp1.x) * ku[e & 1], (e < 2 ? kp0.y : kp1.y) * qs[e & 1]);
                    }
                }
            }
        }
        if (masked) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int t = (int)fdiv(tile * ROWS + nt * 8 + 2 * j + c, a.by_group);
                    const int hi = upper(a, seq, t), lo = lower(a, seq, t);
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const int tok = tok0 + 16 * q + 8 * r + g;
                            if (tok < lo || tok >= hi) y[q][nt][2 * r + c] = -INFINITY;
                        }
                }
            // a token past the end has no scales (its bytes are whatever the page or the ring held),
            // one before every row's window none that count
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    if (const int tok = tok0 + 16 * q + 8 * r + g; tok >= end || tok < first) vp[q][r] = make_float2(0.0f, 0.0f);
        }
        // A token held as NaN makes the rows that see it NaN, and no others: its scales
        // leave the sums (0 * NaN is not 0) and a NaN joins what is added to each output.
        const float steps = (vp[0][0].x + vp[0][1].x) + (vp[1][0].x + vp[1][1].x);
        if (__any_sync(0xffffffffu, !(steps < INFINITY))) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    if (!(vp[q][r].x < INFINITY)) {
                        vp[q][r] = make_float2(0.0f, 0.0f);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int c = 0; c < 2; ++c)
                                if (y[q][nt][2 * r + c] != -INFINITY) lowsum[nt][c] = NAN;
                    }
        }
        // The reference m moves only where a logit passes it by 2^kSlack, and the steps' cap
        // only past eight times a power of two: moving the running state costs half a
        // tile's work, and following every new maximum of eight rows did so in two
        // tiles of three (attn of 131071 tokens: 44 against 33 us).
        bool grow = false;
        float vmax = fmaxf(fmaxf(vp[0][0].x, vp[0][1].x), fmaxf(vp[1][0].x, vp[1][1].x));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float t = fmaxf(fmaxf(y[0][nt][c], y[0][nt][2 + c]), fmaxf(y[1][nt][c], y[1][nt][2 + c]));
                grow = grow || t > m[nt][c] + kSlack;
            }
        if (__any_sync(0xffffffffu, grow || vmax >= vcap)) {
            vmax = lanes_max(vmax, 32);
            float move = 1.0f;
            if (vmax >= vcap && vmax > 0.0f) {
                const int e = (int)(__float_as_uint(vmax) >> 23) - 127;  // 2^e <= vmax < 2^(e+1)
                move = vcap > 0.0f ? ldexpf(1.0f, vexp - e) : 1.0f;
                vexp = e;
                vcap = ldexpf(1.0f, e + 3);
                vscale = ldexpf(1.0f, kStepBits - e);
            } else if (vcap == 0.0f) {
                vcap = 0x1p-30f;  // only zero steps so far
                vexp = -33;
                vscale = ldexpf(1.0f, kStepBits + 33);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float t = fmaxf(fmaxf(y[0][nt][c], y[0][nt][2 + c]), fmaxf(y[1][nt][c], y[1][nt][2 + c]));
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, x));
                    const float mn = fmaxf(m[nt][c], t - LEAD);
                    const float f = m[nt][c] == -INFINITY ? 0.0f : ex2(m[nt][c] - mn);
                    m[nt][c] = mn;
                    l[nt][c] *= f;
                    lowsum[nt][c] *= f;
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        o[k][nt][c] *= f * move;
                        o[k][nt][2 + c] *= f * move;
                    }
                }
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const uint8_t *blk = st + q * BB;
            uint32_t pb[PARTS][NT][2];
            const float vs0 = vp[q][0].x * vscale, vs1 = vp[q][1].x * vscale;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float mm = m[nt][e & 1];
                    const float p = ex2(y[q][nt][e] - (mm == -INFINITY ? 0.0f : mm));
                    l[nt][e & 1] += p;
                    lowsum[nt][e & 1] = fmaf(p, e < 2 ? vp[q][0].y : vp[q][1].y, lowsum[nt][e & 1]);
                    w[e] = p * (e < 2 ? vs0 : vs1);
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint32_t hi = pack_half2(w[2 * r], w[2 * r + 1]);
                    pb[0][nt][r] = transpose8x8(hi);
                    if constexpr (SPLIT) {
                        const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                        // the rest, below 2^4 against a largest of 2^15
                        pb[PARTS - 1][nt][r] = transpose8x8(pack_half2(w[2 * r] - h.x, w[2 * r + 1] - h.y));
                    }
                }
            }
            // second product: pairs j and j + 4 of tokens, slice g of dims
            constexpr int VW = D / 128 > 0 ? D / 64 : 1;  // words of 8 dims a token has in a slice: 1, 2, 4
            uint32_t v0[2 * VW], v1[2 * VW];  // [token parity][word]
            const uint8_t *vr = blk + kv4_v_off(D) + j * D + g * (D / 8);
            if constexpr (D == 64) {
                *reinterpret_cast<uint2 *>(v0) = *reinterpret_cast<const uint2 *>(vr);
                *reinterpret_cast<uint2 *>(v1) = *reinterpret_cast<const uint2 *>(vr + 4 * D);
            } else {
#pragma unroll
                for (int x = 0; x < VW / 2; ++x) {
                    reinterpret_cast<uint4 *>(v0)[x] = reinterpret_cast<const uint4 *>(vr)[x];
                    reinterpret_cast<uint4 *>(v1)[x] = reinterpret_cast<const uint4 *>(vr + 4 * D)[x];
                }
            }
#pragma unroll
            for (int w = 0; w < VW; ++w)
#pragma unroll
                for (int pr = 0; pr < 2; ++pr) {
                    const uint32_t sel = pr ? 0x7632u : 0x5410u;  // (even, odd) token: low or high 16 bits
                    const uint32_t e0 = __byte_perm(v0[w], v0[VW + w], sel), e1 = __byte_perm(v1[w], v1[VW + w], sel);
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const uint32_t x0 = hf ? e0 >> 8 : e0, x1 = hf ? e1 >> 8 : e1;
                        const uint32_t a0 = centred_even(x0, bias), a1 = centred_odd(x0, bias);
                        const uint32_t a2 = centred_even(x1, bias), a3 = centred_odd(x1, bias);
#pragma unroll
                        for (int p = 0; p < PARTS; ++p)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16816(o[4 * w + 2 * pr + hf][nt], a0, a1, a2, a3, pb[p][nt][0], pb[p][nt][1]);
                    }
                }
        }
        __syncwarp();  // every lane has read the stage
        if (issued < mine) issue(issued++);
        if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
        }
    }
    if (!alive) {
        // let what is in flight land before the block's shared memory goes: the
        // stages from the one that did not come
        if (lane == 0) atomicOr(a.status, kStatusTimeout);
        do {
            mbar_wait_bounded(bar_s + 8 * stage, phase);
            if (++stage == STAGES) {
                stage = 0;
                phase ^= 1;
            }
        } while (stage != fill);
    }
    pdl_wait();
    if (!__syncthreads_and(alive)) return;

    // ---- join the warps.  o: dims 2k of slice g in elements 0, 1 and 2k + 1 in 2, 3,
    // in units of 2^E (16 times that for the odd ones)
    const float even = ldexpf(1.0f, vexp - kStepBits), odd = even * 0.0625f;
    float *stat = reinterpret_cast<float *>(smem);            // [kWarps][ROWS][2]: maximum, sum
    float *buf = stat + kWarps * ROWS * 2;                    // [kWarps][ROWS][D / PASS]
    constexpr int kRoom = kWarps * STAGES * SB - kWarps * ROWS * 8;
    constexpr int kNeed = kWarps * ROWS * D * 4;
    constexpr int PASS = kNeed <= kRoom ? 1 : kNeed <= 2 * kRoom ? 2 : 4;  // parts of the dims joined at a time
    static_assert(kNeed <= 4 * kRoom, "join buffer");
    constexpr int KP = KS / PASS, DP = D / PASS;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) {
                l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], x);
                lowsum[nt][c] += __shfl_xor_sync(0xffffffffu, lowsum[nt][c], x);
            }
            if (g == 0) {
                float *q = stat + (warp * ROWS + nt * 8 + 2 * j + c) * 2;
                q[0] = m[nt][c];
                q[1] = l[nt][c];
            }
        }
    const int64_t all_rows = a.Tq * a.Hq;
#pragma unroll
    for (int ps = 0; ps < PASS; ++ps) {
        if (ps > 0) __syncthreads();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                // this lane's 2 KP dims of this part: 2 KP g .. of it
                float *q = buf + ((warp * ROWS + nt * 8 + 2 * j + c) * 8 + g) * (2 * KP);
#pragma unroll
                for (int k = 0; k < KP; ++k) {
                    q[2 * k] = fmaf(o[ps * KP + k][nt][c], even, lowsum[nt][c]);
                    q[2 * k + 1] = fmaf(o[ps * KP + k][nt][2 + c], odd, lowsum[nt][c]);
                }
            }
        __syncthreads();
        for (int x = threadIdx.x; x < rows * (DP / 2); x += kWarps * 32) {
            const int row = x / (DP / 2), d2 = x % (DP / 2) * 2;
            float mm = -INFINITY, ll = 0.0f, v0 = 0.0f, v1 = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, stat[(w * ROWS + row) * 2]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float mw = stat[(w * ROWS + row) * 2];
                // (a warp that saw nothing: m = -inf, sum and output 0; a NaN sum stays a NaN)
                const float f = mw == -INFINITY ? 1.0f : ex2(mw - mm);
                const float2 v = *reinterpret_cast<const float2 *>(buf + (w * ROWS + row) * DP + d2);
                ll = fmaf(stat[(w * ROWS + row) * 2 + 1], f, ll);
                v0 = fmaf(v.x, f, v0);
                v1 = fmaf(v.y, f, v1);
            }
            // dims of this part: 2 KP of every slice of 2 KS
            const int d = d2 / (2 * KP) * (2 * KS) + ps * 2 * KP + d2 % (2 * KP);
            if (!seg.whole) {
                // the first segment of a block starts inside an item or is slot 1's like any other
                float *slot = a.part + (2 * (int64_t)blockIdx.x + (seg.unit0 == 0 ? 1 : 0)) * (ROWS * (D + 2));
                *reinterpret_cast<float2 *>(slot + row * D + d) = make_float2(v0, v1);
                if (d == 0) *reinterpret_cast<float2 *>(slot + ROWS * D + row * 2) = make_float2(mm, ll);
            } else {
                const int full_row = tile * ROWS + row, t = (int)fdiv(full_row, a.by_group);
                const int hq = kvh * a.G + full_row - t * a.G;
                const int64_t q = (int64_t)(seq.q0 + t) * a.Hq + hq;
                const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
                T *out = reinterpret_cast<T *>(a.O) + (int64_t)(seq.q0 + t) * a.os_tok + hq * a.os_head + d;
                if (a.vec) {
                    Vec<T, 2> v;
                    v.v[0] = from_f<T>(v0 * inv);
                    v.v[1] = from_f<T>(v1 * inv);
                    store_vec(out, v);
                } else {
                    out[0] = from_f<T>(v0 * inv);
                    out[1] = from_f<T>(v1 * inv);
                }
                if (d == 0 && a.lse) a.lse[q] = ll == 0.0f ? -INFINITY : (mm + log2f(ll)) * kLn2;
            }
        }
    }
    // the ring takes copies again: after every thread's last look at the join's buffers
    __syncthreads();
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
}

// Joins the partial outputs of an item's rows: 8 warps, W of them a row (1 or 8), each
// every W-th partial with a running maximum of its own, a lane D/32 dims; then a row's
// warps in order.  Items with few partials (many items) take a warp a row, few items
// with many partials all eight.
// U: partials of a row a warp has in flight.  R: rows a warp has, all in flight (W = 1).
template <typename T, int D, int U, int R>
__global__ void __launch_bounds__(256) kv4_join_kernel(const __grid_constant__ AttnArgs a, int rows_of_tile, int W)
{
    constexpr int E = D / 32, F = E < 4 ? E : 4;
    __shared__ float sums[8][D], stat[8][2];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rows_here = 8 / W * R, sub = warp % W;
    // blockIdx.x = ((b * Hkv + kvh) * row_tiles + tile) * (rows_of_tile / rows_here) + part
    const unsigned parts = rows_of_tile / rows_here, item = blockIdx.x / parts;
    const int row = (int)(blockIdx.x - item * parts) * rows_here + warp / W;  // and every 8th after it
    const int2 job = a.job[item];
    const unsigned bh = item / a.row_tiles;
    const int tile = (int)(item - bh * a.row_tiles), b = (int)(bh / a.Hkv), kvh = (int)(bh - b * a.Hkv);
    const Seq seq = sequence(a, b, false);
    if (tile * rows_of_tile >= seq.n * a.G) return;  // not an item: its job was not noted
    const int n = job.y;
    if (!job_in_grid(job.x, n, a.grid)) {
        if (threadIdx.x == 0) atomicOr(a.status, kStatusTimeout);
        return;
    }
    if (n == 1) return;  // one block had the whole item and wrote its output
    const int stride = rows_of_tile * (D + 2);
    // partial p: the item's first block holds it in its slot 1, the others in slot 0
    const float *first = a.part + (int64_t)2 * job.x * stride;
    float mm[R], ll[R], v[R][E];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        mm[r] = -INFINITY;
        ll[r] = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) v[r][e] = 0.0f;
    }
    for (int p0 = sub; p0 < n; p0 += U * W) {
        Vec<float, F> x[R][U][E / F];
        float2 ms[R][U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int p = p0 + u * W;
            const float *q = first + (int64_t)(p == 0 ? 1 : 2 * p) * stride;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                ms[r][u] = make_float2(-INFINITY, 0.0f);
                if (p < n) ms[r][u] = *reinterpret_cast<const float2 *>(q + rows_of_tile * D + (row + 8 * r) * 2);
#pragma unroll
                for (int e = 0; e < E / F; ++e)
                    if (p < n)
                        x[r][u][e] = *reinterpret_cast<const Vec<float, F> *>(q + (row + 8 * r) * D + lane * E + e * F);
                    else
                        x[r][u][e] = {};
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float top = mm[r];
#pragma unroll
            for (int u = 0; u < U; ++u) top = fmaxf(top, ms[r][u].x);
            const float f0 = mm[r] == -INFINITY ? 1.0f : ex2(mm[r] - top);
            ll[r] *= f0;
#pragma unroll
            for (int e = 0; e < E; ++e) v[r][e] *= f0;
            mm[r] = top;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float f = ms[r][u].x == -INFINITY ? 1.0f : ex2(ms[r][u].x - top);  // a share that saw nothing holds zeros
                ll[r] = fmaf(ms[r][u].y, f, ll[r]);
#pragma unroll
                for (int e = 0; e < E; ++e) v[r][e] = fmaf(x[r][u][e / F].v[e % F], f, v[r][e]);
            }
        }
    }
    if (W > 1) {  // (R = 1)
#pragma unroll
        for (int e = 0; e < E; ++e) sums[warp][lane * E + e] = v[0][e];
        if (lane == 0) {
            stat[warp][0] = mm[0];
            stat[warp][1] = ll[0];
        }
        __syncthreads();
        if (sub != 0) return;
        float top = mm[0];
        for (int w = 1; w < W; ++w) top = fmaxf(top, stat[warp + w][0]);
        const float f0 = mm[0] == -INFINITY ? 1.0f : ex2(mm[0] - top);
        ll[0] *= f0;
#pragma unroll
        for (int e = 0; e < E; ++e) v[0][e] *= f0;
        for (int w = 1; w < W; ++w) {
            const float mw = stat[warp + w][0], f = mw == -INFINITY ? 1.0f : ex2(mw - top);
            ll[0] = fmaf(stat[warp + w][1], f, ll[0]);
#pragma unroll
            for (int e = 0; e < E; ++e) v[0][e] = fmaf(sums[warp + w][lane * E + e], f, v[0][e]);
        }
        mm[0] = top;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int full_row = tile * rows_of_tile + row + 8 * r;
        if (full_row >= seq.n * a.G) return;
        const int t = (int)fdiv(full_row, a.by_group), hq = kvh * a.G + full_row - t * a.G;
        const int64_t q = (int64_t)(seq.q0 + t) * a.Hq + hq;
        const float inv = ll[r] == 0.0f ? 0.0f : 1.0f / ll[r];
        T *out = reinterpret_cast<T *>(a.O) + (int64_t)(seq.q0 + t) * a.os_tok + hq * a.os_head + lane * E;
        if (a.vec && E * sizeof(T) <= 16) {
            Vec<T, E> o;
#pragma unroll
            for (int e = 0; e < E; ++e) o.v[e] = from_f<T>(v[r][e] * inv);
            store_vec(out, o);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) out[e] = from_f<T>(v[r][e] * inv);
        }
        if (lane == 0 && a.lse) a.lse[q] = ll[r] == 0.0f ? -INFINITY : (mm[r] + log2f(ll[r])) * kLn2;
    }
}

// Column tiles for a sequence's rows (its queries x the heads of a group).
// fp32 needs twice the registers for q, D = 256 twice those for the output.
int pick_nt(int64_t rows, int D, bool f32)
{
    return rows > 8 && D != 256 && !f32 ? 2 : 1;
}

// Bytes of the partial slots and of the items' jobs.  For any element type: the most.
size_t attn_workspace(int32_t B, int32_t max_q, int32_t Hq, int32_t Hkv, int32_t D)
{
    const int64_t rows = (int64_t)max_q * (Hq / Hkv);
    size_t slots = 2 * kMostBlocks * (size_t)(rows > 8 ? 16 : 8) * (D + 2) * sizeof(float);
    if (chunk_attn_fits(TM_BF16, rows, D) && chunk_attn_slots_bytes(D) > slots) slots = chunk_attn_slots_bytes(D);
    return slots + (size_t)B * Hkv * ((size_t)rows + 7) / 8 * sizeof(int2);
}

template <typename T, int D>
tm_status join_items(AttnArgs &a, int rows_of_tile, int sms, cudaStream_t s)
{
    const int64_t items = (int64_t)a.B * a.Hkv * a.row_tiles;
    int W = 1, rows = 1;  // warps of a row, rows of a warp
    const void *k = (const void *)kv4_join_kernel<T, D, D == 256 ? 4 : 8, 1>;
    if constexpr (sizeof(T) == 2 && D != 256) {
        // An item has about sms / items + 1 partials.  256 rows a tile, D 128, the whole call:
        // 64 items 87.7 us with four rows a warp, 90.5 with eight partials of one; 32 items
        // 67.7 against 64.0; 16 items 55.9 against 45.4.
        if (rows_of_tile == kChunkRows && 4 * items >= sms) {
            k = (const void *)kv4_join_kernel<T, D, 2, 4>;
            rows = 4;
        }
    }
    if (rows_of_tile != kChunkRows) {
        W = items >= sms ? 1 : 8;
        if (W == 1) k = (const void *)kv4_join_kernel<T, D, 2, 1>;
    }
    void *jargs[] = {(void *)&a, &rows_of_tile, &W};
    return launch_dependent(k, dim3((unsigned)(items * rows_of_tile / (8 / W * rows))), dim3(256), jargs, 0, s);
}

template <typename T, int D, int NT>
tm_status launch_attn(AttnArgs &a, int dev, int sms, bool join, cudaStream_t s, bool pdl)
{
    const void *k = (const void *)kv4_attn_kernel<T, D, NT>;
    static std::atomic<bool> ready[kMaxDevices];  // once a device
    if (!ready[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, attn_smem<D>()) != cudaSuccess) {
            cudaGetLastError();
            return TM_ERR_CUDA;
        }
        ready[dev].store(true, std::memory_order_release);
    }
    int64_t blocks = (int64_t)sms * blocks_per_sm<T, D, NT>();
    if (blocks > kMostBlocks) blocks = kMostBlocks;
    a.grid = (int)blocks;
    void *args[] = {(void *)&a};
    tm_status st = launch_kernel(k, dim3((unsigned)blocks), dim3(kWarps * 32), args, attn_smem<D>(), s, pdl);
    if (st != TM_OK || !join) return st;
    return join_items<T, D>(a, NT * 8, sms, s);
}

template <typename T>
tm_status launch_attn(int D, int nt, AttnArgs &a, int dev, int sms, bool join, cudaStream_t s, bool pdl)
{
    if constexpr (sizeof(T) == 2) {
        if (nt == 2)
            return D == 64 ? launch_attn<T, 64, 2>(a, dev, sms, join, s, pdl)
                           : launch_attn<T, 128, 2>(a, dev, sms, join, s, pdl);
    }
    return D == 64    ? launch_attn<T, 64, 1>(a, dev, sms, join, s, pdl)
           : D == 128 ? launch_attn<T, 128, 1>(a, dev, sms, join, s, pdl)
                      : launch_attn<T, 256, 1>(a, dev, sms, join, s, pdl);
}

bool attn_shape_ok(int32_t B, int64_t Tq, int32_t max_q, int64_t max_len, int32_t Hq, int32_t Hkv)
{
    return B >= 0 && Tq >= 0 && max_q >= 0 && max_len >= 0 && max_len <= (1 << 30) && Hkv > 0 && Hq > 0 &&
           Hq % Hkv == 0 && Hq <= 65536 && Tq <= INT32_MAX && max_q <= (1 << 24) / (Hq / Hkv);
}

}  // namespace

tm_status launch_chunk_join(int D, int32_t xtype, AttnArgs &a, int sms, cudaStream_t s)
{
    if (xtype == TM_F16) return D == 64 ? join_items<__half, 64>(a, kChunkRows, sms, s) : join_items<__half, 128>(a, kChunkRows, sms, s);
    return D == 64 ? join_items<__nv_bfloat16, 64>(a, kChunkRows, sms, s)
                   : join_items<__nv_bfloat16, 128>(a, kChunkRows, sms, s);
}

}  // namespace libtm

using namespace libtm;

extern "C" size_t tm_kv4_attention_workspace_bytes(int32_t B, int64_t Tq, int32_t max_q, int64_t max_len, int32_t Hq,
                                                   int32_t Hkv, int32_t D)
{
    if (!attn_shape_ok(B, Tq, max_q, max_len, Hq, Hkv) || !kv4_head_ok(D) || B == 0 || Tq == 0 || max_q == 0) return 0;
    return max_len <= kUnit ? 0 : attn_workspace(B, max_q, Hq, Hkv, D);
}

extern "C" tm_status tm_kv4_attention(const void *Q, int64_t qs_tok, int64_t qs_head, void *O, int64_t os_tok,
                                      int64_t os_head, float *lse, const void *pool, int64_t pages, int32_t page,
                                      const int32_t *table, int64_t ldt, const int32_t *lens, const int32_t *qstart,
                                      int32_t B, int64_t Tq, int32_t max_q, int64_t max_len, int32_t Hq, int32_t Hkv,
                                      int32_t D, float scale, int32_t window, int32_t xtype, void *workspace,
                                      size_t ws_bytes, uint32_t flags, tm_stream_t stream)
{
    const int e = elem_bytes(xtype);
    if (e == 0 || (flags & ~(TM_ATTN_FULL | TM_PDL))) return TM_ERR_INVALID_ARG;
    if (!attn_shape_ok(B, Tq, max_q, max_len, Hq, Hkv) || window < 0) return TM_ERR_INVALID_ARG;
    if ((flags & TM_ATTN_FULL) && window > 0) return TM_ERR_INVALID_ARG;
    if (!kv4_head_ok(D) || page <= 0 || page % 16 != 0) return TM_ERR_UNSUPPORTED_TILE;
    const Heads q = {Q, qs_tok, qs_head}, o = {O, os_tok, os_head};
    if (!heads_ok(q, Tq, Hq, D) || !heads_ok(o, Tq, Hq, D)) return TM_ERR_INVALID_ARG;
    if (!kv4_pool_ok(pool, pages, page, Hkv, D)) return TM_ERR_INVALID_ARG;
    if (B == 0 || Tq == 0) return TM_OK;
    if (max_q < 1 || lens == nullptr || (qstart == nullptr && Tq != B)) return TM_ERR_INVALID_ARG;
    if (ldt < (max_len + page - 1) / page || (max_len > 0 && (table == nullptr || pages == 0)) || ldt > INT64_MAX / 8 / B)
        return TM_ERR_INVALID_ARG;
    if (!aligned_to(Q, e) || !aligned_to(O, e) || !aligned_to(pool, 16) || !aligned_to(lse, 4) || !aligned_to(table, 4) ||
        !aligned_to(lens, 4) || !aligned_to(qstart, 4))
        return TM_ERR_MISALIGNED;
    // one unit an item at most: every item is one block's, nothing to join
    const bool join = max_len > kUnit;
    const size_t need = join ? attn_workspace(B, max_q, Hq, Hkv, D) : 0;
    if (need > 0 && (workspace == nullptr || ws_bytes < need || !aligned_to(workspace, 16))) return TM_ERR_WORKSPACE;
    const int64_t pb = (int64_t)tm_kv4_page_bytes(Hkv, D, page);
    const Span so = heads_span(o, Tq, Hq, D, e), sl = span_of(lse, Tq * Hq, lse ? 1 : 0, Tq * Hq, 4),
               sw = need ? span_of(workspace, (int64_t)need, 1, (int64_t)need, 1) : Span{0, 0};
    const Span ins[] = {heads_span(q, Tq, Hq, D, e), span_of(pool, pages * pb, 1, pages * pb, 1),
                        span_of(table, ldt, B, ldt, 4), span_of(lens, B, 1, B, 4), span_of(qstart, B + 1, 1, B + 1, 4)};
    for (const Span &s : ins)
        if (meets(so, s) || meets(sl, s) || meets(sw, s)) return TM_ERR_INVALID_ARG;
    if (meets(so, sl) || meets(so, sw) || meets(sl, sw)) return TM_ERR_INVALID_ARG;
    const int64_t most_rows = (int64_t)max_q * (Hq / Hkv);
    const bool chunk = chunk_attn_fits(xtype, most_rows, D);
    const int nt = pick_nt(most_rows, D, e == 4), rows_of_tile = chunk ? kChunkRows : nt * 8;
    const int64_t row_tiles = (most_rows + rows_of_tile - 1) / rows_of_tile;
    // the units of all items, and the join's grid, fit 31 bits (with room for a block's share)
    if (row_tiles > (1 << 30) / rows_of_tile / ((int64_t)B * Hkv) ||
        (max_len / kUnit + 4) > (1 << 30) / ((int64_t)B * Hkv * row_tiles))
        return TM_ERR_INVALID_ARG;
    const DevInfo *dev;
    tm_status st = device_info(&dev);
    if (st != TM_OK) return st;
    AttnArgs a = {};
    a.Q = Q;
    a.O = O;
    a.lse = lse;
    a.pool = reinterpret_cast<const uint8_t *>(pool);
    a.table = table;
    a.lens = lens;
    a.qstart = qstart;
    a.part = reinterpret_cast<float *>(workspace);
    a.job = join ? reinterpret_cast<int2 *>(reinterpret_cast<char *>(workspace) +
                                           (chunk ? chunk_attn_slots_bytes(D)
                                                  : 2 * (size_t)kMostBlocks * nt * 8 * (D + 2) * sizeof(float)))
                 : nullptr;
    a.qs_tok = qs_tok;
    a.qs_head = qs_head;
    a.os_tok = os_tok;
    a.os_head = os_head;
    a.pages = pages;
    a.page_bytes = pb;
    a.ldt = ldt;
    a.Tq = Tq;
    a.max_len = max_len;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    a.window = window_of(window, max_len);
    a.full = (flags & TM_ATTN_FULL) ? 1 : 0;
    a.vec = heads_vec(q, e) && heads_vec(o, e) ? 1 : 0;
    a.blocks_per_page = page / 16;
    a.by_page = make_fastdiv((uint32_t)a.blocks_per_page);
    a.by_group = make_fastdiv((uint32_t)a.G);
    a.max_q = max_q;
    a.row_tiles = (int)row_tiles;
    // Row tiles by what they see, if the queries are a good part of the tokens and items have
    // several units.  32 heads on 8, D 128, counting all alike / by what they see, us: 8192
    // queries on 8192 tokens 1248 / 746, two of 4096 on 4096 585 / 401, 2048 on 8192 354 / 322,
    // four of 1024 on 4096 321 / 306, four of 1024 on 1024 107 / 107; four of 512 on 4096 173 / 180,
    // eight of 512 on 512 75 / 86.  (With more queries than tokens the tiles' ends would pass
    // max_len, the bound above.)
    a.tile_step = -1;
    if (chunk && !a.full && a.window == 0 && kChunkRows % a.G == 0 && max_len > 4 * kUnit && max_q <= max_len &&
        4 * (int64_t)max_q >= max_len)
        for (a.tile_step = 0; a.G << a.tile_step < kChunkRows;) ++a.tile_step;  // kChunkRows / G, a power of two
    a.bias = 0x64006400u;
    a.scale = scale;
    a.status = dev->status;
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) {
        cudaGetLastError();
        return TM_ERR_CUDA;
    }
    cudaStream_t s = as_stream(stream);
    const bool pdl = (flags & TM_PDL) != 0;
    if (chunk) return launch_chunk_attn(D, xtype, a, device, dev->sms, join, s, pdl);
    return xtype == TM_F32   ? launch_attn<float>(D, nt, a, device, dev->sms, join, s, pdl)
           : xtype == TM_F16 ? launch_attn<__half>(D, nt, a, device, dev->sms, join, s, pdl)
                             : launch_attn<__nv_bfloat16>(D, nt, a, device, dev->sms, join, s, pdl);
}
