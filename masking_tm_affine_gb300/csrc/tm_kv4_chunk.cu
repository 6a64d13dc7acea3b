// tm_kv4_chunk.cu -- attention over the 4-bit cache for many query rows (the chunks
// of a prompt): the same mathematics as tm_kv4_attn.cu, on tcgen05.
//
// The least it has to do is 4 D flops and one exponential for each (query row, token).
// An item's row tile is 256 rows (queries x the heads that share a KV head), two
// halves of 128, walked over 128 tokens at a time:
//
//   loader warp      bulk copies of the tile's eight cache blocks
//   4 unpack warps   codes -> fp16 in shared memory, once for both halves: K as the
//                    whole numbers c, V as the values low + c step
//   2 MMA warps      a half each, so that neither waits for the other's softmax:
//                    S = Q K^T  [128 rows, 64 tokens], both operands in shared memory,
//                    half a tile ahead of the softmax;
//                    O += P V   [128 rows, D], P from tensor memory, 32 tokens at a time
//   2 x 4 warps      a half each, a thread a row: S from tensor memory, softmax, P back
//                    into the columns S came from
//
// What bounds it: the softmax warps, two to a scheduler, by the latency of their chain
// (read S, maximum, exponentials, write P): 256 queries on 2 sequences of 4 100 to 8 192
// tokens, 32 heads on 8, D 128, bf16, the whole call 88 us, about 70 of them this kernel's,
// 60 of those its tiles, about 5800 cycles each, of which the products need 1024.  There
// the tensor cores are 28% busy, the issue slots 49%, the exponential unit 14%.
// 2048 queries on 8192 tokens: 319 us, 755 TFLOP/s; 8192 on 8192: 745 us, 738.
// On the way, the first of these calls: one warp issuing both halves' products in turn
// 109 us, 124 with S made half a tile ahead; two warps, S of a tile made after the tile
// before, 107, ahead 99; the softmax step's loop unrolled 118 instead of 89 (the roles'
// code outgrows the instruction caches); an exponent of Q common to the tile, which the
// halves exchanged before the first product, 90.
//
// Shared memory: Q and K are K-major, V is MN-major (a token's dims contiguous), all in
// 128-byte swizzled panels of 64 dims; a word's eight dims lie in the order 0 4 1 5 2 6
// 3 7, the order its nibbles come in (Q is written in the same order, O is read back
// in it).  Tensor memory: S of both halves in columns 0 .. 255, O in 256 .. 511.
//
// K's scales stay outside its product, as in tm_kv4_attn.cu, so that logits keep fp32's
// accuracy; a thread multiplies them in, two floats a token.  V's are multiplied into
// its operand, which rounds each value to fp16, off by 2^-11 of itself like the
// probabilities; the exponent of the largest value so far comes off first, so that the
// rounding does not depend on V's size.  That value may be a token's that a row does not
// see: it goes in at 2^9 and more, so that what lies 2^20 below it (fp16's steps and lows reach
// no further from 1) still keeps 2^-13 of itself.
//
// A thread has a whole row, so its maximum and sums need no exchange.  The reference
// lies 2^7 below the maximum that set it: probabilities go up from 2^7 in fp16, so that
// those of 2^-21 and more of the maximum keep fp16's eleven bits, and what vanishes lies
// below 2^-32 of it (a long context holds 10^5 of them).  It moves only where a logit
// passes that maximum by 2^8, and V's exponent only past a power of two well above it: O
// is then scaled in tensor memory, which almost never happens after a segment's first
// tile.
//
// Every wait is bounded.  One that runs out sets the abort flag, which every role
// looks at; outstanding copies and products are waited for before the block ends.
#include <atomic>

#include "tm_kv4_attn.cuh"

namespace libtm {
namespace {

constexpr int kTok = 128;            // tokens of a tile
constexpr int kStep = 32, kSteps = kTok / kStep;  // tokens of one step of the second product
constexpr int kUnpackWarps = 4;
constexpr int kThreads2 = 16 * 32;   // warps 0-7 softmax, 8-11 unpack, 12 and 14 MMA, 13 loader (15 idle)
// Registers: 128 a thread at launch (all there are); the softmax warps, which hold a
// step of S and P of a row, take what the others give: 2 x 168 + 2 x 88 = 4 x 128.
// (152 and 104: 90.5 us for 88.5.)
constexpr int kSoftmaxRegs = 168, kOtherRegs = 88;
static_assert(2 * kSoftmaxRegs + 2 * kOtherRegs == 4 * 128, "register shares");
constexpr int kHead = 7;  // 2^(kHead + kSlack) is the largest probability, below fp16's 2^16
static_assert(kHead + kSlack <= 15, "probabilities in fp16");
constexpr int kValueBits = 9;  // the largest value lies in [2^9, 2^12) of fp16's 2^16
constexpr int kRawStages = 2, kOpStages = 3, kParStages = 2;

template <int D>
struct ChunkSmem {
    alignas(1024) uint8_t q[2][D / 64][128 * 128];           // [half][panel]: 128 rows of 128 bytes
    alignas(1024) uint8_t op[kOpStages][D / 64 * 128 * 128];  // K tiles: panels as Q; V tiles: [8 tokens][panel]
    alignas(128) uint8_t raw[kRawStages][kTok / 16 * kv4_block_bytes(D)];
    alignas(16) float kpar[kParStages][kTok / 2][4];  // K's scales, two tokens at a time: steps, lows
    int vexp[kParStages];
    uint32_t vnan[kParStages][kTok / 32];  // tokens whose V is held as NaN
    alignas(8) uint64_t raw_full[kRawStages], raw_free[kRawStages], op_full[kOpStages], op_free[kOpStages],
        par_full[kParStages], par_free[kParStages], q_full, s_full[2][2], p_full[2][kSteps], o_done[2][kSteps], done;
    uint32_t tmem;
    int abort;
};

__device__ __forceinline__ void bar_init(uint64_t *b, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t *b)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(b)) : "memory");
}

// Wait for a phase; false after the limit, or once any role has given up.
__device__ __forceinline__ bool bar_wait(uint64_t *b, uint32_t parity, volatile int *abort, unsigned *status)
{
    const uint32_t at = smem_u32(b);
    if (mbar_try_wait(at, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(at, parity)) {
        if (*abort) return false;
        if (clock64() - t0 > kWaitCycles) {
            *abort = 1;
            atomicOr(status, kStatusTimeout);
            return false;
        }
    }
    return true;
}

// A counter of a ring's uses: stage and the parity of its next completion.
struct Turn {
    uint32_t stage = 0, phase = 0;
    __device__ __forceinline__ void next(uint32_t stages)
    {
        if (++stage == stages) {
            stage = 0;
            phase ^= 1;
        }
    }
};

// Shared-memory descriptors, 128-byte swizzle (layout 2), version 1.  K-major: groups
// of 8 rows 1024 bytes apart.  MN-major: panels of 64 columns `panel` bytes apart,
// groups of 8 rows of the other extent `group` bytes apart.
__device__ __forceinline__ uint64_t desc_k(uint32_t at)
{
    return (uint64_t)((at >> 4) & 0x3FFF) | (1ull << 16) | ((1024ull >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t at, uint32_t panel, uint32_t group)
{
    return (uint64_t)((at >> 4) & 0x3FFF) | ((uint64_t)(panel >> 4) << 16) | ((uint64_t)(group >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
}

// Instruction descriptor, kind::f16: D fp32 (bits 4-5 = 1), A and B fp16 (0), B
// MN-major (bit 16), N >> 3 at bit 17, M >> 4 at bit 24.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn)
{
    return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t da, uint64_t db, uint32_t id, bool acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(da), "l"(db), "r"(id), "r"((uint32_t)acc)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t db, uint32_t id, bool acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(db), "r"(id), "r"((uint32_t)acc)
        : "memory");
}
// One lane of the warp, the same at every call.  The compiler knows that code under
// this has one active lane and can keep descriptors in uniform registers.
__device__ __forceinline__ bool elect()
{
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e)::"memory");
    return e != 0;
}
__device__ __forceinline__ void commit(uint64_t *b)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(b))
                 : "memory");
}

// 32 columns of this warp's 32 rows, a row a lane.
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at));
}
// The loads' end, for registers that were named before it.
__device__ __forceinline__ void tmem_load_wait(uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.wait::ld.sync.aligned;"
        : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
          "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
          "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
          "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t at, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at));
}
__device__ __forceinline__ void tmem_load_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_store16(uint32_t at, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2 *>(&x); }
__device__ __forceinline__ uint32_t as_bits(__half2 x) { return *reinterpret_cast<const uint32_t *>(&x); }

// Eight codes of a word as whole numbers in fp16, in the order 0 4 1 5 2 6 3 7.  Even
// nibbles: 1024 + c less 1024; odd ones: (1024 + 16 c) / 16 less 64.  Exact.
__device__ __forceinline__ uint4 unpack8(uint32_t w, uint32_t bias)
{
    const __half2 e0 = as_half2(0x64006400u), sx = as_half2(0x2c002c00u), o0 = as_half2(0xd400d400u);  // 1024, 1/16, -64
    const uint32_t v = w >> 8;
    return make_uint4(as_bits(__hsub2(as_half2((w & 0x000f000fu) | bias), e0)),
                      as_bits(__hfma2(as_half2((w & 0x00f000f0u) | bias), sx, o0)),
                      as_bits(__hsub2(as_half2((v & 0x000f000fu) | bias), e0)),
                      as_bits(__hfma2(as_half2((v & 0x00f000f0u) | bias), sx, o0)));
}

// The values they stand for, rounded once.
__device__ __forceinline__ uint4 scaled8(uint4 c, __half2 step, __half2 low)
{
    return make_uint4(as_bits(__hfma2(as_half2(c.x), step, low)), as_bits(__hfma2(as_half2(c.y), step, low)),
                      as_bits(__hfma2(as_half2(c.z), step, low)), as_bits(__hfma2(as_half2(c.w), step, low)));
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair2(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 both(uint64_t p)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ void st_shared(uint32_t at, uint4 v)
{
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads2, 1) kv4_chunk_kernel(const __grid_constant__ AttnArgs a)
{
    constexpr int BB = kv4_block_bytes(D), PANELS = D / 64;
    constexpr uint32_t kS = 0, kO = 256;  // first columns of S and O in tensor memory
    extern __shared__ __align__(1024) unsigned char raw_smem[];
    using Smem = ChunkSmem<D>;
    // (an offset, not a rounded address: the compiler has to see shared memory)
    Smem &s = *reinterpret_cast<Smem *>(raw_smem + ((1024 - (smem_u32(raw_smem) & 1023)) & 1023));
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Run run;
    const bool work = find_run(a, kChunkRows, warp == 0, run);
    if (!work) {  // the same for every warp
        pdl_wait();
        return;
    }
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < kRawStages; ++i) {
            bar_init(&s.raw_full[i], 1);
            bar_init(&s.raw_free[i], kUnpackWarps * 32);
        }
        for (int i = 0; i < kOpStages; ++i) {
            bar_init(&s.op_full[i], kUnpackWarps * 32);
            bar_init(&s.op_free[i], 2);
        }
        for (int i = 0; i < kParStages; ++i) {
            bar_init(&s.par_full[i], kUnpackWarps * 32);
            bar_init(&s.par_free[i], 256);
        }
        bar_init(&s.q_full, 256);
        // [half of the rows][step of a tile's tokens]: each completes once a tile, so the
        // parity of the tile's number tells a completion from the one before
        for (int i = 0; i < 2; ++i) {
            bar_init(&s.s_full[i][0], 1);
            bar_init(&s.s_full[i][1], 1);
            for (int h = 0; h < kSteps; ++h) {
                bar_init(&s.p_full[i][h], 128);
                bar_init(&s.o_done[i][h], 1);
            }
        }
        bar_init(&s.done, 2);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        s.abort = 0;
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = s.tmem;
    volatile int *abort = &s.abort;
    auto wait = [&](uint64_t *b, uint32_t parity) { return bar_wait(b, parity, abort, a.status); };

    // Each split is taken in its own branch, so that the registers of either are known to
    // the compiler all the way through it.
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 13) {
        // ---------------- loader: lane i copies block i of a tile
        Turn raw;
        uint32_t issued = 0;
        bool ok = true;
        while (ok && run.pos < run.stop) {
            const Segment g = next_segment(a, kChunkRows, run);
            const int32_t *trow = a.table + (int64_t)run.b * a.ldt;
            run.pos += g.count;
            for (int tok = g.c0; tok < g.c1; tok += kTok) {
                const int blk = tok / 16 + lane;
                const bool in = lane < kTok / 16 && blk * 16 < g.end;
                int page = 0, at = 0;
                if (in) {
                    const int e = (int)fdiv(blk, a.by_page);
                    at = blk - e * a.blocks_per_page;
                    page = trow[e];
                    if (page < 0 || page >= a.pages) {
                        atomicOr(a.status, kStatusIndex);
                        page = 0;
                    }
                }
                const unsigned who = __ballot_sync(0xffffffffu, in);
                if (issued >= kRawStages && !wait(&s.raw_free[raw.stage], raw.phase ^ 1)) ok = false;
                ok = __all_sync(0xffffffffu, ok) && !*abort;
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const uint32_t bar = smem_u32(&s.raw_full[raw.stage]);
                if (lane == 0)
                    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar),
                                 "r"((uint32_t)__popc(who) * BB)
                                 : "memory");
                __syncwarp();
                if (in)
                    asm volatile(
                        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                            smem_u32(s.raw[raw.stage]) + lane * BB),
                        "l"(a.pool + page * a.page_bytes + ((int64_t)g.kvh * a.blocks_per_page + at) * BB), "r"(BB), "r"(bar)
                        : "memory");
                raw.next(kRawStages);
                ++issued;
            }
        }
        // nothing may still be landing when the block leaves
        const uint32_t first = issued > kRawStages ? issued - kRawStages : 0;
        for (uint32_t i = first; i < issued; ++i)
            mbar_wait_bounded(smem_u32(&s.raw_full[i % kRawStages]), (i / kRawStages) & 1);
    } else if (warp == 12 || warp == 14) {
        // ---------------- MMA issuers, one for each half of the rows: the warp together, one lane
        // of it issuing
        const int i = __shfl_sync(0xffffffffu, (warp - 12) / 2, 0);
        constexpr uint32_t id_s = idesc_f16(128, kTok / 2, false), id_o = idesc_f16(128, D, true);
        const uint32_t base = __shfl_sync(0xffffffffu, tmem, 0), acc_s = base + kS + 128 * i, acc_o = base + kO + 128 * i;
        const uint64_t q = desc_k(smem_u32(s.q[i][0]));
        const uint32_t ops = smem_u32(s.op[0]);
        constexpr uint32_t kOpBytes = sizeof(s.op[0]);
        auto wait = [&](uint64_t *b, uint32_t parity) { return __all_sync(0xffffffffu, bar_wait(b, parity, abort, a.status)) != 0; };
        Turn k;                        // the next K
        uint32_t segs = 0, count = 0;  // segments with tokens, tiles
        bool ok = true;
        // S for the first or second 64 tokens of the tile whose K is at `at`
        auto score = [&](int part, Turn at) {
            const uint64_t kd = desc_k(ops + at.stage * kOpBytes + part * (kTok / 2 * 128));
            if (elect()) {
#pragma unroll
                for (int x = 0; x < D / 16; ++x)
                    mma_ss(acc_s + 64 * part, q + (x / 4) * 1024 + (x % 4) * 2, kd + (x / 4) * 1024 + (x % 4) * 2, id_s, x > 0);
                commit(&s.s_full[i][part]);
                if (part == 1) commit(&s.op_free[at.stage]);
            }
        };
        while (__any_sync(0xffffffffu, ok && run.pos < run.stop)) {
            const Segment g = next_segment(a, kChunkRows, run);
            run.pos += g.count;
            const int tiles = __shfl_sync(0xffffffffu, (g.c1 - g.c0 + kTok - 1) / kTok, 0);
            if (tiles == 0) continue;
            ok = wait(&s.q_full, segs & 1) && wait(&s.op_full[k.stage], k.phase);
            if (!ok) break;
            ++segs;
            fence_after();
            score(0, k);
            for (int t = 0; t < tiles; ++t, ++count) {
                const Turn k0 = k;  // this tile's K
                Turn v = k;
                v.next(kOpStages);
                k = v;
                k.next(kOpStages);  // the next tile's
                const uint64_t vd = desc_mn(ops + v.stage * kOpBytes, 1024, PANELS * 1024);
#pragma unroll
                for (int h = 0; h < kSteps; ++h) {
                    // S is made half a tile ahead of the softmax, into the columns whose P is done
                    // with: the second half of this tile, while the softmax is at the first, then the
                    // first half of the next
                    if (h == 0) {
                        ok = t == 0 || wait(&s.o_done[i][kSteps - 1], (count - 1) & 1);
                        if (!ok) break;
                        fence_after();
                        score(1, k0);
                    } else if (h == 2 && t + 1 < tiles) {
                        ok = wait(&s.op_full[k.stage], k.phase) && wait(&s.o_done[i][1], count & 1);
                        if (!ok) break;
                        fence_after();
                        score(0, k);
                    }
                    if (h == 0) ok = ok && wait(&s.op_full[v.stage], v.phase);
                    ok = ok && wait(&s.p_full[i][h], count & 1);
                    if (!ok) break;
                    fence_after();
                    if (elect()) {
#pragma unroll
                        for (int x = 0; x < kStep / 16; ++x)
                            mma_ts(acc_o, acc_s + 64 * (h / 2) + kStep / 2 * (h % 2) + 8 * x, vd + (h * (kStep / 8) + 2 * x) * (PANELS * 64), id_o,
                                   h > 0 || x > 0 || t > 0);
                        commit(&s.o_done[i][h]);
                        if (h == kSteps - 1) commit(&s.op_free[v.stage]);
                    }
                }
                if (!ok) break;
            }
        }
        if (elect()) commit(&s.done);  // every product issued, also after an abort
        if (!mbar_wait_bounded(smem_u32(&s.done), 0)) {
            *abort = 1;
            atomicOr(a.status, kStatusTimeout);
        }
    } else if (warp < 12) {
        // ---------------- unpack
        const int t = threadIdx.x - 256, w = warp - 8;
        const uint32_t bias = a.bias;
        Turn raw, op, par;
        uint32_t ops = 0, pars = 0;
        bool ok = true;
        auto wait_all = [&](uint64_t *b, uint32_t parity) { return __all_sync(0xffffffffu, wait(b, parity)) != 0; };
        while (ok && run.pos < run.stop) {
            const Segment g = next_segment(a, kChunkRows, run);
            run.pos += g.count;
            if (g.c1 <= g.c0) continue;
            int vexp = 0;
            float vcap = 0.0f;
            for (int tok = g.c0; ok && tok < g.c1; tok += kTok) {
                ok = wait_all(&s.raw_full[raw.stage], raw.phase);
                if (!ok) break;
                const uint8_t *src = s.raw[raw.stage];
                // ---- scales: V's largest magnitude in the tile, by every warp for itself
                float vmax = 0.0f;
                unsigned nans[kTok / 32];
#pragma unroll
                for (int x = 0; x < kTok / 32; ++x) {
                    const int tt = x * 32 + lane;
                    const float2 vp = half2_at(src + (tt / 16) * BB + kv4_vs_off(D) + 4 * (tt % 16));
                    const bool in = tok + tt < g.end, bad = in && !(vp.x < INFINITY);
                    if (in && !bad) vmax = fmaxf(vmax, fmaxf(fabsf(vp.y), fabsf(fmaf(15.0f, vp.x, vp.y))));
                    nans[x] = __ballot_sync(0xffffffffu, bad);
                }
                vmax = lanes_max(vmax, 32);
                if (vmax >= vcap) {
                    vexp = vmax > 0.0f ? (int)(__float_as_uint(vmax) >> 23) - 127 : -24;  // 2^e <= vmax < 2^(e+1)
                    vcap = ldexpf(1.0f, vexp + 3);
                }
                const float vscale = ldexpf(1.0f, kValueBits - vexp);  // values below 2^(kValueBits + 3)
                if (pars >= kParStages) ok = wait_all(&s.par_free[par.stage], par.phase ^ 1);
                if (!ok) break;
                {
                    const uint8_t *blk = src + (t / 16) * BB;
                    // a token past the end has no scales (its bytes are whatever the ring held)
                    const float2 kp = tok + t < g.end ? half2_at(blk + kv4_ks_off(D) + 4 * (t % 16)) : make_float2(0.0f, 0.0f);
                    s.kpar[par.stage][t / 2][t % 2] = kp.x;
                    s.kpar[par.stage][t / 2][2 + t % 2] = kp.y;
                    if (t < kTok / 32) s.vnan[par.stage][t] = t == 0 ? nans[0] : t == 1 ? nans[1] : t == 2 ? nans[2] : nans[3];
                    if (t == 0) s.vexp[par.stage] = vexp;
                }
                bar_arrive(&s.par_full[par.stage]);
                par.next(kParStages);
                ++pars;
                // ---- K: a lane takes a quarter of a token's row (lanes of equal quarter together:
                // their stores then fall on different banks)
                if (ops >= kOpStages) ok = wait_all(&s.op_free[op.stage], op.phase ^ 1);
                if (!ok) break;
                uint32_t dst = smem_u32(s.op[op.stage]);
                {
                    const int j = lane >> 3, gr = lane & 7;
                    constexpr int LW = D / 32;  // words of a quarter row
                    // (rolled: the four roles' loops share the instruction caches)
#pragma unroll 1
                    for (int i = 0; i < kTok / 8 / kUnpackWarps; ++i) {
                        const int row = w * (kTok / kUnpackWarps) + i * 8 + gr;
                        const uint8_t *p = src + (row / 16) * BB + (row % 16) * (D / 2) + j * (D / 8);
                        uint32_t c[LW];
                        if constexpr (LW == 4)
                            *reinterpret_cast<uint4 *>(c) = *reinterpret_cast<const uint4 *>(p);
                        else
                            *reinterpret_cast<uint2 *>(c) = *reinterpret_cast<const uint2 *>(p);
#pragma unroll
                        for (int x = 0; x < LW; ++x) {
                            const int chunk = j * LW + x;  // of 8 dims
                            st_shared(dst + (chunk / 8) * 16384 + row * 128 + ((chunk % 8) ^ (row & 7)) * 16, unpack8(c[x], bias));
                        }
                    }
                }
                fence_async();
                bar_arrive(&s.op_full[op.stage]);
                op.next(kOpStages);
                ++ops;
                // ---- V: a lane takes a slice (D/8 dims) of a token pair
                if (ops >= kOpStages) ok = wait_all(&s.op_free[op.stage], op.phase ^ 1);
                if (!ok) break;
                dst = smem_u32(s.op[op.stage]);
                {
                    const int r = lane & 7, pr = lane >> 3;
                    constexpr int LW = D / 64;  // words a token has in a slice
#pragma unroll 1
                    for (int i = 0; i < kTok / 8 / kUnpackWarps; ++i) {
                        const int pair = w * (kTok / 2 / kUnpackWarps) + i * 4 + pr;  // of 64
                        const uint8_t *p = src + (pair / 8) * BB + kv4_v_off(D) + (pair % 8) * D + r * (D / 8);
                        uint32_t c[2 * LW];
                        if constexpr (LW == 2)
                            *reinterpret_cast<uint4 *>(c) = *reinterpret_cast<const uint4 *>(p);
                        else
                            *reinterpret_cast<uint2 *>(c) = *reinterpret_cast<const uint2 *>(p);
#pragma unroll
                        for (int o = 0; o < 2; ++o) {
                            const int token = 2 * pair + o;
                            float2 vp = half2_at(src + (token / 16) * BB + kv4_vs_off(D) + 4 * (token % 16));
                            if (tok + token >= g.end || !(vp.x < INFINITY)) vp = make_float2(0.0f, 0.0f);
                            const __half2 step = __float2half2_rn(vp.x * vscale), low = __float2half2_rn(vp.y * vscale);
#pragma unroll
                            for (int x = 0; x < LW; ++x) {
                                const int chunk = r * LW + x;
                                st_shared(dst + (token / 8) * (PANELS * 1024) + (chunk / 8) * 1024 + (token % 8) * 128 +
                                              ((chunk % 8) ^ (token % 8)) * 16,
                                          scaled8(unpack8(c[o * LW + x], bias), step, low));
                            }
                        }
                    }
                }
                bar_arrive(&s.raw_free[raw.stage]);
                raw.next(kRawStages);
                fence_async();
                bar_arrive(&s.op_full[op.stage]);
                op.next(kOpStages);
                ++ops;
            }
        }
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        // ---------------- softmax: half i, thread r of it has row 128 i + r of the tile
        const int i = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + kS + 128 * i, to = tmem + lanes + kO + 128 * i;
        Turn par;
        uint32_t count = 0;  // tiles
        bool ok = true;
        while (ok && run.pos < run.stop) {
            const Segment g = next_segment(a, kChunkRows, run);
            const Seq seq = run.seq;
            if (a.job && g.last && threadIdx.x == 0) {
                pdl_wait();
                note_job(a, run, g);
            }
            run.pos += g.count;
            const int row = 128 * i + r, full_row = g.tile * kChunkRows + row;
            const bool live = row < g.rows;
            const int t = live ? (int)fdiv(full_row, a.by_group) : 0, hq = g.kvh * a.G + full_row - t * a.G;
            // ---- Q into shared memory, a warp its own 32 rows; then a thread its row: scaled in
            // place by a power of two of its own (one row's infinity leaves the others as they are)
            const bool any = g.c1 > g.c0;
            float qsum = 0.0f, unit = 1.0f;  // logits in base 2 are z unit
            const uint32_t rows_at = smem_u32(s.q[i][0]) + (warp & 3) * (32 * 128);
            // the 16 bytes x of row rl of this warp's
            auto piece = [&](int rl, int x) { return rows_at + rl * 128 + (x / 8) * 16384 + ((x % 8) ^ (rl & 7)) * 16; };
            auto lds = [](uint32_t at, uint32_t *w) {
                asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                             : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                             : "r"(at)
                             : "memory");
            };
            if (any) {
                if (a.vec) {
                    constexpr int kLanes = D / 8;
                    const int x = lane % kLanes;
#pragma unroll
                    for (int r0 = 0; r0 < 32; r0 += 32 / kLanes) {
                        const int rl = r0 + lane / kLanes, rw = 128 * i + (warp & 3) * 32 + rl;
                        const int fr = g.tile * kChunkRows + min(rw, g.rows - 1);
                        const int tq = (int)fdiv(fr, a.by_group), hh = g.kvh * a.G + fr - tq * a.G;
                        const T *p = reinterpret_cast<const T *>(a.Q) + (int64_t)(seq.q0 + tq) * a.qs_tok + (int64_t)hh * a.qs_head + 8 * x;
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(piece(rl, x)), "l"(p), "r"(rw < g.rows ? 16 : 0)
                                     : "memory");
                    }
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    __syncwarp();
                } else {
                    const T *p = reinterpret_cast<const T *>(a.Q) + (int64_t)(seq.q0 + t) * a.qs_tok + (int64_t)hq * a.qs_head;
#pragma unroll 1
                    for (int x = 0; x < D / 8; ++x) {
                        Vec<T, 8> v;
#pragma unroll
                        for (int e = 0; e < 8; ++e) v.v[e] = live ? p[8 * x + e] : from_f<T>(0.0f);
                        const uint32_t *w = reinterpret_cast<const uint32_t *>(&v);
                        st_shared(piece(lane, x), make_uint4(w[0], w[1], w[2], w[3]));
                    }
                }
                float top = 0.0f;
#pragma unroll 4
                for (int x = 0; x < D / 8; ++x) {
                    Vec<T, 8> v;
                    lds(piece(lane, x), reinterpret_cast<uint32_t *>(&v));
#pragma unroll
                    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(to_f(v.v[e])));
                }
                const int qe = max(-100, min((int)(__float_as_uint(top) >> 23) - 127, 127));
                // (a negative scale turns q's sign: z below then grows with the logit)
                const float up = copysignf(ldexpf(1.0f, 14 - qe), a.scale);
                unit = fmaxf(fabsf(a.scale) * kLog2eF * ldexpf(1.0f, qe - 14), 1e-37f);
#pragma unroll 4
                for (int x = 0; x < D / 8; ++x) {
                    Vec<T, 8> v;
                    float f[8];
                    lds(piece(lane, x), reinterpret_cast<uint32_t *>(&v));
                    widen(v, f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        f[e] *= up;
                        qsum += f[e];
                    }
                    st_shared(piece(lane, x), make_uint4(pack_half2(f[0], f[4]), pack_half2(f[1], f[5]), pack_half2(f[2], f[6]),
                                                         pack_half2(f[3], f[7])));
                }
                fence_async();
                bar_arrive(&s.q_full);
            }

            // ---- this row's keys [lo, hi), and where all of this warp's rows see all
            const int lo = live ? lower(a, seq, t) : 0, hi = live ? upper(a, seq, t) : g.c1;
            const int safe0 = __reduce_max_sync(0xffffffffu, lo), safe1 = __reduce_min_sync(0xffffffffu, hi);
            float m = -INFINITY, l = 0.0f, poison = 0.0f;  // reference, sum, what joins the outputs: 0 or NaN
            int vexp = 0;
            bool first = true;
            for (int tok = g.c0; ok && tok < g.c1; tok += kTok) {
                ok = wait(&s.par_full[par.stage], par.phase);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const float4 *kpar = reinterpret_cast<const float4 *>(s.kpar[par.stage]);
                const int e_new = s.vexp[par.stage];
                const uint32_t nan0 = s.vnan[par.stage][0] | s.vnan[par.stage][1] | s.vnan[par.stage][2] | s.vnan[par.stage][3];
                // One step: logits, the reference, probabilities back to tensor memory.  `acc`
                // holds its columns of S.
                auto step = [&](int h, uint32_t (&acc)[kStep]) {
                    float z[kStep], top = -INFINITY;
#pragma unroll
                    for (int c = 0; c < kStep; c += 2) {
                        const float4 kp = kpar[(kStep * h + c) / 2];
                        const float2 zz = both(fma2(pair2(__uint_as_float(acc[c]), __uint_as_float(acc[c + 1])), pair2(kp.x, kp.y),
                                                    mul2(pair2(kp.z, kp.w), pair2(qsum, qsum))));
                        z[c] = zz.x;
                        z[c + 1] = zz.y;
                    }
                    const int t0 = tok + kStep * h;
                    if (t0 < safe0 || t0 + kStep > safe1) {
#pragma unroll
                        for (int c = 0; c < kStep; ++c)
                            if (t0 + c < lo || t0 + c >= hi) z[c] = -INFINITY;
                    }
#pragma unroll
                    for (int c = 0; c < kStep; c += 2) top = fmaxf(top, fmaxf(z[c], z[c + 1]));
                    top *= unit;
                    if (__any_sync(0xffffffffu, top > m + (kHead + kSlack)) || e_new != vexp) {
                        const float mn = fmaxf(m, top - kHead);
                        const float f = m == -INFINITY ? 0.0f : ex2(m - mn);
                        m = mn;
                        l *= f;
                        if (!first) {
                            // O is this warp's once the last step handed over is done
                            ok = h ? wait(&s.o_done[i][h - 1], count & 1) : wait(&s.o_done[i][kSteps - 1], (count - 1) & 1);
                            ok = __all_sync(0xffffffffu, ok);
                            if (!ok) return;
                            fence_after();
                            const float move = f * ldexpf(1.0f, vexp - e_new);
#pragma unroll 1
                            for (int c = 0; c < D; c += 16) {
                                uint32_t o[16];
                                tmem_load16(to + c, o);
                                tmem_load_wait();
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * move);
                                tmem_store16(to + c, o);
                            }
                            tmem_store_wait();
                        }
                        vexp = e_new;
                    }
                    first = false;
                    // a token held as NaN makes the rows that see it NaN, and no others
                    if (nan0 != 0) {
#pragma unroll
                        for (int c = 0; c < kStep; ++c)
                            if ((s.vnan[par.stage][h] >> c & 1) && z[c] != -INFINITY) poison = NAN;
                    }
                    const float ref = m == -INFINITY ? 0.0f : m;
                    uint32_t p[kStep / 2];
                    uint64_t sum = 0;
#pragma unroll
                    for (int c = 0; c < kStep; c += 2) {
                        const float2 x = both(fma2(pair2(z[c], z[c + 1]), pair2(unit, unit), pair2(-ref, -ref)));
                        const float p0 = ex2(x.x), p1 = ex2(x.y);
                        sum = add2(sum, pair2(p0, p1));
                        p[c / 2] = pack_half2(p0, p1);
                    }
                    const float2 sums = both(sum);
                    l += sums.x + sums.y;
                    tmem_store16(ts + 64 * (h / 2) + kStep / 2 * (h % 2), p);
                    tmem_store_wait();
                    fence_before();
                    bar_arrive(&s.p_full[i][h]);
                };
#pragma unroll 1
                for (int h = 0; ok && h < kSteps; ++h) {
                    if (h % 2 == 0) {
                        ok = __all_sync(0xffffffffu, wait(&s.s_full[i][h / 2], count & 1));
                        if (!ok) break;
                        fence_after();
                    }
                    uint32_t acc[kStep];
                    tmem_load(ts + kStep * h, acc);
                    tmem_load_wait();
                    step(h, acc);
                }
                if (!ok) break;
                bar_arrive(&s.par_free[par.stage]);
                par.next(kParStages);
                ++count;
            }
            // ---- the segment's end
            pdl_wait();
            if (ok && any) {
                ok = wait(&s.o_done[i][kSteps - 1], (count - 1) & 1);
                ok = __all_sync(0xffffffffu, ok);
                fence_after();
            }
            if (!ok) break;
            const float back = ldexpf(1.0f, vexp - kValueBits), inv = l == 0.0f ? 0.0f : 1.0f / l;
            float *slot = a.part + (2 * (int64_t)blockIdx.x + (g.unit0 == 0 ? 1 : 0)) * (kChunkRows * (D + 2));
            // O goes out through this warp's rows of Q's shared memory (which the products are done
            // with), D/2 columns at a time, so that a warp writes whole rows
            const float scale = g.whole ? back * inv : back, join = g.whole ? poison * inv : poison;
#pragma unroll 1
            for (int c = 0; c < D; c += D / 2) {
#pragma unroll 1
                for (int cc = 0; cc < D / 2; cc += 32) {
                    uint32_t o[32];
                    if (any) {
                        tmem_load(to + c + cc, o);
                        tmem_load_wait();
                    }
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        float f[8];  // columns come in the order 0 4 1 5 2 6 3 7 of a word's dims
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            f[(e & 1) * 4 + (e >> 1)] = any ? fmaf(__uint_as_float(o[8 * x + e]), scale, join) : 0.0f;
                        const int pc = cc / 4 + 2 * x;
                        st_shared(piece(lane, pc), make_uint4(as_u(f[0]), as_u(f[1]), as_u(f[2]), as_u(f[3])));
                        st_shared(piece(lane, pc + 1), make_uint4(as_u(f[4]), as_u(f[5]), as_u(f[6]), as_u(f[7])));
                    }
                }
                __syncwarp();
                constexpr int kLanes = D / 2 / 8, kRowsIt = 32 / kLanes;  // 8 columns a lane
                const int part = lane % kLanes;
#pragma unroll 2
                for (int x = 0; x < 32; x += kRowsIt) {
                    const int rl = x + lane / kLanes, rw = 128 * i + (warp & 3) * 32 + rl;
                    float f[8];
                    lds(piece(rl, 2 * part), reinterpret_cast<uint32_t *>(f));
                    lds(piece(rl, 2 * part + 1), reinterpret_cast<uint32_t *>(f + 4));
                    if (rw >= g.rows) continue;
                    if (!g.whole) {
                        float4 *q = reinterpret_cast<float4 *>(slot + rw * D + c + 8 * part);
                        q[0] = make_float4(f[0], f[1], f[2], f[3]);
                        q[1] = make_float4(f[4], f[5], f[6], f[7]);
                    } else {
                        const int fr = g.tile * kChunkRows + rw, tq = (int)fdiv(fr, a.by_group), hh = g.kvh * a.G + fr - tq * a.G;
                        T *out = reinterpret_cast<T *>(a.O) + (int64_t)(seq.q0 + tq) * a.os_tok + (int64_t)hh * a.os_head + c + 8 * part;
                        Vec<T, 8> vo;
                        narrow(f, vo);
                        if (a.vec) {
                            store_vec(out, vo);
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e) out[e] = vo.v[e];
                        }
                    }
                }
                __syncwarp();
            }
            if (live && !g.whole) *reinterpret_cast<float2 *>(slot + kChunkRows * D + row * 2) = make_float2(m, l);
            if (live && g.whole && a.lse)
                a.lse[(int64_t)(seq.q0 + t) * a.Hq + hq] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
            fence_before();  // the reads of O, before the next segment's P lets products write it
        }
    }
    pdl_wait();
    fence_before();
    __syncthreads();
    if (warp == 12) {
        __syncwarp();
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

template <typename T, int D>
tm_status launch_chunk(AttnArgs &a, int device, int sms, cudaStream_t s, bool pdl)
{
    const void *k = (const void *)kv4_chunk_kernel<T, D>;
    constexpr size_t smem = sizeof(ChunkSmem<D>) + 1024;
    static_assert(smem <= 227 * 1024, "shared memory");
    static std::atomic<bool> ready[kMaxDevices];
    if (!ready[device].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) {
            cudaGetLastError();
            return TM_ERR_CUDA;
        }
        ready[device].store(true, std::memory_order_release);
    }
    const unsigned blocks = (unsigned)(sms < kMostBlocks / 4 ? sms : kMostBlocks / 4);
    a.grid = (int)blocks;
    void *args[] = {(void *)&a};
    return launch_kernel(k, dim3(blocks), dim3(kThreads2), args, smem, s, pdl);
}

}  // namespace

bool chunk_attn_fits(int32_t xtype, int64_t rows, int D)
{
    // Whole calls, mma.sync kernel against this one, heads 4 to a KV head.  D 128, 64 rows:
    // 2 sequences of 8192 tokens 35 / 39 us, 32 of 4096 148 / 195, one of 65536 88 / 105;
    // 96 rows: 46 / 39, 213 / 196, 122 / 105.  D 64, 2 of 8192: 64 rows 27 / 37 us,
    // 128 rows 37 / 35.
    return xtype != TM_F32 && ((D == 128 && rows >= 96) || (D == 64 && rows >= 128));
}

size_t chunk_attn_slots_bytes(int D) { return 2 * (size_t)(kMostBlocks / 4) * kChunkRows * (D + 2) * sizeof(float); }

tm_status launch_chunk_attn(int D, int32_t xtype, AttnArgs &a, int device, int sms, bool join, cudaStream_t s, bool pdl)
{
    const tm_status st = xtype == TM_F16 ? (D == 64 ? launch_chunk<__half, 64>(a, device, sms, s, pdl)
                                                    : launch_chunk<__half, 128>(a, device, sms, s, pdl))
                                         : (D == 64 ? launch_chunk<__nv_bfloat16, 64>(a, device, sms, s, pdl)
                                                    : launch_chunk<__nv_bfloat16, 128>(a, device, sms, s, pdl));
    if (st != TM_OK || !join) return st;
    return launch_chunk_join(D, xtype, a, sms, s);
}

}  // namespace libtm
