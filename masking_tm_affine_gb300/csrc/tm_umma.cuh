// tm_umma.cuh -- what the products on operands of 16 and 8 bits share: barriers with
// bounded waits, TMA loads, tcgen05 allocation, products, commits and reads, for one
// CTA or a CTA pair; and the rows of each expert.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "tm_device.cuh"

namespace libtm {

// ---------------------------------------------------------------- barriers
__device__ __forceinline__ void mbar_init(uint64_t *b, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t *b)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(b)) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint64_t *b, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(b)), "r"(bytes) : "memory");
}
// The same on a barrier of any CTA of the cluster, by its cluster address.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The same where only the order of this thread's tensor memory reads matters, which are
// over when it is issued: no fence at cluster scope.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Relaxed: it publishes nothing but the count (a release at cluster scope a stage costs a
// fence each: 412 us for the 8192 x 4096 x 4096 product in 16 bits).
__device__ __forceinline__ void mbar_expect_cluster(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// A wait on a phase that other CTAs of the cluster complete.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Wait for a phase of `b`.  False after the limit, or once any role of this CTA has
// given up; the first to give up records it.
template <bool CLUSTER = false>
__device__ __forceinline__ bool role_wait(uint64_t *b, uint32_t parity, int *abort_flag, unsigned *status)
{
    const uint32_t bar = smem_u32(b);
    auto look = [&] { return CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity); };
    if (look()) return true;
    const long long t0 = clock64();
    while (!look()) {
        if (*(volatile const int *)abort_flag != 0) return false;
        if (clock64() - t0 > kWaitCycles) {
            atomicOr(status, kStatusTimeout);
            *(volatile int *)abort_flag = 1;
            return false;
        }
    }
    return true;
}

// The same by a whole warp, which goes on or gives up together.
template <bool CLUSTER = false>
__device__ __forceinline__ bool warp_wait(uint64_t *b, uint32_t parity, int *abort_flag, unsigned *status)
{
    return __all_sync(0xffffffffu, role_wait<CLUSTER>(b, parity, abort_flag, status)) != 0;
}

// One lane of a converged warp, the same every time.  Warps that copy or multiply stay together and elect:
// the instructions' operands then live in uniform registers (by a lane in a branch of its own each
// stage cost the 16-bit products a tenth of their time).
__device__ __forceinline__ bool elect()
{
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e)::"memory");
    return e != 0;
}

// Place in a ring of barriers: the slot, and the parity of the phase to wait for.
struct Turn {
    uint32_t slot = 0, phase = 0;
    __device__ __forceinline__ void next(uint32_t slots)
    {
        if (++slot == slots) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

// ---------------------------------------------------------------- copies
__device__ __forceinline__ void tensormap_prefetch(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d_hint(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar,
                                                 uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4}],"
        " [%5], %6;" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy)
        : "memory");
}
// Into this CTA's memory, counted on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
            dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_4d_pair(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

// ---------------------------------------------------------------- tensor cores
// Shared-memory operands in rows of 128 bytes, 128-byte swizzle (layout 2), version 1.
// K-major: groups of 8 rows 1024 bytes apart.  MN-major: panels of 64 elements of the
// outer extent `panel` bytes apart, groups of 8 of the summed extent 1024 bytes apart.
__device__ __forceinline__ uint64_t operand_k(uint32_t at)
{
    return (uint64_t)((at >> 4) & 0x3FFF) | (1ull << 16) | ((1024ull >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t operand_mn(uint32_t at, uint32_t panel)
{
    return (uint64_t)((at >> 4) & 0x3FFF) | ((uint64_t)(panel >> 4) << 16) | ((1024ull >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// Instruction descriptor: D fp32 (bits 4-5 = 1), the types of A and B (bits 7-9 and
// 10-12; kind::f16: 0 fp16, 1 bf16; kind::f8f6f4: 0 e4m3), MN-major A (15) and B (16),
// N >> 3 at bit 17, M >> 4 at bit 24.
__host__ __device__ constexpr uint32_t instruction(uint32_t type, bool a_mn, bool b_mn, uint32_t M, uint32_t N)
{
    return (1u << 4) | (type << 7) | (type << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((N >> 3) << 17) |
           ((M >> 4) << 24);
}

template <bool F8, bool PAIR>
__device__ __forceinline__ void umma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool acc)
{
#define TM_UMMA(GROUP, KIND)                                                                                        \
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"                                                   \
                 "tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), \
                 "r"(id), "r"((uint32_t)acc)                                                                         \
                 : "memory")
    if constexpr (F8 && PAIR)
        TM_UMMA("2", "f8f6f4");
    else if constexpr (F8)
        TM_UMMA("1", "f8f6f4");
    else if constexpr (PAIR)
        TM_UMMA("2", "f16");
    else
        TM_UMMA("1", "f16");
#undef TM_UMMA
}

// Arrive on `b` (in both CTAs of a pair, whose ranks are the bits of `ranks`) once every
// product issued so far by this thread has completed.
template <bool PAIR>
__device__ __forceinline__ void umma_done(uint64_t *b, uint32_t ranks = 3)
{
    if constexpr (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_u32(b)),
            "h"((uint16_t)ranks)
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(b))
                     : "memory");
}

// Tensor memory, taken and given back by one whole warp (in each CTA of a pair).
template <bool PAIR>
__device__ __forceinline__ void acc_alloc(uint32_t *dst, uint32_t cols)
{
    if constexpr (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
}
template <bool PAIR>
__device__ __forceinline__ void acc_free(uint32_t at, uint32_t cols)
{
    if constexpr (PAIR)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols) : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols) : "memory");
}

__device__ __forceinline__ void acc_load32(uint32_t at, float (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
          "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
          "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(at));
}
// All reads of this warp have arrived; the registers are named so that no use moves ahead.
__device__ __forceinline__ void acc_load_wait(float (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]),
                   "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]),
                   "+f"(r[16]), "+f"(r[17]), "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]), "+f"(r[23]),
                   "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]), "+f"(r[28]), "+f"(r[29]), "+f"(r[30]), "+f"(r[31])::
                     "memory");
}
__device__ __forceinline__ void acc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void acc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// sum += m * 32 columns of the accumulator, two columns an operation.  One statement: the
// values pass from the read to the additions in registers that nothing else names, which
// saves the moves that separate statements took (8192 x 8192 x 4096: 255 us, so 234).
__device__ __forceinline__ void add_columns(uint32_t at, uint64_t *s, uint64_t m)
{
#define TM_ADD(I, A, B) "mov.b64 p, {t" #A ", t" #B "};\n\tfma.rn.f32x2 %" #I ", p, %17, %" #I ";\n\t"
    asm volatile(
        "{\n\t.reg .b32 t<32>;\n\t.reg .b64 p;\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {t0, t1, t2, t3, t4, t5, t6, t7, t8, t9, t10, t11, t12, t13, t14, t15, t16, "
        "t17, t18, t19, t20, t21, t22, t23, t24, t25, t26, t27, t28, t29, t30, t31}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;\n\t" TM_ADD(0, 0, 1) TM_ADD(1, 2, 3) TM_ADD(2, 4, 5) TM_ADD(3, 6, 7) TM_ADD(4, 8, 9)
            TM_ADD(5, 10, 11) TM_ADD(6, 12, 13) TM_ADD(7, 14, 15) TM_ADD(8, 16, 17) TM_ADD(9, 18, 19) TM_ADD(10, 20, 21)
                TM_ADD(11, 22, 23) TM_ADD(12, 24, 25) TM_ADD(13, 26, 27) TM_ADD(14, 28, 29) TM_ADD(15, 30, 31) "}"
        : "+l"(s[0]), "+l"(s[1]), "+l"(s[2]), "+l"(s[3]), "+l"(s[4]), "+l"(s[5]), "+l"(s[6]), "+l"(s[7]), "+l"(s[8]),
          "+l"(s[9]), "+l"(s[10]), "+l"(s[11]), "+l"(s[12]), "+l"(s[13]), "+l"(s[14]), "+l"(s[15])
        : "r"(at), "l"(m)
        : "memory");
#undef TM_ADD
}

// 16-bit operands: how much of a sum the tensor cores add before it leaves them.
constexpr int kRunSums = 512;

// ---------------------------------------------------------------- joins
// A tile's sum cut over the pairs of a cluster: each output warp pushes its runs of 32 columns to
// the CTA (of its own rank in the pair) whose pair owns them, into [pair][8 warps][4 / S runs][8][32 lanes] x
// 16 bytes, 128 KB in the rings' place.  The owner adds them in the order of the pairs.
__device__ __forceinline__ uint32_t join_slot(int pair, int warp, int run, int S, int lane)
{
    return (uint32_t)(((pair * 8 + warp) * (4 / S) + run % (4 / S)) * 8 * 32 + lane) * 16u;
}
__device__ __forceinline__ void join_push(const float (&v)[32], uint32_t inbox, uint64_t *bar, int pair, int warp, int run, int S,
                                          uint32_t rank)
{
    const uint32_t to = (uint32_t)(run / (4 / S)) * 2u + rank, lane = threadIdx.x & 31u;
    const uint32_t dst = cluster_addr(inbox + join_slot(pair, warp, run, S, (int)lane), to), b = cluster_addr(smem_u32(bar), to);
#pragma unroll
    for (int c = 0; c < 32; c += 4)
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                         dst + (uint32_t)c * 128u),
                     "r"(as_u(v[c])), "r"(as_u(v[c + 1])), "r"(as_u(v[c + 2])), "r"(as_u(v[c + 3])), "r"(b)
                     : "memory");
}
__device__ __forceinline__ void join_sum(float (&v)[32], const unsigned char *inbox, int warp, int run, int S)
{
#pragma unroll
    for (int c = 0; c < 32; ++c) v[c] = 0.0f;
    for (int pair = 0; pair < S; ++pair) {
        const unsigned char *from = inbox + join_slot(pair, warp, run, S, (int)(threadIdx.x & 31u));
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
            const float4 u = *reinterpret_cast<const float4 *>(from + c * 128);
            v[c] += u.x, v[c + 1] += u.y, v[c + 2] += u.z, v[c + 3] += u.w;
        }
    }
}

// ---------------------------------------------------------------- rows of the experts
constexpr int kMaxExperts = 1024;

// The rows of each expert in shared memory, and how many tiles of `tile` rows come before
// it.  Borders that leave [0, T], fall, or lie before an earlier one give an expert no
// rows and set the status word: no row has two experts, whatever the borders are.
struct Experts {
    int first[kMaxExperts], count[kMaxExperts], before[kMaxExperts + 1];
};

// All threads of the block; ends with a __syncthreads.
__device__ __forceinline__ void experts_read(Experts &x, const int32_t *starts, int E, int T, int tile, unsigned *status)
{
    if (starts == nullptr) {  // one expert
        if (threadIdx.x == 0) {
            x.first[0] = x.before[0] = 0;
            x.count[0] = T;
            x.before[1] = T / tile + (T % tile != 0);
        }
        __syncthreads();
        return;
    }
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        x.first[e] = starts[e];
        x.count[e] = starts[e + 1];  // the upper border, until the scan below
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = (int)threadIdx.x;
        int sum = 0, past = 0;  // tiles, and the highest border, before these 32
        bool all = true;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            const int lo = e < E ? x.first[e] : 0, hi = e < E ? x.count[e] : 0;
            int m = lo;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, m, o);
                if (lane >= o && u > m) m = u;
            }
            if (past > m) m = past;
            const bool ok = m <= lo && lo <= hi && hi <= T;  // m <= lo: nothing earlier lies above, nor zero
            int v = ok && e < E ? (hi - lo) / tile + ((hi - lo) % tile != 0) : 0;
            if (e < E) {
                x.first[e] = ok ? lo : 0;
                x.count[e] = ok ? hi - lo : 0;
                all = all && ok;
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += u;
            }
            if (e < E) x.before[e + 1] = sum + v;
            sum += __shfl_sync(0xffffffffu, v, 31);
            past = __shfl_sync(0xffffffffu, m, 31);
        }
        if (lane == 0) x.before[0] = 0;
        if (!all && blockIdx.x == 0) atomicOr(status, kStatusIndex);
    }
    __syncthreads();
}

}  // namespace libtm
