// tm_wide.cu -- 16-bit products grouped by expert, for experts with many rows: the output,
// the gradient of the rows and the gradient of the weights.
//
//   forward           y[t, n]    = sum_k x[t, k]  w_e[n, k]
//   rows' gradient    dx[t, k]   = sum_n dy[t, n] w_e[n, k]
//   weights' gradient dw_e[n, k] = sum_t dy[t, n] x[t, k]     over the rows t of expert e
//
// One kernel: out[c, r] = sum_s wide[c, s] tall[r, s], a tile 256 of r by up to 256 of c,
// shared by a CTA pair (tcgen05 cta_group::2: each CTA stages its 128 of the tall operand
// and half of the wide one, 32 KB a stage of 64 of the sum, six stages; two
// accumulators of 256 columns, so that one run's addition and one tile's output overlap the next one's products).
// The tall operand (r) runs along the tensor memory's lanes and c along its columns, so
// that a warp's 32 lanes hold 32 neighbours of an output row: outputs leave as coalesced
// stores of 64 or 128 bytes with no way through shared memory, whatever their
// alignment, and a row past an expert's end is one that is not stored.  Nothing is
// transposed first: an operand whose summed extent is the outer one is read MN-major.  A stage
// comes in as few copies as there can be, one of 16 KB an operand where the extents allow it:
// with four of 4 KB the copies bound the kernel (8192 x 4096 x 4096: 182 us, with one 156; now 146, at 93 % of the
// tensor pipe, and the weights' gradient 167).
//
// The rows of an expert end anywhere.  Along c that costs nothing (the product's extent is
// a multiple of 64 of rows, the others are not stored).  Where rows are summed (the
// weights' gradient) a last stage of r < 64 rows runs ceil(r / 16) products, and a warp
// clears the rows between r and the next 16 in both operands first: they are
// the next expert's, or whatever lies there.
#include <mutex>

#include "tm_products.h"
#include "tm_umma.cuh"

namespace libtm {
namespace {

// Warp 0 copies, 1 multiplies, 2 clears rows, 4 to 11 make outputs.  Sums leave the tensor
// cores every kRunSums and are added in registers (tm_thin.cu says why), 128 a thread of the output warps,
// which so are whole warpgroups and take registers from the others: 4 warps of 96 and 8 of 200 are
// 63488, of the 64512 that 384 threads of 168 start with.  To 16 bits, cold, against sums that stay in the
// tensor cores: 8192 x 4096 x 4096 146 us either way, its gradients 146 and 164 (146 and 163); weights' gradient of
// 64 experts of 2048 x 2048, 128 rows each, 110 (107), 32 rows each 105 (101).
constexpr int kWideThreads = 384, kClear = 2, kOut = 4;
constexpr int kFewRegs = 96, kManyRegs = 200;
constexpr int kRun = kRunSums / 64;  // stages
constexpr int kStages = 6;
constexpr uint32_t kHalf = 128 * 128;       // bytes of one operand a stage and CTA: 128 of its outer extent by 64 of the sum
constexpr uint32_t kPanel = 64 * 128;       // MN-major: 64 of the outer extent by 64 of the sum
constexpr uint32_t kStageBytes = 2 * kHalf;
constexpr int kGroup = 8;                   // c tiles that run at the same time, for the sake of L2

enum Mode { kForward = 0, kRows = 1, kWeights = 2 };

struct WideArgs {
    void *out;
    int64_t ldo;
    const int32_t *starts;
    unsigned *status;
    int otype, E, T;
    int R, C;    // extents of r, and of c where c is not an expert's rows
    int rtiles, ctiles;  // of 256 of r, of `width` of c (ctiles: weights' gradient)
    int width;           // of a tile along c: 256, 128 or 64
    FastDiv by_block, by_expert;  // kGroup * rtiles; rtiles * ctiles
    int steps;   // stages a tile (not of the weights' gradient)
    int tall_panels, wide_panels;  // MN-major operands whose two panels come in one copy
    uint32_t id;
};

struct WideSmem {
    alignas(8) uint64_t full[kStages], empty[kStages], tail[kStages], acc_full[2], acc_empty[2], done, inbox;
    uint32_t tmem;
    int abort;
    Experts x;
};

// A tile: expert, first of r and c, how many of c, the rows summed (weights' gradient).
struct Tile {
    int e, r0, c0, n, s0, steps, last;  // last: rows of the last stage, 64 if it is whole
    int kb, ke;                         // this pair's stages
};

template <int MODE>
struct Walk {
    const WideArgs &a;
    const Experts &x;
    const int pair, S;  // of the S pairs that share a tile's sum
    int e = 0;
    __device__ Walk(const WideArgs &args, const Experts &experts, int p, int pairs) : a(args), x(experts), pair(p), S(pairs) {}
    __device__ Tile at(int item)
    {
        Tile t;
        int cts, local;
        if constexpr (MODE == kWeights) {
            const int per = a.rtiles * a.ctiles;
            e = (int)fdiv((uint32_t)item, a.by_expert);
            local = item - e * per;
            cts = a.ctiles;
        } else {
            while ((int64_t)x.before[e + 1] * a.rtiles <= item) ++e;
            cts = x.before[e + 1] - x.before[e];
            local = item - x.before[e] * a.rtiles;
        }
        // blocks of kGroup tiles of c; within one, c is the faster
        const int block = (int)fdiv((uint32_t)local, a.by_block), in = local - block * kGroup * a.rtiles;
        const int wide = cts - block * kGroup < kGroup ? cts - block * kGroup : kGroup;
        const int rt = wide == kGroup ? in / kGroup : in / wide, ct = block * kGroup + in - rt * wide;
        t.e = e;
        t.r0 = rt * 256;
        if constexpr (MODE == kWeights) {
            t.c0 = ct * a.width;
            t.n = a.C - t.c0 < a.width ? a.C - t.c0 : a.width;
            t.s0 = x.first[e];
            t.steps = (x.count[e] + 63) / 64;
            t.last = x.count[e] - (t.steps - 1) * 64;
        } else {
            const int left = x.count[e] - ct * a.width;
            t.c0 = x.first[e] + ct * a.width;
            t.n = left < a.width ? left : a.width;
            t.s0 = 0;
            t.steps = a.steps;
            t.last = 64;
        }
        t.kb = S == 1 ? 0 : t.steps * pair / S;
        t.ke = S == 1 ? t.steps : t.steps * (pair + 1) / S;
        return t;
    }
};

// SPLIT (weights' gradient): a cluster of S pairs (2 or 4) has one tile, each pair its part of the sum.
template <int MODE, typename O, bool SPLIT>
__global__ void __launch_bounds__(kWideThreads, 1)
    wide_kernel(const __grid_constant__ CUtensorMap mtall, const __grid_constant__ CUtensorMap mwide,
                const __grid_constant__ CUtensorMap mwide_all, const WideArgs a, const int pairs)
{
    constexpr bool A_MN = MODE != kForward, B_MN = MODE == kWeights;
    extern __shared__ __align__(1024) unsigned char raw[];
    unsigned char *ring = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    __shared__ WideSmem s;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = SPLIT ? pairs : 1;
    const uint32_t rank = cluster_rank() & 1u, even = SPLIT ? cluster_rank() & ~1u : 0u;  // in the pair; its even CTA
    const int pair = (int)even / 2, unit = (int)blockIdx.x / (2 * S), units = (int)gridDim.x / (2 * S);

    if (warp == 1) acc_alloc<true>(&s.tmem, 512);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&s.full[i], 2);  // each CTA says what it copies, or that its last rows are cleared
            mbar_init(&s.empty[i], 1);
            mbar_init(&s.tail[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.acc_full[i], 1);
            mbar_init(&s.acc_empty[i], 16);
        }
        mbar_init(&s.done, 1);
        mbar_init(&s.inbox, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        s.abort = 0;
    }
    experts_read(s.x, a.starts, a.E, a.T, a.width, a.status);
    acc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist
    acc_fence_after();
    pdl_trigger();  // only now: a dependent's CTA could take the tensor memory that this one waits for
    const uint32_t tmem = s.tmem;
    const int items = MODE == kWeights ? a.E * a.rtiles * a.ctiles : s.x.before[a.E] * a.rtiles;
    Walk<MODE> walk(a, s.x, pair, S);

    // in the branches themselves: behind one of its own the compiler counts on the smaller share everywhere
    auto fewer_registers = [] { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs)); };
    if (warp == 0) {
        fewer_registers();
        {
            Turn t;
            uint32_t used = 0, tails = 0;  // tails: slots whose last filling was counted on `tail`
            uint32_t tail_parity = 0;
            bool ok = true;
            for (int item = unit; ok && item < items; item += units) {
                const Tile w = walk.at(item);
                const int r = w.r0 + (int)rank * 128;
                // the wide operand's share of this CTA: half of the product's extent
                const int half = B_MN ? a.width / 2 : (w.n + 63) / 64 * 32, c = w.c0 + (int)rank * half;
                const uint32_t bytes = kHalf + (uint32_t)half * 128u;
                for (int k = w.kb; k < w.ke; ++k) {
                    if (used >= kStages && !warp_wait(&s.empty[t.slot], t.phase ^ 1u, &s.abort, a.status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t at = smem_u32(ring) + t.slot * kStageBytes;
                    const int k0 = w.s0 + k * 64;
                    const bool cut = MODE == kWeights && k == w.steps - 1 && w.last % 16 != 0;
                    if (cut) {
                        tails |= 1u << t.slot;
                        tail_parity ^= 1u << t.slot;
                    } else {
                        tails &= ~(1u << t.slot);
                    }
                    if (!elect()) {
                        // the others wait below
                    } else if (cut) {
                        if constexpr (MODE == kWeights) {
                            const uint32_t bar = smem_u32(&s.tail[t.slot]);
                            mbar_expect(&s.tail[t.slot], bytes);
                            if (a.tall_panels)
                                tma_load_4d(at, &mtall, 0, k0, r / 64, 0, bar);
                            else
                                for (int p = 0; p < 2; ++p) tma_load_2d(at + p * kPanel, &mtall, r + 64 * p, k0, bar);
                            if (a.wide_panels)
                                tma_load_4d(at + kHalf, &mwide, 0, k0, c / 64, 0, bar);
                            else
                                for (int p = 0; p < half / 64; ++p) tma_load_2d(at + kHalf + p * kPanel, &mwide, c + 64 * p, k0, bar);
                        }
                    } else {
                        const uint32_t bar = cluster_addr(smem_u32(&s.full[t.slot]), even);
                        mbar_expect_cluster(bar, bytes);
                        if constexpr (MODE == kWeights) {
                            if (a.tall_panels)
                                tma_load_4d_pair(at, &mtall, 0, k0, r / 64, 0, bar);
                            else
                                for (int p = 0; p < 2; ++p) tma_load_2d_pair(at + p * kPanel, &mtall, r + 64 * p, k0, bar);
                            if (a.wide_panels)
                                tma_load_4d_pair(at + kHalf, &mwide, 0, k0, c / 64, 0, bar);
                            else
                                for (int p = 0; p < half / 64; ++p) tma_load_2d_pair(at + kHalf + p * kPanel, &mwide, c + 64 * p, k0, bar);
                        } else {
                            if constexpr (A_MN) {
                                if (a.tall_panels)
                                    tma_load_4d_pair(at, &mtall, 0, k0, r / 64, w.e, bar);
                                else
                                    for (int p = 0; p < 2; ++p) tma_load_3d_pair(at + p * kPanel, &mtall, r + 64 * p, k0, w.e, bar);
                            } else {
                                tma_load_3d_pair(at, &mtall, k0, r, w.e, bar);
                            }
                            if (half == a.width / 2)
                                tma_load_2d_pair(at + kHalf, &mwide_all, k0, c, bar);
                            else
                                for (int b = 0; b < half; b += 32)
                                    tma_load_2d_pair(at + kHalf + (uint32_t)b * 128u, &mwide, k0, c + b, bar);
                        }
                    }
                    __syncwarp();
                    ++used;
                    t.next(kStages);
                }
            }
            // nothing may still be landing when the pair leaves: the last filling of each slot
            for (uint32_t i = 0; i < (uint32_t)kStages && i < used; ++i) {
                if (tails >> i & 1u)
                    mbar_wait_bounded(smem_u32(&s.tail[i]), (tail_parity >> i & 1u) ^ 1u);
                if (rank == 0) mbar_wait_bounded(smem_u32(&s.full[i]), ((used - i + kStages - 1) / kStages - 1) & 1u);
            }
        }
    } else if (warp == 1) {
        fewer_registers();
        if (rank == 0) {
            Turn t, acc;
            uint32_t runs = 0;
            bool ok = true;
            for (int item = unit; ok && item < items; item += units) {
                const Tile w = walk.at(item);
                const uint32_t id = a.id | ((B_MN ? (uint32_t)a.width : (uint32_t)((w.n + 63) / 64 * 64)) >> 3) << 17;
                for (int k = w.kb; ok && k < w.ke;) {
                    // a run of the sum into the next accumulator
                    const int end = w.ke - k > kRun ? k + kRun : w.ke;
                    ok = runs < 2 || warp_wait(&s.acc_empty[acc.slot], acc.phase ^ 1u, &s.abort, a.status);
                    const uint32_t d = tmem + acc.slot * 256;
                    bool add = false;
                    for (; ok && k < end; ++k) {
                        // a cut stage's rows were cleared by the pair's threads; others are the copies' alone
                        const bool last = MODE == kWeights && k == w.steps - 1;
                        ok = last && w.last % 16 != 0 ? warp_wait<true>(&s.full[t.slot], t.phase, &s.abort, a.status)
                                                      : warp_wait(&s.full[t.slot], t.phase, &s.abort, a.status);
                        if (!ok) break;
                        acc_fence_after();
                        const uint32_t at = smem_u32(ring) + t.slot * kStageBytes;
                        const int js = last ? (w.last + 15) / 16 : 4;
                        if (elect()) {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (MODE != kWeights || j < js)
                                    umma<false, true>(d, A_MN ? operand_mn(at + j * 2048, kPanel) : operand_k(at + j * 32),
                                                      B_MN ? operand_mn(at + kHalf + j * 2048, kPanel) : operand_k(at + kHalf + j * 32),
                                                      id, j != 0 || add);
                            umma_done<true>(&s.empty[t.slot], 3u << even);
                            if (k + 1 == end) umma_done<true>(&s.acc_full[acc.slot], 3u << even);
                        }
                        __syncwarp();
                        add = true;
                        t.next(kStages);
                    }
                    acc.next(2);
                    ++runs;
                }
            }
            if (elect()) umma_done<true>(&s.done, 3u << even);
            __syncwarp();
            mbar_wait_bounded(smem_u32(&s.done), 0);
        }
    } else if (warp >= kOut) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
        // two warps a 32 lanes: one takes the even runs of 32 columns, the other the odd
        const int q = warp & 3, odd = (warp - kOut) >> 2;
        const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
        const uint32_t free0 = cluster_addr(smem_u32(&s.acc_empty[0]), even), free1 = cluster_addr(smem_u32(&s.acc_empty[1]), even);
        O *out = reinterpret_cast<O *>(a.out);
        Turn acc;
        bool waited = false;
        for (int item = unit; item < items; item += units) {
            const Tile w = walk.at(item);
            const int r = w.r0 + (int)rank * 128 + q * 32 + lane;
            O *const first = out + ((MODE == kWeights ? (int64_t)w.e * a.C : 0) + w.c0) * a.ldo + r;
            bool ok = true;
            auto ready = [&] {
                ok = __all_sync(0xffffffffu, role_wait(&s.acc_full[acc.slot], acc.phase, &s.abort, a.status));
                acc_fence_after();
                return ok;
            };
            auto give_back = [&] {
                acc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(acc.slot ? free1 : free0);
                acc.next(2);
            };
            auto store = [&](const float(&v)[32], int c0) {
                O *p = first + c0 * a.ldo;
                if (c0 + 32 <= w.n) {
                    if (r < a.R) {
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            *p = from_f<O>(v[c]);
                            p += a.ldo;
                        }
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        if (c0 + c < w.n && r < a.R) *p = from_f<O>(v[c]);
                        p += a.ldo;
                    }
                }
            };
            uint64_t sum[64];  // runs of 32 columns, pairs of them
#pragma unroll
            for (int i = 0; i < 64; ++i) sum[i] = 0;
            auto get = [&](int i, float(&v)[32]) {  // columns 32 odd + 64 i on
#pragma unroll
                for (int c = 0; c < 16; ++c) unpack2(sum[16 * i + c], v[2 * c], v[2 * c + 1]);
            };
            const uint64_t one = pack2(1.0f, 1.0f);
            for (int k = w.kb; k < w.ke && ready(); k += kRun) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (64 * i < a.width) add_columns(lanes + acc.slot * 256 + 32 * odd + 64 * i, sum + 16 * i, one);
                give_back();
            }
            if constexpr (SPLIT) {  // the parts of the sum meet
                const int own = pair * (4 / S), mine = warp - kOut;
                if (warp == kOut && lane == 0) {
                    uint32_t runs = 0;
                    for (int i = 0; i < 4 / S; ++i) runs += (64 * (own + i) < w.n) + (64 * (own + i) + 32 < w.n);
                    mbar_expect(&s.inbox, runs * (uint32_t)S * 16384u);
                }
                __syncwarp();
                cluster_sync();  // every ring is done with, every inbox ready
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (32 * odd + 64 * i < w.n) {
                        float v[32];
                        get(i, v);
                        join_push(v, smem_u32(ring), &s.inbox, pair, mine, i, S, rank);
                    }
                ok = __all_sync(0xffffffffu, role_wait<true>(&s.inbox, 0, &s.abort, a.status));
                if (!ok) break;
                pdl_wait();
                for (int i = own; i < own + 4 / S; ++i)
                    if (32 * odd + 64 * i < w.n) {
                        float v[32];
                        join_sum(v, ring, mine, i, S);
                        store(v, 32 * odd + 64 * i);
                    }
                break;
            }
            if (!ok) break;
            if (!waited) pdl_wait();
            waited = true;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (32 * odd + 64 * i < w.n) {
                    float v[32];
                    get(i, v);
                    store(v, 32 * odd + 64 * i);
                }
        }
    } else {
        fewer_registers();
        // rows past an expert's end, up to the next 16 of the sum, in the stage that holds its last rows
        Turn t;
        uint32_t parity = 0;
        for (int item = unit; MODE == kWeights && warp == kClear && item < items; item += units) {
            const Tile w = walk.at(item);
            if (w.kb == w.ke) continue;
            for (int k = w.kb; k + 1 < w.ke; ++k) t.next(kStages);
            if (w.last % 16 != 0 && w.ke == w.steps) {
                if (!__all_sync(0xffffffffu, role_wait(&s.tail[t.slot], parity >> t.slot & 1u, &s.abort, a.status))) break;
                parity ^= 1u << t.slot;
                const uint32_t at = smem_u32(ring) + t.slot * kStageBytes;
                const int upto = (w.last + 15) / 16 * 16;
                // a row of the sum is 128 bytes in each of the four panels: 8 lanes a row, 4 panels at once
                for (int row = w.last; row < upto; ++row)
                    asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(at + (uint32_t)(lane >> 3) * kPanel +
                                                                                (uint32_t)row * 128u + (uint32_t)(lane & 7) * 16u),
                                 "r"(0)
                                 : "memory");
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(cluster_addr(smem_u32(&s.full[t.slot]), even));
            }
            t.next(kStages);
        }
    }
    __syncwarp();
    if (SPLIT && unit < items && warp < kOut) cluster_sync();  // the joins' own
    pdl_wait();
    acc_fence_before();
    __syncthreads();
    cluster_sync();  // the pair's products, copies and arrivals are over
    if (warp == 1) {
        __syncwarp();
        acc_fence_after();
        acc_free<true>(tmem, 512);
    }
}

constexpr size_t kWideSmem = kStages * kStageBytes + 1024;

// One instance of the kernel on a device: its shared memory allowed, and how many clusters of 2 and
// 4 pairs can be there at once.
struct Instance {
    std::once_flag once;
    bool good;
    int fit2, fit4;
};

template <int MODE, typename O, bool SPLIT>
tm_status instance(const Instance **out)
{
    static Instance each[kMaxDevices];
    const void *k = (const void *)wide_kernel<MODE, O, SPLIT>;
    int d = 0;
    if (cudaGetDevice(&d) != cudaSuccess || d < 0 || d >= kMaxDevices) return TM_ERR_CUDA;
    Instance &i = each[d];
    std::call_once(i.once, [&] {
        i.good = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kWideSmem) == cudaSuccess;
        i.fit2 = i.fit4 = 0;
        for (int S = 2; i.good && SPLIT && S <= 4; S *= 2) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(2 * S);
            cfg.blockDim = dim3(kWideThreads);
            cfg.dynamicSmemBytes = kWideSmem;
            cudaLaunchAttribute attr;
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = (unsigned)(2 * S);
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(S == 2 ? &i.fit2 : &i.fit4, k, &cfg) != cudaSuccess) (S == 2 ? i.fit2 : i.fit4) = 0;
        }
        cudaGetLastError();
    });
    *out = &i;
    return i.good ? TM_OK : TM_ERR_CUDA;
}

template <int MODE, typename O, bool SPLIT>
tm_status launch_pairs(const CUtensorMap &tall, const CUtensorMap &wide, const CUtensorMap &all, const WideArgs &a, int S, int64_t units,
                       cudaStream_t s, bool pdl)
{
    const Instance *i;
    const tm_status st = instance<MODE, O, SPLIT>(&i);
    if (st != TM_OK) return st;
    void *args[] = {const_cast<CUtensorMap *>(&tall), const_cast<CUtensorMap *>(&wide), const_cast<CUtensorMap *>(&all),
                    const_cast<WideArgs *>(&a), &S};
    return launch_kernel((const void *)wide_kernel<MODE, O, SPLIT>, dim3((unsigned)(2 * S * units)),
                         dim3(kWideThreads), args, kWideSmem, s, pdl, (unsigned)(2 * S));
}

// steps: stages of an average sum (weights' gradient).  Few long sums are shared by pairs while all the
// clusters are there at once: a join costs about 5 us, a stage 0.27.  One expert of 1024 x 1024 in fp32,
// 2048 rows: 15.6 us a pair a tile, 16.0 two; 4096 rows: 24.0, 20.2; 8192 rows: 40.8, 28.5.  Of 512 x 520, four
// pairs a tile: 2048 rows 15.2, 4096 rows 17.3, 8192 rows 21.6 us.  The other products with as few
// tiles and sums as long go to the small tiles (tm_experts.cu).
template <int MODE, typename O>
tm_status launch_wide(const CUtensorMap &tall, const CUtensorMap &wide, const CUtensorMap &all, const WideArgs &a, int64_t items,
                      int64_t steps, const DevInfo &dev, cudaStream_t s, bool pdl)
{
    if constexpr (MODE == kWeights)
        if (steps >= 32) {
            const Instance *i;
            const tm_status st = instance<MODE, O, true>(&i);
            if (st != TM_OK) return st;
            const int S = items <= i->fit4 ? 4 : items <= i->fit2 && steps >= 48 ? 2 : 1;
            if (S > 1) return launch_pairs<MODE, O, true>(tall, wide, all, a, S, items, s, pdl);
        }
    const int64_t pairs = dev.sms / 2;
    return launch_pairs<MODE, O, false>(tall, wide, all, a, 1, items < pairs ? items : pairs, s, pdl);
}

template <int MODE>
tm_status launch_typed(const CUtensorMap &tall, const CUtensorMap &wide, const CUtensorMap &all, const WideArgs &a, int64_t items,
                       int64_t steps, const DevInfo &dev, cudaStream_t s, bool pdl)
{
    if (items > (1 << 30)) return TM_ERR_UNSUPPORTED_TILE;
    if constexpr (MODE != kRows)  // always to 16 bits
        if (a.otype == TM_F32) return launch_wide<MODE, float>(tall, wide, all, a, items, steps, dev, s, pdl);
    if (a.otype == TM_F16) return launch_wide<MODE, __half>(tall, wide, all, a, items, steps, dev, s, pdl);
    return launch_wide<MODE, __nv_bfloat16>(tall, wide, all, a, items, steps, dev, s, pdl);
}

int tiles256(int64_t n) { return (int)((n + 255) / 256); }

// The width of a tile along c: 128 or 64 where all such tiles run at once, on SMs that would have nothing to do; more
// of them would only read more.  16 bits, cold: 5 experts of 520 x 1000, 200 rows each, forward 16.4 us with 256 and 14.3 with
// 128; 512 x 512, 1000 rows, 12.3 and with 64 10.7.
template <typename F>
int width_of(F tiles, int least, const DevInfo &dev)
{
    int w = 256;
    while (w > least && tiles(w / 2) <= dev.sms / 2) w /= 2;
    return w;
}

}  // namespace

tm_status wide_product(const Product &p, const DevInfo &dev, cudaStream_t s, bool pdl)
{
    WideArgs a = {};
    a.out = p.out;
    a.ldo = p.ldo;
    a.starts = p.starts;
    a.status = dev.status;
    a.otype = p.otype;
    a.E = p.E;
    a.T = (int)p.T;
    a.R = (int)p.F;
    a.rtiles = tiles256(p.F);
    const int64_t busy = p.E < p.T ? p.E : p.T;
    auto tiles = [&](int w) { return ((p.T + w - 1) / w + busy) * a.rtiles; };
    a.width = width_of([&](int w) { return tiles_of(p, w) * a.rtiles; }, 64, dev);
    a.by_block = a.by_expert = make_fastdiv((uint32_t)(kGroup * a.rtiles));
    a.steps = (int)((p.R + 63) / 64);
    a.id = instruction(p.kind == kProductBF16 ? 1u : 0u, p.w_mn, false, 256, 0);
    a.tall_panels = p.w_mn && p.F % 64 == 0 && p.R > 0;
    CUtensorMap tall, wide, all;
    if (a.tall_panels ? !panels_map(&tall, p.w, p.F, p.R, p.ldw, p.E)
                      : !rows_map(&tall, p.kind, p.w, p.w_mn ? p.F : p.R, p.w_mn ? p.R : p.F, p.ldw, p.E, p.w_mn ? 64 : 128))
        return TM_ERR_CUDA;
    if (!rows_map(&wide, p.kind, p.x, p.R, p.T, p.ldx, 0, 32) || !rows_map(&all, p.kind, p.x, p.R, p.T, p.ldx, 0, a.width / 2)) return TM_ERR_CUDA;
    return p.w_mn ? launch_typed<kRows>(tall, wide, all, a, tiles(a.width), a.steps, dev, s, pdl)
                  : launch_typed<kForward>(tall, wide, all, a, tiles(a.width), a.steps, dev, s, pdl);
}

tm_status wide_weights(ProductKind kind, const void *dy, int64_t lddy, const void *x, int64_t ldx, void *dw, int64_t lddw,
                       int32_t wtype, const int32_t *starts, int32_t E, int64_t T, int64_t N, int64_t K, const DevInfo &dev,
                       cudaStream_t s, bool pdl)
{
    WideArgs a = {};
    a.out = dw;
    a.ldo = lddw;
    a.starts = starts;
    a.status = dev.status;
    a.otype = wtype;
    a.E = E;
    a.T = (int)T;
    a.R = (int)K;
    a.C = (int)N;
    a.rtiles = tiles256(K);
    // long sums are shared by pairs instead (one of 1024 x 512, 3000 rows: 20.8 us, narrow 24.6)
    a.width = T / 64 / E >= 32 ? 256 : width_of([&](int w) { return (int64_t)E * a.rtiles * ((N + w - 1) / w); }, 128, dev);
    a.ctiles = (int)((N + a.width - 1) / a.width);
    a.by_block = make_fastdiv((uint32_t)(kGroup * a.rtiles));
    a.by_expert = make_fastdiv((uint32_t)((int64_t)a.rtiles * a.ctiles < (1 << 30) ? a.rtiles * a.ctiles : 1));  // more tiles are refused
    a.id = instruction(kind == kProductBF16 ? 1u : 0u, true, true, 256, 0);
    a.tall_panels = K % 64 == 0 && T > 0;
    a.wide_panels = N % 64 == 0 && T > 0 && a.width == 256;  // two panels a CTA
    CUtensorMap tall, wide;
    if (a.tall_panels ? !panels_map(&tall, x, K, T, ldx, 0) : !rows_map(&tall, kind, x, K, T, ldx, 0, 64)) return TM_ERR_CUDA;
    if (a.wide_panels ? !panels_map(&wide, dy, N, T, lddy, 0) : !rows_map(&wide, kind, dy, N, T, lddy, 0, 64)) return TM_ERR_CUDA;
    return launch_typed<kWeights>(tall, wide, wide, a, (int64_t)E * a.rtiles * a.ctiles, T / 64 / E, dev, s, pdl);
}

}  // namespace libtm
