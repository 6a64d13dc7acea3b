// tm_thin.cu -- products whose experts have few rows: out[t, f] = sum_r x[t, r] w_e[f, r].
//
// What bounds it is reading each busy expert's weights once.  So the weights are the
// tall operand: a tile is 128 features by up to BT rows of x, the rows along N of the
// tensor cores' product, where an extent is any multiple of 16 (a tile of 5 rows costs
// 16).  TMA fills a ring of stages of 16 KB of weights.  A CTA has one tile and two or
// three CTAs share an SM, so that one's start and end hide behind the others' copies and a free SM takes the next
// tile: CTAs that stay, one an SM with all of its memory, read at 5.3 TB/s.
// Few tiles are cut along the sum over a cluster of S CTAs: each
// pushes its partial rows to the CTA that owns them (st.async into its shared memory),
// which adds them in rank order and stores: one launch, no workspace, the same bits
// every time.  256 rows over 48 experts of 2048 x 4096 in 8 bits: 67 us, 6.0 TB/s; 64 rows over 24 in 16 bits: 67 us, 6.0.
//
// Sums.  The tensor cores' additions lose up to 2^-23 of the sum each, always towards zero, so a
// sum of 16-bit products leaves them after kRunSums of it and is added in registers, rounded to nearest (over
// 8192 rows of a weights' gradient: 2.5e-6 of the result without, 2e-7 with; 131072 terms of one sign
// lose 4e-4 of their sum without, nearly an output's rounding to fp16, and 3e-6 with).  e4m3: one accumulator for each 128 of the
// sum, read out, multiplied by both scales and added in fp32 registers while the next ones are made.
#include <mutex>

#include "tm_products.h"
#include "tm_umma.cuh"

namespace libtm {

bool rows_map_of(CUtensorMap *m, int e, const void *p, int64_t inner, int64_t rows, int64_t ld, int64_t E, int box)
{
    if (inner <= 0 || rows <= 0) inner = rows = 1, ld = 16;  // nothing to read: a map that no tile asks for
    const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)(E > 0 ? E : 1)};
    const cuuint64_t strides[2] = {(cuuint64_t)(ld * e), (cuuint64_t)(ld * e * rows)};
    const cuuint32_t boxes[3] = {(cuuint32_t)(128 / e), (cuuint32_t)box, 1};
    const cuuint32_t steps[3] = {1, 1, 1};
    auto encode = tensor_map_encoder();
    if (encode == nullptr) return false;
    return encode(m, e == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : e == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : CU_TENSOR_MAP_DATA_TYPE_UINT32, E > 0 ? 3 : 2,
                  const_cast<void *>(p), dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool panels_map(CUtensorMap *m, const void *p, int64_t inner, int64_t rows, int64_t ld, int64_t E)
{
    const cuuint64_t dims[4] = {64, (cuuint64_t)rows, (cuuint64_t)(inner / 64), (cuuint64_t)(E > 0 ? E : 1)};
    const cuuint64_t strides[3] = {(cuuint64_t)(ld * 2), 128, (cuuint64_t)(ld * 2 * rows)};
    const cuuint32_t boxes[4] = {64, 64, 2, 1};
    const cuuint32_t steps[4] = {1, 1, 1, 1};
    auto encode = tensor_map_encoder();
    if (encode == nullptr) return false;
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<void *>(p), dims, strides, boxes, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

constexpr int kMaxStages = 10;
constexpr uint32_t kTall = 128 * 128;  // bytes of weights a stage

struct ThinArgs {
    void *out;
    int64_t ldo;
    const int32_t *starts;
    const float *sa, *sb;
    unsigned *status;
    int otype, E, T, F, ftiles;
    int steps;   // stages a tile: 128 bytes of the sum each
    int stages;  // of the ring
    int group;
    uint32_t id;  // the instruction without its N
};

// The forms.  F8: e4m3.
template <bool F8, int BT>
struct Thin {
    static constexpr int kOutWarps = BT <= 32 ? 4 : 8;  // behind warp 0, which copies, and warp 1, which multiplies
    static constexpr int kThreads = 64 + 32 * kOutWarps;
    static constexpr int kCols = BT * 4 / kOutWarps;    // columns of an output warp
    // Three CTAs an SM with tiles of 32 rows, stages of 20 KB; one with 128, stages of 32 KB and 64 sums a thread.
    static constexpr int kCtas = BT <= 32 ? 3 : 1;
    // Stages of the ring, by how many CTAs an SM there are: a tile alone there has all of the memory (16 rows
    // by 2048 x 8192 in 16 bits, cold: 18.5 us with 3 stages, 16.0 with 10; 4096 x 4096 14.1 and 13.4)
    static constexpr int stages(int ctas) { return BT > 32 ? 6 : ctas <= 1 ? 10 : ctas == 2 ? 5 : 3; }
    static constexpr int kRun = F8 ? 1 : kRunSums / 64;  // stages a run
    static constexpr int kAccs = BT <= 32 ? 4 : 2;  // accumulators that take turns over a tile's runs
};

template <bool F8, int BT>
struct ThinSmem {
    using F = Thin<F8, BT>;
    alignas(8) uint64_t full[kMaxStages], empty[kMaxStages], acc_full[4], acc_empty[4], inbox, done;
    uint32_t tmem;
    int abort;
    int e, row, n;  // the tile: expert, first row, how many (0: none)
    alignas(16) float scale[F::kOutWarps][2][F8 ? F::kCols : 4];  // each output warp's own
    int starts[kMaxExperts + 1];
};

__device__ __forceinline__ void store_one(void *out, int64_t at, int type, float v)
{
    if (type == TM_F32)
        reinterpret_cast<float *>(out)[at] = v;
    else if (type == TM_F16)
        reinterpret_cast<__half *>(out)[at] = __float2half_rn(v);
    else
        reinterpret_cast<__nv_bfloat16 *>(out)[at] = __float2bfloat16_rn(v);
}

// One warp: the expert and rows of row tile `tile`.  The rules of experts_read.
template <typename S>
__device__ __forceinline__ void find_tile(S &s, const ThinArgs &a, int tile, int BT)
{
    const int lane = threadIdx.x & 31;
    if (a.starts == nullptr) {
        const int left = a.T - tile * BT;
        if (lane == 0) s.e = 0, s.row = tile * BT, s.n = left < 0 ? 0 : left < BT ? left : BT;
        return;
    }
    int sum = 0, past = 0;
    bool all = true, found = false;
    for (int e0 = 0; e0 < a.E && (!found || blockIdx.x == 0); e0 += 32) {
        const int e = e0 + lane;
        const int lo = e < a.E ? s.starts[e] : 0, hi = e < a.E ? s.starts[e + 1] : 0;
        int m = lo;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, m, o);
            if (lane >= o && u > m) m = u;
        }
        if (past > m) m = past;
        const bool ok = m <= lo && lo <= hi && hi <= a.T;
        all = all && (ok || e >= a.E);
        const int own = ok && e < a.E ? (hi - lo) / BT + ((hi - lo) % BT != 0) : 0;
        int v = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        const int local = tile - (sum + v - own);
        if (local >= 0 && local < own) {
            const int row = lo + local * BT;
            s.e = e, s.row = row, s.n = hi - row < BT ? hi - row : BT;
        }
        found = found || __any_sync(0xffffffffu, local >= 0 && local < own);
        sum += __shfl_sync(0xffffffffu, v, 31);
        past = __shfl_sync(0xffffffffu, m, 31);
    }
    if (!found && lane == 0) s.n = 0;
    if (!all && blockIdx.x == 0) atomicOr(a.status, kStatusIndex);
    __syncwarp();
}

template <bool F8, bool MN, int BT>
__global__ void __launch_bounds__(Thin<F8, BT>::kThreads)
    thin_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mx_all,
                const ThinArgs a, const int S)
{
    constexpr uint32_t kStage = kTall + BT * 128;
    using F = Thin<F8, BT>;
    const uint32_t stages = (uint32_t)a.stages;
    constexpr int kStep = F8 ? 128 : 64;  // elements of the sum a stage
    constexpr int kAccs = F::kAccs, kRun = F::kRun, CW = F::kCols;
    // weights are read once, or by a few tiles at about the same time: they are the first L2 gives up, not
    // lines still to be written back (32 experts of 2048 x 4096 in 16 bits, 64 rows: 63.5 us without, 55.6 with)
    const uint64_t pol = l2_evict_first_policy();
    extern __shared__ __align__(1024) unsigned char raw[];
    unsigned char *ring = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    // with S > 1: [S][4 warps][BT / S / 4][32 lanes][4 rows] partial sums of the rows this CTA owns, in
    // the ring's place once every CTA of the cluster is done with its own
    float *inbox = reinterpret_cast<float *>(ring);
    static_assert(BT * 128 * 4 <= 3 * kStage, "inbox");
    __shared__ ThinSmem<F8, BT> s;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = S > 1 ? (int)cluster_rank() : 0;
    const int item = (int)blockIdx.x / S;
    // row tiles of the experts in order; all features of one, then the next
    const int tile = item / a.ftiles, f0 = (item - tile * a.ftiles) * 128;
    const int k0 = (int)((int64_t)a.steps * rank / S), k1 = (int)((int64_t)a.steps * (rank + 1) / S);

    if (threadIdx.x == 0) {
        tensormap_prefetch(&mw);
        tensormap_prefetch(&mx);
        for (int i = 0; i < a.stages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < kAccs; ++i) {
            mbar_init(&s.acc_full[i], 1);
            mbar_init(&s.acc_empty[i], F::kOutWarps);
        }
        mbar_init(&s.done, 1);
        mbar_init(&s.inbox, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        s.abort = 0;
    }
    if (a.starts != nullptr) {
        for (int e = threadIdx.x; e <= a.E; e += F::kThreads) s.starts[e] = a.starts[e];
        __syncthreads();
    }
    if (warp == 0) find_tile(s, a, tile, BT);
    if (warp == 1) acc_alloc<false>(&s.tmem, kAccs * BT);
    acc_fence_before();
    __syncthreads();
    acc_fence_after();
    pdl_trigger();  // only now: a dependent's CTA could take the tensor memory that this one waits for
    const int e = s.e, row0 = s.row, n = s.n;
    const uint32_t tmem = s.tmem;
    // an output warp: 32 features, CW columns from cb on
    const int q = warp & 3, f = f0 + q * 32 + lane, part = (warp - 2) >> 2, cb = part * CW;
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
    bool ok = true;
    float sum[CW];

    if (warp == 0) {
        if (n > 0) {
            // few copies a stage: rows in boxes of 32, or all 128 in one
            const bool whole = BT > 32 && n > 96;
            const uint32_t boxes = whole ? 4 : (uint32_t)(n + 31) / 32;
            Turn t;
            uint32_t used = 0;
            for (int k = k0; k < k1; ++k) {
                if (used >= stages && !warp_wait(&s.empty[t.slot], t.phase ^ 1u, &s.abort, a.status)) break;
                const uint32_t bar = smem_u32(&s.full[t.slot]), at = smem_u32(ring) + t.slot * kStage;
                if (elect()) {
                    mbar_expect(&s.full[t.slot], kTall + boxes * 4096u);
                    if constexpr (MN) {
                        tma_load_3d_hint(at, &mw, f0, k * kStep, e, bar, pol);
                        tma_load_3d_hint(at + kTall / 2, &mw, f0 + 64, k * kStep, e, bar, pol);
                    } else {
                        tma_load_3d_hint(at, &mw, k * kStep, f0, e, bar, pol);
                    }
                    if (whole)
                        tma_load_2d(at + kTall, &mx_all, k * kStep, row0, bar);
                    else
                        for (uint32_t b = 0; b < boxes; ++b) tma_load_2d(at + kTall + b * 4096u, &mx, k * kStep, row0 + 32 * (int)b, bar);
                }
                __syncwarp();
                ++used;
                t.next(stages);
            }
            // nothing may still be landing when the CTA leaves: the last filling of each slot
            for (uint32_t i = 0; i < stages && i < used; ++i)
                mbar_wait_bounded(smem_u32(&s.full[i]), ((used - i + stages - 1) / stages - 1) & 1u);
        }
    } else if (warp == 1) {
        if (n > 0) {
            const uint32_t id = a.id | ((uint32_t)((n + 15) / 16 * 2) << 17);
            Turn t, acc;
            int in_run = 0;
            uint32_t runs = 0;
            for (int k = k0; k < k1; ++k) {
                if (in_run == 0 && runs >= (uint32_t)kAccs &&
                    !warp_wait(&s.acc_empty[acc.slot], acc.phase ^ 1u, &s.abort, a.status))
                    break;
                if (!warp_wait(&s.full[t.slot], t.phase, &s.abort, a.status)) break;
                acc_fence_after();
                const uint32_t at = smem_u32(ring) + t.slot * kStage, d = tmem + acc.slot * BT;
                ++in_run;
                const bool end = in_run == kRun || k + 1 == k1;
                if (elect()) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        umma<F8, false>(d, MN ? operand_mn(at + j * 2048, kTall / 2) : operand_k(at + j * 32),
                                        operand_k(at + kTall + j * 32), id, j != 0 || in_run != 1);
                    umma_done<false>(&s.empty[t.slot]);
                    if (end) umma_done<false>(&s.acc_full[acc.slot]);
                }
                __syncwarp();
                t.next(stages);
                if (end) {
                    acc.next(kAccs);
                    in_run = 0;
                    ++runs;
                }
            }
            // every product issued has completed before the tensor memory is given back
            if (elect()) umma_done<false>(&s.done);
            __syncwarp();
            mbar_wait_bounded(smem_u32(&s.done), 0);
        }
    } else if (n > 0) {
#pragma unroll
        for (int c = 0; c < CW; ++c) sum[c] = 0.0f;
        // e4m3: this warp's copy of the rows' factors; the next block's are on their way meanwhile
        const int G = a.steps;  // scales of a row
        const float *sb = F8 ? a.sb + ((int64_t)e * a.ftiles + f0 / 128) * G : nullptr;
        float fa[CW / 32], fb = 0.0f;
        auto fetch = [&](int k) {
            if (!F8 || k >= k1) return;
            fb = __ldg(sb + k);
#pragma unroll
            for (int i = 0; i < CW / 32; ++i) {
                const int t = cb + i * 32 + lane;
                const int64_t row = row0 + (t < n ? t : 0);
                fa[i] = __ldg(a.sa + (a.group ? row * G + k : row));
            }
        };
        Turn acc;
        fetch(k0);
        for (int k = k0; k < k1; k += kRun) {
            float *factor = s.scale[warp - 2][k & 1];
            if constexpr (F8) {
#pragma unroll
                for (int i = 0; i < CW / 32; ++i) factor[i * 32 + lane] = fa[i] * fb;
                fetch(k + 1);
                __syncwarp();
            }
            ok = __all_sync(0xffffffffu, role_wait(&s.acc_full[acc.slot], acc.phase, &s.abort, a.status));
            if (!ok) break;
            acc_fence_after();
#pragma unroll
            for (int c0 = 0; c0 < CW; c0 += 32) {
                if (cb + c0 < n) {
                    float v[32];
                    acc_load32(lanes + acc.slot * BT + cb + c0, v);
                    acc_load_wait(v);
#pragma unroll
                    for (int c = 0; c < 32; c += 4) {
                        if constexpr (F8) {
                            const float4 m = *reinterpret_cast<const float4 *>(factor + c0 + c);
                            sum[c0 + c] = __fmaf_rn(v[c], m.x, sum[c0 + c]);
                            sum[c0 + c + 1] = __fmaf_rn(v[c + 1], m.y, sum[c0 + c + 1]);
                            sum[c0 + c + 2] = __fmaf_rn(v[c + 2], m.z, sum[c0 + c + 2]);
                            sum[c0 + c + 3] = __fmaf_rn(v[c + 3], m.w, sum[c0 + c + 3]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i) sum[c0 + c + i] += v[c + i];
                        }
                    }
                }
            }
            acc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.acc_empty[acc.slot]);
            acc.next(kAccs);
        }
    }
    __syncwarp();
    // rows of a tile that this CTA owns; its inbox expects them from every rank
    const int share = ((n + S - 1) / S + 3) & ~3, own0 = rank * share;  // whole fours: a push is 16 bytes
    const int own = own0 < n ? (n - own0 < share ? n - own0 : share) : 0;
    if (S > 1) {
        if (threadIdx.x == 0 && n > 0) mbar_expect(&s.inbox, (uint32_t)(S * ((own + 3) & ~3)) * 512u);
        __syncwarp();
        cluster_sync();  // every ring is done with, every inbox ready
    }
    if (warp >= 2 && n > 0) {
        pdl_wait();
        if (ok) {
#pragma unroll
            for (int i0 = 0; i0 < CW; i0 += 32) {
                const int c0 = cb + i0;
                if (c0 >= n) break;
                float v[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) v[c] = sum[i0 + c];
                if (S == 1) {
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (c0 + c < n && f < a.F) store_one(a.out, (int64_t)(row0 + c0 + c) * a.ldo + f, a.otype, v[c]);
                } else {
                    int to = c0 / share, at = c0 - to * share;  // owner of row c0 + c, and its place there
#pragma unroll
                    for (int c = 0; c < 32; c += 4) {
                        if (c0 + c < n) {
                            const uint32_t dst = smem_u32(inbox + (((rank * 4 + q) * (BT / S / 4) + at / 4) * 32 + lane) * 4);
                            asm volatile(
                                "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                                    cluster_addr(dst, (uint32_t)to)),
                                "r"(as_u(v[c])), "r"(as_u(v[c + 1])), "r"(as_u(v[c + 2])), "r"(as_u(v[c + 3])),
                                "r"(cluster_addr(smem_u32(&s.inbox), (uint32_t)to))
                                : "memory");
                            at += 4;
                            if (at == share) {
                                at = 0;
                                ++to;
                            }
                        }
                    }
                }
            }
            if (S > 1 && __all_sync(0xffffffffu, role_wait<true>(&s.inbox, 0, &s.abort, a.status)))
                for (int c = 4 * part; c < own; c += F::kOutWarps) {
                    float4 v = {0.0f, 0.0f, 0.0f, 0.0f};
                    for (int r = 0; r < S; ++r) {
                        const float4 u = *reinterpret_cast<const float4 *>(inbox + (((r * 4 + q) * (BT / S / 4) + c / 4) * 32 + lane) * 4);
                        v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
                    }
                    const float w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (c + i < own && f < a.F) store_one(a.out, (int64_t)(row0 + own0 + c + i) * a.ldo + f, a.otype, w[i]);
                }
        }
    }
    __syncwarp();
    pdl_wait();
    acc_fence_before();
    __syncthreads();
    if (S > 1) cluster_sync();  // no peer still writes to this inbox
    if (warp == 1) {
        __syncwarp();
        acc_fence_after();
        acc_free<false>(tmem, kAccs * BT);
    }
}

template <bool F8, bool MN, int BT>
tm_status launch_thin(const Product &p, const DevInfo &dev, cudaStream_t s, bool pdl)
{
    using F = Thin<F8, BT>;
    constexpr size_t kStage = kTall + BT * 128;
    static_assert(F::stages(1) * kStage + 1024 + sizeof(ThinSmem<F8, BT>) <= 227 * 1024 && F::stages(1) <= kMaxStages, "shared memory");
    static_assert(F::kCtas == 1 || F::kCtas * (F::stages(F::kCtas) * kStage + sizeof(ThinSmem<F8, BT>) + 2048) <= 228 * 1024,
                  "shared memory");
    static_assert(F::kCtas * F::kAccs * BT <= 512, "tensor memory");
    const void *k = (const void *)thin_kernel<F8, MN, BT>;
    static std::once_flag once[kMaxDevices];
    static bool good[kMaxDevices];
    int d = 0;
    if (cudaGetDevice(&d) != cudaSuccess || d < 0 || d >= kMaxDevices) return TM_ERR_CUDA;
    std::call_once(once[d], [&] {
        good[d] = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)(F::stages(1) * kStage + 1024)) == cudaSuccess;
        if (!good[d]) cudaGetLastError();
    });
    if (!good[d]) return TM_ERR_CUDA;
    ThinArgs a = {};
    a.out = p.out;
    a.ldo = p.ldo;
    a.starts = p.starts;
    a.sa = p.sa;
    a.sb = p.sb;
    a.status = dev.status;
    a.otype = p.otype;
    a.E = p.E;
    a.T = (int)p.T;
    a.F = (int)p.F;
    a.ftiles = (int)((p.F + 127) / 128);
    a.steps = (int)((p.R + (F8 ? 127 : 63)) / (F8 ? 128 : 64));
    a.group = p.group;
    a.id = instruction(p.kind == kProductBF16 ? 1u : 0u, MN, false, 128, 0);
    // tiles: at least one for each expert that has rows (how many have is not known here), and no more than `most`
    const int64_t busy = p.E < p.T ? p.E : p.T, rt = (p.T + BT - 1) / BT;
    const int64_t tiles = (rt > busy ? rt : busy) * a.ftiles, most = (p.starts == nullptr ? rt : rt + busy) * a.ftiles;
    if (most > (1 << 30)) return TM_ERR_UNSUPPORTED_TILE;
    // S CTAs a tile, up to two an SM in all.  32 tiles of a 4096 x 4096 matrix in 8 bits, 16 rows: S 1
    // 21.5 us, 2 18.6, 4 15.0, 8 14.8; 128 rows: 35.8, 35.6, 25.0, 47.6
    int S = 1;
    while (S < 4 && tiles * S <= (int64_t)dev.sms && a.steps >= 4 * S) S *= 2;
    a.stages = F::stages((int)(most * S > 3 * (int64_t)dev.sms ? 3 : (most * S + dev.sms - 1) / dev.sms));
    CUtensorMap mw, mx, mx_all;
    if (!rows_map(&mw, p.kind, p.w, MN ? p.F : p.R, MN ? p.R : p.F, p.ldw, p.E, MN ? 64 : 128) ||
        !rows_map(&mx, p.kind, p.x, p.R, p.T, p.ldx, 0, 32) || !rows_map(&mx_all, p.kind, p.x, p.R, p.T, p.ldx, 0, BT))
        return TM_ERR_CUDA;
    void *args[] = {&mw, &mx, &mx_all, &a, &S};
    return launch_kernel(k, dim3((unsigned)(most * S)), dim3(F::kThreads), args, a.stages * kStage + 1024, s, pdl, (unsigned)S);
}

}  // namespace

tm_status thin_product(const Product &p, const DevInfo &dev, cudaStream_t s, bool pdl)
{
    const bool few = p.T <= 32 * (int64_t)p.E;
    if (p.kind == kProductE4M3) return few ? launch_thin<true, false, 32>(p, dev, s, pdl) : launch_thin<true, false, 128>(p, dev, s, pdl);
    if (p.w_mn) return few ? launch_thin<false, true, 32>(p, dev, s, pdl) : launch_thin<false, true, 128>(p, dev, s, pdl);
    return few ? launch_thin<false, false, 32>(p, dev, s, pdl) : launch_thin<false, false, 128>(p, dev, s, pdl);
}

}  // namespace libtm
