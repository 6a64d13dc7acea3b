// tm_thin.cu -- products whose experts have few rows: out[t, f] = sum_r x[t, r] w_e[f, r].
//
// What bounds it is reading each busy expert's weights once.  So the weights are the
// tall operand: a tile is 128 features by up to BT rows of x, the rows along N of the
// tensor cores' product, where an extent is any multiple of 16 (a tile of 5 rows costs
// 16, and copies 16).  One CTA an SM walks tiles; TMA fills a ring of about 190 KB
// (16 KB of weights a stage), which keeps enough bytes in flight for the whole memory
// rate.  Few tiles are cut along the sum over a cluster of S CTAs: each
// pushes its partial rows to the CTA that owns them (st.async into its shared memory),
// which adds them in rank order and stores: one launch, no workspace, the same bits
// every time.
//
// Sums.  16-bit operands: the accumulator stays in tensor memory, fp32.  e4m3: one
// accumulator for each 128 of the sum, read out, multiplied by both scales and added in
// fp32 registers while the next one is made.
#include <mutex>

#include "tm_products.h"
#include "tm_umma.cuh"

namespace libtm {

bool rows_map(CUtensorMap *m, ProductKind kind, const void *p, int64_t inner, int64_t rows, int64_t ld, int64_t E, int box)
{
    const int e = kind == kProductE4M3 ? 1 : 2;
    if (inner <= 0 || rows <= 0) inner = rows = 1, ld = 16;  // nothing to read: a map that no tile asks for
    const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)(E > 0 ? E : 1)};
    const cuuint64_t strides[2] = {(cuuint64_t)(ld * e), (cuuint64_t)(ld * e * rows)};
    const cuuint32_t boxes[3] = {(cuuint32_t)(128 / e), (cuuint32_t)box, 1};
    const cuuint32_t steps[3] = {1, 1, 1};
    auto encode = tensor_map_encoder();
    if (encode == nullptr) return false;
    return encode(m, kind == kProductE4M3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, E > 0 ? 3 : 2,
                  const_cast<void *>(p), dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

constexpr int kThreadsThin = 192;  // warp 0 copies, warp 1 products, warps 2-5 outputs
constexpr int kMaxStages = 12;
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

template <int BT>
struct ThinSmem {
    alignas(8) uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2];
    alignas(8) uint64_t inbox_full, inbox_free, done;
    uint32_t tmem;
    int abort;
    alignas(16) float scale[4][2][BT];  // e4m3: each output warp's own
    Experts x;
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

template <bool F8, bool MN, int BT>
__global__ void __launch_bounds__(kThreadsThin, 1)
    thin_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mx, const ThinArgs a, const int S)
{
    constexpr uint32_t kStage = kTall + BT * 128;
    constexpr int kStep = F8 ? 128 : 64;  // elements of the sum a stage
    extern __shared__ __align__(1024) unsigned char raw[];
    unsigned char *ring = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    float *inbox = reinterpret_cast<float *>(ring + (size_t)a.stages * kStage);  // [S][BT / S][128], with S > 1
    __shared__ ThinSmem<BT> s;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = S > 1 ? (int)cluster_rank() : 0;
    const int unit = (int)blockIdx.x / S, units = (int)gridDim.x / S;
    const uint32_t stages = (uint32_t)a.stages;

    pdl_trigger();
    if (warp == 1) acc_alloc<false>(&s.tmem, 2 * BT);
    if (threadIdx.x == 0) {
        for (int i = 0; i < a.stages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.acc_full[i], 1);
            mbar_init(&s.acc_empty[i], 4);
        }
        mbar_init(&s.done, 1);
        mbar_init(&s.inbox_full, 1);
        mbar_init(&s.inbox_free, 4 * S);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        s.abort = 0;
    }
    experts_read(s.x, a.starts, a.E, a.T, BT, a.status);
    acc_fence_before();
    __syncthreads();
    if (S > 1) cluster_sync();  // every inbox and its barriers exist
    acc_fence_after();
    const uint32_t tmem = s.tmem;
    const int items = s.x.before[a.E] * a.ftiles;
    const int k0 = (int)((int64_t)a.steps * rank / S), k1 = (int)((int64_t)a.steps * (rank + 1) / S);

    // item i: row tile i / ftiles (experts in order), feature tile i % ftiles
    struct At {
        int e, row, n, f0;
    };
    int e_next = 0;
    auto find = [&](int item) {
        const int tile = item / a.ftiles;
        while (s.x.before[e_next + 1] <= tile) ++e_next;
        const int r0 = (tile - s.x.before[e_next]) * BT, left = s.x.count[e_next] - r0;
        return At{e_next, s.x.first[e_next] + r0, left < BT ? left : BT, (item % a.ftiles) * 128};
    };

    if (warp == 0) {
        if (lane == 0) {
            Turn t;
            uint32_t used = 0;
            bool ok = true;
            for (int item = unit; ok && item < items; item += units) {
                const At w = find(item);
                const uint32_t boxes = (uint32_t)(w.n + 15) / 16;
                for (int k = k0; k < k1; ++k) {
                    if (used >= stages && !role_wait(&s.empty[t.slot], t.phase ^ 1u, &s.abort, a.status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = smem_u32(&s.full[t.slot]), at = smem_u32(ring) + t.slot * kStage;
                    mbar_expect(&s.full[t.slot], kTall + boxes * 2048u);
                    if constexpr (MN) {
                        tma_load_3d(at, &mw, w.f0, k * kStep, w.e, bar);
                        tma_load_3d(at + kTall / 2, &mw, w.f0 + 64, k * kStep, w.e, bar);
                    } else {
                        tma_load_3d(at, &mw, k * kStep, w.f0, w.e, bar);
                    }
                    for (uint32_t b = 0; b < boxes; ++b)
                        tma_load_2d(at + kTall + b * 2048u, &mx, k * kStep, w.row + 16 * (int)b, bar);
                    ++used;
                    t.next(stages);
                }
            }
            // nothing may still be landing when the CTA leaves: the last filling of each slot
            for (uint32_t i = 0; i < stages && i < used; ++i)
                mbar_wait_bounded(smem_u32(&s.full[i]), ((used - i + stages - 1) / stages - 1) & 1u);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            Turn t, acc;
            uint32_t runs = 0;
            bool ok = true;
            auto take = [&] {  // the next accumulator, once it has been read out
                if (runs >= 2 && !role_wait(&s.acc_empty[acc.slot], acc.phase ^ 1u, &s.abort, a.status)) return false;
                acc_fence_after();
                ++runs;
                return true;
            };
            for (int item = unit; ok && item < items; item += units) {
                const At w = find(item);
                if (k0 == k1) continue;
                const uint32_t id = a.id | ((uint32_t)((w.n + 15) / 16 * 2) << 17);
                if (!F8 && !take()) break;
                for (int k = k0; k < k1; ++k) {
                    if (F8 && !take()) {
                        ok = false;
                        break;
                    }
                    if (!role_wait(&s.full[t.slot], t.phase, &s.abort, a.status)) {
                        ok = false;
                        break;
                    }
                    acc_fence_after();
                    const uint32_t at = smem_u32(ring) + t.slot * kStage, d = tmem + acc.slot * BT;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        umma<F8, false>(d, MN ? operand_mn(at + j * 2048, kTall / 2) : operand_k(at + j * 32),
                                        operand_k(at + kTall + j * 32), id, j != 0 || (!F8 && k != k0));
                    umma_done<false>(&s.empty[t.slot]);
                    t.next(stages);
                    if (F8) {
                        umma_done<false>(&s.acc_full[acc.slot]);
                        acc.next(2);
                    }
                }
                if (!F8 && ok) {
                    umma_done<false>(&s.acc_full[acc.slot]);
                    acc.next(2);
                }
            }
            // every product issued has completed before the tensor memory is given back
            umma_done<false>(&s.done);
            mbar_wait_bounded(smem_u32(&s.done), 0);
        }
    } else {
        const int q = warp & 3, thread = (warp - 2) * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
        const int G = (a.steps * kStep) / 128;  // e4m3: scales of a row
        Turn acc, box;
        uint32_t sent = 0;
        bool ok = true, waited = false;
        for (int item = unit; ok && item < items; item += units) {
            const At w = find(item);
            const int f = w.f0 + q * 32 + lane;
            float sum[F8 ? BT : 32];
            if constexpr (F8) {
#pragma unroll
                for (int c = 0; c < BT; ++c) sum[c] = 0.0f;
                const float *sb = a.sb + ((int64_t)w.e * a.ftiles + w.f0 / 128) * G;
                // this warp's copy of the rows' factors; the next block's are on their way meanwhile
                float fa[BT / 32], fb = 0.0f;
                auto fetch = [&](int k) {
                    if (k >= k1) return;
                    fb = __ldg(sb + k);
#pragma unroll
                    for (int i = 0; i < BT / 32; ++i) {
                        const int t = i * 32 + lane;
                        const int64_t row = w.row + (t < w.n ? t : 0);
                        fa[i] = __ldg(a.sa + (a.group ? row * G + k : row));
                    }
                };
                fetch(k0);
                for (int k = k0; k < k1; ++k) {
                    float *factor = s.scale[q][k & 1];
#pragma unroll
                    for (int i = 0; i < BT / 32; ++i) factor[i * 32 + lane] = fa[i] * fb;
                    fetch(k + 1);
                    __syncwarp();
                    ok = __all_sync(0xffffffffu, role_wait(&s.acc_full[acc.slot], acc.phase, &s.abort, a.status));
                    if (!ok) break;
                    acc_fence_after();
#pragma unroll
                    for (int c0 = 0; c0 < BT; c0 += 32) {
                        if (c0 < w.n) {
                            float v[32];
                            acc_load32(lanes + acc.slot * BT + c0, v);
                            acc_load_wait(v);
#pragma unroll
                            for (int c = 0; c < 32; c += 4) {
                                const float4 m = *reinterpret_cast<const float4 *>(factor + c0 + c);
                                sum[c0 + c] = __fmaf_rn(v[c], m.x, sum[c0 + c]);
                                sum[c0 + c + 1] = __fmaf_rn(v[c + 1], m.y, sum[c0 + c + 1]);
                                sum[c0 + c + 2] = __fmaf_rn(v[c + 2], m.z, sum[c0 + c + 2]);
                                sum[c0 + c + 3] = __fmaf_rn(v[c + 3], m.w, sum[c0 + c + 3]);
                            }
                        }
                    }
                    acc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s.acc_empty[acc.slot]);
                    acc.next(2);
                }
                if (!ok) break;
            } else if (k0 < k1) {
                ok = __all_sync(0xffffffffu, role_wait(&s.acc_full[acc.slot], acc.phase, &s.abort, a.status));
                if (!ok) break;
                acc_fence_after();
            }
            if (!waited) {
                pdl_wait();
                waited = true;
            }
            // with S > 1: this item's inbox expects the rows this CTA owns, from every rank
            const int share = (w.n + S - 1) / S, own0 = rank * share;
            const int own = own0 < w.n ? (w.n - own0 < share ? w.n - own0 : share) : 0;
            if (S > 1) {
                if (thread == 0) mbar_expect(&s.inbox_full, (uint32_t)(S * own) * 512u);
                if (sent > 0) {
                    ok = __all_sync(0xffffffffu, role_wait<true>(&s.inbox_free, box.phase ^ 1u, &s.abort, a.status));
                    if (!ok) break;
                }
            }
#pragma unroll
            for (int c0 = 0; c0 < BT; c0 += 32) {
                if (c0 >= w.n) break;
                float v[32];
                if constexpr (F8) {
#pragma unroll
                    for (int c = 0; c < 32; ++c) v[c] = sum[c0 + c];
                } else if (k0 < k1) {
                    acc_load32(lanes + acc.slot * BT + c0, v);
                    acc_load_wait(v);
                } else {
#pragma unroll
                    for (int c = 0; c < 32; ++c) v[c] = 0.0f;
                }
                if (S == 1) {
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (c0 + c < w.n && f < a.F) store_one(a.out, (int64_t)(w.row + c0 + c) * a.ldo + f, a.otype, v[c]);
                } else {
                    int to = c0 / share, at = c0 - to * share;  // owner of row c0 + c, and its place there
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        if (c0 + c < w.n) {
                            const uint32_t dst = smem_u32(inbox + ((size_t)rank * (BT / S) + at) * 128 + q * 32 + lane);
                            asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(
                                             cluster_addr(dst, (uint32_t)to)),
                                         "r"(as_u(v[c])), "r"(cluster_addr(smem_u32(&s.inbox_full), (uint32_t)to))
                                         : "memory");
                            if (++at == share) {
                                at = 0;
                                ++to;
                            }
                        }
                    }
                }
            }
            if (!F8 && k0 < k1) {
                acc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.acc_empty[acc.slot]);
                acc.next(2);
            }
            if (S > 1) {
                ok = __all_sync(0xffffffffu, role_wait<true>(&s.inbox_full, box.phase, &s.abort, a.status));
                if (!ok) break;
                for (int c = 0; c < own; ++c) {
                    float v = 0.0f;
                    for (int r = 0; r < S; ++r) v += inbox[((size_t)r * (BT / S) + c) * 128 + q * 32 + lane];
                    if (f < a.F) store_one(a.out, (int64_t)(w.row + own0 + c) * a.ldo + f, a.otype, v);
                }
                __syncwarp();
                if (lane < S) mbar_arrive_cluster(cluster_addr(smem_u32(&s.inbox_free), (uint32_t)lane));
                box.phase ^= 1u;
                ++sent;
            }
        }
    }
    pdl_wait();
    acc_fence_before();
    __syncthreads();
    if (S > 1) cluster_sync();  // no peer still writes to this inbox or signals these barriers
    if (warp == 1) {
        __syncwarp();
        acc_fence_after();
        acc_free<false>(tmem, 2 * BT);
    }
}

// Clusters of S that can be resident at once, for this kernel and its shared memory.
struct Fit {
    const void *kernel;
    int S, clusters;
};
std::mutex g_fit_mu;
Fit g_fit[kMaxDevices][64];

tm_status clusters_that_fit(const void *k, int S, size_t smem, int *clusters)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return TM_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_fit_mu);
    Fit *free_slot = nullptr;
    for (Fit &f : g_fit[dev]) {
        if (f.kernel == k && f.S == S) {
            *clusters = f.clusters;
            return TM_OK;
        }
        if (f.kernel == nullptr) {
            free_slot = &f;
            break;
        }
    }
    // the instance's most, whatever S: set before any launch of it
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) {
        cudaGetLastError();
        return TM_ERR_CUDA;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)S);
    cfg.blockDim = dim3(kThreadsThin);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)S;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        return TM_ERR_CUDA;
    }
    if (free_slot != nullptr) *free_slot = {k, S, n};
    *clusters = n;
    return TM_OK;
}

// Static shared memory is at most 14 KB; ring and inbox take the rest of 227 KB.
constexpr size_t kThinSmem = 208 * 1024;

template <bool F8, bool MN, int BT>
tm_status launch_thin(const Product &p, const DevInfo &dev, cudaStream_t s, bool pdl)
{
    static_assert(sizeof(ThinSmem<BT>) + kThinSmem <= 227 * 1024, "shared memory");
    constexpr size_t kStage = kTall + BT * 128, kInbox = BT * 128 * 4;
    const void *k = (const void *)thin_kernel<F8, MN, BT>;
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
    // tiles: at least one for each expert that has rows (how many have is not known here)
    const int64_t busy = p.E < p.T ? p.E : p.T, rt = (p.T + BT - 1) / BT;
    const int64_t tiles = (rt > busy ? rt : busy) * a.ftiles, most = (rt + busy) * a.ftiles;
    if (most > (1 << 30)) return TM_ERR_UNSUPPORTED_TILE;
    // S CTAs a tile: the rounds of tiles times a round's length, in stages; a round costs
    // about 4 stages that nothing hides, a join 3 more
    int S = 1;
    int64_t best = INT64_MAX;
    for (int c = 1; c <= 8 && c <= BT / 4; c *= 2) {
        if (c > 1 && a.steps < 2 * c) break;
        const int64_t rounds = (tiles + dev.sms / c - 1) / (dev.sms / c);
        const int64_t cost = rounds * ((a.steps + c - 1) / c) + 4 + (c > 1 ? 3 * rounds : 0);
        if (cost < best) best = cost, S = c;
    }
    int clusters = 0;
    const tm_status st = clusters_that_fit(k, S, kThinSmem, &clusters);
    if (st != TM_OK) return st;
    a.stages = (int)((kThinSmem - 1024 - (S > 1 ? kInbox : 0)) / kStage);
    if (a.stages > kMaxStages) a.stages = kMaxStages;
    CUtensorMap mw, mx;
    if (!rows_map(&mw, p.kind, p.w, MN ? p.F : p.R, MN ? p.R : p.F, p.ldw, p.E, MN ? 64 : 128) ||
        !rows_map(&mx, p.kind, p.x, p.R, p.T, p.ldx, 0, 16))
        return TM_ERR_CUDA;
    const int64_t grid = (most < clusters ? most : clusters) * S;
    void *args[] = {&mw, &mx, &a, &S};
    return launch_kernel(k, dim3((unsigned)grid), dim3(kThreadsThin), args, kThinSmem, s, pdl, (unsigned)S);
}

}  // namespace

tm_status thin_product(const Product &p, const DevInfo &dev, cudaStream_t s, bool pdl)
{
    const bool few = p.T <= 32 * (int64_t)p.E;
    if (p.kind == kProductE4M3)
        return few ? launch_thin<true, false, 32>(p, dev, s, pdl) : launch_thin<true, false, 128>(p, dev, s, pdl);
    if (p.w_mn) return few ? launch_thin<false, true, 32>(p, dev, s, pdl) : launch_thin<false, true, 128>(p, dev, s, pdl);
    return few ? launch_thin<false, false, 32>(p, dev, s, pdl) : launch_thin<false, false, 128>(p, dev, s, pdl);
}

}  // namespace libtm
