// tm_wide8.cu -- the 8-bit product for experts with many rows:
//
//   c[t, n] = sum_b sa[t, b] sb[n / 128, b] * sum_{k in b} a[t, k] b[n, k]
//
// A CTA pair takes a tile of 256 rows t by 256 columns n (128 where that leaves SMs without a tile), or a CTA
// one of 128 by 128 where experts have few rows; a stage of the ring is one block of 128 of the sum, up to 16 KB of
// each operand a CTA.  Rows lie along the tensor memory's lanes
// here: then a block's two scales are one factor a thread (its row's, times that of the 128
// columns the thread holds), and adding a block is one packed fp32 operation for two
// outputs.  The tensor cores make a block's sums in one accumulator of 256 columns while
// eight warps read the other, multiply and add: 128 sums a thread, in registers.  That
// addition is what the kernel must keep up with: 256 by 256 by 128 takes the tensor cores
// about 512 cycles, and a CTA's share of it 128 x 256 reads and additions, 256 cycles each at best.  8192 x 8192 x
// 4096: 220 us, 2.5 PFLOP/s; products and copies without the additions take 174 to 181.
//
// Outputs leave through shared memory: whole warps' rows by TMA, so that the warps are back
// at the next tile's sums early; rows that another expert's follow, or outputs off TMA's 16-byte
// grid, by rows (stored by each thread from its own registers, 1001 rows of 1000 columns in fp32 took 15 us).
#include <mutex>

#include "tm_products.h"
#include "tm_umma.cuh"

namespace libtm {
namespace {

constexpr int kThreads8 = 384;  // warp 0 copies, 1 products, 2-3 none, 4-11 sums and outputs
constexpr int kStages8 = 4;
constexpr uint32_t kHalf8 = 128 * 128;
constexpr uint32_t kStage8 = 2 * kHalf8;
constexpr int kGroup8 = 8;                 // row tiles that run at the same time, for the sake of L2
constexpr uint32_t kOutWarp = 2 * 32 * 128;  // a warp's outputs on their way: 32 rows of two pieces of 128 bytes
// 384 threads start with 168 registers each: 64512.  4 warps of 120 and 8 of 184 are 62464.
constexpr int kFewRegs = 120, kManyRegs = 184;

struct Wide8Args {
    void *out;
    int64_t ldo;
    const int32_t *starts;
    const float *sa, *sb;
    unsigned *status;
    int E, T, N, ntiles, steps, group;
    int by_copy;  // outputs on a grid TMA can store to
    uint32_t id;
};

struct Wide8Smem {
    alignas(8) uint64_t full[kStages8], empty[kStages8], acc_full[2], acc_empty[2], done;
    uint32_t tmem;
    int abort;
    Experts x;
};

struct Tile8 {
    int e, row, n, n0;  // expert, first row and how many, first column
};

template <int RT, int NT>
struct Walk8 {
    const Wide8Args &a;
    const Experts &x;
    int e = 0;
    __device__ Walk8(const Wide8Args &args, const Experts &experts) : a(args), x(experts) {}
    __device__ Tile8 at(int item)
    {
        while ((int64_t)x.before[e + 1] * a.ntiles <= item) ++e;
        const int tiles = x.before[e + 1] - x.before[e], local = item - x.before[e] * a.ntiles;
        const int block = local / (kGroup8 * a.ntiles), in = local - block * kGroup8 * a.ntiles;
        const int wide = tiles - block * kGroup8 < kGroup8 ? tiles - block * kGroup8 : kGroup8;
        const int r = (block * kGroup8 + in % wide) * RT, left = x.count[e] - r;
        return {e, x.first[e] + r, left < RT ? left : RT, in / wide * NT};
    }
};

// Staged rows to where another expert's rows follow, or off the copies' grid: two rows of 256 bytes at once on
// the grid, else row by row, neighbours by neighbours.  Out of line: what the sums' loop has for registers is not to depend
// on it.  (64 experts of 2048 x 4096 with 47 rows each, element by element: 152 us, so 131.)
template <int E>
__device__ __noinline__ void rows_out(const unsigned char *staged, void *out, int64_t ldo, int rows, int cols, bool on_grid)
{
    auto from = [&](int i, int at) { return staged + (at >> 7) * (kOutWarp / 2) + i * 128 + ((at >> 4 & 7) ^ (i & 7)) * 16 + (at & 15); };
    const int lane = threadIdx.x & 31;
    if (on_grid) {
        const int at = (lane & 15) * 16;
        if (at >= cols * E) return;
#pragma unroll 2
        for (int i = lane >> 4; i < rows; i += 2)
            *reinterpret_cast<uint4 *>(reinterpret_cast<char *>(out) + i * ldo * E + at) = *reinterpret_cast<const uint4 *>(from(i, at));
        return;
    }
    for (int c = lane; c < 256 / E && c < cols; c += 32)
#pragma unroll 2
        for (int i = 0; i < rows; ++i) {
            if constexpr (E == 4)
                reinterpret_cast<uint32_t *>(out)[i * ldo + c] = *reinterpret_cast<const uint32_t *>(from(i, c * E));
            else
                reinterpret_cast<uint16_t *>(out)[i * ldo + c] = *reinterpret_cast<const uint16_t *>(from(i, c * E));
        }
}

// NT: columns of a tile, 256 or 128.  PAIR: two CTAs a tile of 256 rows; else one a tile of 128 (by 128).
template <typename O, int NT, bool PAIR>
__global__ void __launch_bounds__(kThreads8, 1)
    wide8_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                 const __grid_constant__ CUtensorMap mc, const Wide8Args a)
{
    extern __shared__ __align__(1024) unsigned char raw[];
    unsigned char *ring = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    unsigned char *outs = ring + kStages8 * kStage8;
    __shared__ Wide8Smem s;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    static_assert(PAIR || NT == 128, "a stage holds 128 rows of each operand");
    constexpr int C = PAIR ? 2 : 1, BR = NT / C;  // CTAs a tile; a CTA's rows of b
    const uint32_t rank = PAIR ? cluster_rank() : 0;
    const int unit = (int)blockIdx.x / C, units = (int)gridDim.x / C;

    if (warp == 1) acc_alloc<PAIR>(&s.tmem, 512);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages8; ++i) {
            mbar_init(&s.full[i], C);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.acc_full[i], 1);
            mbar_init(&s.acc_empty[i], 8 * C);
        }
        mbar_init(&s.done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        s.abort = 0;
    }
    experts_read(s.x, a.starts, a.E, a.T, 128 * C, a.status);
    acc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();
    acc_fence_after();
    pdl_trigger();  // only now: a dependent's CTA could take the tensor memory that this one waits for
    const uint32_t tmem = s.tmem;
    const int items = s.x.before[a.E] * a.ntiles;
    Walk8<128 * C, NT> walk(a, s.x);

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
        if (warp == 0) {
            // one row tile an expert: its weights are read once
            const uint64_t pol = PAIR ? 0 : l2_evict_first_policy();
            Turn t;
            uint32_t used = 0;
            bool ok = true;
            for (int item = unit; ok && item < items; item += units) {
                const Tile8 w = walk.at(item);
                const int row = w.row + (int)rank * 128, n = w.n0 + (int)rank * BR;
                for (int k = 0; k < a.steps; ++k) {
                    if (used >= kStages8 && !warp_wait(&s.empty[t.slot], t.phase ^ 1u, &s.abort, a.status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t at = smem_u32(ring) + t.slot * kStage8, bar = cluster_addr(smem_u32(&s.full[t.slot]), 0);
                    if (elect()) {
                        mbar_expect_cluster(bar, kHalf8 + BR * 128);
                        if constexpr (PAIR) {
                            tma_load_2d_pair(at, &ma, k * 128, row, bar);
                            tma_load_3d_pair(at + kHalf8, &mb, k * 128, n, w.e, bar);
                        } else {
                            tma_load_2d(at, &ma, k * 128, row, smem_u32(&s.full[t.slot]));
                            tma_load_3d_hint(at + kHalf8, &mb, k * 128, n, w.e, smem_u32(&s.full[t.slot]), pol);
                        }
                    }
                    __syncwarp();
                    ++used;
                    t.next(kStages8);
                }
            }
            // nothing may still be landing when the pair leaves: the last filling of each slot
            if (rank == 0)
                for (uint32_t i = 0; i < (uint32_t)kStages8 && i < used; ++i)
                    mbar_wait_bounded(smem_u32(&s.full[i]), ((used - i + kStages8 - 1) / kStages8 - 1) & 1u);
        } else if (warp == 1 && rank == 0) {
            Turn t, acc;
            uint32_t runs = 0;
            bool ok = true;
            for (int item = unit; ok && item < items; item += units) {
                for (int k = 0; k < a.steps; ++k) {
                    if ((runs >= 2 && !warp_wait(&s.acc_empty[acc.slot], acc.phase ^ 1u, &s.abort, a.status)) ||
                        !warp_wait(&s.full[t.slot], t.phase, &s.abort, a.status)) {
                        ok = false;
                        break;
                    }
                    ++runs;
                    acc_fence_after();
                    const uint32_t at = smem_u32(ring) + t.slot * kStage8, d = tmem + acc.slot * 256;
                    if (elect()) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            umma<true, PAIR>(d, operand_k(at + j * 32), operand_k(at + kHalf8 + j * 32), a.id, j != 0);
                        umma_done<PAIR>(&s.empty[t.slot]);
                        umma_done<PAIR>(&s.acc_full[acc.slot]);
                    }
                    __syncwarp();
                    t.next(kStages8);
                    acc.next(2);
                }
            }
            if (elect()) umma_done<PAIR>(&s.done);
            __syncwarp();
            mbar_wait_bounded(smem_u32(&s.done), 0);
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
        constexpr int CW = NT / 2;  // columns of a warp
        const int q = warp & 3, half = (warp - 4) >> 2;  // lanes 32 q .., columns CW half ..
        const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(half * CW);
        const uint32_t free0 = cluster_addr(smem_u32(&s.acc_empty[0]), 0), free1 = cluster_addr(smem_u32(&s.acc_empty[1]), 0);
        unsigned char *mine = outs + (warp - 4) * kOutWarp;
        const int NB = (a.N + 127) / 128;
        Turn acc;
        bool waited = false, ok = true;
        for (int item = unit; ok && item < items; item += units) {
            const Tile8 w = walk.at(item);
            const int r = (int)rank * 128 + q * 32 + lane;  // of the tile
            const bool live = r < w.n;
            const int64_t row = (int64_t)w.row + r;
            const int n = w.n0 + half * CW;
            const float *sa = a.sa + (live ? (a.group ? row * a.steps : row) : 0);
            const float *sb = a.sb + ((int64_t)w.e * NB + (n < a.N ? n / 128 : 0)) * a.steps;
            uint64_t sum[CW / 2];
#pragma unroll
            for (int i = 0; i < CW / 2; ++i) sum[i] = 0;
            // the next block's factors are on their way while this one is added
            float fa = a.steps > 0 ? __ldg(sa) : 0.0f, fb = a.steps > 0 ? __ldg(sb) : 0.0f;
            for (int k = 0; k < a.steps; ++k) {
                const float f = fa * fb;
                const uint64_t m = pack2(f, f);
                if (k + 1 < a.steps) {
                    fa = __ldg(sa + (a.group ? k + 1 : 0));
                    fb = __ldg(sb + k + 1);
                }
                ok = __all_sync(0xffffffffu, role_wait(&s.acc_full[acc.slot], acc.phase, &s.abort, a.status));
                if (!ok) break;
                acc_fence_after();
                const uint32_t at = lanes + acc.slot * 256;
#pragma unroll
                for (int c = 0; c < CW / 32; ++c) add_columns(at + 32 * c, sum + 16 * c, m);
                acc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(acc.slot ? free1 : free0);
                acc.next(2);
            }
            if (!ok) break;
            if (!waited) {
                pdl_wait();
                waited = true;
            }
            if (n >= a.N) continue;
            // the warp's 32 rows go through its staging rows of 256 bytes, two pieces of 128 in the copy's
            // swizzle: 128 columns in 16 bits, 64 in fp32
            const int row0 = w.row + (int)rank * 128 + q * 32, rows = w.n - ((int)rank * 128 + q * 32);
            auto room = [&] {  // the last copy has read the staging rows
                if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                __syncwarp();
            };
            auto put = [&](int i, const uint32_t(&u)[4]) {  // 16 bytes, the i-th of the lane's row
                const uint32_t at = smem_u32(mine) + (uint32_t)(i >> 3) * (kOutWarp / 2) + (uint32_t)lane * 128u +
                                    (uint32_t)(((i & 7) ^ (lane & 7)) * 16);
                asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]) : "memory");
            };
            auto out = [&](int first) {  // columns first .. from the staging rows
                constexpr int e = sizeof(O);
                if (a.by_copy && rows >= 32) {
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) {
#pragma unroll
                        for (int p = 0; p < (CW * e > 128 ? 2 : 1); ++p)
                            if (first + p * (128 / e) < a.N)
                                asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(&mc),
                                             "r"(first + p * (128 / e)), "r"(row0), "r"(smem_u32(mine) + (uint32_t)p * (kOutWarp / 2))
                                             : "memory");
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    }
                    __syncwarp();
                    return;
                }
                __syncwarp();
                rows_out<sizeof(O)>(mine, reinterpret_cast<O *>(a.out) + (int64_t)row0 * a.ldo + first, a.ldo, rows < 32 ? rows : 32,
                                    a.N - first < CW ? a.N - first : CW, a.by_copy != 0);
                __syncwarp();
            };
            if (rows <= 0) continue;
            if constexpr (sizeof(O) == 4) {
#pragma unroll
                for (int half64 = 0; half64 < CW / 64; ++half64) {
                    if (n + 64 * half64 >= a.N) break;
                    room();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float v[4];
                        unpack2(sum[32 * half64 + 2 * i], v[0], v[1]);
                        unpack2(sum[32 * half64 + 2 * i + 1], v[2], v[3]);
                        const uint32_t u[4] = {as_u(v[0]), as_u(v[1]), as_u(v[2]), as_u(v[3])};
                        put(i, u);
                    }
                    out(n + 64 * half64);
                }
            } else {
                room();
#pragma unroll
                for (int i = 0; i < CW / 8; ++i) {
                    uint32_t u[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float lo, hi;
                        unpack2(sum[4 * i + j], lo, hi);
                        if constexpr (std::is_same<O, __half>::value)
                            asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(u[j]) : "f"(hi), "f"(lo));
                        else
                            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u[j]) : "f"(hi), "f"(lo));
                    }
                    put(i, u);
                }
                out(n);
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }
    pdl_wait();
    acc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();
    if (warp == 1) {
        __syncwarp();
        acc_fence_after();
        acc_free<PAIR>(tmem, 512);
    }
}

constexpr size_t kWide8Smem = kStages8 * kStage8 + 8 * kOutWarp + 1024;

template <typename O, int NT, bool PAIR>
tm_status launch_wide8_as(const CUtensorMap &ma, const CUtensorMap &mb, const CUtensorMap &mc, const Wide8Args &a, int64_t units,
                       cudaStream_t s, bool pdl)
{
    const void *k = (const void *)wide8_kernel<O, NT, PAIR>;
    static std::once_flag once[kMaxDevices];
    static bool good[kMaxDevices];
    int d = 0;
    if (cudaGetDevice(&d) != cudaSuccess || d < 0 || d >= kMaxDevices) return TM_ERR_CUDA;
    std::call_once(once[d], [&] {
        good[d] = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kWide8Smem) == cudaSuccess;
        if (!good[d]) cudaGetLastError();
    });
    if (!good[d]) return TM_ERR_CUDA;
    void *args[] = {const_cast<CUtensorMap *>(&ma), const_cast<CUtensorMap *>(&mb), const_cast<CUtensorMap *>(&mc),
                    const_cast<Wide8Args *>(&a)};
    return launch_kernel(k, dim3((unsigned)(units * (PAIR ? 2 : 1))), dim3(kThreads8), args, kWide8Smem, s, pdl, PAIR ? 2 : 1);
}

template <typename O>
tm_status launch_wide8(const CUtensorMap &ma, const CUtensorMap &mb, const CUtensorMap &mc, const Wide8Args &a, int nt, bool pair, int64_t units,
                       cudaStream_t s, bool pdl)
{
    if (!pair) return launch_wide8_as<O, 128, false>(ma, mb, mc, a, units, s, pdl);
    return nt == 256 ? launch_wide8_as<O, 256, true>(ma, mb, mc, a, units, s, pdl) : launch_wide8_as<O, 128, true>(ma, mb, mc, a, units, s, pdl);
}

}  // namespace

tm_status wide8_product(const Product &p, const DevInfo &dev, cudaStream_t s, bool pdl)
{
    Wide8Args a = {};
    a.out = p.out;
    a.ldo = p.ldo;
    a.starts = p.starts;
    a.sa = p.sa;
    a.sb = p.sb;
    a.status = dev.status;
    a.E = p.E;
    a.T = (int)p.T;
    a.N = (int)p.F;
    // a tile a CTA where experts have 128 rows on average (64 experts of 2048 x 4096, 64 rows each: 129 us by pairs,
    // 111 so; 8 of 4096 x 4096, 100 rows each: 47 and 37; 64 of 2048 x 2048 with uneven rows, 128 on average: 75
    // and 80; all 8192 rows one expert's: 43 and 55).  Else narrow tiles where all of them run at once, on SMs that
    // would have nothing to do (one of 4096 x 4096, 512 rows: 24.6 us with 256 columns and 20.5 with 128; 1000 rows of
    // 2048 x 7168: 34.8 and 28.7).
    const bool pair = p.T > 128 * (int64_t)p.E;
    const int64_t busy = p.E < p.T ? p.E : p.T, rt = pair ? 256 : 128, rtiles = (p.T + rt - 1) / rt + busy;
    const int64_t at_once = pair ? dev.sms / 2 : dev.sms;
    const int nt = !pair || tiles_of(p, 256) * ((p.F + 127) / 128) <= at_once ? 128 : 256;
    a.ntiles = (int)((p.F + nt - 1) / nt);
    a.steps = (int)((p.R + 127) / 128);
    a.group = p.group;
    a.id = instruction(0, false, false, (uint32_t)rt, (uint32_t)nt);
    // TMA clips what it stores at whole 16 bytes: N must end on them
    const int eo = elem_bytes(p.otype), grid = 16 / eo;
    a.by_copy = aligned_to(p.out, 16) && p.ldo % grid == 0 && p.F % grid == 0;
    CUtensorMap ma, mb, mc;
    if (!rows_map(&ma, p.kind, p.x, p.R, p.T, p.ldx, 0, 128) ||
        !rows_map(&mb, p.kind, p.w, p.R, p.F, p.ldw, p.E, pair ? nt / 2 : nt))
        return TM_ERR_CUDA;
    if (a.by_copy ? !rows_map_of(&mc, eo, p.out, p.F, p.T, p.ldo, 0, 32) : (mc = ma, false)) return TM_ERR_CUDA;
    const int64_t items = rtiles * a.ntiles;
    if (items > (1 << 30)) return TM_ERR_UNSUPPORTED_TILE;
    const int64_t units = items < at_once ? items : at_once;
    if (p.otype == TM_F32) return launch_wide8<float>(ma, mb, mc, a, nt, pair, units, s, pdl);
    if (p.otype == TM_F16) return launch_wide8<__half>(ma, mb, mc, a, nt, pair, units, s, pdl);
    return launch_wide8<__nv_bfloat16>(ma, mb, mc, a, nt, pair, units, s, pdl);
}

}  // namespace libtm
