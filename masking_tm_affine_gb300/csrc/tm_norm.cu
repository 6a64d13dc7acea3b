// tm_norm.cu -- root-mean-square norm of rows, with the residual's addition
// before it and an optional 8-bit output with scales, and its gradient.
//
//   h = x + r,   s = 1 / sqrt(mean_j h_j^2 + eps),   y_j = h_j s w_j
//   e4m3 output: scale_g = max_{j in g} |y_j| / 448, code_j = e4m3(y_j / scale_g)
//
//   n = h s,  c = mean_j dy_j w_j n_j
//   dx_j = s (dy_j w_j - n_j c) + dr_j,   dw_j = sum_rows dy_j n_j
//
// Both are bound by HBM (about 5 and 10 flops per element of 4 to 8 bytes
// moved), so a row is read once and lives in registers between its statistics
// and its output: L lanes share it (a power of two, 8 lanes up to a block of
// 1024), each holding K vectors of EW elements.
//
// Two forms.  Few rows, rows off the 16-byte grid, very short and very long ones:
// a block a row (or several short rows), straight from memory.  Many rows: as many
// blocks as the GPU holds walk them, each with a ring of row copies (bulk copies of
// one row of one tensor) in flight ahead of the row it works on; in the first form a
// block's loads, reduction and stores follow one another and too few rows fit an SM
// to cover that.  Lane l's k-th vector is
// (w K + k) 32 + l of the row (w the warp within the row): every access of a
// warp is one run of 512 bytes, and a scale group of 32, 64 or 128 columns is a
// run of lanes of one warp (or, with single elements, of one lane's registers).
// All sums are fp32, in a fixed order.
//
// Measured, bf16: 8192 x 8192 with a residual to e4m3 by 128 columns 82 us, 85% of the
// rate of a copy of the same bytes; 8192 x 4096 with a residual, both directions, 97 us,
// 81%; 32 x 4096 to e4m3 3.1 us on the device.
#include "tm_host.h"

#include <cuda_fp8.h>

#include <atomic>

#include "tm_elem.cuh"

namespace libtm {
namespace {

constexpr int kMaxCols = 32768;  // what a block of 1024 lanes holds in registers

// Largest block an instance of the norm and of its gradient is launched with (see
// pick_lanes).
template <int EW, int K>
constexpr int kNormLanes = (EW == 1 && K > 8) || (EW == 4 && K >= 4) ? 1024 : 512;
template <int EW, int K>
constexpr int kGradLanes = (EW == 1 && K > 8) || (EW == 4 && K > 4) ? 1024 : 512;

// Sum over the L lanes of a row.  L > 32: through shared memory, warps added
// in order, one barrier per call (the caller alternates between two buffers,
// so a second call cannot overwrite what a slow warp still reads).
__device__ __forceinline__ float row_sum(float x, int L, float *buf)
{
    x = lanes_sum(x, L < 32 ? L : 32);
    if (L > 32) {
        const int warp = threadIdx.x >> 5, W = L >> 5, base = warp / W * W;
        if ((threadIdx.x & 31) == 0) buf[warp] = x;
        __syncthreads();
        x = buf[base];
        for (int w = 1; w < W; ++w) x += buf[base + w];
    }
    return x;
}

__device__ __forceinline__ float row_max(float x, int L, float *buf)
{
    x = lanes_max(x, L < 32 ? L : 32);
    if (L > 32) {
        const int warp = threadIdx.x >> 5, W = L >> 5, base = warp / W * W;
        if ((threadIdx.x & 31) == 0) buf[warp] = x;
        __syncthreads();
        x = buf[base];
        for (int w = 1; w < W; ++w) x = fmaxf(x, buf[base + w]);
    }
    return x;
}

// A lane's first column; its k-th vector is k * 32 * EW columns on (rows of fewer
// than 32 lanes have one vector a lane).
template <int EW, int K>
__device__ __forceinline__ int first_column(int ln)
{
    return K == 1 ? ln * EW : ((ln >> 5) * K * 32 + (ln & 31)) * EW;
}

// A lane's vectors of a row from p (its first), zeros past the end: `left` columns
// from there.
template <typename T, int EW, int K>
__device__ __forceinline__ void load_row(const T *p, int left, Vec<T, EW> (&v)[K])
{
#pragma unroll
    for (int k = 0; k < K; ++k) load_vec_if(p + k * 32 * EW, k * 32 * EW < left, v[k]);
}

// A lane's weights, ones if there are none.
template <typename WT, int EW, int K>
__device__ __forceinline__ void load_weights(const void *W, int j0, int left, Vec<WT, EW> (&v)[K])
{
    if (W != nullptr) {
        load_row<WT, EW, K>(reinterpret_cast<const WT *>(W) + j0, left, v);
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < EW; ++e) v[k].v[e] = from_f<WT>(1.0f);
    }
}

template <typename T, int EW>
__device__ __forceinline__ void store_row_vec(T *p, int k, int left, const float (&f)[EW])
{
    Vec<T, EW> o;
    narrow(f, o);
    store_vec_if(p + k * 32 * EW, k * 32 * EW < left, o);
}

template <int EW>
__device__ __forceinline__ void store_e4m3(uint8_t *p, bool ok, const float (&y)[EW])
{
    if constexpr (EW == 1) {
        if (ok) *p = __nv_cvt_float_to_fp8(y[0], __NV_SATFINITE, __NV_E4M3);
    } else {
        Vec<uint8_t, EW> o;
#pragma unroll
        for (int e = 0; e < EW; e += 2) {
            const uint16_t c = __nv_cvt_float2_to_fp8x2(make_float2(y[e], y[e + 1]), __NV_SATFINITE, __NV_E4M3);
            *reinterpret_cast<uint16_t *>(&o.v[e]) = c;
        }
        store_vec_if(p, ok, o);
    }
}

struct NormArgs {
    const void *X, *R, *W;
    void *H, *Y;
    float *scales, *rstd;
    int64_t ldx, ldr, ldh, ldy, M;
    int N, L, group, group_log;
    float eps, inv_n;
    unsigned *status;
};

// What maps a largest magnitude of `top` (of h w) to 448, and what a code of 1 then
// stands for (s = 1 / rms).  448 / top passes fp32's range below 2^-119: values of a group
// below kTiny are lifted by 2^100 first (lift_tiny), and the factor is that of the lifted ones.
constexpr float kTiny = 0x1p-100f, kLift = 0x1p100f;
__device__ __forceinline__ float e4m3_factor(float top)
{
    return top > 0.0f ? 448.0f / (top < kTiny ? top * kLift : top) : 1.0f;
}
__device__ __forceinline__ float e4m3_scale(float top, float s) { return top > 0.0f ? top * s * (1.0f / 448.0f) : 1.0f; }

// By whole warps: one vote a row, next to always with no such group.
template <int EW, int K>
__device__ __forceinline__ void lift_tiny(const float (&top)[K], float (&h)[K][EW])
{
    bool tiny = false;
#pragma unroll
    for (int k = 0; k < K; ++k) tiny = tiny || (top[k] > 0.0f && top[k] < kTiny);
    if (!__any_sync(0xffffffffu, tiny)) return;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < EW; ++e) h[k][e] *= top[k] < kTiny ? kLift : 1.0f;
}

// What follows a row's sum: 1 / rms, h, y.  `h` is overwritten.
template <typename T, typename WT, int EW, int K, bool E4M3>
__device__ __forceinline__ void finish_row(const NormArgs &a, int64_t row, bool live, int ln, int j0, int left, float ss,
                                           float (&h)[K][EW], const Vec<WT, EW> (&w)[K], float *buf)
{
    const float s = rsqrtf(fmaf(ss, a.inv_n, a.eps));
    if (live && a.rstd && ln == 0) a.rstd[row] = s;
    if (a.H) {
        T *out = reinterpret_cast<T *>(a.H) + row * a.ldh + j0;
#pragma unroll
        for (int k = 0; k < K; ++k) store_row_vec<T, EW>(out, k, left, h[k]);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float f[EW];
        widen(w[k], f);
#pragma unroll
        for (int e = 0; e < EW; ++e) h[k][e] *= f[e];
    }
    if constexpr (!E4M3) {
        T *out = reinterpret_cast<T *>(a.Y) + row * a.ldy + j0;
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int e = 0; e < EW; ++e) h[k][e] *= s;
            store_row_vec<T, EW>(out, k, left, h[k]);
        }
    } else {
        // codes are h w 448 / max|h w|: 1 / rms cancels, and enters the scale alone
        uint8_t *out = reinterpret_cast<uint8_t *>(a.Y) + row * a.ldy + j0;
        float top[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            top[k] = 0.0f;
#pragma unroll
            for (int e = 0; e < EW; ++e) top[k] = fmaxf(top[k], fabsf(h[k][e]));
        }
        if (a.group == 0) {
            float t = 0.0f;
#pragma unroll
            for (int k = 0; k < K; ++k) t = fmaxf(t, top[k]);
            t = row_max(t, a.L, buf);
            if (live && ln == 0) a.scales[row] = e4m3_scale(t, s);
#pragma unroll
            for (int k = 0; k < K; ++k) top[k] = t;
        } else {
            // a group is group / EW lanes of one k (EW > 1), or all 32 lanes of group / 32
            // consecutive k (EW = 1)
            const int64_t ng = (a.N + a.group - 1) >> a.group_log;
            float *scales = a.scales + row * ng;
            if constexpr (EW > 1) {
                const int lanes = a.group / EW;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    top[k] = lanes_max(top[k], lanes);
                    if (k * 32 * EW < left && (ln & (lanes - 1)) == 0)
                        scales[(j0 + k * 32 * EW) >> a.group_log] = e4m3_scale(top[k], s);
                }
            } else {
                float m[K];
#pragma unroll
                for (int k = 0; k < K; ++k) m[k] = lanes_max(top[k], 32);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    float t = 0.0f;
#pragma unroll
                    for (int q = 0; q < K; ++q)
                        if (q >> (a.group_log - 5) == k >> (a.group_log - 5)) t = fmaxf(t, m[q]);
                    const int j = j0 + k * 32;
                    if (k * 32 < left && (j & (a.group - 1)) == 0) scales[j >> a.group_log] = e4m3_scale(t, s);
                    top[k] = t;
                }
            }
        }
        lift_tiny<EW, K>(top, h);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float f = e4m3_factor(top[k]);
#pragma unroll
            for (int e = 0; e < EW; ++e) h[k][e] *= f;
            store_e4m3<EW>(out + k * 32 * EW, k * 32 * EW < left, h[k]);
        }
    }
}

// A row's h (x + r, or x) in fp32 and its sum of squares over this lane.
template <typename T, int EW, int K>
__device__ __forceinline__ float add_rows(const Vec<T, EW> (&x)[K], const Vec<T, EW> (&r)[K], bool two, float (&h)[K][EW])
{
    float ss = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) widen(x[k], h[k]);
    if (two) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float f[EW];
            widen(r[k], f);
#pragma unroll
            for (int e = 0; e < EW; ++e) h[k][e] += f[e];
        }
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < EW; ++e) ss = fmaf(h[k][e], h[k][e], ss);
    return ss;
}

// First form: one block per blockDim.x / L rows.
template <typename T, typename WT, int EW, int K, bool E4M3>
__global__ void __launch_bounds__(kNormLanes<EW, K>) rmsnorm_kernel(const __grid_constant__ NormArgs a)
{
    __shared__ float buf[2][32];
    pdl_trigger();
    const int L = a.L, ln = threadIdx.x & (L - 1);
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / L) + threadIdx.x / L;
    const int j0 = first_column<EW, K>(ln);
    const int left = row < a.M ? a.N - j0 : 0;  // a row past the end has no columns
    float h[K][EW], ss;
    {
        Vec<T, EW> v[K], r[K];
        load_row<T, EW, K>(reinterpret_cast<const T *>(a.X) + row * a.ldx + j0, left, v);
        if (a.R) load_row<T, EW, K>(reinterpret_cast<const T *>(a.R) + row * a.ldr + j0, left, r);
        ss = add_rows<T, EW, K>(v, r, a.R != nullptr, h);
    }
    Vec<WT, EW> w[K];
    load_weights<WT, EW, K>(a.W, j0, a.N - j0, w);
    ss = row_sum(ss, L, buf[0]);
    pdl_wait();  // loads may run ahead of the kernel before, stores may not
    finish_row<T, WT, EW, K, E4M3>(a, row, row < a.M, ln, j0, left, ss, h, w, buf[1]);
}

// ---------------------------------------------------------------- the ring of row copies
// A stage holds `slots` rows of each of `tensors` tensors, row bytes each (a multiple
// of 16).  The first slots * tensors threads issue a copy each; thread 0 announces
// the bytes.  Waits are bounded: a warp whose stage does not come marks the status word
// and stores nothing more.  A warp gives up together, and the threads that copy are one
// warp (slots * tensors <= 8 * 3): the bytes announced for a stage are those copied.
struct Ring {
    uint32_t data, bars;  // shared addresses
    uint32_t row_bytes, slots, tensors, stages;
};

__device__ __forceinline__ void ring_init(const Ring &g)
{
    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < g.stages; ++s)
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(g.bars + 8 * s) : "memory");
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncthreads();
}

// Rows r0 .. of the tensors at `base` (this thread's tensor) into stage s.
__device__ __forceinline__ void ring_issue(const Ring &g, uint32_t s, const char *base, int64_t ld_bytes, int64_t r0,
                                           int64_t M, uint64_t policy)
{
    const uint32_t bar = g.bars + 8 * s, tid = threadIdx.x;
    const int64_t rows = M - r0 < g.slots ? M - r0 : g.slots;
    if (tid == 0)
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar),
                     "r"((uint32_t)rows * g.tensors * g.row_bytes)
                     : "memory");
    if (tid < g.slots * g.tensors) {
        const uint32_t slot = tid % g.slots;
        if (slot < rows)
            asm volatile(
                "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], "
                "%4;" ::"r"(g.data + (s * g.tensors * g.slots + tid) * g.row_bytes),
                "l"(base + (r0 + slot) * ld_bytes), "r"(g.row_bytes), "r"(bar), "l"(policy)
                : "memory");
    }
}

// Let what a block has in flight land before its shared memory goes: every stage
// from `stage` on, each wait bounded.
__device__ __forceinline__ void ring_drain(const Ring &g, uint32_t stage, uint32_t phase)
{
    for (uint32_t s = 0; s < g.stages; ++s) {
        mbar_wait_bounded(g.bars + 8 * stage, phase);
        if (++stage == g.stages) {
            stage = 0;
            phase ^= 1;
        }
    }
}

// A lane's vectors of a row in a stage (shared address of its first), zeros past the end.
template <typename T, int EW, int K>
__device__ __forceinline__ void ring_row(uint32_t at, int left, Vec<T, EW> (&v)[K])
{
    static_assert(EW * sizeof(T) == 16, "vector access");
#pragma unroll
    for (int k = 0; k < K; ++k) {
        uint32_t *u = reinterpret_cast<uint32_t *>(&v[k]);
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
            "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
            "@p ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];\n\t}"
            : "=&r"(u[0]), "=&r"(u[1]), "=&r"(u[2]), "=&r"(u[3])
            : "r"(at + k * 32 * 16), "r"((uint32_t)(k * 32 * EW < left))
            : "memory");
    }
}

constexpr int kMostStages = 6;

// Second form: block b takes rows (b + i gridDim.x) slots .. for i = 0, 1, ...
template <typename T, typename WT, int EW, int K, bool E4M3>
__global__ void __launch_bounds__(512) rmsnorm_ring_kernel(const __grid_constant__ NormArgs a, int stages)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t bars[kMostStages];
    __shared__ float buf[2][2][32];
    pdl_trigger();
    const int L = a.L, ln = threadIdx.x & (L - 1), slot = threadIdx.x / L, slots = blockDim.x / L;
    const int tensors = a.R ? 2 : 1;
    const Ring g = {smem_u32(smem), smem_u32(bars), (uint32_t)(a.N * sizeof(T)), (uint32_t)slots, (uint32_t)tensors,
                    (uint32_t)stages};
    ring_init(g);
    const bool second = (int)threadIdx.x >= slots;  // which tensor this thread copies
    const char *base = reinterpret_cast<const char *>(second ? a.R : a.X);
    const int64_t ld = (second ? a.ldr : a.ldx) * (int64_t)sizeof(T);
    const uint64_t policy = l2_evict_first_policy();
    const int64_t step = (int64_t)gridDim.x * slots;
    int64_t next = (int64_t)blockIdx.x * slots;  // first row of the next copies
    for (int s = 0; s < stages && next < a.M; ++s, next += step) ring_issue(g, s, base, ld, next, a.M, policy);
    const int j0 = first_column<EW, K>(ln);
    Vec<WT, EW> w[K];
    load_weights<WT, EW, K>(a.W, j0, a.N - j0, w);
    pdl_wait();
    int stage = 0, turn = 0;
    uint32_t phase = 0;
    bool alive = true;
    for (int64_t r0 = (int64_t)blockIdx.x * slots; r0 < a.M; r0 += step) {
        alive = alive && __all_sync(0xffffffffu, mbar_wait_bounded(g.bars + 8 * stage, phase));
        const int64_t row = r0 + slot;
        const int left = row < a.M ? a.N - j0 : 0;
        float h[K][EW], ss;
        {
            Vec<T, EW> v[K], r[K];
            const uint32_t at = g.data + (stage * tensors * slots + slot) * g.row_bytes + j0 * (int)sizeof(T);
            ring_row<T, EW, K>(at, left, v);
            if (a.R) ring_row<T, EW, K>(at + slots * g.row_bytes, left, r);
            ss = add_rows<T, EW, K>(v, r, a.R != nullptr, h);
        }
        if (L > 32) {
            ss = row_sum(ss, L, buf[0][turn]);  // its barrier: every thread has read the stage
        } else {
            ss = row_sum(ss, L, nullptr);
            __syncthreads();
        }
        if (next < a.M && alive) ring_issue(g, stage, base, ld, next, a.M, policy);
        next += step;
        finish_row<T, WT, EW, K, E4M3>(a, row, alive && row < a.M, ln, j0, alive ? left : 0, ss, h, w, buf[1][turn]);
        turn ^= 1;
        if (++stage == stages) {
            stage = 0;
            phase ^= 1;
        }
    }
    if (!alive) {
        atomicOr(a.status, kStatusTimeout);
        ring_drain(g, stage, phase);
    }
}

struct NormBwdArgs {
    const void *DY, *H, *W, *DR;
    const float *rstd;
    void *DX;
    float *part;  // [gridDim.x, N]: each block's share of dw
    int64_t lddy, ldh, lddr, lddx, M;
    int N, L;
    float inv_n;
    unsigned *status;
};

// A lane's share of c = mean(dy w n) / s before the sum over lanes, and its part of dw.
template <typename T, typename WT, int EW, int K>
__device__ __forceinline__ float grad_sums(const Vec<T, EW> (&vy)[K], const Vec<T, EW> (&vh)[K], const Vec<WT, EW> (&w)[K],
                                           float s, float (&dw)[K][EW])
{
    float c = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float fy[EW], fh[EW], fw[EW];
        widen(vy[k], fy);
        widen(vh[k], fh);
        widen(w[k], fw);
#pragma unroll
        for (int e = 0; e < EW; ++e) {
            const float p = fy[e] * (fh[e] * s);
            c = fmaf(p, fw[e], c);
            dw[k][e] += p;
        }
    }
    return c;
}

// dx of a lane's vectors: s (dy w - h c) + dr, with c = mean(dy w n) s.
template <typename T, typename WT, int EW, int K>
__device__ __forceinline__ void grad_row(T *out, int left, const Vec<T, EW> (&vy)[K], const Vec<T, EW> (&vh)[K],
                                         const Vec<T, EW> (&vr)[K], bool dr, const Vec<WT, EW> (&w)[K], float s, float c)
{
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float fy[EW], fh[EW], fw[EW], o[EW];
        widen(vy[k], fy);
        widen(vh[k], fh);
        widen(w[k], fw);
#pragma unroll
        for (int e = 0; e < EW; ++e) o[e] = s * fmaf(fy[e], fw[e], -(fh[e] * c));
        if (dr) {
            float fr[EW];
            widen(vr[k], fr);
#pragma unroll
            for (int e = 0; e < EW; ++e) o[e] += fr[e];
        }
        store_row_vec<T, EW>(out, k, left, o);
    }
}

// A block's row of partial dw: the slots' registers meet in acc ([N], zeroed), in order.
template <int EW, int K>
__device__ __forceinline__ void store_dw(float *acc, float *out, int N, int slots, int slot, int j0, const float (&dw)[K][EW])
{
    for (int q = 0; q < slots; ++q) {
        if (slot == q) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int j = j0 + k * 32 * EW;
                if (j < N) {
#pragma unroll
                    for (int e = 0; e < EW; ++e) acc[j + e] += dw[k][e];
                }
            }
        }
        __syncthreads();
    }
    for (int j = threadIdx.x; j < N; j += blockDim.x) out[j] = acc[j];
}

// The gradient.  A block walks rows blockIdx.x, + gridDim.x, ... in each of its
// blockDim.x / L slots, adding dy n into its own columns' dw: in registers, or for the
// longest rows (a lane's share would not fit) in its own words of shared memory.  Its
// weights stay in registers.  At the end the slots' sums meet in shared memory and one
// row of partials goes out; a second launch adds the blocks' rows in order.
template <typename T, typename WT, int EW, int K>
__global__ void __launch_bounds__(kGradLanes<EW, K>) rmsnorm_bwd_kernel(const __grid_constant__ NormBwdArgs a)
{
    constexpr bool kRegs = EW == 1 ? K <= 8 : K <= 4;  // beyond, a row is the whole block's
    extern __shared__ float acc[];  // [N] floats, zeroed here
    __shared__ float buf[2][32];
    pdl_trigger();
    const int L = a.L, ln = threadIdx.x & (L - 1), slots = blockDim.x / L, slot = threadIdx.x / L;
    const int j0 = first_column<EW, K>(ln);
    for (int j = threadIdx.x; j < a.N; j += blockDim.x) acc[j] = 0.0f;
    float dw[K][EW];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < EW; ++e) dw[k][e] = 0.0f;
    Vec<WT, EW> w[K];
    if constexpr (kRegs) load_weights<WT, EW, K>(a.W, j0, a.N - j0, w);
    __syncthreads();
    bool wrote = false;
    int turn = 0;
    // the same number of steps for every slot: row_sum holds a barrier
    for (int64_t r0 = (int64_t)blockIdx.x * slots; r0 < a.M; r0 += (int64_t)gridDim.x * slots, turn ^= 1) {
        const int64_t row = r0 + slot;
        const int left = row < a.M ? a.N - j0 : 0;
        Vec<T, EW> vy[K], vh[K], vr[K];
        load_row<T, EW, K>(reinterpret_cast<const T *>(a.DY) + row * a.lddy + j0, left, vy);
        load_row<T, EW, K>(reinterpret_cast<const T *>(a.H) + row * a.ldh + j0, left, vh);
        if (a.DR) load_row<T, EW, K>(reinterpret_cast<const T *>(a.DR) + row * a.lddr + j0, left, vr);
        const float s = row < a.M ? a.rstd[row] : 0.0f;
        if constexpr (!kRegs) load_weights<WT, EW, K>(a.W, j0, a.N - j0, w);
        float c = grad_sums<T, WT, EW, K>(vy, vh, w, s, dw);
        if constexpr (!kRegs) {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int e = 0; e < EW; ++e) {
                    if (k * 32 * EW < left) acc[j0 + k * 32 * EW + e] += dw[k][e];
                    dw[k][e] = 0.0f;
                }
        }
        c = row_sum(c, L, buf[turn]) * a.inv_n * s;
        if (!wrote) pdl_wait();
        wrote = true;
        grad_row<T, WT, EW, K>(reinterpret_cast<T *>(a.DX) + row * a.lddx + j0, left, vy, vh, vr, a.DR != nullptr, w, s, c);
    }
    if (!wrote) pdl_wait();
    if (a.part == nullptr) return;
    float *out = a.part + (int64_t)blockIdx.x * a.N;
    if constexpr (kRegs) {
        store_dw<EW, K>(acc, out, a.N, slots, slot, j0, dw);
    } else {
        __syncthreads();
        for (int j = threadIdx.x; j < a.N; j += blockDim.x) out[j] = acc[j];
    }
}

// The same with the rows' copies in a ring ahead of the block.
template <typename T, typename WT, int EW, int K>
__global__ void __launch_bounds__(512) rmsnorm_bwd_ring_kernel(const __grid_constant__ NormBwdArgs a, int stages)
{
    extern __shared__ __align__(128) uint8_t smem[];  // the ring; at the end [N] floats
    __shared__ __align__(8) uint64_t bars[kMostStages];
    __shared__ float buf[2][32];
    pdl_trigger();
    const int L = a.L, ln = threadIdx.x & (L - 1), slots = blockDim.x / L, slot = threadIdx.x / L;
    const int tensors = a.DR ? 3 : 2;
    const Ring g = {smem_u32(smem), smem_u32(bars), (uint32_t)(a.N * sizeof(T)), (uint32_t)slots, (uint32_t)tensors,
                    (uint32_t)stages};
    ring_init(g);
    const int which = threadIdx.x / slots;  // the tensor this thread copies
    const char *base = reinterpret_cast<const char *>(which == 0 ? a.DY : which == 1 ? a.H : a.DR);
    const int64_t ld = (which == 0 ? a.lddy : which == 1 ? a.ldh : a.lddr) * (int64_t)sizeof(T);
    const uint64_t policy = l2_evict_first_policy();
    const int64_t step = (int64_t)gridDim.x * slots;
    int64_t next = (int64_t)blockIdx.x * slots;
    for (int s = 0; s < stages && next < a.M; ++s, next += step) ring_issue(g, s, base, ld, next, a.M, policy);
    const int j0 = first_column<EW, K>(ln);
    float dw[K][EW];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < EW; ++e) dw[k][e] = 0.0f;
    Vec<WT, EW> w[K];
    load_weights<WT, EW, K>(a.W, j0, a.N - j0, w);
    pdl_wait();
    int stage = 0, turn = 0;
    uint32_t phase = 0;
    bool alive = true;
    for (int64_t r0 = (int64_t)blockIdx.x * slots; r0 < a.M; r0 += step, turn ^= 1) {
        const int64_t row = r0 + slot;
        const float s = row < a.M ? __ldg(a.rstd + row) : 0.0f;
        alive = alive && __all_sync(0xffffffffu, mbar_wait_bounded(g.bars + 8 * stage, phase));
        const int left = row < a.M ? a.N - j0 : 0;
        Vec<T, EW> vy[K], vh[K], vr[K];
        const uint32_t at = g.data + (stage * tensors * slots + slot) * g.row_bytes + j0 * (int)sizeof(T);
        ring_row<T, EW, K>(at, left, vy);
        ring_row<T, EW, K>(at + slots * g.row_bytes, left, vh);
        if (a.DR) ring_row<T, EW, K>(at + 2 * slots * g.row_bytes, left, vr);
        float c = grad_sums<T, WT, EW, K>(vy, vh, w, s, dw);
        c = row_sum(c, L, buf[turn]) * a.inv_n * s;
        if (L <= 32) __syncthreads();  // (with more lanes row_sum's barrier): every thread has read the stage
        if (next < a.M && alive) ring_issue(g, stage, base, ld, next, a.M, policy);
        next += step;
        grad_row<T, WT, EW, K>(reinterpret_cast<T *>(a.DX) + row * a.lddx + j0, alive ? left : 0, vy, vh, vr,
                               a.DR != nullptr, w, s, c);
        if (++stage == stages) {
            stage = 0;
            phase ^= 1;
        }
    }
    if (!alive) {
        atomicOr(a.status, kStatusTimeout);
        ring_drain(g, stage, phase);
    }
    if (a.part == nullptr) return;
    float *acc = reinterpret_cast<float *>(smem);
    __syncthreads();
    for (int j = threadIdx.x; j < a.N; j += blockDim.x) acc[j] = 0.0f;
    __syncthreads();
    store_dw<EW, K>(acc, a.part + (int64_t)blockIdx.x * a.N, a.N, slots, slot, j0, dw);
}

// dw[j] = sum over the P blocks' partial rows: 16 columns x 32 lanes a block (64
// bytes a row of partials; few columns, so that enough blocks run), each lane every
// 32nd row in order with 8 loads in flight, then the lanes in order.
constexpr int kDwCols = 16;
template <typename WT>
__global__ void __launch_bounds__(512) rmsnorm_dw_kernel(const float *__restrict__ part, WT *__restrict__ dw, int P, int N)
{
    __shared__ float s[32][kDwCols + 1];
    pdl_trigger();
    pdl_wait();
    const int col = threadIdx.x % kDwCols, ln = threadIdx.x / kDwCols;
    const int j = blockIdx.x * kDwCols + col;
    float t = 0.0f;
    if (j < N) {
        int p = ln;
        for (; p + 7 * 32 < P; p += 8 * 32) {
            float v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = __ldcg(part + (int64_t)(p + 32 * u) * N + j);
#pragma unroll
            for (int u = 0; u < 8; ++u) t += v[u];
        }
        float v[7];
#pragma unroll
        for (int u = 0; u < 7; ++u) v[u] = p + 32 * u < P ? __ldcg(part + (int64_t)(p + 32 * u) * N + j) : 0.0f;
#pragma unroll
        for (int u = 0; u < 7; ++u) t += v[u];
    }
    s[ln][col] = t;
    __syncthreads();
    if (ln == 0 && j < N) {
#pragma unroll
        for (int q = 1; q < 32; ++q) t += s[q][col];
        dw[j] = from_f<WT>(t);
    }
}

// Lanes a row (L) and vectors of EW a lane (K) for nv vectors: about `want`
// vectors a lane, at least `least` lanes.  Up to 512 lanes of 1, 2 or 4 vectors (8
// single elements); rows beyond that take the instances with more vectors a lane
// or 1024 lanes, whose registers are scarce.
void pick_lanes(int64_t nv, int want, int least, int EW, bool grad, int *L, int *K)
{
    const int most = EW == 1 ? 8 : 4;
    int l = least;
    while (l < 512 && (int64_t)l * (l < 32 ? 1 : want) < nv) l *= 2;
    if ((int64_t)l * most < nv) {
        *L = EW == 8 ? 512 : 1024;
        *K = EW == 1 ? 32 : EW == 4 && !grad && nv <= 4096 ? 4 : 8;
        return;
    }
    int k = EW == 1 ? 8 : 1;
    while ((int64_t)l * k < nv) k *= 2;
    *L = l;
    *K = k;
}

// A kernel instance and the dynamic shared memory its launches may ask for: its most over all
// sizes, allowed once a device (the limit belongs to the instance, so a call that set its own
// size could take it from under a call of another host thread).
struct Instance {
    const void *k;
    int most;
    mutable std::atomic<bool> ready[kMaxDevices];
};

constexpr int kRingBytes = 222 * 1024;

template <auto KERNEL, int MOST = 0>
const Instance *instance()
{
    static const Instance i = {(const void *)KERNEL, MOST, {}};
    return &i;
}

tm_status allow_smem(const Instance &i)
{
    if (i.most == 0) return TM_OK;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return TM_ERR_CUDA;
    }
    if (i.ready[dev].load(std::memory_order_acquire)) return TM_OK;
    if (cudaFuncSetAttribute(i.k, cudaFuncAttributeMaxDynamicSharedMemorySize, i.most) != cudaSuccess) {
        cudaGetLastError();
        return TM_ERR_CUDA;
    }
    i.ready[dev].store(true, std::memory_order_release);
    return TM_OK;
}

template <typename T, typename WT, int EW, bool E4M3>
const Instance *norm_kernel(int K)
{
    if constexpr (EW == 1)
        return K <= 8 ? instance<rmsnorm_kernel<T, WT, 1, 8, E4M3>>() : instance<rmsnorm_kernel<T, WT, 1, 32, E4M3>>();
    else
        return K == 1   ? instance<rmsnorm_kernel<T, WT, EW, 1, E4M3>>()
               : K == 2 ? instance<rmsnorm_kernel<T, WT, EW, 2, E4M3>>()
               : K == 4 ? instance<rmsnorm_kernel<T, WT, EW, 4, E4M3>>()
                        : instance<rmsnorm_kernel<T, WT, EW, 8, E4M3>>();
}

template <typename T, typename WT, int EW>
const Instance *norm_bwd_kernel(int K)
{
    if constexpr (EW == 1)
        return K <= 8 ? instance<rmsnorm_bwd_kernel<T, WT, 1, 8>, kMaxCols * 4>()
                      : instance<rmsnorm_bwd_kernel<T, WT, 1, 32>, kMaxCols * 4>();
    else
        return K == 1   ? instance<rmsnorm_bwd_kernel<T, WT, EW, 1>, kMaxCols * 4>()
               : K == 2 ? instance<rmsnorm_bwd_kernel<T, WT, EW, 2>, kMaxCols * 4>()
               : K == 4 ? instance<rmsnorm_bwd_kernel<T, WT, EW, 4>, kMaxCols * 4>()
                        : instance<rmsnorm_bwd_kernel<T, WT, EW, 8>, kMaxCols * 4>();
}

template <typename T, typename WT>
const Instance *norm_pick(bool vec, bool ring, bool e4, int K)
{
    constexpr int EW = 16 / sizeof(T);
    if (ring) {
        if (e4)
            return K == 1   ? instance<rmsnorm_ring_kernel<T, WT, EW, 1, true>, kRingBytes>()
                   : K == 2 ? instance<rmsnorm_ring_kernel<T, WT, EW, 2, true>, kRingBytes>()
                            : instance<rmsnorm_ring_kernel<T, WT, EW, 4, true>, kRingBytes>();
        return K == 1   ? instance<rmsnorm_ring_kernel<T, WT, EW, 1, false>, kRingBytes>()
               : K == 2 ? instance<rmsnorm_ring_kernel<T, WT, EW, 2, false>, kRingBytes>()
                        : instance<rmsnorm_ring_kernel<T, WT, EW, 4, false>, kRingBytes>();
    }
    if (vec) return e4 ? norm_kernel<T, WT, EW, true>(K) : norm_kernel<T, WT, EW, false>(K);
    return e4 ? norm_kernel<T, WT, 1, true>(K) : norm_kernel<T, WT, 1, false>(K);
}

template <typename T, typename WT>
const Instance *norm_bwd_pick(bool vec, bool ring, int K)
{
    constexpr int EW = 16 / sizeof(T);
    if (ring)
        return K == 1   ? instance<rmsnorm_bwd_ring_kernel<T, WT, EW, 1>, kRingBytes>()
               : K == 2 ? instance<rmsnorm_bwd_ring_kernel<T, WT, EW, 2>, kRingBytes>()
                        : instance<rmsnorm_bwd_ring_kernel<T, WT, EW, 4>, kRingBytes>();
    return vec ? norm_bwd_kernel<T, WT, EW>(K) : norm_bwd_kernel<T, WT, 1>(K);
}

// The ring's shape for rows of nv vectors, `tensors` of them a row: 256 lanes a block
// where a row needs no more, `want` vectors a lane, two blocks an SM (one if a row's
// copies are too large), and as many stages as their shared memory holds.  (Registers are
// not counted: a block of 512 threads of more than 64 fits an SM once, and the second
// round of blocks follows the first.)  False if
// the ring does not fit, or if there are fewer steps than blocks.  Measured (bf16 with
// a residual, first form / ring, us): norm 8192 x 8192 122 / 91, 1024 x 8192 19.6 /
// 14.6, 2048 x 4096 18.7 / 14.9, 8192 x 1024 17.3 / 15.0, 4096 x 1024 10.5 / 10.7;
// gradient 135 / 103, 31.0 / 24.9, 24.8 / 20.9, 22.9 / 21.0, 16.6 / 15.2.
struct RingPlan {
    int L, K, threads, per_sm, stages;
    int64_t blocks;
    size_t smem;
};

bool ring_plan(int64_t M, int64_t nv, int tensors, int want, int sms, RingPlan *p)
{
    if (nv < 64) return false;  // copies of less than 1 KB
    int l = 32;
    while (l < 512 && (int64_t)l * want < nv) l *= 2;
    int k = 1;
    while ((int64_t)l * k < nv) k *= 2;
    if (k > 4) return false;
    p->L = l;
    p->K = k;
    p->threads = l < 256 ? 256 : l;
    const int64_t slots = p->threads / l, stage = slots * tensors * nv * 16;
    p->per_sm = stage * 2 <= 110 * 1024 ? 2 : 1;
    const int64_t room = p->per_sm == 2 ? 110 * 1024 : kRingBytes;
    p->stages = (int)(room / stage);
    if (p->stages < 2) return false;
    if (p->stages > kMostStages) p->stages = kMostStages;
    p->smem = (size_t)(p->stages * stage);
    const int64_t most = (int64_t)sms * p->per_sm;
    p->blocks = (M + slots - 1) / slots;
    if (p->blocks < most) return false;
    p->blocks = most;
    return true;
}

constexpr int64_t kBwdBlocks = 608;  // dw partial rows at most: 152 SMs x 4 blocks

struct BwdPlan {
    int L, K, threads;
    int64_t blocks;
};

BwdPlan bwd_plan(int64_t M, int64_t N, int EW)
{
    BwdPlan p;
    const int64_t nv = (N + EW - 1) / EW;
    pick_lanes(nv, EW == 1 ? 8 : 16 / EW, EW == 1 ? 32 : 8, EW, true, &p.L, &p.K);
    p.threads = p.L < 256 ? 256 : p.L;
    const int64_t per = p.threads / p.L;
    p.blocks = (M + per - 1) / per;
    if (p.blocks > kBwdBlocks) p.blocks = kBwdBlocks;
    return p;
}

bool type_ok(int32_t t) { return elem_bytes(t) != 0; }

}  // namespace
}  // namespace libtm

using namespace libtm;

extern "C" tm_status tm_rmsnorm(const void *X, int64_t ldx, const void *R, int64_t ldr, void *H, int64_t ldh,
                                const void *W, int64_t M, int64_t N, float eps, void *Y, int64_t ldy, float *scales,
                                float *rstd, int32_t xtype, int32_t wtype, int32_t ytype, int32_t group,
                                uint32_t flags, tm_stream_t stream)
{
    const bool e4 = ytype == TM_E4M3;
    if (!type_ok(xtype) || (wtype != xtype && wtype != TM_F32) || (!e4 && ytype != xtype)) return TM_ERR_INVALID_ARG;
    if (flags & ~TM_PDL) return TM_ERR_INVALID_ARG;
    if (!(eps >= 0.0f)) return TM_ERR_INVALID_ARG;
    if (!valid_rows(X, ldx, M, N) || !valid_rows(Y, ldy, M, N)) return TM_ERR_INVALID_ARG;
    if (R != nullptr && !valid_rows(R, ldr, M, N)) return TM_ERR_INVALID_ARG;
    if (H != nullptr && !valid_rows(H, ldh, M, N)) return TM_ERR_INVALID_ARG;
    if (group != 0 && (!e4 || (group != 32 && group != 64 && group != 128))) return TM_ERR_UNSUPPORTED_TILE;
    if (N > kMaxCols) return TM_ERR_UNSUPPORTED_TILE;
    if (e4 ? (M > 0 && N > 0 && scales == nullptr) : scales != nullptr) return TM_ERR_INVALID_ARG;
    const int e = elem_bytes(xtype), we = elem_bytes(wtype);
    if (!aligned_to(X, e) || !aligned_to(R, e) || !aligned_to(H, e) || !aligned_to(W, we) || !aligned_to(scales, 4) ||
        !aligned_to(rstd, 4) || (!e4 && !aligned_to(Y, e)))
        return TM_ERR_MISALIGNED;
    if (M == 0 || N == 0) return TM_OK;
    const Span sx = span_of(X, ldx, M, N, e), sr = span_of(R, ldr, M, N, e), sh = span_of(H, ldh, M, N, e);
    const Span sy = span_of(Y, ldy, M, N, e4 ? 1 : e), sw = span_of(W, N, W ? 1 : 0, N, we);
    const int64_t ng = group ? (N + group - 1) / group : 1;
    const Span ss = span_of(scales, ng, scales ? M : 0, ng, 4), sd = span_of(rstd, 1, rstd ? M : 0, 1, 4);
    // In place: H or Y may be X or R exactly (same base, same ld, same type);
    // every other overlap of an output with anything is refused.
    auto clash = [&](const void *o, int64_t ldo, const Span &so, bool same_type, const void *p, int64_t ldp,
                     const Span &sp) { return meets(so, sp) && !(same_type && o == p && ldo == ldp); };
    if (clash(H, ldh, sh, true, X, ldx, sx) || clash(H, ldh, sh, true, R, ldr, sr) ||
        clash(Y, ldy, sy, !e4, X, ldx, sx) || clash(Y, ldy, sy, !e4, R, ldr, sr))
        return TM_ERR_INVALID_ARG;
    const Span outs[] = {sh, sy, ss, sd};
    for (int i = 0; i < 4; ++i) {
        if (meets(outs[i], sw)) return TM_ERR_INVALID_ARG;
        if (i >= 2 && (meets(outs[i], sx) || meets(outs[i], sr))) return TM_ERR_INVALID_ARG;
        for (int k = 0; k < i; ++k)
            if (meets(outs[i], outs[k])) return TM_ERR_INVALID_ARG;
    }

    const int EWv = 16 / e;
    const bool vec = N % EWv == 0 && ldx % EWv == 0 && aligned_to(X, 16) &&
                     (!R || (ldr % EWv == 0 && aligned_to(R, 16))) && (!H || (ldh % EWv == 0 && aligned_to(H, 16))) &&
                     ldy % EWv == 0 && aligned_to(Y, e4 ? EWv : 16) && (!W || aligned_to(W, 16));
    const int EW = vec ? EWv : 1;
    const int64_t nv = (N + EW - 1) / EW;
    int L, K;
    if (vec) {
        // few rows: one vector a lane, the shortest chain; many: four, so that
        // each lane has that many loads in flight
        pick_lanes(nv, M <= 304 ? 1 : 4, group ? 32 : 8, EW, false, &L, &K);
    } else {
        pick_lanes(nv, 8, 32, 1, false, &L, &K);
    }
    const DevInfo *dev;
    tm_status st = device_info(&dev);
    if (st != TM_OK) return st;
    int threads = L < 128 ? 128 : L;
    int64_t blocks = (M + threads / L - 1) / (threads / L);
    RingPlan rp;
    const bool ring = vec && ring_plan(M, nv, R ? 2 : 1, 4, dev->sms, &rp);
    if (ring) {
        L = rp.L;
        K = rp.K;
        threads = rp.threads;
        blocks = rp.blocks;
    }
    if (blocks > INT32_MAX) return TM_ERR_INVALID_ARG;
    NormArgs a = {X, R, W, H, Y, scales, rstd, ldx, ldr, ldh, ldy, M, (int)N, L, group,
                  group == 32 ? 5 : group == 64 ? 6 : 7, eps, 1.0f / (float)N, dev->status};
    const bool wf = wtype == TM_F32;
    const Instance *k =
        xtype == TM_F32 ? norm_pick<float, float>(vec, ring, e4, K)
        : xtype == TM_F16
            ? (wf ? norm_pick<__half, float>(vec, ring, e4, K) : norm_pick<__half, __half>(vec, ring, e4, K))
            : (wf ? norm_pick<__nv_bfloat16, float>(vec, ring, e4, K)
                  : norm_pick<__nv_bfloat16, __nv_bfloat16>(vec, ring, e4, K));
    void *args[] = {&a, &rp.stages};
    const size_t smem = ring ? rp.smem : 0;
    st = allow_smem(*k);
    if (st != TM_OK) return st;
    return launch_kernel(k->k, dim3((unsigned)blocks), dim3(threads), args, smem, as_stream(stream), (flags & TM_PDL) != 0);
}

extern "C" size_t tm_rmsnorm_bwd_workspace_bytes(int64_t M, int64_t N)
{
    if (M <= 0 || N <= 0 || N > kMaxCols) return 0;
    return (size_t)(M < kBwdBlocks ? M : kBwdBlocks) * (size_t)N * sizeof(float);
}

extern "C" tm_status tm_rmsnorm_bwd(const void *DY, int64_t lddy, const void *H, int64_t ldh, const void *W,
                                    const float *rstd, const void *DR, int64_t lddr, void *DX, int64_t lddx, void *DW,
                                    int64_t M, int64_t N, int32_t xtype, int32_t wtype, void *workspace,
                                    size_t ws_bytes, uint32_t flags, tm_stream_t stream)
{
    if (!type_ok(xtype) || (wtype != xtype && wtype != TM_F32)) return TM_ERR_INVALID_ARG;
    if (flags & ~TM_PDL) return TM_ERR_INVALID_ARG;
    if (!valid_rows(DY, lddy, M, N) || !valid_rows(H, ldh, M, N) || !valid_rows(DX, lddx, M, N))
        return TM_ERR_INVALID_ARG;
    if (DR != nullptr && !valid_rows(DR, lddr, M, N)) return TM_ERR_INVALID_ARG;
    if (M > 0 && N > 0 && rstd == nullptr) return TM_ERR_INVALID_ARG;
    if (N > kMaxCols) return TM_ERR_UNSUPPORTED_TILE;
    const int e = elem_bytes(xtype), we = elem_bytes(wtype);
    if (!aligned_to(DY, e) || !aligned_to(H, e) || !aligned_to(DR, e) || !aligned_to(DX, e) || !aligned_to(W, we) ||
        !aligned_to(DW, we) || !aligned_to(rstd, 4))
        return TM_ERR_MISALIGNED;
    if (N == 0) return TM_OK;
    const size_t need = tm_rmsnorm_bwd_workspace_bytes(M, N);
    if (DW != nullptr && M > 0 && (workspace == nullptr || ws_bytes < need || !aligned_to(workspace, 16)))
        return TM_ERR_WORKSPACE;
    const Span sy = span_of(DY, lddy, M, N, e), sh = span_of(H, ldh, M, N, e), sr = span_of(DR, lddr, M, N, e);
    const Span sx = span_of(DX, lddx, M, N, e), sw = span_of(W, N, W ? 1 : 0, N, we);
    const Span sdw = span_of(DW, N, DW ? 1 : 0, N, we), sd = span_of(rstd, 1, M, 1, 4);
    const Span sws = DW && M > 0 ? span_of(workspace, (int64_t)need, 1, (int64_t)need, 1) : Span{0, 0};
    auto clash = [&](const void *p, int64_t ldp, const Span &sp) { return meets(sx, sp) && !(DX == p && lddx == ldp); };
    if (clash(DY, lddy, sy) || clash(H, ldh, sh) || clash(DR, lddr, sr)) return TM_ERR_INVALID_ARG;
    const Span ins[] = {sy, sh, sr, sw, sd};
    for (const Span &s : ins)
        if (meets(s, sdw) || meets(s, sws)) return TM_ERR_INVALID_ARG;
    if (meets(sx, sw) || meets(sx, sd) || meets(sx, sdw) || meets(sx, sws) || meets(sdw, sws)) return TM_ERR_INVALID_ARG;
    if (M == 0 && DW == nullptr) return TM_OK;

    const int EWv = 16 / e;
    const bool vec = N % EWv == 0 && lddy % EWv == 0 && aligned_to(DY, 16) && ldh % EWv == 0 && aligned_to(H, 16) &&
                     lddx % EWv == 0 && aligned_to(DX, 16) && (!DR || (lddr % EWv == 0 && aligned_to(DR, 16))) &&
                     (!W || aligned_to(W, 16));
    BwdPlan p = bwd_plan(M, N, vec ? EWv : 1);
    const DevInfo *dev;
    tm_status st = device_info(&dev);
    if (st != TM_OK) return st;
    cudaStream_t s = as_stream(stream);
    if (M > 0) {
        RingPlan rp;
        const bool ring = vec && ring_plan(M, N / EWv, DR ? 3 : 2, 16 / EWv, dev->sms, &rp) && rp.blocks <= kBwdBlocks;
        if (ring) p = {rp.L, rp.K, rp.threads, rp.blocks};
        NormBwdArgs a = {DY, H, W, DR, rstd, DX, DW ? reinterpret_cast<float *>(workspace) : nullptr,
                         lddy, ldh, lddr, lddx, M, (int)N, p.L, 1.0f / (float)N, dev->status};
        const bool wf = wtype == TM_F32;
        const Instance *k =
            xtype == TM_F32 ? norm_bwd_pick<float, float>(vec, ring, p.K)
            : xtype == TM_F16
                ? (wf ? norm_bwd_pick<__half, float>(vec, ring, p.K) : norm_bwd_pick<__half, __half>(vec, ring, p.K))
                : (wf ? norm_bwd_pick<__nv_bfloat16, float>(vec, ring, p.K)
                      : norm_bwd_pick<__nv_bfloat16, __nv_bfloat16>(vec, ring, p.K));
        // the ring's stages hold [N] floats for the end: two rows of 2-byte elements or more
        const size_t smem = ring ? rp.smem : (size_t)N * sizeof(float);
        st = allow_smem(*k);
        if (st != TM_OK) return st;
        void *args[] = {&a, &rp.stages};
        st = launch_kernel(k->k, dim3((unsigned)p.blocks), dim3(p.threads), args, smem, s, (flags & TM_PDL) != 0);
        if (st != TM_OK) return st;
    }
    if (DW != nullptr) {
        const float *part = reinterpret_cast<const float *>(workspace);
        int P = M > 0 ? (int)p.blocks : 0, n = (int)N;
        void *args[] = {&part, &DW, &P, &n};
        const void *k = wtype == TM_F32   ? (const void *)rmsnorm_dw_kernel<float>
                        : wtype == TM_F16 ? (const void *)rmsnorm_dw_kernel<__half>
                                          : (const void *)rmsnorm_dw_kernel<__nv_bfloat16>;
        return launch_dependent(k, dim3((unsigned)((N + kDwCols - 1) / kDwCols)), dim3(512), args, 0, s);
    }
    return TM_OK;
}
