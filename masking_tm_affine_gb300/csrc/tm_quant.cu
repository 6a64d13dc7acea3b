// tm_quant.cu -- 8-bit floats with a scale for each run of 128 columns of one row, or for
// each block of 128 by 128.
//
//   top = max |x| over the block,  scale = top / 448,  code = nearest e4m3 to x * 448 / top
//
// Each value is read once and stays in registers between the block's maximum and its codes,
// so memory bounds it: 2 or 4 bytes in, 1 out.
//
// Codes are those of the exact quotient.  In 16 bits quotients often lie exactly on a border
// between two codes, where an error of the last place of q = x * (448 / top) decides wrongly.
// So a value whose q is within 4 places of a border is decided in 64 bits: |x| * 448
// against border * top, both exact there.  Few values take that way.
#include "tm_host.h"
#include "tm_elem.cuh"

namespace libtm {
namespace {

constexpr int kQuantThreads = 256;

// A block's factor 448 / top.  Tops below 2^-60 are lifted by 2^64 (exactly), with their values.
struct Factor {
    float top, by, lift;
};
__device__ __forceinline__ Factor factor_of(float top)
{
    Factor f;
    f.lift = top < 8.6736174e-19f ? 1.8446744e19f : 1.0f;
    f.top = top * f.lift;
    f.by = top > 0.0f ? __fdiv_rn(448.0f, f.top) : 0.0f;
    return f;
}

// x * 448 / top, moved off a border (or onto it, where the quotient lies on it) if fp32 cannot tell its side.
__device__ __forceinline__ float quotient(float x, const Factor &f)
{
    const float z = fabsf(x) * f.lift, q = z * f.by;
    // below 2^-6 codes are multiples of 2^-9: 2^-6 more, and they are spaced as at 2^-6
    const float y = q < 0.015625f ? q + 0.015625f : q;
    const uint32_t u = as_u(y);
    float r = q;
    if (((u & 0xFFFFFu) - 0x7FFFCu) <= 8u) {
        const float edge = as_f((u & 0xFFF00000u) | 0x80000u), m = q < 0.015625f ? edge - 0.015625f : edge;
        const double a = (double)z * 448.0, b = (double)m * (double)f.top;
        r = a > b ? m * (1.0f + 0x1p-18f) : a < b ? m * (1.0f - 0x1p-18f) : m;
    }
    return copysignf(r, x);
}

__device__ __forceinline__ uint32_t codes2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// The maximum of magnitudes; an infinity or NaN makes it infinite.
__device__ __forceinline__ float join(float top, float x)
{
    const float m = fabsf(x);
    return fmaxf(top, m == m ? m : INFINITY);
}

template <int W>
__device__ __forceinline__ void put_codes(uint8_t *p, bool ok, const float (&v)[W], const Factor &f, bool finite)
{
    if constexpr (W == 1) {
        if (ok) *p = finite ? (uint8_t)codes2(quotient(v[0], f), 0.0f) : (uint8_t)0x7F;
    } else {
        uint32_t w[W / 4];
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            w[i] = codes2(quotient(v[4 * i], f), quotient(v[4 * i + 1], f)) |
                   codes2(quotient(v[4 * i + 2], f), quotient(v[4 * i + 3], f)) << 16;
            if (!finite) w[i] = 0x7F7F7F7Fu;
        }
        if (ok) {
            if constexpr (W == 8)
                asm volatile("st.global.v2.b32 [%0], {%1,%2};" ::"l"(p), "r"(w[0]), "r"(w[1]) : "memory");
            else
                st_b32(p, w[0]);
        }
    }
}

struct QuantArgs {
    const void *x;
    uint8_t *y;
    float *scales;
    int64_t ldx, ldy, M, N, cols;  // cols: runs of 128 columns
    int64_t tasks;
};

// One row's runs: L lanes a run, U runs a thread, neighbours in the flat order of all runs.
template <typename T, int W, int U>
__global__ void __launch_bounds__(kQuantThreads) quant_rows(const QuantArgs a)
{
    constexpr int L = W == 1 ? 32 : 128 / W, P = W == 1 ? 4 : 1;  // lanes a run; vectors a lane
    constexpr int kRuns = kQuantThreads / L;
    pdl_trigger();
    const int lane = threadIdx.x % L;
    const int64_t first = (int64_t)blockIdx.x * kRuns * U + threadIdx.x / L;
    Vec<T, W> raw[U][P];
    int64_t row[U], col[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t run = first + u * kRuns;
        const bool live = run < a.tasks;
        row[u] = live ? run / a.cols : a.M;
        col[u] = live ? (run - row[u] * a.cols) * 128 + lane * W : 0;
#pragma unroll
        for (int p = 0; p < P; ++p)
            load_vec_if(reinterpret_cast<const T *>(a.x) + (live ? row[u] * a.ldx + col[u] + p * 32 : 0),
                        live && col[u] + p * 32 < a.N, raw[u][p]);
    }
    pdl_wait();
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float v[P][W], top = 0.0f;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            widen(raw[u][p], v[p]);
#pragma unroll
            for (int e = 0; e < W; ++e) top = join(top, v[p][e]);
        }
        top = lanes_max(top, L);
        const bool finite = top <= 3.402823466e38f, live = row[u] < a.M;
        const Factor f = factor_of(top);
        if (live && lane == 0)
            a.scales[row[u] * a.cols + col[u] / 128] = !finite ? NAN : top > 0.0f ? __fdiv_rn(top, 448.0f) : 1.0f;
#pragma unroll
        for (int p = 0; p < P; ++p)
            put_codes<W>(a.y + (live ? row[u] * a.ldy + col[u] + p * 32 : 0), live && col[u] + p * 32 < a.N, v[p], f, finite);
    }
}

// A block of 128 by 128 values a CTA, 64 a thread.
template <typename T, int W>
__global__ void __launch_bounds__(kQuantThreads, 2) quant_blocks(const QuantArgs a)
{
    constexpr int L = W == 1 ? 32 : 128 / W, P = W == 1 ? 4 : 1, R = kQuantThreads / L, I = 128 / R;
    __shared__ float tops[kQuantThreads / 32];
    pdl_trigger();
    const int lane = threadIdx.x % L, r0 = threadIdx.x / L;
    for (int64_t b = blockIdx.x; b < a.tasks; b += gridDim.x) {
        const int64_t br = b / a.cols, bc = b - br * a.cols, col = bc * 128 + lane * W;
        Vec<T, W> raw[I][P];
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const int64_t row = br * 128 + r0 + i * R;
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const bool ok = row < a.M && col + p * 32 < a.N;
                load_vec_if(reinterpret_cast<const T *>(a.x) + (ok ? row * a.ldx + col + p * 32 : 0), ok, raw[i][p]);
            }
        }
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < I; ++i)
#pragma unroll
            for (int p = 0; p < P; ++p) {
                float v[W];
                widen(raw[i][p], v);
#pragma unroll
                for (int e = 0; e < W; ++e) top = join(top, v[e]);
            }
        top = lanes_max(top, 32);
        if ((threadIdx.x & 31) == 0) tops[threadIdx.x / 32] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kQuantThreads / 32; ++i) top = fmaxf(top, tops[i]);
        __syncthreads();  // read, before the next block's
        const bool finite = top <= 3.402823466e38f;
        const Factor f = factor_of(top);
        pdl_wait();
        if (threadIdx.x == 0) a.scales[b] = !finite ? NAN : top > 0.0f ? __fdiv_rn(top, 448.0f) : 1.0f;
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const int64_t row = br * 128 + r0 + i * R;
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const bool ok = row < a.M && col + p * 32 < a.N;
                float v[W];
                widen(raw[i][p], v);
                put_codes<W>(a.y + (ok ? row * a.ldy + col + p * 32 : 0), ok, v, f, finite);
            }
        }
    }
    pdl_wait();
}

template <typename T, int W>
tm_status launch_quant(const QuantArgs &a, int32_t rows, cudaStream_t s, bool pdl)
{
    void *args[] = {const_cast<QuantArgs *>(&a)};
    if (rows == 128)
        return launch_kernel((const void *)quant_blocks<T, W>, dim3(flat_grid(a.tasks)), dim3(kQuantThreads), args, 0, s, pdl);
    constexpr int U = W == 1 ? 2 : 4, kRuns = kQuantThreads / (W == 1 ? 32 : 128 / W);
    const int64_t blocks = (a.tasks + kRuns * U - 1) / (kRuns * U);
    if (blocks > INT32_MAX) return TM_ERR_UNSUPPORTED_TILE;
    return launch_kernel((const void *)quant_rows<T, W, U>, dim3((unsigned)blocks), dim3(kQuantThreads), args, 0, s, pdl);
}

template <typename T>
tm_status launch_quant_typed(const QuantArgs &a, bool vec, int32_t rows, cudaStream_t s, bool pdl)
{
    return vec ? launch_quant<T, 16 / sizeof(T)>(a, rows, s, pdl) : launch_quant<T, 1>(a, rows, s, pdl);
}

}  // namespace
}  // namespace libtm

using namespace libtm;

extern "C" tm_status tm_quant_e4m3(const void *X, int64_t ldx, int64_t M, int64_t N, void *Y, int64_t ldy, float *scales,
                                   int32_t rows, int32_t xtype, uint32_t flags, tm_stream_t stream)
{
    const int e = elem_bytes(xtype);
    if (e == 0 || (flags & ~(uint32_t)TM_PDL)) return TM_ERR_INVALID_ARG;
    if (!valid_rows(X, ldx, M, N) || !valid_rows(Y, ldy, M, N)) return TM_ERR_INVALID_ARG;
    if (M > 0 && N > 0 && scales == nullptr) return TM_ERR_INVALID_ARG;
    if (rows != 1 && rows != 128) return TM_ERR_UNSUPPORTED_TILE;
    if (!aligned_to(X, (uintptr_t)e) || !aligned_to(scales, 4)) return TM_ERR_MISALIGNED;
    QuantArgs a = {X, reinterpret_cast<uint8_t *>(Y), scales, ldx, ldy, M, N, (N + 127) / 128, 0};
    const int64_t bands = (M + rows - 1) / rows;
    a.tasks = bands * a.cols;
    const Span x = span_of(X, ldx, M, N, e), y = span_of(Y, ldy, M, N, 1), sc = span_of(scales, a.cols, bands, a.cols, 4);
    if (meets(x, y) || meets(x, sc) || meets(y, sc)) return TM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return TM_OK;
    const int w = 16 / e;
    const bool vec = aligned_to(X, 16) && aligned_to(Y, (uintptr_t)w) && ldx % w == 0 && ldy % w == 0 && N % w == 0;
    const bool pdl = (flags & TM_PDL) != 0;
    if (xtype == TM_F32) return launch_quant_typed<float>(a, vec, rows, as_stream(stream), pdl);
    if (xtype == TM_F16) return launch_quant_typed<__half>(a, vec, rows, as_stream(stream), pdl);
    return launch_quant_typed<__nv_bfloat16>(a, vec, rows, as_stream(stream), pdl);
}
