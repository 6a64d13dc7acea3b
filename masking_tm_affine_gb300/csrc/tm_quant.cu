// tm_quant.cu -- 8-bit floats with a scale for each run of 128 columns of one row, or for
// each block of 128 by 128.
//
//   top = max |x| over the block,  scale = top / 448,  code = nearest e4m3 to x * 448 / top
//
// Each value is read once and stays in registers between the block's maximum and its codes,
// so memory bounds it: 2 or 4 bytes in, 1 out.  At 16 bits that leaves about 11 lanes'
// instructions a value on an SM, so the maximum is taken two values at a time on their bits.
// 8192 x 8192 in 16 bits: 34 us by blocks and by rows, 87 % of a copy's rate.
//
// Codes are those of the exact quotient, which q = x * (448 / top) misses by up to 2^-23 of
// itself: wrong where a border between two codes lies between them.
//   16-bit x.  x and top have at most 11 significant bits and a border 5, so x * 448 and border *
//   top are integers below 2^17 on one scale: a quotient lies on a border or at least
//   2^-17 of itself away.  q is made too large by 2^-21 of itself, by way of the factor (all
//   roundings together are 3 * 2^-24 at most), and its last 4 bits, up to 2^-19, are cut: that puts
//   one that belongs on a border back on it, where the conversion takes the even code, and moves
//   no other across.
//   fp32 x.  A q within 4 places of a border is decided in 64 bits: |x| * 448 against
//   border * top, both exact there.  Few values take that way.
#include "tm_host.h"
#include "tm_elem.cuh"

namespace libtm {
namespace {

constexpr int kQuantThreads = 256;

// A block's factor 448 / top.  It passes fp32's range below tops of 2^-119: values of a block whose top is
// below 2^-100 are raised by 2^64 first, which is exact in their own type (fp16 has none as small).
struct Factor {
    float top, by;
};
template <typename T>
constexpr float kMore = sizeof(T) == 2 ? 1.0f + 0x1p-21f : 1.0f;
constexpr float kSmall = 0x1p-100f, kRaise = 0x1p64f;
template <typename T>
__device__ __forceinline__ Factor factor_of(float top)
{
    const float t = top < kSmall ? top * kRaise : top;
    return {t, top > 0.0f ? __fdiv_rn(448.0f, t) * kMore<T> : 0.0f};
}
template <typename T, int W>
__device__ __forceinline__ void raise(Vec<T, W> &r)
{
#pragma unroll
    for (int e = 0; e < W; ++e) r.v[e] = from_f<T>(to_f(r.v[e]) * kRaise);
}

__device__ __forceinline__ float cut(float q) { return as_f(as_u(q) & ~15u); }

// fp32: how far q is from a border, at least; 0 .. 8 within 4 places.  Below 2^-6 codes are
// multiples of 2^-9: 2^-6 more, and they are spaced as at 2^-6.
__device__ __forceinline__ uint32_t places(float q)
{
    const float y = fabsf(q) < 0.015625f ? fabsf(q) + 0.015625f : q;
    return (as_u(y) & 0xFFFFFu) - 0x7FFFCu;
}
// q moved off the border that it is close to, to its side of it (or onto it, where the quotient lies on it).
__device__ __noinline__ float decided(float x, float q, Factor f)
{
    const float p = fabsf(q), z = fabsf(x), y = p < 0.015625f ? p + 0.015625f : p;
    const float edge = as_f((as_u(y) & 0xFFF00000u) | 0x80000u), m = p < 0.015625f ? edge - 0.015625f : edge;
    const double a = (double)z * 448.0, b = (double)m * (double)f.top;
    return copysignf(a > b ? m * (1.0f + 0x1p-18f) : a < b ? m * (1.0f - 0x1p-18f) : m, x);
}

__device__ __forceinline__ uint32_t codes2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// The largest magnitude as the bits of T, which grow with it; two halves at once in 16 bits.
template <typename T, int W>
__device__ __forceinline__ uint32_t join(uint32_t top, const Vec<T, W> &r)
{
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int e = 0; e < W; ++e) top = max(top, as_u(r.v[e]) & 0x7FFFFFFFu);
    } else if constexpr (W == 1) {
        top = max(top, (uint32_t)(*reinterpret_cast<const uint16_t *>(&r) & 0x7FFFu));
    } else {
        const uint32_t *u = reinterpret_cast<const uint32_t *>(&r);
#pragma unroll
        for (int e = 0; e < W / 2; ++e) top = __vmaxu2(top, u[e] & 0x7FFF7FFFu);
    }
    return top;
}
// The maximum over `lanes` lanes, as fp32; infinite or NaN where any value is.
template <typename T>
__device__ __forceinline__ float joined(uint32_t top, int lanes)
{
    if constexpr (sizeof(T) == 2) top = max(top & 0xFFFFu, top >> 16);
    for (int o = lanes >> 1; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    if constexpr (sizeof(T) == 4)
        return as_f(top);
    else {
        const uint16_t h = (uint16_t)top;
        return to_f(*reinterpret_cast<const T *>(&h));
    }
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

template <typename T, int W>
__device__ __forceinline__ void put_codes(uint8_t *p, bool ok, const Vec<T, W> &r, const Factor &f, bool finite)
{
    float v[W], q[W];
    widen(r, v);
    uint32_t close = ~0u;
#pragma unroll
    for (int e = 0; e + 1 < W; e += 2) {
        const uint64_t p = mul2(pack2(v[e], v[e + 1]), pack2(f.by, f.by));
        unpack2(p, q[e], q[e + 1]);
    }
    if constexpr (W == 1) q[0] = v[0] * f.by;
#pragma unroll
    for (int e = 0; e < W; ++e) {
        if constexpr (sizeof(T) == 2)
            q[e] = cut(q[e]);
        else
            close = min(close, places(q[e]));
    }
    if constexpr (sizeof(T) == 4)
        if (close <= 8u) {
#pragma unroll
            for (int e = 0; e < W; ++e)
                if (places(q[e]) <= 8u) q[e] = decided(v[e], q[e], f);
        }
    if constexpr (W == 1) {
        if (ok) *p = finite ? (uint8_t)codes2(q[0], 0.0f) : (uint8_t)0x7F;
    } else if constexpr (W == 2) {
        if (ok) *reinterpret_cast<uint16_t *>(p) = finite ? (uint16_t)codes2(q[0], q[1]) : (uint16_t)0x7F7F;
    } else {
        uint32_t w[W / 4];
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            w[i] = codes2(q[4 * i], q[4 * i + 1]) | codes2(q[4 * i + 2], q[4 * i + 3]) << 16;
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

__device__ __forceinline__ float scale_of(float top, bool finite) { return !finite ? NAN : top > 0.0f ? __fdiv_rn(top, 448.0f) : 1.0f; }

struct QuantArgs {
    const void *x;
    uint8_t *y;
    float *scales;
    int64_t ldx, ldy, M, N;
    int tasks, cols;  // cols: runs of 128 columns
    FastDiv by_cols;
};

// One row's runs, neighbours in the flat order of all runs: 32 values a thread in four vectors, so that a
// run's maximum takes few exchanges between lanes and its address is found once (8192 x 8192 in 16 bits, cold: 36 us; 8
// values a thread of each of four runs, 48).
template <typename T, int W>
__global__ void __launch_bounds__(kQuantThreads) quant_rows(const QuantArgs a)
{
    constexpr int L = 32 / W, P = 4;  // lanes a run; vectors a lane
    pdl_trigger();
    const int lane = threadIdx.x % L, run = (int)blockIdx.x * (kQuantThreads / L) + (int)threadIdx.x / L;
    const bool live = run < a.tasks;
    const int row = live ? (int)fdiv((uint32_t)run, a.by_cols) : 0;
    const int64_t col = live ? (int64_t)(run - row * a.cols) * 128 + lane * W : a.N;
    const T *x = reinterpret_cast<const T *>(a.x) + (live ? row * a.ldx + col : 0);
    Vec<T, W> raw[P];
#pragma unroll
    for (int p = 0; p < P; ++p) load_vec_if(x + p * 32, col + p * 32 < a.N, raw[p]);
    uint32_t bits = 0;
#pragma unroll
    for (int p = 0; p < P; ++p) bits = join(bits, raw[p]);
    const float top = joined<T>(bits, L);
    const bool finite = top <= 3.402823466e38f;
    const Factor f = factor_of<T>(top);
    if (top < kSmall)
#pragma unroll
        for (int p = 0; p < P; ++p) raise(raw[p]);
    pdl_wait();
    if (live && lane == 0) a.scales[run] = scale_of(top, finite);
    uint8_t *y = a.y + (live ? row * a.ldy + col : 0);
#pragma unroll
    for (int p = 0; p < P; ++p) put_codes(y + p * 32, col + p * 32 < a.N, raw[p], f, finite);
}

// A block of 128 by 128 values a CTA, 64 a thread.
template <typename T, int W>
__global__ void __launch_bounds__(kQuantThreads, W == 1 ? 2 : sizeof(T) == 2 ? 5 : 3) quant_blocks(const QuantArgs a)
{
    constexpr int L = W == 1 ? 32 : 128 / W, P = W == 1 ? 4 : 1, R = kQuantThreads / L, I = 128 / R;
    __shared__ float tops[kQuantThreads / 32];
    pdl_trigger();
    const int lane = threadIdx.x % L, r0 = threadIdx.x / L;
    const int br = (int)fdiv(blockIdx.x, a.by_cols), bc = (int)blockIdx.x - br * a.cols, col = bc * 128 + lane * W;
    Vec<T, W> raw[I][P];
#pragma unroll
    for (int i = 0; i < I; ++i) {
        const int64_t row = (int64_t)br * 128 + r0 + i * R;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const bool ok = row < a.M && col + p * 32 < a.N;
            load_vec_if(reinterpret_cast<const T *>(a.x) + (ok ? row * a.ldx + col + p * 32 : 0), ok, raw[i][p]);
        }
    }
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
        for (int p = 0; p < P; ++p) bits = join(bits, raw[i][p]);
    float top = joined<T>(bits, 32);
    // a NaN loses against a number in fmaxf: it counts as an infinity
    if ((threadIdx.x & 31) == 0) tops[threadIdx.x / 32] = top <= 3.402823466e38f ? top : INFINITY;
    __syncthreads();
    top = tops[0];
#pragma unroll
    for (int i = 1; i < kQuantThreads / 32; ++i) top = fmaxf(top, tops[i]);
    const bool finite = top <= 3.402823466e38f;
    const Factor f = factor_of<T>(top);
    if (top < kSmall)
#pragma unroll
        for (int i = 0; i < I; ++i)
#pragma unroll
            for (int p = 0; p < P; ++p) raise(raw[i][p]);
    pdl_wait();
    if (threadIdx.x == 0) a.scales[blockIdx.x] = scale_of(top, finite);
#pragma unroll
    for (int i = 0; i < I; ++i) {
        const int64_t row = (int64_t)br * 128 + r0 + i * R;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const bool ok = row < a.M && col + p * 32 < a.N;
            put_codes(a.y + (ok ? row * a.ldy + col + p * 32 : 0), ok, raw[i][p], f, finite);
        }
    }
}

template <typename T, int W>
tm_status launch_quant(const QuantArgs &a, int32_t rows, cudaStream_t s, bool pdl)
{
    void *args[] = {const_cast<QuantArgs *>(&a)};
    if (rows == 128)
        return launch_kernel((const void *)quant_blocks<T, W>, dim3((unsigned)a.tasks), dim3(kQuantThreads), args, 0, s, pdl);
    constexpr int kRuns = kQuantThreads / (32 / W);
    return launch_kernel((const void *)quant_rows<T, W>, dim3((unsigned)((a.tasks + kRuns - 1) / kRuns)), dim3(kQuantThreads), args, 0, s, pdl);
}

template <typename T>
tm_status launch_quant_typed(const QuantArgs &a, int32_t rows, cudaStream_t s, bool pdl)
{
    // the widest vectors that start, end and step on their own grid (8000 x 8004 in 16 bits: 42 us by fours, 100 by ones)
    auto fits = [&](int w) {
        return aligned_to(a.x, w * sizeof(T)) && aligned_to(a.y, (uintptr_t)w) && a.ldx % w == 0 && a.ldy % w == 0 && a.N % w == 0;
    };
    if constexpr (sizeof(T) == 2)
        if (fits(8)) return launch_quant<T, 8>(a, rows, s, pdl);
    if (fits(4)) return launch_quant<T, 4>(a, rows, s, pdl);
    return fits(2) ? launch_quant<T, 2>(a, rows, s, pdl) : launch_quant<T, 1>(a, rows, s, pdl);
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
    const int64_t bands = (M + rows - 1) / rows, cols = (N + 127) / 128;
    const Span x = span_of(X, ldx, M, N, e), y = span_of(Y, ldy, M, N, 1), sc = span_of(scales, cols, bands, cols, 4);
    if (meets(x, y) || meets(x, sc) || meets(y, sc)) return TM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return TM_OK;
    if (N > (1 << 30) || bands > (1 << 30) / cols) return TM_ERR_UNSUPPORTED_TILE;
    const QuantArgs a = {X, reinterpret_cast<uint8_t *>(Y), scales, ldx, ldy, M, N, (int)(bands * cols), (int)cols,
                         make_fastdiv((uint32_t)cols)};
    const bool pdl = (flags & TM_PDL) != 0;
    if (xtype == TM_F32) return launch_quant_typed<float>(a, rows, as_stream(stream), pdl);
    if (xtype == TM_F16) return launch_quant_typed<__half>(a, rows, as_stream(stream), pdl);
    return launch_quant_typed<__nv_bfloat16>(a, rows, as_stream(stream), pdl);
}
