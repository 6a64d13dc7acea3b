// tm_elem.cuh -- element types of the transformer-block operators (fp32, fp16,
// bf16) and how their vectors move: 16-byte (or narrower) accesses in the
// file's inline PTX, values widened to fp32 in registers and rounded once, to
// nearest, on the way out.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "tm_device.cuh"

namespace libtm {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// W elements of type T as one access: 4, 8, 16 or 32 bytes, aligned to its
// size up to 16 (32 bytes move as two 16-byte accesses); 1 element is a plain load.
template <typename T, int W>
struct alignas(W * sizeof(T) > 16 ? 16 : W * sizeof(T)) Vec {
    T v[W];
};

// Read-only data, each byte read once: past L1.  Zeros where `ok` is false: a
// predicate on the access itself, no branch around it (a warp's branches and the
// moves that join their two sides cost the norms more than their arithmetic).
template <typename T, int W>
__device__ __forceinline__ void load_vec_if(const T *p, bool ok, Vec<T, W> &r)
{
    constexpr int B = W * sizeof(T);
    uint32_t *u = reinterpret_cast<uint32_t *>(&r);
    if constexpr (B % 16 == 0) {
#pragma unroll
        for (int q = 0; q < B / 16; ++q)
            asm volatile(
                "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
                "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
                "@p ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];\n\t}"
                : "=&r"(u[4 * q]), "=&r"(u[4 * q + 1]), "=&r"(u[4 * q + 2]), "=&r"(u[4 * q + 3])
                : "l"(reinterpret_cast<const char *>(p) + 16 * q), "r"((uint32_t)ok));
    } else if constexpr (B == 8) {
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %3, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\t"
            "@p ld.global.nc.L1::no_allocate.v2.b32 {%0,%1}, [%2];\n\t}"
            : "=&r"(u[0]), "=&r"(u[1])
            : "l"(p), "r"((uint32_t)ok));
    } else if constexpr (B == 4) {
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t"
            "@p ld.global.nc.L1::no_allocate.b32 %0, [%1];\n\t}"
            : "=&r"(u[0])
            : "l"(p), "r"((uint32_t)ok));
    } else {
        static_assert(B == 2, "access width");
        uint16_t h;
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.b16 %0, 0;\n\t"
            "@p ld.global.nc.L1::no_allocate.b16 %0, [%1];\n\t}"
            : "=&h"(h)
            : "l"(p), "r"((uint32_t)ok));
        *reinterpret_cast<uint16_t *>(&r) = h;
    }
}

template <typename T, int W>
__device__ __forceinline__ void load_vec(const T *p, Vec<T, W> &r)
{
    load_vec_if(p, true, r);
}

template <typename T, int W>
__device__ __forceinline__ void store_vec_if(T *p, bool ok, const Vec<T, W> &r)
{
    constexpr int B = W * sizeof(T);
    const uint32_t *u = reinterpret_cast<const uint32_t *>(&r);
    if constexpr (B % 16 == 0) {
#pragma unroll
        for (int q = 0; q < B / 16; ++q)
            asm volatile(
                "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t@p st.global.v4.b32 [%0], {%1,%2,%3,%4};\n\t}" ::"l"(
                    reinterpret_cast<char *>(p) + 16 * q),
                "r"(u[4 * q]), "r"(u[4 * q + 1]), "r"(u[4 * q + 2]), "r"(u[4 * q + 3]), "r"((uint32_t)ok)
                : "memory");
    } else if constexpr (B == 8) {
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %3, 0;\n\t@p st.global.v2.b32 [%0], {%1,%2};\n\t}" ::"l"(p),
                     "r"(u[0]), "r"(u[1]), "r"((uint32_t)ok)
                     : "memory");
    } else if constexpr (B == 4) {
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p st.global.b32 [%0], %1;\n\t}" ::"l"(p),
                     "r"(u[0]), "r"((uint32_t)ok)
                     : "memory");
    } else {
        static_assert(B == 2, "access width");
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p st.global.b16 [%0], %1;\n\t}" ::"l"(p),
                     "h"(*reinterpret_cast<const uint16_t *>(&r)), "r"((uint32_t)ok)
                     : "memory");
    }
}

template <typename T, int W>
__device__ __forceinline__ void store_vec(T *p, const Vec<T, W> &r)
{
    store_vec_if(p, true, r);
}

template <typename T, int W>
__device__ __forceinline__ void widen(const Vec<T, W> &r, float (&f)[W])
{
#pragma unroll
    for (int e = 0; e < W; ++e) f[e] = to_f(r.v[e]);
}

// Rounded to nearest, two values an instruction.
template <typename T, int W>
__device__ __forceinline__ void narrow(const float (&f)[W], Vec<T, W> &r)
{
    if constexpr (sizeof(T) == 2 && W % 2 == 0) {
        uint32_t *u = reinterpret_cast<uint32_t *>(&r);
#pragma unroll
        for (int e = 0; e < W / 2; ++e) {
            if constexpr (std::is_same<T, __half>::value)
                asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(u[e]) : "f"(f[2 * e + 1]), "f"(f[2 * e]));
            else
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u[e]) : "f"(f[2 * e + 1]), "f"(f[2 * e]));
        }
    } else {
#pragma unroll
        for (int e = 0; e < W; ++e) r.v[e] = from_f<T>(f[e]);
    }
}

// 2^x, good to two places; 1 / x likewise, for x whose reciprocal is a normal number.
__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Maximum over the `lanes` (a power of two) consecutive lanes that share a row.
__device__ __forceinline__ float lanes_max(float x, int lanes, unsigned mask = 0xffffffffu)
{
    for (int o = lanes >> 1; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(mask, x, o));
    return x;
}

__device__ __forceinline__ float lanes_sum(float x, int lanes, unsigned mask = 0xffffffffu)
{
    for (int o = lanes >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(mask, x, o);
    return x;
}

// ---------------------------------------------------------------- host side
// Size of an element type code (TM_F32 ...), 0 if it is not one of the three.
inline int elem_bytes(int32_t type)
{
    return type == TM_F32 ? 4 : (type == TM_F16 || type == TM_BF16) ? 2 : 0;
}

// Bytes [lo, hi) that a row-major [M, N] tensor of `e`-byte elements touches.
struct Span {
    uintptr_t lo, hi;
};

inline Span span_of(const void *p, int64_t ld, int64_t M, int64_t N, int e)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (p == nullptr || M <= 0 || N <= 0) return {0, 0};
    return {lo, lo + (uintptr_t)(((M - 1) * ld + N) * (int64_t)e)};
}

inline bool meets(const Span &a, const Span &b) { return a.hi > b.lo && b.hi > a.lo; }

// Extents >= 0, ld >= N, addressed bytes within int64, non-NULL when there is work.
inline bool valid_rows(const void *p, int64_t ld, int64_t M, int64_t N)
{
    if (M < 0 || N < 0 || ld < N) return false;
    if (M == 0 || N == 0) return true;
    return p != nullptr && !(ld > 0 && M > (INT64_MAX / 8) / ld);
}

// [T, H, D] tensors: token and head strides in elements, a head's dims contiguous.
struct Heads {
    const void *p;
    int64_t tok, head;
};

inline bool heads_ok(const Heads &x, int64_t T, int64_t H, int64_t D)
{
    if (x.tok < 0 || x.head < 0) return false;
    if (T == 0 || H == 0 || D == 0) return true;
    if (x.p == nullptr) return false;
    const int64_t cap = INT64_MAX / 32;
    return (T <= 1 || x.tok <= cap / T) && (H <= 1 || x.head <= cap / H);
}

inline Span heads_span(const Heads &x, int64_t T, int64_t H, int64_t D, int e)
{
    if (x.p == nullptr || T <= 0 || H <= 0 || D <= 0) return {0, 0};
    const uintptr_t lo = reinterpret_cast<uintptr_t>(x.p);
    return {lo, lo + (uintptr_t)(((T - 1) * x.tok + (H - 1) * x.head + D) * (int64_t)e)};
}

// Whether two [T, H, D] tensors share an element, where their bounding spans
// meet: not if they interleave with the same strides, one token's (or one
// head's) dims of the one lying in the gap of the other.
inline bool heads_meet(const Heads &a, int64_t Ha, const Heads &b, int64_t Hb, int64_t T, int64_t D, int e)
{
    if (!meets(heads_span(a, T, Ha, D, e), heads_span(b, T, Hb, D, e))) return false;
    if (a.tok != b.tok) return true;
    const bool swap = reinterpret_cast<uintptr_t>(a.p) > reinterpret_cast<uintptr_t>(b.p);
    const Heads &x = swap ? b : a, &y = swap ? a : b;
    const int64_t Hx = swap ? Hb : Ha, Hy = swap ? Ha : Hb;
    const int64_t gap = (int64_t)(reinterpret_cast<uintptr_t>(y.p) - reinterpret_cast<uintptr_t>(x.p)) / e;
    if (gap >= (Hx - 1) * x.head + D && (T <= 1 || gap + (Hy - 1) * y.head + D <= x.tok)) return false;
    if (x.head == y.head && gap >= D && gap + D <= x.head && (T <= 1 || x.tok >= (Hx > Hy ? Hx : Hy) * x.head))
        return false;
    return true;
}

// Whether every head of x starts on a 16-byte boundary.
inline bool heads_vec(const Heads &x, int e)
{
    const int w = 16 / e;
    return (reinterpret_cast<uintptr_t>(x.p) & 15) == 0 && x.tok % w == 0 && x.head % w == 0;
}

}  // namespace libtm
