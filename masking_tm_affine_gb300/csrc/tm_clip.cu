// tm_clip.cu -- the norm of many gradients together, and their clipping.
//
//   norm = sqrt(sum over all tensors of g^2),  out = g * min(1, max_norm / (norm + eps))
//
// The tensors are cut into chunks of kChunk elements by the plan, a table on the device, so
// that one launch walks any number of tensors of any sizes and types.  Two launches: sums of
// squares, one a block in a fixed order; then every block adds those sums itself and
// scales its chunks.  The second walks the chunks backwards: what the first read last is
// still in L2.  Memory bounds it: a read, then a read and a write (300 M elements in 16 bits: 282 us, 94 % of a
// copy's rate).  Few chunks by one launch of a cluster were slower: 48 of them 11.6 us, two launches 6.9.
//
// Sums.  A thread's vector of a chunk is squared and added in fp32 and joins the block's
// sum in 64 bits.  Where such a part leaves 2^-80 .. 2^100 (squares below it lose
// bits, above it nears infinity) it is made again in 64 bits, so that a norm is right for
// any gradients whose norm fp32 holds, however small or large.
//
// A gradient off 16 bytes, or whose output is, goes element by element, and one square at a time joins in 64
// bits (300 M elements in 16 bits to another buffer: 288 us, all odd 2080, only the outputs 1030; in 32 bits 563, 2140, 1190).
#include "tm_host.h"
#include "tm_elem.cuh"

namespace libtm {
namespace {

constexpr int kClipThreads = 256;  // of a chunk
constexpr int kClipGroups = 4;     // chunks a block walks at once: one block fills an SM
constexpr int kBlock = kClipThreads * kClipGroups;
constexpr int kChunk = 8192;       // 32 elements a thread, all read together
constexpr int kMostBlocks = 4096;  // sums a workspace holds

struct Chunk {
    const void *src;
    void *dst;
    int32_t count, type;
    int64_t unused;
};
static_assert(sizeof(Chunk) == TM_CLIP_CHUNK_BYTES, "plan entries");

struct ClipArgs {
    const Chunk *plan;
    int64_t chunks;
    double *sums;
    int blocks;  // of the first launch: how many sums there are
    float max_norm, eps;
    float *norm;
};

// Chunks are walked by groups of kClipThreads.
__device__ __forceinline__ unsigned clip_thread() { return threadIdx.x % kClipThreads; }

__device__ __forceinline__ Chunk chunk_at(const Chunk *plan, int64_t i)
{
    const u32x4 a = ldg_v4(plan + i), b = ldg_v4(reinterpret_cast<const char *>(plan + i) + 16);
    Chunk c;
    c.src = reinterpret_cast<const void *>((uint64_t)a.v[1] << 32 | a.v[0]);
    c.dst = reinterpret_cast<void *>((uint64_t)a.v[3] << 32 | a.v[2]);
    c.count = (int32_t)b.v[0];
    c.type = (int32_t)b.v[1];
    return c;
}

template <int W>
__device__ __forceinline__ double square(const float (&v)[W])
{
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < W; ++e) s = __fmaf_rn(v[e], v[e], s);
    if (s == 0.0f || (s > 0x1p-80f && s < 0x1p100f)) {
        if (s != 0.0f) return (double)s;
        bool any = false;
#pragma unroll
        for (int e = 0; e < W; ++e) any |= v[e] != 0.0f;
        if (!any) return 0.0;
    }
    double d = 0.0;
#pragma unroll
    for (int e = 0; e < W; ++e) d = fma((double)v[e], (double)v[e], d);
    return d;
}

template <typename T>
__device__ __forceinline__ double chunk_sum(const Chunk &c)
{
    constexpr int W = 16 / sizeof(T), U = 32 / W;
    const T *p = reinterpret_cast<const T *>(c.src);
    double sum = 0.0;
    if ((reinterpret_cast<uintptr_t>(p) & 15) == 0) {
        const int whole = c.count / W * W;
        for (int i = (int)clip_thread() * W; i < whole; i += kClipThreads * W * U) {
            Vec<T, W> r[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int at = i + u * kClipThreads * W;
                load_vec_if(p + at, at < whole, r[u]);
            }
            float v[U * W];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float t[W];
                widen(r[u], t);
#pragma unroll
                for (int e = 0; e < W; ++e) v[u * W + e] = t[e];
            }
            sum += square(v);
        }
        if (whole + (int)clip_thread() < c.count) {
            const float v[1] = {to_f(p[whole + clip_thread()])};
            sum += square(v);
        }
    } else {
        for (int i = clip_thread(); i < c.count; i += kClipThreads) {
            const float v[1] = {to_f(p[i])};
            sum += square(v);
        }
    }
    return sum;
}

__device__ __forceinline__ double sum_of(const Chunk &c)
{
    return c.type == TM_F32 ? chunk_sum<float>(c) : c.type == TM_F16 ? chunk_sum<__half>(c) : chunk_sum<__nv_bfloat16>(c);
}

// The block's sum, in a fixed order, in every lane of warp 0.  64-bit additions run at 2 lanes a cycle and SM: one
// warp makes them and the norm (blocks of 256 threads that each summed by trees and took their own root and quotient
// cost 20 M elements in 16 bits 26.0 us, where this takes 18.5).
__device__ __forceinline__ double warp_sum(double x)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ double block_sum(double x, double *shared)
{
    shared[threadIdx.x] = x;
    __syncthreads();
    if (threadIdx.x >= 32) return 0.0;
    x = 0.0;
#pragma unroll 8
    for (int i = 0; i < kBlock / 32; ++i) x += shared[i * 32 + threadIdx.x];
    return warp_sum(x);
}

// This group's chunks: the first, and how far apart they are.
struct Share {
    int64_t first, step;
};
__device__ __forceinline__ Share clip_share()
{
    return {(int64_t)(threadIdx.x / kClipThreads) * gridDim.x + blockIdx.x, (int64_t)gridDim.x * kClipGroups};
}

__global__ void __launch_bounds__(kBlock, 1) clip_sums(const ClipArgs a)
{
    __shared__ double shared[kBlock];
    pdl_trigger();
    const Share w = clip_share();
    double sum = 0.0;
    Chunk next = {};
    if (w.first < a.chunks) next = chunk_at(a.plan, w.first);
    for (int64_t i = w.first; i < a.chunks; i += w.step) {
        const Chunk c = next;
        if (i + w.step < a.chunks) next = chunk_at(a.plan, i + w.step);
        sum += sum_of(c);
    }
    sum = block_sum(sum, shared);
    pdl_wait();
    if (threadIdx.x == 0) a.sums[blockIdx.x] = sum;
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const Chunk &c, float f)
{
    constexpr int W = 16 / sizeof(T), U = 32 / W;
    const T *p = reinterpret_cast<const T *>(c.src);
    T *q = reinterpret_cast<T *>(c.dst);
    if (((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(q)) & 15) == 0) {
        const int whole = c.count / W * W;
        for (int i = (int)clip_thread() * W; i < whole; i += kClipThreads * W * U) {
            Vec<T, W> r[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int at = i + u * kClipThreads * W;
                load_vec_if(p + at, at < whole, r[u]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int at = i + u * kClipThreads * W;
                float v[W];
                widen(r[u], v);
#pragma unroll
                for (int e = 0; e < W; ++e) v[e] *= f;
                narrow(v, r[u]);
                store_vec_if(q + at, at < whole, r[u]);
            }
        }
        if (whole + (int)clip_thread() < c.count) q[whole + clip_thread()] = from_f<T>(to_f(p[whole + clip_thread()]) * f);
    } else {
        for (int i = clip_thread(); i < c.count; i += kClipThreads) q[i] = from_f<T>(to_f(p[i]) * f);
    }
}

__device__ __forceinline__ void scale(const Chunk &c, float f)
{
    if (c.dst == nullptr || (f == 1.0f && c.dst == c.src)) return;
    if (c.type == TM_F32)
        chunk_scale<float>(c, f);
    else if (c.type == TM_F16)
        chunk_scale<__half>(c, f);
    else
        chunk_scale<__nv_bfloat16>(c, f);
}

// The factor and the norm, of the whole sum.  An infinite max_norm or nothing at all: no clipping; else a NaN
// stays one.
__device__ __forceinline__ float clip_factor(double sum, const ClipArgs &a, float *norm)
{
    const double root = sqrt(sum), size = root + (double)a.eps, ratio = (double)a.max_norm / size;
    *norm = (float)root;
    return isinf(a.max_norm) || size == 0.0 || ratio >= 1.0 ? 1.0f : (float)ratio;
}

__global__ void __launch_bounds__(kBlock, 1) clip_scale(const ClipArgs a)
{
    __shared__ float factor;
    pdl_trigger();
    const Share w = clip_share();
    Chunk next = {};
    if (a.chunks > w.first) next = chunk_at(a.plan, a.chunks - 1 - w.first);
    pdl_wait();  // the sums
    if (threadIdx.x < 32) {
        double sum = 0.0;
        for (int i = threadIdx.x; i < a.blocks; i += 32) sum += __ldcg(a.sums + i);
        float norm;
        const float f = clip_factor(warp_sum(sum), a, &norm);
        if (threadIdx.x == 0) {
            factor = f;
            if (blockIdx.x == 0) *a.norm = norm;
        }
    }
    __syncthreads();
    const float f = factor;
    for (int64_t i = a.chunks - 1 - w.first; i >= 0; i -= w.step) {
        const Chunk c = next;
        if (i >= w.step) next = chunk_at(a.plan, i - w.step);
        scale(c, f);
    }
}

}  // namespace
}  // namespace libtm

using namespace libtm;

extern "C" int64_t tm_clip_chunks(const int64_t *sizes, int32_t n)
{
    if (n < 0 || (n > 0 && sizes == nullptr)) return -1;
    int64_t chunks = 0;
    for (int32_t i = 0; i < n; ++i) {
        if (sizes[i] < 0 || sizes[i] > INT64_MAX / 64) return -1;
        chunks += (sizes[i] + kChunk - 1) / kChunk;
    }
    return chunks;
}

extern "C" tm_status tm_clip_plan(void *plan, const void *const *grads, void *const *outs, const int64_t *sizes,
                                  const int32_t *types, int32_t n)
{
    const int64_t chunks = tm_clip_chunks(sizes, n);
    if (chunks < 0 || (n > 0 && (grads == nullptr || types == nullptr)) || (chunks > 0 && plan == nullptr)) return TM_ERR_INVALID_ARG;
    for (int32_t i = 0; i < n; ++i) {
        const int e = elem_bytes(types[i]);
        if (e == 0 || (sizes[i] > 0 && grads[i] == nullptr)) return TM_ERR_INVALID_ARG;
        if (!aligned_to(grads[i], (uintptr_t)e) || (outs != nullptr && !aligned_to(outs[i], (uintptr_t)e))) return TM_ERR_MISALIGNED;
        if (outs != nullptr && outs[i] != nullptr && outs[i] != grads[i] &&
            meets(span_of(grads[i], sizes[i], 1, sizes[i], e), span_of(outs[i], sizes[i], 1, sizes[i], e)))
            return TM_ERR_INVALID_ARG;
    }
    Chunk *c = reinterpret_cast<Chunk *>(plan);
    for (int32_t i = 0; i < n; ++i) {
        const int e = elem_bytes(types[i]);
        for (int64_t at = 0; at < sizes[i]; at += kChunk) {
            const int64_t left = sizes[i] - at;
            c->src = reinterpret_cast<const char *>(grads[i]) + at * e;
            c->dst = outs == nullptr || outs[i] == nullptr ? nullptr : reinterpret_cast<char *>(outs[i]) + at * e;
            c->count = (int32_t)(left < kChunk ? left : kChunk);
            c->type = types[i];
            c->unused = 0;
            ++c;
        }
    }
    return TM_OK;
}

extern "C" size_t tm_clip_workspace_bytes(void) { return kMostBlocks * sizeof(double); }

extern "C" tm_status tm_clip_grads(const void *plan, int64_t chunks, float max_norm, float eps, float *norm, void *workspace,
                                   size_t ws_bytes, uint32_t flags, tm_stream_t stream)
{
    if (chunks < 0 || (chunks > 0 && plan == nullptr) || norm == nullptr || !(max_norm >= 0.0f) || !(eps >= 0.0f) ||
        (flags & ~(uint32_t)TM_PDL))
        return TM_ERR_INVALID_ARG;
    if (!aligned_to(plan, 16) || !aligned_to(norm, 4)) return TM_ERR_MISALIGNED;
    if (workspace == nullptr || ws_bytes < tm_clip_workspace_bytes() || !aligned_to(workspace, 16)) return TM_ERR_WORKSPACE;
    const Span p = span_of(plan, TM_CLIP_CHUNK_BYTES, chunks, TM_CLIP_CHUNK_BYTES, 1);
    const Span w = span_of(workspace, (int64_t)ws_bytes, 1, (int64_t)tm_clip_workspace_bytes(), 1), m = span_of(norm, 1, 1, 1, 4);
    if (meets(p, w) || meets(p, m) || meets(w, m)) return TM_ERR_INVALID_ARG;
    const DevInfo *dev;
    tm_status st = device_info(&dev);
    if (st != TM_OK) return st;
    // a block an SM, and a chunk each before any has two
    const int64_t most = dev->sms < kMostBlocks ? dev->sms : kMostBlocks;
    const unsigned grid = (unsigned)(chunks < 1 ? 1 : chunks < most ? chunks : most);
    ClipArgs a = {reinterpret_cast<const Chunk *>(plan), chunks, reinterpret_cast<double *>(workspace), (int)grid, max_norm, eps, norm};
    void *args[] = {&a};
    st = launch_kernel((const void *)clip_sums, dim3(grid), dim3(kBlock), args, 0, as_stream(stream), (flags & TM_PDL) != 0);
    if (st != TM_OK) return st;
    return launch_dependent((const void *)clip_scale, dim3(grid), dim3(kBlock), args, 0, as_stream(stream));
}
