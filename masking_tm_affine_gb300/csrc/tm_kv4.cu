// tm_kv4.cu -- writing to and reading back from the 4-bit paged cache.
//
// Append: rotate q and k, hold k and v as codes (see tm.h for the format).
// Bound by HBM: q is read and written, k and v read, their (D + 8) / 2 bytes a
// vector written.  A block takes one token: its rot/2 sines and cosines go to
// shared memory once, then every group of D/16 lanes takes a head, 16 values a
// lane as two runs of 8 (the halves of 8 pairs), so a run's codes are one
// 32-bit store and a vector's minimum and maximum are two or three shuffles.
//
// Exact codes.  fp32 leaves a rotated value off by up to about 2^-22 of its
// pair's size, which moves a code only where (x - low) / step is that close to
// a half, and step or low only where they are that close to a midpoint of two
// fp16 numbers.  Those cases are found by bounds on the fp32 error (about one
// value in 10^5 and one vector in 300) and decided by the same formula in fp64,
// on the lanes concerned alone: fp64 runs at 1/64 of the fp32 rate here, and
// deciding every value in it would take longer than the whole launch.
#include "tm_host.h"

#include "tm_kv4.cuh"
#include "tm_rope.cuh"

namespace libtm {
namespace {

struct AppendArgs {
    const void *Q, *K, *V;
    void *QO;
    int64_t qs_tok, qs_head, qos_tok, qos_head, ks_tok, ks_head, vs_tok, vs_head;
    const int64_t *pos, *slots;
    const uint64_t *turns;
    uint8_t *pool;
    int64_t slots_in_pool, page_bytes;
    int page, Hq, Hkv, rot;
    float gain;
    unsigned *status;
};

template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T *p, float (&f)[8])
{
    if constexpr (VEC) {
        Vec<T, 8> v;
        load_vec(p, v);
        widen(v, f);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = to_f(p[e]);
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T *p, const float (&f)[8])
{
    Vec<T, 8> v;
    narrow(f, v);
    if constexpr (VEC) {
        store_vec(p, v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = v.v[e];
    }
}

// fp16 of a value by way of fp32, clamped to fp16's range.
__device__ __forceinline__ __half held_half(float x) { return __float2half_rn(fminf(fmaxf(x, -65504.0f), 65504.0f)); }
__device__ __forceinline__ __half held_half_d(double x) { return held_half((float)x); }

// One element of a rotated pair in fp64: a cos - b sin (first) or a sin + b cos.
__device__ __noinline__ double exact_rotated(float a, float b, int64_t fraction, float gain, bool first)
{
    double s, c;
    sincospi((double)fraction * 0x1p-63, &s, &c);
    const double r = first ? (double)a * c - (double)b * s : (double)a * s + (double)b * c;
    return r * (double)gain;
}

__device__ __noinline__ int exact_code(double x, float low, float step)
{
    const double t = rint((x - (double)low) / (double)step);
    return (int)fmin(fmax(t, 0.0), 15.0);
}

// A vector's 16 values in one lane: the fp32 values, the error each may have,
// and what computes value i in fp64.
template <int LANES, typename Exact>
__device__ __forceinline__ void hold_vector(const float (&x)[2][8], const float (&err)[2][8], Exact exact,
                                            uint32_t (&word)[2], __half2 &params)
{
    const unsigned lane = threadIdx.x & 31;
    const unsigned mask = LANES == 32 ? 0xffffffffu : ((1u << LANES) - 1) << (lane / LANES * LANES);
    // minimum and maximum, how far each may be off, and whether all are finite
    float lo = INFINITY, hi = -INFINITY, worst = 0.0f, size = 0.0f;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            lo = fminf(lo, x[u][e]);
            hi = fmaxf(hi, x[u][e]);
            worst = fmaxf(worst, err[u][e]);
            size += fabsf(x[u][e]);
        }
    const bool bad = __any_sync(mask, !(size < INFINITY));
    lo = -lanes_max(-lo, LANES, mask);
    hi = lanes_max(hi, LANES, mask);
    worst = lanes_max(worst, LANES, mask);
    if (bad || !(hi - lo < INFINITY)) {
        word[0] = word[1] = 0;
        params = __halves2half2(__ushort_as_half(0x7fff), __ushort_as_half(0x7fff));
        return;
    }
    const float s = (hi - lo) * (1.0f / 15.0f);
    const float es = worst * (2.0f / 15.0f) + s * 0x1p-21f, el = worst + fabsf(lo) * 0x1p-23f;
    __half step = held_half(s), low = held_half(lo);
    const bool unsure = __half_as_ushort(held_half(s - es)) != __half_as_ushort(held_half(s + es)) ||
                        __half_as_ushort(held_half(lo - el)) != __half_as_ushort(held_half(lo + el));
    if (unsure) {  // the same for every lane of the vector
        // the values that may be the extremes, in fp64
        double dlo = INFINITY, dhi = -INFINITY;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (x[u][e] - err[u][e] <= lo + worst || x[u][e] + err[u][e] >= hi - worst) {
                    const double d = exact(u, e);
                    dlo = fmin(dlo, d);
                    dhi = fmax(dhi, d);
                }
            }
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) {
            dlo = fmin(dlo, __shfl_xor_sync(mask, dlo, o));
            dhi = fmax(dhi, __shfl_xor_sync(mask, dhi, o));
        }
        step = held_half_d((dhi - dlo) / 15.0);
        low = held_half_d(dlo);
    }
    const float fs = __half2float(step), fl = __half2float(low);
    const float inv = fs > 0.0f ? 1.0f / fs : 0.0f;
    word[0] = word[1] = 0;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float d = x[u][e] - fl, t = d * inv;
            const float r = rintf(t);
            // the value's error, the difference's rounding and the product's
            const float et = (err[u][e] + fabsf(d) * 0x1p-23f) * inv + fabsf(t) * 0x1p-22f;
            int c = (int)fminf(fmaxf(r, 0.0f), 15.0f);
            if (fs > 0.0f && fabsf(t - r) + et >= 0.5f && t > -1.0f && t < 16.0f) c = exact_code(exact(u, e), fl, fs);
            word[u] |= (uint32_t)c << (4 * e);
        }
    params = __halves2half2(step, low);
}

template <typename T, int D, bool VEC, bool INTER>
__global__ void __launch_bounds__(512) kv4_append_kernel(const __grid_constant__ AppendArgs a)
{
    constexpr int LANES = D / 16;
    __shared__ float2 cs[D / 2];
    pdl_trigger();
    const int64_t t = blockIdx.x;
    const int64_t slot = a.slots[t];
    const int64_t pos = a.rot > 0 ? a.pos[t] : 0;
    for (int i = threadIdx.x; i < a.rot / 2; i += blockDim.x) cs[i] = pair_rotation(pos, a.turns[i], a.gain, 1.0f);
    __syncthreads();
    const bool held = slot >= 0 && slot < a.slots_in_pool;
    if (!held && slot != -1 && threadIdx.x == 0 && blockIdx.y == 0) atomicOr(a.status, kStatusIndex);
    uint8_t *block = nullptr;  // of KV head 0
    int r = 0;
    if (held) {
        const int64_t pg = slot / a.page;
        const int at = (int)(slot - pg * a.page);
        block = a.pool + pg * a.page_bytes + (int64_t)(at / 16) * kv4_block_bytes(D);
        r = at % 16;
    }
    const int ln = threadIdx.x % LANES, half = a.rot / 2;
    const bool turned = ln < a.rot / 16;  // this lane's 16 dims are 8 pairs
    const int d0 = !turned || INTER ? 16 * ln : 8 * ln, d1 = !turned || INTER ? d0 + 8 : d0 + half;
    const int heads = a.Hq + 2 * a.Hkv, slots = blockDim.x / LANES;
    bool waited = false;
    for (int h = blockIdx.y * slots + threadIdx.x / LANES; h < heads; h += gridDim.y * slots) {
        const T *p;
        const bool q = h < a.Hq, k = !q && h < a.Hq + a.Hkv;
        if (q)
            p = reinterpret_cast<const T *>(a.Q) + t * a.qs_tok + h * a.qs_head;
        else if (k)
            p = reinterpret_cast<const T *>(a.K) + t * a.ks_tok + (h - a.Hq) * a.ks_head;
        else
            p = reinterpret_cast<const T *>(a.V) + t * a.vs_tok + (h - a.Hq - a.Hkv) * a.vs_head;
        const bool turn = turned && (q || k);
        const int o0 = q || k ? d0 : 16 * ln, o1 = q || k ? d1 : 16 * ln + 8;
        float x[2][8];
        load8<T, VEC>(p + o0, x[0]);
        load8<T, VEC>(p + o1, x[1]);
        float in[2][8], err[2][8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            in[0][e] = x[0][e];
            in[1][e] = x[1][e];
            err[0][e] = err[1][e] = 0.0f;
        }
        if (turn) {
            float2 rot8[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) rot8[e] = cs[8 * ln + e];
            rotate_pairs<8, INTER>(x[0], x[1], rot8);
            // |cos|, |sin| are off by at most 2.1e-7 (the argument's rounding
            // pi 2^-25, sincospif's last place, the gain's rounding), the products
            // and the sum add 2^-23 of |a| + |b|: 3.3e-7 in all, below 1.5 * 2^-22
            const float ge = fabsf(a.gain) * 0x1.8p-22f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if constexpr (INTER) {
                    err[e / 4][e % 4 * 2] = err[e / 4][e % 4 * 2 + 1] =
                        (fabsf(in[e / 4][e % 4 * 2]) + fabsf(in[e / 4][e % 4 * 2 + 1])) * ge;
                } else {
                    err[0][e] = err[1][e] = (fabsf(in[0][e]) + fabsf(in[1][e])) * ge;
                }
            }
        }
        if (!waited) pdl_wait();
        waited = true;
        if (q) {
            T *o = reinterpret_cast<T *>(a.QO) + t * a.qos_tok + h * a.qos_head;
            store8<T, VEC>(o + o0, x[0]);
            store8<T, VEC>(o + o1, x[1]);
            continue;
        }
        if (!held) continue;
        auto exact = [&](int u, int e) -> double {
            if (!turn) return (double)in[u][e];
            float pa, pb;
            int pair;
            bool first;
            if constexpr (INTER) {
                pair = 4 * u + e / 2;
                first = e % 2 == 0;
                pa = in[u][e / 2 * 2];
                pb = in[u][e / 2 * 2 + 1];
            } else {
                pair = e;
                first = u == 0;
                pa = in[0][e];
                pb = in[1][e];
            }
            return exact_rotated(pa, pb, turn_fraction(pos, a.turns[8 * ln + pair]), a.gain, first);
        };
        uint32_t word[2];
        __half2 params;
        hold_vector<LANES>(x, err, exact, word, params);
        const int kvh = k ? h - a.Hq : h - a.Hq - a.Hkv;
        uint8_t *b = block + (int64_t)kvh * (a.page / 16) * kv4_block_bytes(D);
        if (k) {
            *reinterpret_cast<uint32_t *>(b + kv4_k_word(D, r, o0)) = word[0];
            *reinterpret_cast<uint32_t *>(b + kv4_k_word(D, r, o1)) = word[1];
            if (ln == 0) *reinterpret_cast<__half2 *>(b + kv4_ks_off(D) + 4 * r) = params;
        } else {
            *reinterpret_cast<uint32_t *>(b + kv4_v_word(D, r, o0)) = word[0];
            *reinterpret_cast<uint32_t *>(b + kv4_v_word(D, r, o1)) = word[1];
            if (ln == 0) *reinterpret_cast<__half2 *>(b + kv4_vs_off(D) + 4 * r) = params;
        }
    }
    if (!waited) pdl_wait();
}

struct GatherArgs {
    const uint8_t *pool;
    const int64_t *slots;
    void *K, *V;
    int64_t slots_in_pool, page_bytes, ks_tok, ks_head, vs_tok, vs_head, T;
    int page, Hkv;
    FastDiv by_heads;
    unsigned *status;
};

// Bound by HBM: D/2 + 4 bytes read and D elements written a vector.  A group of
// D/16 lanes takes one (token, head), 16 values of K and 16 of V a lane.
template <typename T, int D, bool VEC>
__global__ void __launch_bounds__(256) kv4_gather_kernel(const __grid_constant__ GatherArgs a)
{
    constexpr int LANES = D / 16;
    pdl_trigger();
    const int ln = threadIdx.x % LANES;
    const int64_t item = (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
    if (item < a.T * a.Hkv) {
        const int64_t t = item <= INT32_MAX ? (int64_t)fdiv((uint32_t)item, a.by_heads) : item / a.Hkv;
        const int h = (int)(item - t * a.Hkv);
        const int64_t slot = a.slots[t];
        const bool held = slot >= 0 && slot < a.slots_in_pool;
        if (!held && slot != -1 && ln == 0) atomicOr(a.status, kStatusIndex);
        uint32_t kw[2] = {0, 0}, vw[2] = {0, 0};
        float2 kp = {0.0f, 0.0f}, vp = {0.0f, 0.0f};
        if (held) {
            const int64_t pg = slot / a.page;
            const int at = (int)(slot - pg * a.page), r = at % 16;
            const uint8_t *b = a.pool + pg * a.page_bytes + ((int64_t)h * (a.page / 16) + at / 16) * kv4_block_bytes(D);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                kw[u] = ld_nc_b32(b + kv4_k_word(D, r, 16 * ln + 8 * u));
                vw[u] = ld_nc_b32(b + kv4_v_word(D, r, 16 * ln + 8 * u));
            }
            const uint32_t ks = ld_nc_b32(b + kv4_ks_off(D) + 4 * r), vs = ld_nc_b32(b + kv4_vs_off(D) + 4 * r);
            kp = __half22float2(*reinterpret_cast<const __half2 *>(&ks));
            vp = __half22float2(*reinterpret_cast<const __half2 *>(&vs));
        }
        pdl_wait();
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float k8[8], v8[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                k8[e] = fmaf((float)(kw[u] >> (4 * e) & 15u), kp.x, kp.y);
                v8[e] = fmaf((float)(vw[u] >> (4 * e) & 15u), vp.x, vp.y);
            }
            if (a.K)
                store8<T, VEC>(reinterpret_cast<T *>(a.K) + t * a.ks_tok + h * a.ks_head + 16 * ln + 8 * u, k8);
            if (a.V)
                store8<T, VEC>(reinterpret_cast<T *>(a.V) + t * a.vs_tok + h * a.vs_head + 16 * ln + 8 * u, v8);
        }
    }
    pdl_wait();
}

template <typename T, int D>
const void *append_kernel(bool vec, bool inter)
{
    if (vec)
        return inter ? (const void *)kv4_append_kernel<T, D, true, true>
                     : (const void *)kv4_append_kernel<T, D, true, false>;
    return inter ? (const void *)kv4_append_kernel<T, D, false, true>
                 : (const void *)kv4_append_kernel<T, D, false, false>;
}

template <typename T>
const void *append_kernel(int D, bool vec, bool inter)
{
    return D == 64    ? append_kernel<T, 64>(vec, inter)
           : D == 128 ? append_kernel<T, 128>(vec, inter)
                      : append_kernel<T, 256>(vec, inter);
}

template <typename T>
const void *gather_kernel(int D, bool vec)
{
    if (vec)
        return D == 64    ? (const void *)kv4_gather_kernel<T, 64, true>
               : D == 128 ? (const void *)kv4_gather_kernel<T, 128, true>
                          : (const void *)kv4_gather_kernel<T, 256, true>;
    return D == 64    ? (const void *)kv4_gather_kernel<T, 64, false>
           : D == 128 ? (const void *)kv4_gather_kernel<T, 128, false>
                      : (const void *)kv4_gather_kernel<T, 256, false>;
}

}  // namespace
}  // namespace libtm

using namespace libtm;

extern "C" size_t tm_kv4_page_bytes(int32_t Hkv, int32_t D, int32_t page)
{
    if (Hkv <= 0 || !kv4_head_ok(D) || page <= 0 || page % 16 != 0) return 0;
    return (size_t)Hkv * (page / 16) * kv4_block_bytes(D);
}

extern "C" tm_status tm_kv4_append(const void *Q, int64_t qs_tok, int64_t qs_head, void *QO, int64_t qos_tok,
                                   int64_t qos_head, int32_t Hq, const void *K, int64_t ks_tok, int64_t ks_head,
                                   const void *V, int64_t vs_tok, int64_t vs_head, const int64_t *pos,
                                   const uint64_t *turns, const int64_t *slots, void *pool, int64_t pages,
                                   int32_t page, int64_t T, int32_t Hkv, int32_t D, int32_t rot, float gain,
                                   int32_t xtype, uint32_t flags, tm_stream_t stream)
{
    const int e = elem_bytes(xtype);
    if (e == 0 || (flags & ~(TM_ROPE_INTERLEAVED | TM_PDL))) return TM_ERR_INVALID_ARG;
    if (T < 0 || Hq < 0 || Hkv < 0 || rot < 0 || rot > D) return TM_ERR_INVALID_ARG;
    if (!kv4_head_ok(D) || rot % 16 != 0 || page <= 0 || page % 16 != 0) return TM_ERR_UNSUPPORTED_TILE;
    if (Hq > 65536 || Hkv > 65536 || T > INT32_MAX) return TM_ERR_INVALID_ARG;
    const Heads q = {Q, qs_tok, qs_head}, qo = {QO, qos_tok, qos_head}, k = {K, ks_tok, ks_head}, v = {V, vs_tok, vs_head};
    if (!heads_ok(q, T, Hq, D) || !heads_ok(qo, T, Hq, D) || !heads_ok(k, T, Hkv, D) || !heads_ok(v, T, Hkv, D))
        return TM_ERR_INVALID_ARG;
    if (!kv4_pool_ok(pool, pages, page, Hkv, D)) return TM_ERR_INVALID_ARG;
    if (T == 0 || Hq + Hkv == 0) return TM_OK;
    if (slots == nullptr || (rot > 0 && (pos == nullptr || turns == nullptr))) return TM_ERR_INVALID_ARG;
    if (!aligned_to(Q, e) || !aligned_to(QO, e) || !aligned_to(K, e) || !aligned_to(V, e) || !aligned_to(pool, 16) ||
        !aligned_to(pos, 8) || !aligned_to(turns, 8) || !aligned_to(slots, 8))
        return TM_ERR_MISALIGNED;
    const int64_t pb = (int64_t)tm_kv4_page_bytes(Hkv, D, page);
    const Span sq = heads_span(q, T, Hq, D, e), so = heads_span(qo, T, Hq, D, e), sk = heads_span(k, T, Hkv, D, e),
               sv = heads_span(v, T, Hkv, D, e), sp = span_of(pool, pages * pb, 1, pages * pb, 1),
               ss = span_of(slots, T, 1, T, 8), spos = rot ? span_of(pos, T, 1, T, 8) : Span{0, 0},
               st_ = rot ? span_of(turns, rot / 2, 1, rot / 2, 8) : Span{0, 0};
    if (meets(sq, so) && !(Q == QO && qs_tok == qos_tok && qs_head == qos_head)) return TM_ERR_INVALID_ARG;
    const Span ins[] = {ss, spos, st_};
    for (const Span &s : ins)
        if (meets(so, s) || meets(sp, s)) return TM_ERR_INVALID_ARG;
    if (Hq > 0 && Hkv > 0 && (heads_meet(qo, Hq, k, Hkv, T, D, e) || heads_meet(qo, Hq, v, Hkv, T, D, e)))
        return TM_ERR_INVALID_ARG;
    if (meets(sp, sq) || meets(sp, so) || meets(sp, sk) || meets(sp, sv)) return TM_ERR_INVALID_ARG;

    const bool vec = (Hq == 0 || (heads_vec(q, e) && heads_vec(qo, e))) && (Hkv == 0 || (heads_vec(k, e) && heads_vec(v, e)));
    const DevInfo *dev;
    tm_status st = device_info(&dev);
    if (st != TM_OK) return st;
    AppendArgs a = {Q, K, V, QO, qs_tok, qs_head, qos_tok, qos_head, ks_tok, ks_head, vs_tok, vs_head, pos, slots, turns,
                    reinterpret_cast<uint8_t *>(pool), pages * page, pb, page, Hq, Hkv, rot, gain, dev->status};
    const int lanes = D / 16;
    const int heads = Hq + 2 * Hkv;
    int threads = (heads * lanes + 31) / 32 * 32;
    threads = threads > 512 ? 512 : threads;
    // few tokens: heads split over blocks, each of at least a warp's heads
    int split = 1;
    while (threads > 64 && T * split * 2 <= dev->sms) {
        split *= 2;
        threads = (threads / 2 + 31) / 32 * 32;
    }
    const bool inter = (flags & TM_ROPE_INTERLEAVED) != 0;
    const void *kern = xtype == TM_F32   ? append_kernel<float>(D, vec, inter)
                       : xtype == TM_F16 ? append_kernel<__half>(D, vec, inter)
                                         : append_kernel<__nv_bfloat16>(D, vec, inter);
    void *args[] = {&a};
    return launch_kernel(kern, dim3((unsigned)T, (unsigned)split), dim3((unsigned)threads), args, 0, as_stream(stream),
                         (flags & TM_PDL) != 0);
}

extern "C" tm_status tm_kv4_gather(const void *pool, int64_t pages, int32_t page, const int64_t *slots, void *K,
                                   int64_t ks_tok, int64_t ks_head, void *V, int64_t vs_tok, int64_t vs_head,
                                   int64_t T, int32_t Hkv, int32_t D, int32_t xtype, uint32_t flags,
                                   tm_stream_t stream)
{
    const int e = elem_bytes(xtype);
    if (e == 0 || (flags & ~TM_PDL) || T < 0 || Hkv < 0) return TM_ERR_INVALID_ARG;
    if (!kv4_head_ok(D) || page <= 0 || page % 16 != 0) return TM_ERR_UNSUPPORTED_TILE;
    const Heads k = {K, ks_tok, ks_head}, v = {V, vs_tok, vs_head};
    if ((K && !heads_ok(k, T, Hkv, D)) || (V && !heads_ok(v, T, Hkv, D))) return TM_ERR_INVALID_ARG;
    if (!kv4_pool_ok(pool, pages, page, Hkv, D) || Hkv > 65536 || T > INT64_MAX / 65536) return TM_ERR_INVALID_ARG;
    if (T == 0 || Hkv == 0 || (!K && !V)) return TM_OK;
    if (slots == nullptr) return TM_ERR_INVALID_ARG;
    if (!aligned_to(K, e) || !aligned_to(V, e) || !aligned_to(pool, 16) || !aligned_to(slots, 8)) return TM_ERR_MISALIGNED;
    const int64_t pb = (int64_t)tm_kv4_page_bytes(Hkv, D, page);
    const Span sk = heads_span(k, T, Hkv, D, e), sv = heads_span(v, T, Hkv, D, e), ss = span_of(slots, T, 1, T, 8),
               sp = span_of(pool, pages * pb, 1, pages * pb, 1);
    if ((K && V && heads_meet(k, Hkv, v, Hkv, T, D, e)) || meets(sk, ss) || meets(sv, ss) || meets(sk, sp) || meets(sv, sp)) return TM_ERR_INVALID_ARG;
    const bool vec = (!K || heads_vec(k, e)) && (!V || heads_vec(v, e));
    const int64_t per = 256 / (D / 16), blocks = (T * Hkv + per - 1) / per;
    if (blocks > INT32_MAX) return TM_ERR_INVALID_ARG;
    const DevInfo *dev;
    tm_status st = device_info(&dev);
    if (st != TM_OK) return st;
    GatherArgs a = {reinterpret_cast<const uint8_t *>(pool), slots, K, V, pages * page, pb, ks_tok, ks_head, vs_tok,
                    vs_head, T, page, Hkv, make_fastdiv((uint32_t)Hkv), dev->status};
    const void *kern = xtype == TM_F32   ? gather_kernel<float>(D, vec)
                       : xtype == TM_F16 ? gather_kernel<__half>(D, vec)
                                         : gather_kernel<__nv_bfloat16>(D, vec);
    void *args[] = {&a};
    return launch_kernel(kern, dim3((unsigned)blocks), dim3(256), args, 0, as_stream(stream), (flags & TM_PDL) != 0);
}
