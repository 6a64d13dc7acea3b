// tm_kv4.cu -- writing to and reading back from the 4-bit paged cache.
//
// Append: rotate q and k, hold k and v as codes (see tm.h for the format).
// Bound by HBM: q is read and written, k and v read, their (D + 8) / 2 bytes a
// vector written.  A warp takes a token and a run of its heads; its rot/2 sines
// and cosines are computed once (two a lane) and passed through shared memory, so
// no block-wide barrier is needed.  A group of D/16 lanes takes a head, 16 values
// a lane as two runs of 8 (the halves of 8 pairs, whose sines and cosines stay in
// registers over the heads): a run's codes are one 32-bit store and a vector's
// minimum and maximum two or three shuffles.  The next heads' values are loaded
// before the present ones are worked on.
//
// Exact codes.  fp32 leaves a rotated value off by up to about 2^-22 of its
// pair's size, which moves a code only where (x - low) / step is that close to
// a half, and step or low only where they are that close to a midpoint of two
// fp16 numbers.  One bound a vector finds those cases (a few vectors in a
// thousand); after its heads a warp goes through those again, in a second routine
// (out of the loop, whose registers a call in it would spill) that decides the values
// concerned, and only those, by the same formula in pairs of floats, good to 2^-41
// (fp64 runs at 1/64 of the fp32 rate here).  8192 tokens, 32 heads of 128 and 8 KV
// heads, bf16: 41 us, where its bytes need 26; issue slots 66% busy.
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
    int64_t slots_in_pool, page_bytes, T;
    int page, Hq, Hkv, rot, split;
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

// Largest and smallest of three, NaN if any is.
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float min3(float a, float b, float c)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ void extremes(const float (&x)[2][8], float &lo, float &hi)
{
    lo = hi = x[0][0];
#pragma unroll
    for (int i = 1; i < 15; i += 2) {
        lo = min3(lo, x[i / 8][i % 8], x[(i + 1) / 8][(i + 1) % 8]);
        hi = max3(hi, x[i / 8][i % 8], x[(i + 1) / 8][(i + 1) % 8]);
    }
    lo = min3(lo, x[1][7], x[1][7]);
    hi = max3(hi, x[1][7], x[1][7]);
}

// Of the vector that LANES lanes hold.
template <int LANES>
__device__ __forceinline__ void vector_extremes(const float (&x)[2][8], unsigned mask, float &lo, float &hi)
{
    extremes(x, lo, hi);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
        const float l = __shfl_xor_sync(mask, lo, o), h = __shfl_xor_sync(mask, hi, o);
        lo = min3(lo, l, l);
        hi = max3(hi, h, h);
    }
}

// How far any rotated value of a vector may be off in fp32, from the largest
// |a| + |b| of its pairs.  |cos|, |sin| are off by at most 1.5e-7 (the argument's
// rounding pi 2^-27, sincospif's last place, the gain's rounding), the products and
// the sum add 2^-23 of |a| + |b|: 2.7e-7 in all, below 1.15 * 2^-22.
template <int LANES>
__device__ __forceinline__ float vector_error(float pair, float gain, unsigned mask)
{
    return lanes_max(pair, LANES, mask) * fabsf(gain) * 0x1.28p-22f;
}

// The largest |a| + |b| of a lane's pairs, before they are turned.
template <bool INTER>
__device__ __forceinline__ float largest_pair(const float (&x)[2][8])
{
    float m[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        m[e] = INTER ? fabsf(x[e / 4][e % 4 * 2]) + fabsf(x[e / 4][e % 4 * 2 + 1]) : fabsf(x[0][e]) + fabsf(x[1][e]);
    return fmaxf(max3(m[0], m[1], m[2]), max3(max3(m[3], m[4], m[5]), m[6], m[7]));
}

// Bounds of a vector's fp32 errors: `err` is how far any of its values may be
// off.  Of the step and the low:
// (three roundings of the step: the difference, 1/15 and the product).
struct Doubt {
    float step, low;
};
__device__ __forceinline__ Doubt doubt_of(float err, float s, float lo)
{
    return {err * (2.0f / 15.0f) + s * 0x1.8p-23f, err + fabsf(lo) * 0x1p-24f};
}
__device__ __forceinline__ bool params_unsure(float err, float s, float lo)
{
    const Doubt u = doubt_of(err, s, lo);
    return __half_as_ushort(held_half(s - u.step)) != __half_as_ushort(held_half(s + u.step)) ||
           __half_as_ushort(held_half(lo - u.low)) != __half_as_ushort(held_half(lo + u.low));
}

// ---------------------------------------------------------------- pairs of floats
// h + l with |l| at most half the last place of h: 48 bits, from the error-free sum
// (Knuth) and product (one fused multiply-add) of two floats.
struct Pair {
    float h, l;
};

__device__ __forceinline__ Pair sum_of(float a, float b)
{
    const float s = __fadd_rn(a, b), t = __fadd_rn(s, -a);
    return {s, __fadd_rn(__fadd_rn(a, -__fadd_rn(s, -t)), __fadd_rn(b, -t))};
}
__device__ __forceinline__ Pair product_of(float a, float b)
{
    const float p = __fmul_rn(a, b);
    return {p, __fmaf_rn(a, b, -p)};
}
__device__ __forceinline__ Pair add(Pair a, Pair b)
{
    const Pair s = sum_of(a.h, b.h), t = sum_of(a.l, b.l), u = sum_of(s.h, __fadd_rn(s.l, t.h));
    return sum_of(u.h, __fadd_rn(u.l, t.l));
}
__device__ __forceinline__ Pair mul(Pair a, Pair b)
{
    const Pair p = product_of(a.h, b.h);
    return sum_of(p.h, __fmaf_rn(a.h, b.l, __fmaf_rn(a.l, b.h, p.l)));
}
__device__ __forceinline__ bool less(Pair a, Pair b) { return a.h < b.h || (a.h == b.h && a.l < b.l); }

// cos and sin of a signed fraction of a turn (units of 2^-64), good to about 2^-41:
// the nearest quarter turn comes off exactly, then Taylor's series over [-pi/4, pi/4],
// its first terms in pairs, the others (below 2^-20 of the result) in floats.
__device__ __forceinline__ void exact_rotation(int64_t fraction, Pair &c, Pair &s)
{
    const uint64_t f = (uint64_t)fraction, quarter = (f + (1ull << 61)) >> 62;
    const int64_t r = (int64_t)(f - (quarter << 62));  // |r| <= 2^61
    const float rh = (float)(int32_t)(r >> 32);
    const int64_t rest = r - ((int64_t)(int32_t)rh << 32);  // |rest| < 2^38
    const float rl = (float)(int32_t)(rest >> 8);
    const Pair x = mul(sum_of(rh * 0x1p-32f, rl * 0x1p-56f), {0x1.921fb6p+2f, -0x1.777a5cp-23f});  // 2 pi
    const Pair z = mul(x, x);
    const float zh = z.h;
    // sin x = x - x^3 (1/3! - z/5! + z^2/7! - z^3 (1/9! - z/11! + z^2/13!))
    float t = fmaf(zh, fmaf(zh, 1.6059044e-10f, -2.5052108e-8f), 2.7557319e-6f);
    Pair u = add({0x1.a01a02p-13f, -0x1.7f97fap-39f}, {-zh * t, 0.0f});
    u = mul(z, u);
    u = add({0x1.111112p-7f, -0x1.dddddep-32f}, {-u.h, -u.l});
    u = mul(z, u);
    u = add({0x1.555556p-3f, -0x1.555556p-28f}, {-u.h, -u.l});
    u = mul(mul(x, z), u);
    const Pair sn = add(x, {-u.h, -u.l});
    // cos x = 1 - z (1/2 - z/4! + z^2/6! - z^3 (1/8! - z/10! + z^2/12! - z^3/14!))
    t = fmaf(zh, fmaf(zh, fmaf(zh, -1.1470746e-11f, 2.0876757e-9f), -2.7557319e-7f), 2.4801587e-5f);
    u = add({0x1.6c16c2p-10f, -0x1.27d27ep-35f}, {-zh * t, 0.0f});
    u = mul(z, u);
    u = add({0x1.555556p-5f, -0x1.555556p-30f}, {-u.h, -u.l});
    u = mul(z, u);
    u = add({0.5f, 0.0f}, {-u.h, -u.l});
    u = mul(z, u);
    const Pair cn = add({1.0f, 0.0f}, {-u.h, -u.l});
    c = quarter & 1 ? Pair{-sn.h, -sn.l} : cn;
    s = quarter & 1 ? cn : sn;
    if (quarter & 2) {
        c = {-c.h, -c.l};
        s = {-s.h, -s.l};
    }
}

// Value i (0 .. 15) of a lane to 2^-41 of its pair's size, from the tensor.
template <typename T, bool INTER>
__device__ __noinline__ Pair exact_value(const T *p, int o0, int o1, bool turn, int64_t pos, const uint64_t *turns,
                                         float gain, int i)
{
    if (!turn) return {to_f(i < 8 ? p[o0 + i] : p[o1 + i - 8]), 0.0f};
    const int pair = INTER ? i / 2 : i % 8;
    const bool first = INTER ? i % 2 == 0 : i < 8;
    const float a = to_f(INTER ? (pair < 4 ? p[o0 + 2 * pair] : p[o1 + 2 * pair - 8]) : p[o0 + pair]);
    const float b = to_f(INTER ? (pair < 4 ? p[o0 + 2 * pair + 1] : p[o1 + 2 * pair - 7]) : p[o1 + pair]);
    Pair c, s;
    exact_rotation(turn_fraction(pos, turns[pair]), c, s);
    const Pair r = first ? add(mul({a, 0.0f}, c), mul({-b, 0.0f}, s)) : add(mul({a, 0.0f}, s), mul({b, 0.0f}, c));
    return mul(r, {gain, 0.0f});
}

// (x - low) / step to the nearest whole number in 0 .. 15, a tie to the even one:
// k from floats is at most one off, and k step is exact.
__device__ __forceinline__ int exact_code(Pair x, float low, float step)
{
    const Pair d = add(x, {-low, 0.0f});
    float k = fminf(fmaxf(rintf(d.h / step), 0.0f), 15.0f);
    const Pair r = add(d, {-k * step, 0.0f});
    const Pair up = add(r, {-0.5f * step, 0.0f}), down = add(r, {0.5f * step, 0.0f});
    const bool odd = (int)k & 1;
    if (up.h > 0.0f || (up.h == 0.0f && odd))
        k += 1.0f;
    else if (down.h < 0.0f || (down.h == 0.0f && odd))
        k -= 1.0f;
    return (int)fminf(fmaxf(k, 0.0f), 15.0f);
}

// The slow path: two words of codes and (step, low), whatever is in doubt in pairs.
// Called by all D/16 lanes of a vector without NaN or infinity.
template <typename T, int D, bool VEC, bool INTER>
__device__ __noinline__ uint3 hold_exactly(const T *p, int o0, int o1, bool rotated, bool turn, int64_t pos, const uint64_t *turns,
                                           float gain, const float2 *table)
{
    constexpr int LANES = D / 16;
    const unsigned lane = threadIdx.x & 31, mask = LANES == 32 ? 0xffffffffu : ((1u << LANES) - 1) << (lane / LANES * LANES);
    float x[2][8];
    float2 cs[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) cs[e] = turn ? table[e] : make_float2(1.0f, 0.0f);
    load8<T, VEC>(p + o0, x[0]);
    load8<T, VEC>(p + o1, x[1]);
    float err = 0.0f, lo, hi;
    if (rotated) err = vector_error<LANES>(turn ? largest_pair<INTER>(x) : 0.0f, gain, mask);
    if (turn) rotate_pairs<8, INTER>(x[0], x[1], cs);
    vector_extremes<LANES>(x, mask, lo, hi);
    const float s = (hi - lo) * (1.0f / 15.0f);
    __half step = held_half(s), low = held_half(lo);
    if (params_unsure(err, s, lo)) {  // the same for every lane of the vector
        uint32_t extreme = 0;  // the values that may be the minimum or the maximum
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (x[i / 8][i % 8] <= lo + 2 * err || x[i / 8][i % 8] >= hi - 2 * err) extreme |= 1u << i;
        Pair least = {INFINITY, 0.0f}, most = {-INFINITY, 0.0f};
        for (; extreme; extreme &= extreme - 1) {
            const Pair d = exact_value<T, INTER>(p, o0, o1, turn, pos, turns, gain, __ffs(extreme) - 1);
            least = less(d, least) ? d : least;
            most = less(most, d) ? d : most;
        }
        __syncwarp(mask);
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) {
            const Pair l = {__shfl_xor_sync(mask, least.h, o), __shfl_xor_sync(mask, least.l, o)};
            const Pair m = {__shfl_xor_sync(mask, most.h, o), __shfl_xor_sync(mask, most.l, o)};
            least = less(l, least) ? l : least;
            most = less(most, m) ? m : most;
        }
        // a fifteenth of the spread: the quotient of the first part, and what it leaves
        const Pair d = add(most, {-least.h, -least.l});
        const float q = d.h / 15.0f, rest = fmaf(-q, 15.0f, d.h) + d.l;
        step = held_half(sum_of(q, rest * (1.0f / 15.0f)).h);
        low = held_half(least.h);
    }
    const float fs = __half2float(step), fl = __half2float(low);
    const float inv = fs > 0.0f ? 1.0f / fs : 0.0f;
    uint32_t word[2] = {0, 0}, close = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float d = x[i / 8][i % 8] - fl, t = d * inv, r = rintf(t);
        // the value's error, the difference's rounding and the product's
        const float et = (err + fabsf(d) * 0x1p-23f) * inv + fabsf(t) * 0x1p-22f;
        if (fs > 0.0f && fabsf(t - r) + et >= 0.5f && t > -1.0f && t < 16.0f) close |= 1u << i;
        word[i / 8] |= (uint32_t)fminf(fmaxf(r, 0.0f), 15.0f) << (i % 8 * 4);
    }
    for (; close; close &= close - 1) {
        const int i = __ffs(close) - 1, sh = i % 8 * 4;
        const uint32_t c = (uint32_t)exact_code(exact_value<T, INTER>(p, o0, o1, turn, pos, turns, gain, i), fl, fs) << sh;
        if (i < 8)
            word[0] = (word[0] & ~(15u << sh)) | c;
        else
            word[1] = (word[1] & ~(15u << sh)) | c;
    }
    const __half2 params = __halves2half2(step, low);
    return make_uint3(word[0], word[1], *reinterpret_cast<const uint32_t *>(&params));
}

constexpr int kAppendWarps = 1;

// One warp a task: a token (blockIdx.x) and one of the `split` parts (blockIdx.y) of
// its passes of 512 / D heads.
template <typename T, int D, bool VEC, bool INTER>
__global__ void __launch_bounds__(kAppendWarps * 32, 24) kv4_append_kernel(const __grid_constant__ AppendArgs a)
{
    constexpr int LANES = D / 16, PER = 32 / LANES;  // lanes a head, heads a pass
    __shared__ float2 table[kAppendWarps][D / 2];
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, ln = lane % LANES;
    const int64_t t = (int64_t)blockIdx.x * kAppendWarps + warp;
    const int part = blockIdx.y;
    if (t >= a.T) {
        pdl_wait();
        return;
    }
    // passes over the query heads, then the key heads, then the value heads
    const int nq = (a.Hq + PER - 1) / PER, nk = (a.Hkv + PER - 1) / PER, passes = nq + 2 * nk;
    const int pass0 = passes * part / a.split, pass1 = passes * (part + 1) / a.split;

    const int half = a.rot / 2;
    const bool turned = ln < a.rot / 16;  // this lane's 16 dims are 8 pairs
    const int q0 = !turned || INTER ? 16 * ln : 8 * ln, q1 = !turned || INTER ? q0 + 8 : q0 + half;
    // This lane's two runs of its head of a pass; false past the last head.
    const int hl = lane / LANES, v0 = 8 * ln, v1 = v0 + D / 2;  // (a warp's accesses stay contiguous)
    const T *q_base = reinterpret_cast<const T *>(a.Q) + t * a.qs_tok, *k_base = reinterpret_cast<const T *>(a.K) + t * a.ks_tok,
            *v_base = reinterpret_cast<const T *>(a.V) + t * a.vs_tok;
    auto source = [&](int pass, const T *&p0, const T *&p1) -> bool {
        if (pass < nq) {
            const int h = pass * PER + hl;
            p0 = q_base + h * a.qs_head + q0;
            p1 = p0 + (q1 - q0);
            return h < a.Hq;
        }
        pass -= nq;
        if (pass < nk) {
            const int h = pass * PER + hl;
            p0 = k_base + h * a.ks_head + q0;
            p1 = p0 + (q1 - q0);
            return h < a.Hkv;
        }
        const int h = (pass - nk) * PER + hl;
        p0 = v_base + h * a.vs_head + v0;
        p1 = p0 + D / 2;
        return h < a.Hkv;
    };
    // Vectors of the next kDepth - 1 passes are on their way to shared memory (every lane
    // copies and reads its own 2 x 8 values, so nothing has to be waited for but its own
    // copies); off the 16-byte grid they are read when they are needed.
    constexpr int kDepth = 4, kParts = 8 * sizeof(T) / 16;  // 16-byte parts of a run
    __shared__ __align__(16) uint4 ring[VEC ? kAppendWarps * kDepth * 2 * kParts * 32 : 1];
    uint4 *mine = ring + (VEC ? warp * (kDepth * 2 * kParts * 32) + lane : 0);
    auto copy = [&](int pass) {
        if constexpr (VEC) {
            const T *p0, *p1;
            if (pass < pass1 && source(pass, p0, p1)) {
                uint4 *d = mine + (pass - pass0) % kDepth * (2 * kParts * 32);
#pragma unroll
                for (int i = 0; i < kParts; ++i) {
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(d + i * 32)),
                                 "l"(reinterpret_cast<const char *>(p0) + 16 * i)
                                 : "memory");
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(d + (kParts + i) * 32)),
                                 "l"(reinterpret_cast<const char *>(p1) + 16 * i)
                                 : "memory");
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    };
    auto take = [&](int pass, float (&x)[2][8]) {
        if constexpr (VEC) {
            copy(pass + kDepth - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
            const uint4 *d = mine + (pass - pass0) % kDepth * (2 * kParts * 32);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                Vec<T, 8> v;
#pragma unroll
                for (int i = 0; i < kParts; ++i) reinterpret_cast<uint4 *>(&v)[i] = d[(u * kParts + i) * 32];
                widen(v, x[u]);
            }
        } else {
            const T *p0, *p1;
            if (source(pass, p0, p1)) {
                load8<T, false>(p0, x[0]);
                load8<T, false>(p1, x[1]);
            }
        }
    };
    for (int i = 0; i < kDepth - 1; ++i) copy(pass0 + i);
    const int64_t slot = a.slots[t], pos = a.rot > 0 ? a.pos[t] : 0;
    for (int i = lane; i < half; i += 32) table[warp][i] = pair_rotation(pos, a.turns[i], a.gain, 1.0f);
    __syncwarp();
    float2 cs[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) cs[e] = turned ? table[warp][8 * ln + e] : make_float2(1.0f, 0.0f);

    const bool held = slot >= 0 && slot < a.slots_in_pool;
    if (!held && slot != -1 && lane == 0 && part == 0) atomicOr(a.status, kStatusIndex);
    uint8_t *block = nullptr;  // of KV head 0
    int r = 0;
    if (held) {
        const int64_t pg = slot <= INT32_MAX ? (int64_t)((uint32_t)slot / (uint32_t)a.page) : slot / a.page;
        const int at = (int)(slot - pg * a.page);
        block = a.pool + pg * a.page_bytes + (int64_t)(at / 16) * kv4_block_bytes(D);
        r = at % 16;
    }
    const int64_t head_bytes = (int64_t)(a.page / 16) * kv4_block_bytes(D);
    pdl_wait();

    // Hold a vector and store it at its words of a block, its (step, low) at `at`.
    const unsigned mask = LANES == 32 ? 0xffffffffu : ((1u << LANES) - 1) << (lane / LANES * LANES);
    // True if fp32 could not decide all of it; err: how far any of its values may be off.
    auto hold = [&](float (&x)[2][8], float err, uint8_t *w0, uint8_t *w1, uint8_t *at) -> bool {
        float lo, hi;
        vector_extremes<LANES>(x, mask, lo, hi);  // NaN if any value is
        bool unsure = false;
        uint32_t word[2];
        __half2 params;
        if (!(hi - lo < INFINITY)) {
            word[0] = word[1] = 0;
            params = __halves2half2(__ushort_as_half(0x7fff), __ushort_as_half(0x7fff));
        } else {
            const float s = (hi - lo) * (1.0f / 15.0f);
            const __half step = held_half(s), low = held_half(lo);
            unsure = params_unsure(err, s, lo);
            const float fs = __half2float(step), fl = __half2float(low);
            const float inv = fs > 0.0f ? 1.0f / fs : 0.0f;
            // t = (x - low) / step as 15 times a value cut to [0, 1]; adding 1.5 * 2^23
            // rounds it to a whole number, in the low bits of the sum
            const float m15 = inv * (1.0f / 15.0f), magic = 12582912.0f;
            float off = 0.0f;  // the largest distance from a whole number
            word[0] = word[1] = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float t15 = __saturatef((x[i / 8][i % 8] - fl) * m15);
                const float sum = fmaf(t15, 15.0f, magic), whole = sum - magic;
                off = fmaxf(off, fabsf(fmaf(t15, 15.0f, -whole)));
                word[i / 8] += __float_as_uint(sum) << (i % 8 * 4);
            }
            word[0] -= 0x4b400000u * 0x11111111u;
            word[1] -= 0x4b400000u * 0x11111111u;
            params = __halves2half2(step, low);
            // the values' error, and what t, at most 14.5 where it matters, is off by: m15 by 2.54 2^-24
            // of itself (three roundings, over every fp16 step), the difference by 2^-24, the cut
            // value, below 1, by 2^-25: 14.5 * 3.54 + 15 / 2 of 2^-24, below 15 * 4
            const float et = err * inv + 15.0f * 0x1p-22f;
            unsure = unsure || off + et >= 0.5f;
        }
        *reinterpret_cast<uint32_t *>(w0) = word[0];
        *reinterpret_cast<uint32_t *>(w1) = word[1];
        if (ln == 0) *reinterpret_cast<__half2 *>(at) = params;
        return __any_sync(mask, unsure);
    };
    float x[2][8];
    for (int pass = pass0; pass < min(pass1, nq); ++pass) {
        take(pass, x);
        if (turned) rotate_pairs<8, INTER>(x[0], x[1], cs);
        const int h = pass * PER + hl;
        if (h < a.Hq) {
            T *o = reinterpret_cast<T *>(a.QO) + t * a.qos_tok + h * a.qos_head;
            store8<T, VEC>(o + q0, x[0]);
            store8<T, VEC>(o + q1, x[1]);
        }
    }
    if (!held) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        return;
    }
    // Keys and values in one loop: two would not fit the instruction cache together.
    uint32_t again = 0;  // passes to go through again, from the first of keys or values
    const int first = max(pass0, nq), kw0 = kv4_k_word(D, r, q0), kw1 = kv4_k_word(D, r, q1),
              vw0 = kv4_v_word(D, r, v0), vw1 = kv4_v_word(D, r, v1);
    for (int pass = first; pass < pass1; ++pass) {
        take(pass, x);
        const bool k = pass < nq + nk;
        const int h = (pass - nq - (k ? 0 : nk)) * PER + hl;
        if (h < a.Hkv) {  // whole groups of lanes
            float err = 0.0f;
            if (k && a.rot > 0) {
                err = vector_error<LANES>(turned ? largest_pair<INTER>(x) : 0.0f, a.gain, mask);
                if (turned) rotate_pairs<8, INTER>(x[0], x[1], cs);
            }
            uint8_t *b = block + h * head_bytes;
            if (hold(x, err, b + (k ? kw0 : vw0), b + (k ? kw1 : vw1), b + (k ? kv4_ks_off(D) : kv4_vs_off(D)) + 4 * r))
                again |= 1u << (pass - first);
        }
    }
    for (; again; again &= again - 1) {
        const int pass = first + __ffs(again) - 1;
        const bool k = pass < nq + nk;
        const int h = (pass - nq - (k ? 0 : nk)) * PER + hl;
        const T *p = k ? k_base + h * a.ks_head : v_base + h * a.vs_head;
        const bool turn = k && turned;
        const uint3 w = hold_exactly<T, D, VEC, INTER>(p, k ? q0 : v0, k ? q1 : v1, k && a.rot > 0, turn, pos,
                                                       a.turns + 8 * ln, a.gain, &table[warp][turn ? 8 * ln : 0]);
        uint8_t *b = block + h * head_bytes;
        *reinterpret_cast<uint32_t *>(b + (k ? kw0 : vw0)) = w.x;
        *reinterpret_cast<uint32_t *>(b + (k ? kw1 : vw1)) = w.y;
        if (ln == 0) *reinterpret_cast<uint32_t *>(b + (k ? kv4_ks_off(D) : kv4_vs_off(D)) + 4 * r) = w.z;
    }
}

struct GatherArgs {
    const uint8_t *pool;
    const int64_t *slots;
    void *K, *V;
    int64_t slots_in_pool, page_bytes, ks_tok, ks_head, vs_tok, vs_head, T;
    int page, Hkv;
    FastDiv by_heads, by_page;
    unsigned *status;
};

// Bound by HBM: D/2 + 4 bytes read and D elements written a vector.  A group of D/8
// lanes takes a (token, head) item, 8 values of K and 8 of V a lane: a word read and a
// 16-byte vector written each, contiguous over the lanes (16 values a lane wrote every
// other 16 bytes at a time: 14.9 against 12.4 us for 8192 tokens of 8 heads of 128).  A
// thread asks for all of its items' words before it works on the first.
constexpr int kGatherItems = 4;

template <typename T, int D, bool VEC>
__global__ void __launch_bounds__(256) kv4_gather_kernel(const __grid_constant__ GatherArgs a)
{
    constexpr int LANES = D / 8, PER = 256 / LANES;
    pdl_trigger();
    const int d = threadIdx.x % LANES * 8;
    const int64_t item0 = (int64_t)blockIdx.x * (PER * kGatherItems) + threadIdx.x / LANES;
    uint32_t kw[kGatherItems], vw[kGatherItems], ks[kGatherItems], vs[kGatherItems];
    int64_t tok[kGatherItems], slot[kGatherItems];
    int head[kGatherItems];
#pragma unroll
    for (int i = 0; i < kGatherItems; ++i) {
        const int64_t item = item0 + i * PER;
        const bool in = item < a.T * a.Hkv;
        tok[i] = item <= INT32_MAX ? (int64_t)fdiv((uint32_t)item, a.by_heads) : item / a.Hkv;
        head[i] = (int)(item - tok[i] * a.Hkv);
        slot[i] = in ? a.slots[tok[i]] : -1;
        tok[i] = in ? tok[i] : -1;
    }
#pragma unroll
    for (int i = 0; i < kGatherItems; ++i) {
        kw[i] = vw[i] = ks[i] = vs[i] = 0;  // slot -1: zeros
        if (slot[i] >= 0 && slot[i] < a.slots_in_pool) {
            const int64_t pg = slot[i] <= INT32_MAX ? (int64_t)fdiv((uint32_t)slot[i], a.by_page) : slot[i] / a.page;
            const int at = (int)(slot[i] - pg * a.page), r = at % 16;
            const uint8_t *b =
                a.pool + pg * a.page_bytes + ((int64_t)head[i] * (a.page / 16) + at / 16) * kv4_block_bytes(D);
            kw[i] = ld_nc_b32(b + kv4_k_word(D, r, d));
            vw[i] = ld_nc_b32(b + kv4_v_word(D, r, d));
            ks[i] = ld_nc_b32(b + kv4_ks_off(D) + 4 * r);
            vs[i] = ld_nc_b32(b + kv4_vs_off(D) + 4 * r);
        } else if (slot[i] != -1 && d == 0) {
            atomicOr(a.status, kStatusIndex);
        }
    }
    pdl_wait();
#pragma unroll
    for (int i = 0; i < kGatherItems; ++i) {
        if (tok[i] < 0) continue;
        const float2 kp = __half22float2(*reinterpret_cast<const __half2 *>(&ks[i]));
        const float2 vp = __half22float2(*reinterpret_cast<const __half2 *>(&vs[i]));
        float k8[8], v8[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            k8[e] = fmaf((float)(kw[i] >> (4 * e) & 15u), kp.x, kp.y);
            v8[e] = fmaf((float)(vw[i] >> (4 * e) & 15u), vp.x, vp.y);
        }
        if (a.K) store8<T, VEC>(reinterpret_cast<T *>(a.K) + tok[i] * a.ks_tok + head[i] * a.ks_head + d, k8);
        if (a.V) store8<T, VEC>(reinterpret_cast<T *>(a.V) + tok[i] * a.vs_tok + head[i] * a.vs_head + d, v8);
    }
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
    // Tasks: about two rounds of the warps the GPU holds, each at least one pass of heads.
    const int64_t per = 512 / D, passes = (Hq + per - 1) / per + 2 * ((Hkv + per - 1) / per), want = 40LL * dev->sms;
    int64_t split = (want + T - 1) / T;
    if (split * 32 < passes) split = (passes + 31) / 32;  // a task notes its passes in 32 bits
    if (split > passes) split = passes;
    AppendArgs a = {Q, K, V, QO, qs_tok, qs_head, qos_tok, qos_head, ks_tok, ks_head, vs_tok, vs_head, pos, slots, turns,
                    reinterpret_cast<uint8_t *>(pool), pages * page, pb, T, page, Hq, Hkv, rot, (int)split, gain,
                    dev->status};
    const int64_t blocks = (T + kAppendWarps - 1) / kAppendWarps;
    if (split > 65535) return TM_ERR_INVALID_ARG;
    const bool inter = (flags & TM_ROPE_INTERLEAVED) != 0;
    const void *kern = xtype == TM_F32   ? append_kernel<float>(D, vec, inter)
                       : xtype == TM_F16 ? append_kernel<__half>(D, vec, inter)
                                         : append_kernel<__nv_bfloat16>(D, vec, inter);
    void *args[] = {&a};
    return launch_kernel(kern, dim3((unsigned)blocks, (unsigned)split), dim3(kAppendWarps * 32), args, 0, as_stream(stream),
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
    const int64_t per = 256 / (D / 8) * kGatherItems, blocks = (T * Hkv + per - 1) / per;
    if (blocks > INT32_MAX) return TM_ERR_INVALID_ARG;
    const DevInfo *dev;
    tm_status st = device_info(&dev);
    if (st != TM_OK) return st;
    GatherArgs a = {reinterpret_cast<const uint8_t *>(pool), slots, K, V, pages * page, pb, ks_tok, ks_head, vs_tok,
                    vs_head, T, page, Hkv, make_fastdiv((uint32_t)Hkv), make_fastdiv((uint32_t)page), dev->status};
    const void *kern = xtype == TM_F32   ? gather_kernel<float>(D, vec)
                       : xtype == TM_F16 ? gather_kernel<__half>(D, vec)
                                         : gather_kernel<__nv_bfloat16>(D, vec);
    void *args[] = {&a};
    return launch_kernel(kern, dim3((unsigned)blocks), dim3(256), args, 0, as_stream(stream), (flags & TM_PDL) != 0);
}
