// tm_rope.cu -- rotary positions.
//
//   (a, b) -> gain (a cos t - b sin t, a sin t + b cos t),  t = pos * f_i
//
// Bound by HBM: each element is read and written once, against three flops.
// What could cost more is the sine and cosine (about 40 instructions a pair), so a
// warp takes a token and a run of its heads, computes the token's rot/2 pairs once
// (two or so a lane, exchanged through shared memory) and keeps the P pairs of its
// own place in registers over the heads.  A lane moves two vectors of P elements,
// the two halves of P pairs; rot/2P lanes take a head, as many heads as fit a warp
// at a time.  (Tables read from shared memory for each head instead cost a four-way
// bank conflict a read: 40 heads of 128, 8192 tokens, 30.9 against 26.1 us by the profiler.
// In a stream: 31 us, 79% of the rate of a copy of the same bytes.)
#include <cmath>

#include "tm_host.h"

#include "tm_rope.cuh"

namespace libtm {
namespace {

constexpr int kRopeWarps = 4;

struct RopeArgs {
    const void *X;
    void *Y;
    int64_t xs_tok, xs_head, ys_tok, ys_head;
    const int64_t *pos;
    const uint64_t *turns;
    int64_t T;
    int H, D, rot, heads, rest;  // heads of a task; whether dims from rot on are copied
    float gain, sign;
};

// One warp a task: a token (blockIdx.x) and `heads` of its heads (blockIdx.y).
template <typename T, int P, bool INTER>
__global__ void __launch_bounds__(kRopeWarps * 32) rope_kernel(const __grid_constant__ RopeArgs a)
{
    constexpr int kChunk = 32 * P;  // pairs a warp holds at a time
    __shared__ float2 table[kRopeWarps][kChunk];
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * kRopeWarps + warp;
    if (t >= a.T) {
        pdl_wait();
        return;
    }
    const int h0 = blockIdx.y * a.heads, h1 = min(h0 + a.heads, a.H);
    const T *x = reinterpret_cast<const T *>(a.X) + t * a.xs_tok;
    T *y = reinterpret_cast<T *>(a.Y) + t * a.ys_tok;
    const int half = a.rot / 2, groups = half / P;
    const int64_t pos = half ? a.pos[t] : 0;
    bool waited = false;
    for (int g0 = 0; g0 < groups; g0 += 32) {  // one round unless P is small and the head long
        const int gn = min(32, groups - g0), per = 32 / gn;  // lanes a head, heads at a time
        const int hl = lane / gn, gl = lane - hl * gn;
        const bool in = hl < per;
        const int i = P * (g0 + gl);  // this lane's first pair
        const int o0 = INTER ? 2 * i : i, o1 = INTER ? o0 + P : o0 + half;
        // the first heads' loads go out before the sines
        constexpr int U = 2;  // heads a lane works on at a time, and has in flight behind them
        Vec<T, P> va[2][U], vb[2][U];
        float2 cs[P];
        const int64_t xs = per * a.xs_head, ys = per * a.ys_head;
        const T *xp = x + (h0 + hl) * a.xs_head + o0;
        T *yp = y + (h0 + hl) * a.ys_head + o0;
        int left = in ? h1 - h0 - hl : 0;  // heads from this lane's next on
        auto fetch = [&](int left, Vec<T, P> (&fa)[U], Vec<T, P> (&fb)[U]) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                load_vec_if(xp, u * per < left, fa[u]);
                load_vec_if(xp + (o1 - o0), u * per < left, fb[u]);
                xp += xs;
            }
        };
        auto turn = [&](const Vec<T, P> (&fa)[U], const Vec<T, P> (&fb)[U]) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float lo[P], hi[P];
                widen(fa[u], lo);
                widen(fb[u], hi);
                rotate_pairs<P, INTER>(lo, hi, cs);
                Vec<T, P> o;
                narrow(lo, o);
                store_vec_if(yp, u * per < left, o);
                narrow(hi, o);
                store_vec_if(yp + (o1 - o0), u * per < left, o);
                yp += ys;
            }
            left -= U * per;
        };
        fetch(left, va[0], vb[0]);
        __syncwarp();
        for (int q = lane; q < gn * P; q += 32) table[warp][q] = pair_rotation(pos, a.turns[P * g0 + q], a.gain, a.sign);
        __syncwarp();
#pragma unroll
        for (int q = 0; q < P; ++q) cs[q] = table[warp][P * gl + q];
        if (!waited) pdl_wait();
        waited = true;
        const int rounds = (h1 - h0 + U * per - 1) / (U * per);
        for (int i = 0; i < rounds; i += 2) {
            fetch(i + 1 < rounds ? left - U * per : 0, va[1], vb[1]);
            turn(va[0], vb[0]);
            if (i + 1 < rounds) {
                fetch(i + 2 < rounds ? left - U * per : 0, va[0], vb[0]);
                turn(va[1], vb[1]);
            }
        }
    }
    if (!waited) pdl_wait();
    if (a.rest) {
        const int per = (a.D - a.rot) / P;
        for (int i = lane; i < (h1 - h0) * per; i += 32) {
            const int h = i / per, o = a.rot + P * (i - h * per);
            Vec<T, P> v;
            load_vec(x + (h0 + h) * a.xs_head + o, v);
            store_vec(y + (h0 + h) * a.ys_head + o, v);
        }
    }
}

template <typename T, int P>
const void *rope_pick(bool inter)
{
    return inter ? (const void *)rope_kernel<T, P, true> : (const void *)rope_kernel<T, P, false>;
}

template <typename T>
const void *rope_width(int P, bool inter)
{
    if constexpr (sizeof(T) == 2)
        if (P == 8) return rope_pick<T, 8>(inter);
    return P == 4 ? rope_pick<T, 4>(inter) : P == 2 ? rope_pick<T, 2>(inter) : rope_pick<T, 1>(inter);
}

}  // namespace
}  // namespace libtm

using namespace libtm;

extern "C" tm_status tm_rope_turns(uint64_t *turns, int32_t rot, float base, int32_t scaling, float factor, float low,
                                   float high, int64_t orig)
{
    if (turns == nullptr || rot < 2 || rot % 2 != 0 || !(base > 1.0f) || !std::isfinite(base)) return TM_ERR_INVALID_ARG;
    if (scaling < TM_ROPE_PLAIN || scaling > TM_ROPE_BY_DIM) return TM_ERR_INVALID_ARG;
    if (scaling != TM_ROPE_PLAIN && !(factor >= 1.0f && std::isfinite(factor))) return TM_ERR_INVALID_ARG;
    if (scaling == TM_ROPE_BASE && rot == 2) return TM_ERR_INVALID_ARG;
    const bool ramp = scaling == TM_ROPE_BY_TURNS || scaling == TM_ROPE_BY_DIM;
    if (ramp && !(orig > 0 && low > 0.0f && high > low && std::isfinite(high))) return TM_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586476925286766559;
    double b = base;
    if (scaling == TM_ROPE_BASE) b *= std::pow((double)factor, (double)rot / (rot - 2));
    // BY_DIM: the real index at which a pair makes n turns within orig positions
    auto index_of = [&](double n) { return rot * std::log((double)orig / (n * two_pi)) / (2.0 * std::log(b)); };
    double d0 = 0.0, d1 = 0.0;
    if (scaling == TM_ROPE_BY_DIM) {
        d0 = std::fmax(std::floor(index_of(high)), 0.0);
        d1 = std::fmin(std::ceil(index_of(low)), rot - 1.0);
        if (d1 <= d0) d1 = d0 + 0.001;
    }
    for (int i = 0; i < rot / 2; ++i) {
        double f = std::exp(-2.0 * i / rot * std::log(b));
        if (scaling == TM_ROPE_LINEAR) f /= factor;
        if (ramp) {
            double keep;  // share of the unscaled frequency
            if (scaling == TM_ROPE_BY_TURNS)
                keep = ((double)orig * f / two_pi - low) / ((double)high - low);
            else
                keep = 1.0 - (i - d0) / (d1 - d0);
            keep = std::fmin(std::fmax(keep, 0.0), 1.0);
            f = keep * f + (1.0 - keep) * f / factor;
        }
        // f <= 1 radian, so f / 2 pi * 2^64 < 2^62
        turns[i] = (uint64_t)std::llrint(std::ldexp(f / two_pi, 64));
    }
    return TM_OK;
}

extern "C" tm_status tm_rope(const void *X, int64_t xs_tok, int64_t xs_head, void *Y, int64_t ys_tok, int64_t ys_head,
                             const int64_t *pos, const uint64_t *turns, int64_t T, int32_t H, int32_t D, int32_t rot,
                             float gain, int32_t xtype, uint32_t flags, tm_stream_t stream)
{
    const int e = elem_bytes(xtype);
    if (e == 0 || (flags & ~(TM_ROPE_INTERLEAVED | TM_ROPE_INVERSE | TM_PDL))) return TM_ERR_INVALID_ARG;
    if (T < 0 || H < 0 || D < 0 || rot < 0 || rot % 2 != 0 || rot > D) return TM_ERR_INVALID_ARG;
    if (D > 1024) return TM_ERR_UNSUPPORTED_TILE;
    const Heads x = {X, xs_tok, xs_head}, y = {Y, ys_tok, ys_head};
    if (!heads_ok(x, T, H, D) || !heads_ok(y, T, H, D)) return TM_ERR_INVALID_ARG;
    if (T == 0 || H == 0 || D == 0) return TM_OK;
    if (rot > 0 && (pos == nullptr || turns == nullptr)) return TM_ERR_INVALID_ARG;
    if (!aligned_to(X, e) || !aligned_to(Y, e) || !aligned_to(pos, 8) || !aligned_to(turns, 8)) return TM_ERR_MISALIGNED;
    const Span sx = heads_span(x, T, H, D, e), sy = heads_span(y, T, H, D, e);
    if (meets(sx, sy) && !(X == Y && xs_tok == ys_tok && xs_head == ys_head)) return TM_ERR_INVALID_ARG;
    if (rot > 0 && (meets(sy, span_of(pos, T, 1, T, 8)) || meets(sy, span_of(turns, rot / 2, 1, rot / 2, 8))))
        return TM_ERR_INVALID_ARG;

    // The widest vector that every head's start, the pairs' halves and the
    // copied rest allow.
    int P = 16 / e;
    auto fits = [&](int p) {
        return p == 1 || (rot / 2 % p == 0 && (D - rot) % p == 0 && aligned_to(X, (uintptr_t)p * e) &&
                          aligned_to(Y, (uintptr_t)p * e) && xs_tok % p == 0 && xs_head % p == 0 && ys_tok % p == 0 &&
                          ys_head % p == 0);
    };
    while (!fits(P)) P /= 2;
    const DevInfo *dev;
    tm_status st = device_info(&dev);
    if (st != TM_OK) return st;
    // Tasks: at least about two rounds of the warps the GPU holds, each of some heads.
    int64_t split = (48LL * dev->sms + T - 1) / T;
    if (split > H) split = H;
    const int heads = (int)((H + split - 1) / split);
    split = (H + heads - 1) / heads;
    const int64_t blocks = (T + kRopeWarps - 1) / kRopeWarps;
    if (blocks > INT32_MAX || split > 65535) return TM_ERR_INVALID_ARG;
    RopeArgs a = {X, Y, xs_tok, xs_head, ys_tok, ys_head, pos, turns, T, H, D, rot, heads, X != Y && rot < D, gain,
                  (flags & TM_ROPE_INVERSE) ? -1.0f : 1.0f};
    const bool inter = (flags & TM_ROPE_INTERLEAVED) != 0;
    const void *k = xtype == TM_F32   ? rope_width<float>(P, inter)
                    : xtype == TM_F16 ? rope_width<__half>(P, inter)
                                      : rope_width<__nv_bfloat16>(P, inter);
    void *args[] = {&a};
    return launch_kernel(k, dim3((unsigned)blocks, (unsigned)split), dim3(kRopeWarps * 32), args, 0, as_stream(stream),
                         (flags & TM_PDL) != 0);
}
