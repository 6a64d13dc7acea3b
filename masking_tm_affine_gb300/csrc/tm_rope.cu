// tm_rope.cu -- rotary positions.
//
//   (a, b) -> gain (a cos t - b sin t, a sin t + b cos t),  t = pos * f_i
//
// Bound by HBM: each element is read and written once, against three flops.
// What could cost more is the sine and cosine (about 40 instructions a pair),
// so a block takes a run of tokens, computes each token's rot/2 pairs once
// into shared memory and then walks the tokens' heads with them: with 40 heads
// of 128 that is half an instruction an element.  A lane moves two vectors of
// P elements, the two halves of P pairs.
#include <cmath>

#include "tm_host.h"

#include "tm_rope.cuh"

namespace libtm {
namespace {

struct RopeArgs {
    const void *X;
    void *Y;
    int64_t xs_tok, xs_head, ys_tok, ys_head;
    const int64_t *pos;
    const uint64_t *turns;
    int64_t T;
    int H, D, rot, tokens;  // tokens per block
    float gain, sign;
    FastDiv by_items, by_groups;  // items of a token; pair groups of a head
};

// Items of a token: H heads x (rot / 2P rotated groups + (D - rot) / P copied
// vectors).  blockIdx.x walks token runs, blockIdx.y splits the items of a run
// (few tokens, many heads).
template <typename T, int P, bool INTER>
__global__ void __launch_bounds__(256) rope_kernel(const __grid_constant__ RopeArgs a)
{
    extern __shared__ float2 cs[];  // [tokens][rot / 2]
    pdl_trigger();
    const int half = a.rot / 2;
    const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
    const int n = (int)(a.T - t0 < a.tokens ? a.T - t0 : a.tokens);
    for (int i = threadIdx.x; i < n * half; i += blockDim.x) {
        const int t = i / half, q = i - t * half;
        cs[i] = pair_rotation(a.pos[t0 + t], a.turns[q], a.gain, a.sign);
    }
    __syncthreads();
    const int groups = half / P, per_head = groups + (a.D - a.rot) / P, items = a.H * per_head;
    bool waited = false;
    for (int i = blockIdx.y * blockDim.x + threadIdx.x; i < n * items; i += gridDim.y * blockDim.x) {
        const int t = (int)fdiv((uint32_t)i, a.by_items), it = i - t * items;
        const int h = (int)fdiv((uint32_t)it, a.by_groups), g = it - h * per_head;
        const T *x = reinterpret_cast<const T *>(a.X) + (t0 + t) * a.xs_tok + h * a.xs_head;
        T *y = reinterpret_cast<T *>(a.Y) + (t0 + t) * a.ys_tok + h * a.ys_head;
        if (g < groups) {
            const int o0 = INTER ? 2 * P * g : P * g, o1 = INTER ? o0 + P : o0 + half;
            Vec<T, P> va, vb;
            load_vec(x + o0, va);
            load_vec(x + o1, vb);
            float lo[P], hi[P];
            float2 r[P];
#pragma unroll
            for (int q = 0; q < P; ++q) r[q] = cs[t * half + P * g + q];
            widen(va, lo);
            widen(vb, hi);
            rotate_pairs<P, INTER>(lo, hi, r);
            narrow(lo, va);
            narrow(hi, vb);
            if (!waited) pdl_wait();
            waited = true;
            store_vec(y + o0, va);
            store_vec(y + o1, vb);
        } else {
            const int o = a.rot + P * (g - groups);
            Vec<T, P> v;
            load_vec(x + o, v);
            if (!waited) pdl_wait();
            waited = true;
            store_vec(y + o, v);
        }
    }
    if (!waited) pdl_wait();
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
    const int per_head = rot / 2 / P + (D - rot) / P;
    const int64_t items = (int64_t)H * per_head;
    if (items > (1 << 24)) return TM_ERR_INVALID_ARG;
    const DevInfo *dev;
    tm_status st = device_info(&dev);
    if (st != TM_OK) return st;
    // Tokens per block: enough items for several rounds of the block, while
    // every SM keeps some blocks; few tokens split their items over blocks.
    int tokens = 1;
    while (tokens < 16 && tokens * rot <= 4096 && tokens * items < 2048 && T / (2 * tokens) >= 4LL * dev->sms) tokens *= 2;
    const int64_t blocks = (T + tokens - 1) / tokens;
    if (blocks > INT32_MAX) return TM_ERR_INVALID_ARG;
    int64_t split = 1;
    while (split < 64 && blocks * split < 2LL * dev->sms && split * 256 < tokens * items) split *= 2;
    RopeArgs a = {X, Y, xs_tok, xs_head, ys_tok, ys_head, pos, turns, T, H, D, rot, tokens, gain,
                  (flags & TM_ROPE_INVERSE) ? -1.0f : 1.0f, make_fastdiv((uint32_t)items),
                  make_fastdiv((uint32_t)per_head)};
    const bool inter = (flags & TM_ROPE_INTERLEAVED) != 0;
    const void *k = xtype == TM_F32   ? rope_width<float>(P, inter)
                    : xtype == TM_F16 ? rope_width<__half>(P, inter)
                                      : rope_width<__nv_bfloat16>(P, inter);
    void *args[] = {&a};
    return launch_kernel(k, dim3((unsigned)blocks, (unsigned)split), dim3(256), args,
                         (size_t)tokens * (rot / 2) * sizeof(float2), as_stream(stream), (flags & TM_PDL) != 0);
}
