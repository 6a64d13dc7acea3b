// tm_rope.cuh -- the rotation shared by tm_rope and the cache append.
//
// Angles.  turns_i is the pair's frequency in turns a position, times 2^64, so
// p * turns_i in wrapping 64-bit integers is the exact fraction of a turn at
// position p (for |p| up to 2^63; the only error is turns_i's own rounding,
// p * 2^-65 turns).  Read as a signed number it is the angle in units of
// 2^-63 * pi within [-pi, pi).
// fp32 angles formed as p * f_i would be off by 0.03 radians at p = 2^20.
#pragma once

#include "tm_elem.cuh"

namespace libtm {

__device__ __forceinline__ int64_t turn_fraction(int64_t pos, uint64_t turns)
{
    return (int64_t)((uint64_t)pos * turns);
}

// (cos, sin) * gain of a pair; sign -1 turns back.
__device__ __forceinline__ float2 pair_rotation(int64_t pos, uint64_t turns, float gain, float sign)
{
    // The nearest quarter turn comes off exactly, in integers, so that what is rounded is
    // at most an eighth of a turn.  The upper 32 bits are enough (2^-32 of a turn) and
    // convert at full rate, 64 bits do not.
    const uint32_t f = (uint32_t)((uint64_t)turn_fraction(pos, turns) >> 32);
    const uint32_t quarter = (f + 0x20000000u) >> 30;
    float s, c;
    sincospif((float)(int32_t)(f - (quarter << 30)) * 0x1p-31f, &s, &c);
    const float u = quarter & 1 ? -s : c, v = quarter & 1 ? c : s;
    const float g = quarter & 2 ? -gain : gain;
    return make_float2(u * g, v * g * sign);
}

// A lane's P pairs: `lo` and `hi` hold its two vectors of P elements.  Half
// layout: pair q is (lo[q], hi[q]).  Interleaved: the 2P elements are
// contiguous, pair q is elements 2q and 2q + 1 of them.
template <int P, bool INTER>
__device__ __forceinline__ void rotate_pairs(float (&lo)[P], float (&hi)[P], const float2 (&cs)[P])
{
#pragma unroll
    for (int q = 0; q < P; ++q) {
        float *a, *b;
        if constexpr (INTER && P > 1) {
            a = 2 * q < P ? &lo[2 * q] : &hi[2 * q - P];
            b = 2 * q + 1 < P ? &lo[2 * q + 1] : &hi[2 * q + 1 - P];
        } else {
            a = &lo[q];
            b = &hi[q];
        }
        const float x = *a, y = *b;
        *a = fmaf(x, cs[q].x, -(y * cs[q].y));
        *b = fmaf(x, cs[q].y, y * cs[q].x);
    }
}

}  // namespace libtm
