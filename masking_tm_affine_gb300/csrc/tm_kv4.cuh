// tm_kv4.cuh -- the layout of the 4-bit paged cache (described in tm.h), shared
// by the append, the gather and the attention.
#pragma once

#include <cstdint>

namespace libtm {

// Blocks of 16 tokens of one KV head: K codes, V codes, K scales, V scales.
// All byte offsets inside a block; 16 (D + 8) bytes, a multiple of 128 for
// every D, so a block (and any run of blocks of a page) is one bulk copy.
constexpr int kBlockTokens = 16;

__host__ __device__ constexpr int kv4_block_bytes(int D) { return 16 * (D + 8); }
__host__ __device__ constexpr int kv4_v_off(int D) { return 8 * D; }
__host__ __device__ constexpr int kv4_ks_off(int D) { return 16 * D; }
__host__ __device__ constexpr int kv4_vs_off(int D) { return 16 * D + 64; }

// Byte offset within a block of the 4 bytes that hold dims d .. d + 7 (d a
// multiple of 8) of token r.
__host__ __device__ constexpr int kv4_k_word(int D, int r, int d) { return r * (D / 2) + d / 2; }
__host__ __device__ constexpr int kv4_v_word(int D, int r, int d)
{
    return kv4_v_off(D) + (r >> 1) * D + d / (D / 8) * (D / 8) + (r & 1) * (D / 16) + d % (D / 8) / 2;
}

inline bool kv4_head_ok(int D) { return D == 64 || D == 128 || D == 256; }

// Largest pool the kernels address, in tokens (a slot number fits 62 bits with
// room for its byte offset at any supported shape).
inline bool kv4_pool_ok(const void *pool, int64_t pages, int32_t page, int32_t Hkv, int32_t D)
{
    if (pages < 0 || Hkv < 0) return false;
    if (pages == 0 || Hkv == 0) return true;
    const int64_t pb = (int64_t)Hkv * (page / 16) * kv4_block_bytes(D);
    return pool != nullptr && pages <= INT64_MAX / 4 / pb;
}

}  // namespace libtm
