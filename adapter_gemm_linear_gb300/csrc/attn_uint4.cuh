// The 4-bit cache (LORA_KV_UINT4): where its codes and scales are, and how codes
// become floating point.
//
// A tile of 16 tokens is D/64 blocks of 64 dimensions, each 512 bytes: 32 pieces of
// 16 bytes, piece 4 g + q being what lane 4 g + q of a warp feeds to the matrix
// instructions (attn_decode4.cu):
//   K: dimensions 16 q .. 16 q + 15 of tokens t = 4 (g / 2) + g % 2 (two words) and t + 2;
//      a word has eight dimensions, d in nibble (d / 2) + 4 (d % 2);
//   V: tokens 4 q .. 4 q + 3 of dimensions 4 g, 4 g + 2, 4 g + 32, 4 g + 34 (a word each)
//      and the next, which have the high nibbles; token t in byte 0, 2, 1, 3 for t = 0 .. 3.
// Two values that a matrix instruction takes side by side are 16 bits apart, so
//   w & 0x000F000F,  w & 0x00F000F0,  (w >> 8) & 0x000F000F,  (w >> 8) & 0x00F000F0
// are its four pairs as f16 subnormals: code * 2^-24, and code * 2^-20 in the second
// and fourth.  No other instruction is needed; the matrix instructions take
// subnormals exactly, and the powers of two come out of the sums.
#pragma once

#include "attn_device.cuh"

namespace lora {

constexpr int kBlockDims = 64;                                   // dimensions of a scale
constexpr int kBlockBytes = kKvTile * kBlockDims / 2;            // codes of a block
constexpr uint32_t kNibbles0 = 0x000F000Fu, kNibbles1 = 0x00F000F0u;
constexpr float kCode0 = 16777216.0f, kCode1 = 1048576.0f;       // 2^24, 2^20: codes from such pairs

// Index of 16-token tile g of (page, head).
__device__ __forceinline__ int64_t tile_index(const KvView &b, int32_t page, int32_t head, int32_t g) {
    return (static_cast<int64_t>(page) * b.heads + head) * (b.page_tokens / kKvTile) + g;
}

// The first token of piece 4 g + q of K (the other: that + 2).
__device__ __forceinline__ int k_token(int g) { return 4 * (g >> 1) + (g & 1); }

// The four pairs of a word.
__device__ __forceinline__ void nibble_pairs(uint32_t w, uint32_t (&f)[4]) {
    const uint32_t h = w >> 8;
    f[0] = w & kNibbles0;
    f[1] = w & kNibbles1;
    f[2] = h & kNibbles0;
    f[3] = h & kNibbles1;
}

__device__ __forceinline__ uint32_t times(uint32_t a, uint32_t b) {  // pairs of f16
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t less(uint32_t a, uint32_t b) {
    const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t at_most(uint32_t a, uint32_t b) {
    const __half2 r = __hmin2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t times_and(uint32_t a, uint32_t b, uint32_t c) {
    const __half2 r = __hfma2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b),
                              *reinterpret_cast<const __half2 *>(&c));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// The eight codes of a word of the 4-bit cache, less LESS, as f16 pairs in the order of
// nibble_pairs: a nibble in the low bits of 1024's f16 is 1024 + code, four bits up 1024 + 16 code.
template <int LESS>
__device__ __forceinline__ void nibbles_less(uint32_t w, uint32_t (&f)[4]) {
    constexpr uint32_t k1024 = LESS ? 0x64086408u : 0x64006400u, k64 = LESS ? 0xD480D480u : 0xD400D400u;  // 1024, -64, and LESS
    static_assert(LESS == 0 || LESS == 8, "the constants");
    uint32_t x[4];
    nibble_pairs(w, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t y = x[i] | 0x64006400u;
        f[i] = i & 1 ? times_and(y, 0x2C002C00u, k64) : less(y, k1024);  // (2C00: 1/16)
    }
}

__device__ __forceinline__ float2 f16_pair(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }

// Whether the values of a (scale, least) pair, s code + m with codes 0 to 15, are f16 numbers.
__device__ __forceinline__ bool are_numbers(uint32_t w) {
    const float2 y = f16_pair(w);
    return fabsf(y.y) < 65520.0f && fabsf(fmaf(15.0f, y.x, y.y)) < 65520.0f;
}

}  // namespace lora
