// What the kernels that turn heads by rotary positions share: 16-byte pieces to
// floats and back, a chunk's angles, and the rotation itself.
#pragma once

#include "attn_internal.h"
#include "lora_device.cuh"

namespace lora {

__device__ __forceinline__ void unpack(const uint4 &q, float (&v)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void unpack(const uint4 &q, float (&v)[4]) {
    v[0] = __uint_as_float(q.x); v[1] = __uint_as_float(q.y); v[2] = __uint_as_float(q.z); v[3] = __uint_as_float(q.w);
}
__device__ __forceinline__ uint4 pack(const float (&v)[8]) {
    __nv_bfloat162 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    return *reinterpret_cast<uint4 *>(h);
}
__device__ __forceinline__ uint4 pack(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}

// Every bit of the low four, twice.
__device__ __forceinline__ uint32_t twice(uint32_t b) {
    return (b & 1u) * 3u | (b >> 1 & 1u) * 12u | (b >> 2 & 1u) * 48u | (b >> 3 & 1u) * 192u;
}

// The VE values in `a`, with those of `b` where `from_b` has their bit.
template <int VE>
__device__ __forceinline__ uint4 replace(const uint4 &a, const uint4 &b, uint32_t from_b) {
    uint32_t m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m[i] = VE == 4 ? (from_b >> i & 1u) * 0xFFFFFFFFu
                       : (from_b >> 2 * i & 1u) * 0xFFFFu | (from_b >> (2 * i + 1) & 1u) * 0xFFFF0000u;
    return make_uint4((a.x & ~m[0]) | (b.x & m[0]), (a.y & ~m[1]) | (b.y & m[1]), (a.z & ~m[2]) | (b.z & m[2]),
                      (a.w & ~m[3]) | (b.w & m[3]));
}

// A chunk is what one thread takes of a head: VE pairs of the rotated
// dimensions (two 16-byte pieces), or one piece of those past them.
struct Chunk {
    bool turn;
    int32_t d0, d1;  // first dimensions of its two pieces (the same where there is one)
};
template <int VE>
__device__ __forceinline__ Chunk chunk_at(const RopeView &a, int32_t c) {
    const int32_t pair_chunks = a.rot_dim / (2 * VE);  // then the dimensions that are copied
    Chunk x;
    x.turn = c < pair_chunks;
    x.d0 = !x.turn ? a.rot_dim + (c - pair_chunks) * VE : a.interleaved ? 2 * c * VE : c * VE;
    x.d1 = !x.turn ? x.d0 : a.interleaved ? x.d0 + VE : x.d0 + a.rot_dim / 2;
    return x;
}

// Cosines and sines of the pairs of chunk c in a row; a bit is set for each pair
// whose position is out of range (recorded).
template <int VE>
__device__ __forceinline__ uint32_t load_angles(const RopeView &a, int32_t c, int64_t row, float (&cs)[VE], float (&sn)[VE]) {
    uint32_t out_of_range = 0;
    const int32_t half = a.rot_dim / 2;
    auto position = [&](int32_t axis) {  // < 0: out of range
        const int32_t p = a.positions[static_cast<int64_t>(axis) * a.rows + row];
        if (p >= 0 && p < a.max_pos) return p;
        record_error(a.status, kDevBadBlock, static_cast<uint32_t>(row));
        return -1;
    };
    const int32_t axis = a.chunk_axis[c];
    if (axis < LORA_ROPE_MAX_AXES) {  // the chunk's pairs follow one axis
        const int32_t p = position(axis);
        const int64_t at = static_cast<int64_t>(max(p, 0)) * half + c * VE;
#pragma unroll
        for (int e = 0; e < VE; e += 4) {
            const float4 x = __ldg(reinterpret_cast<const float4 *>(a.cos_table + at + e));
            const float4 y = __ldg(reinterpret_cast<const float4 *>(a.sin_table + at + e));
            cs[e] = x.x; cs[e + 1] = x.y; cs[e + 2] = x.z; cs[e + 3] = x.w;
            sn[e] = y.x; sn[e + 1] = y.y; sn[e + 2] = y.z; sn[e + 3] = y.w;
        }
        if (p < 0) out_of_range = (1u << VE) - 1u;
    } else {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            const int32_t p = position(a.pair_axis[c * VE + e]);
            const int64_t at = static_cast<int64_t>(max(p, 0)) * half + c * VE + e;
            cs[e] = __ldg(a.cos_table + at);
            sn[e] = __ldg(a.sin_table + at);
            if (p < 0) out_of_range |= 1u << e;
        }
    }
    return out_of_range;
}

// The pairs of (u, v), a chunk's two pieces, turned into (y, w).
template <int VE>
__device__ __forceinline__ void turn_pairs(const float (&u)[VE], const float (&v)[VE], const float (&cs)[VE], const float (&sn)[VE],
                                           bool interleaved, float (&y)[VE], float (&w)[VE]) {
    if (interleaved) {  // (2 e, 2 e + 1): the first half of the pairs in u, the second in v
#pragma unroll
        for (int e = 0; e < VE / 2; ++e) {
            y[2 * e] = u[2 * e] * cs[e] - u[2 * e + 1] * sn[e];
            y[2 * e + 1] = u[2 * e + 1] * cs[e] + u[2 * e] * sn[e];
            w[2 * e] = v[2 * e] * cs[VE / 2 + e] - v[2 * e + 1] * sn[VE / 2 + e];
            w[2 * e + 1] = v[2 * e + 1] * cs[VE / 2 + e] + v[2 * e] * sn[VE / 2 + e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            y[e] = u[e] * cs[e] - v[e] * sn[e];
            w[e] = v[e] * cs[e] + u[e] * sn[e];
        }
    }
}

// Of each chunk of a head the axis that its pairs follow, where they follow one; on the host.
template <int VE>
inline int32_t plan_chunks(RopeView &v) {
    const int32_t pair_chunks = v.rot_dim / (2 * VE);
    for (int32_t c = 0; c < pair_chunks; ++c) {
        v.chunk_axis[c] = v.pair_axis[c * VE];
        for (int32_t e = 1; e < VE; ++e)
            if (v.pair_axis[c * VE + e] != v.chunk_axis[c]) v.chunk_axis[c] = LORA_ROPE_MAX_AXES;
    }
    return pair_chunks + (v.head_dim - v.rot_dim) / VE;
}

}  // namespace lora
