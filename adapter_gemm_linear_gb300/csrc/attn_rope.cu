// Rotary positions on q and k (lora_rope): every pair (x1, x2) of a head's
// rotated dimensions turned by the angle of its axis' position,
//     y1 = x1 c - x2 s,   y2 = x2 c + x1 s.
//
// Bound by memory: each value is read and written once, 3 flops a value.  A
// thread owns one chunk of pairs (16 bytes of x1 and 16 of x2) of one row
// and applies it to several heads, so that the chunk's cosines and sines are
// fetched once for them and the heads' loads are in flight together.  The
// block's shape is (chunk, head group, row), so that no thread divides: with
// an index taken apart by 64-bit divisions and the table read value by value
// the call took 95 us instead of 58 for 8192 rows of 72 heads of 128 (306 MB,
// 5.2 TB/s; now 58.7); one token of each of 64 sequences, 40 heads: 4 us.
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "lora_device.cuh"

namespace lora {

namespace {

constexpr int kRopeThreads = 256;     // of a block, about
constexpr int kRopeMaxThreads = 512;  // (chunks of one head: 256 at most)

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

// Thread (x, y, z): chunk x (a head's row is read in whole lines), head group
// y, row z of the block.  Group j has heads j, j + groups, ..., of which HPT are
// in work at once.
template <typename T, int HPT>
__global__ void __launch_bounds__(kRopeMaxThreads) rope_kernel(const __grid_constant__ RopeView a) {
    constexpr int VE = VecTraits<T>::kElems;  // elements of 16 bytes
    const int32_t pair_chunks = a.rot_dim / (2 * VE);  // then the dimensions that are copied
    const int32_t c = threadIdx.x, j = threadIdx.y, groups = blockDim.y;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.z + threadIdx.z;
    if (row >= a.rows) return;
    const int32_t heads = a.q_heads + a.k_heads;
    const bool turn = c < pair_chunks;
    // element offsets of the chunk's two 16-byte pieces
    const int32_t d0 = !turn ? a.rot_dim + (c - pair_chunks) * VE : a.interleaved ? 2 * c * VE : c * VE;
    const int32_t d1 = !turn ? d0 : a.interleaved ? d0 + VE : d0 + a.rot_dim / 2;

    float cs[VE], sn[VE];
    uint32_t out_of_range = 0;  // a bit a pair: these stay as they are
    if (turn) {
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
        if (a.inverse) {
#pragma unroll
            for (int e = 0; e < VE; ++e) sn[e] = -sn[e];
        }
    }
    for (int32_t h0 = j; h0 < heads; h0 += HPT * groups) {
        uint4 x[HPT][2];
#pragma unroll
        for (int i = 0; i < HPT; ++i) {
            const int32_t h = h0 + i * groups;
            if (h >= heads) continue;
            const bool is_q = h < a.q_heads;
            const HeadsView &in = is_q ? a.q : a.k;
            const T *src = static_cast<const T *>(in.p) + row * in.row + (is_q ? h : h - a.q_heads) * in.head;
            x[i][0] = *reinterpret_cast<const uint4 *>(src + d0);
            if (turn) x[i][1] = *reinterpret_cast<const uint4 *>(src + d1);
        }
#pragma unroll
        for (int i = 0; i < HPT; ++i) {
            const int32_t h = h0 + i * groups;
            if (h >= heads) continue;
            const bool is_q = h < a.q_heads;
            const HeadsView &out = is_q ? a.q_out : a.k_out;
            T *dst = static_cast<T *>(out.p) + row * out.row + (is_q ? h : h - a.q_heads) * out.head;
            if (!turn) {
                *reinterpret_cast<uint4 *>(dst + d0) = x[i][0];
                continue;
            }
            float u[VE], v[VE], y[VE], w[VE];
            unpack(x[i][0], u);
            unpack(x[i][1], v);
            if (a.interleaved) {  // (2 e, 2 e + 1): the first half of the pairs in u, the second in v
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
            uint4 py = pack(y), pw = pack(w);
            if (__builtin_expect(out_of_range != 0, 0)) {
                // (not by a cosine of 1: the other value of a pair may be infinite or NaN)
                py = replace<VE>(py, x[i][0], a.interleaved ? twice(out_of_range) : out_of_range);
                pw = replace<VE>(pw, x[i][1], a.interleaved ? twice(out_of_range >> (VE / 2)) : out_of_range);
            }
            *reinterpret_cast<uint4 *>(dst + d0) = py;
            *reinterpret_cast<uint4 *>(dst + d1) = pw;
        }
    }
}

template <typename T>
cudaError_t launch_typed(RopeView v, cudaStream_t stream) {
    constexpr int VE = VecTraits<T>::kElems;
    const int32_t heads = v.q_heads + v.k_heads;
    const int32_t pair_chunks = v.rot_dim / (2 * VE), chunks = pair_chunks + (v.head_dim - v.rot_dim) / VE;
    for (int32_t c = 0; c < pair_chunks; ++c) {
        v.chunk_axis[c] = v.pair_axis[c * VE];
        for (int32_t e = 1; e < VE; ++e)
            if (v.pair_axis[c * VE + e] != v.chunk_axis[c]) v.chunk_axis[c] = LORA_ROPE_MAX_AXES;
    }
    // One head a thread while that fills less than the machine's resident
    // threads a few times over, else four
    const bool many = static_cast<int64_t>(v.rows) * chunks * heads > 4LL * 2048 * device_sm_count();
    const int32_t wanted = many ? (heads + 3) / 4 : heads, most = kRopeMaxThreads / chunks;
    const int32_t groups = wanted < most ? wanted : most;
    const int32_t per_block = groups * chunks >= kRopeThreads ? 1 : kRopeThreads / (groups * chunks);
    const dim3 block(chunks, groups, per_block < 64 ? per_block : 64);
    const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(v.rows) + block.z - 1) / block.z);
    if (many)
        rope_kernel<T, 4><<<grid, block, 0, stream>>>(v);
    else
        rope_kernel<T, 1><<<grid, block, 0, stream>>>(v);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeView &v, lora_dtype_t dtype, cudaStream_t stream) {
    return dtype == LORA_FP32 ? launch_typed<float>(v, stream) : launch_typed<__nv_bfloat16>(v, stream);
}

}  // namespace lora
