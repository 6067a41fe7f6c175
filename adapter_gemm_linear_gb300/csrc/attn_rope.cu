// Rotary positions on q and k (lora_rope): every pair (x1, x2) of a head's
// rotated dimensions turned by the angle of its axis' position,
//     y1 = x1 c - x2 s,   y2 = x2 c + x1 s.
//
// Bound by memory: each value is read and written once, 3 flops a value.  A
// thread owns one chunk of pairs (16 bytes of x1 and 16 of x2) of one row
// and applies it to several heads, so that the chunk's cosines and sines are
// fetched once for them and the heads' loads are in flight together.
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "lora_device.cuh"

namespace lora {

namespace {

constexpr int kRopeThreads = 256;

template <typename T>
__device__ __forceinline__ void store_vec(T *p, const float *v);
template <>
__device__ __forceinline__ void store_vec<float>(float *p, const float *v) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
template <>
__device__ __forceinline__ void store_vec<__nv_bfloat16>(__nv_bfloat16 *p, const float *v) {
    __nv_bfloat162 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<uint4 *>(h);
}

// Threads: chunk fastest (a head's row is read in whole lines), then the
// head group, then the row.  Head h of group j: h = j + i * groups, i < HPT.
template <typename T, int HPT>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeView a, int32_t groups) {
    constexpr int VE = VecTraits<T>::kElems;  // elements of 16 bytes
    const int32_t pair_chunks = a.rot_dim / (2 * VE);
    const int32_t chunks = pair_chunks + (a.head_dim - a.rot_dim) / VE;  // then the dimensions that are copied
    const int64_t id = static_cast<int64_t>(blockIdx.x) * kRopeThreads + threadIdx.x;
    const int32_t c = static_cast<int32_t>(id % chunks);
    const int64_t rest = id / chunks;
    const int32_t j = static_cast<int32_t>(rest % groups);
    const int64_t row = rest / groups;
    if (row >= a.rows) return;
    const int32_t heads = a.q_heads + a.k_heads;
    const bool turn = c < pair_chunks;
    // element offsets of the chunk's two 16-byte pieces
    const int32_t d0 = !turn ? a.rot_dim + (c - pair_chunks) * VE : a.interleaved ? 2 * c * VE : c * VE;
    const int32_t d1 = !turn ? d0 : a.interleaved ? d0 + VE : d0 + a.rot_dim / 2;

    T *src[HPT], *dst[HPT];
    float x[HPT][2 * VE];
#pragma unroll
    for (int i = 0; i < HPT; ++i) {
        const int32_t h = j + i * groups;
        const bool is_q = h < a.q_heads;
        const HeadsView &in = is_q ? a.q : a.k, &out = is_q ? a.q_out : a.k_out;
        const int32_t hh = is_q ? h : h - a.q_heads;
        src[i] = static_cast<T *>(in.p) + row * in.row + hh * in.head;
        dst[i] = static_cast<T *>(out.p) + row * out.row + hh * out.head;
        if (h < heads) {
            VecTraits<T>::load(src[i] + d0, x[i]);
            if (turn) VecTraits<T>::load(src[i] + d1, x[i] + VE);
        }
    }
    float cs[VE], sn[VE];
    if (turn) {
        const int32_t half = a.rot_dim / 2;
        int32_t axis_last = -1, p = 0;
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            const int32_t axis = a.pair_axis[c * VE + e];
            if (axis != axis_last) {
                p = a.positions[static_cast<int64_t>(axis) * a.rows + row];
                axis_last = axis;
                if (p < 0 || p >= a.max_pos) {
                    record_error(a.status, kDevBadBlock, static_cast<uint32_t>(row));
                    p = -1;
                }
            }
            const int64_t at = static_cast<int64_t>(p) * half + c * VE + e;
            cs[e] = p < 0 ? 1.0f : __ldg(a.cos_table + at);
            sn[e] = p < 0 ? 0.0f : __ldg(a.sin_table + at);
            if (a.inverse) sn[e] = -sn[e];
        }
    }
#pragma unroll
    for (int i = 0; i < HPT; ++i) {
        if (j + i * groups >= heads) continue;
        if (!turn) {
            if (dst[i] != src[i]) store_vec<T>(dst[i] + d0, x[i]);
            continue;
        }
        float y[2 * VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            // the partners of pair e: (e, VE + e) of the halves, (2e, 2e + 1) interleaved
            const float x1 = a.interleaved ? x[i][2 * e] : x[i][e];
            const float x2 = a.interleaved ? x[i][2 * e + 1] : x[i][VE + e];
            const float y1 = x1 * cs[e] - x2 * sn[e], y2 = x2 * cs[e] + x1 * sn[e];
            if (a.interleaved) {
                y[2 * e] = y1;
                y[2 * e + 1] = y2;
            } else {
                y[e] = y1;
                y[VE + e] = y2;
            }
        }
        store_vec<T>(dst[i] + d0, y);
        store_vec<T>(dst[i] + d1, y + VE);
    }
}

template <typename T>
cudaError_t launch_typed(const RopeView &v, cudaStream_t stream) {
    constexpr int VE = VecTraits<T>::kElems;
    const int32_t heads = v.q_heads + v.k_heads;
    const int64_t chunks = v.rot_dim / (2 * VE) + (v.head_dim - v.rot_dim) / VE;
    // One head a thread while that fills less than the machine's resident
    // threads a few times over, else four
    const bool many = v.rows * chunks * heads > 4LL * 2048 * device_sm_count();
    const int32_t groups = many ? (heads + 3) / 4 : heads;
    const int64_t blocks = (v.rows * chunks * groups + kRopeThreads - 1) / kRopeThreads;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    if (many)
        rope_kernel<T, 4><<<static_cast<unsigned>(blocks), kRopeThreads, 0, stream>>>(v, groups);
    else
        rope_kernel<T, 1><<<static_cast<unsigned>(blocks), kRopeThreads, 0, stream>>>(v, groups);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeView &v, lora_dtype_t dtype, cudaStream_t stream) {
    return dtype == LORA_FP32 ? launch_typed<float>(v, stream) : launch_typed<__nv_bfloat16>(v, stream);
}

}  // namespace lora
