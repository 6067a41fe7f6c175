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

#include "attn_rope.cuh"

namespace lora {

namespace {

constexpr int kRopeThreads = 256;     // of a block, about
constexpr int kRopeMaxThreads = 512;  // (chunks of one head: 256 at most)

// Thread (x, y, z): chunk x (a head's row is read in whole lines), head group
// y, row z of the block.  Group j has heads j, j + groups, ..., of which HPT are
// in work at once.
template <typename T, int HPT>
__global__ void __launch_bounds__(kRopeMaxThreads) rope_kernel(const __grid_constant__ RopeView a) {
    constexpr int VE = VecTraits<T>::kElems;  // elements of 16 bytes
    const int32_t c = threadIdx.x, j = threadIdx.y, groups = blockDim.y;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.z + threadIdx.z;
    if (row >= a.rows) return;
    const int32_t heads = a.q_heads + a.k_heads;
    const Chunk chunk = chunk_at<VE>(a, c);
    const bool turn = chunk.turn;
    const int32_t d0 = chunk.d0, d1 = chunk.d1;

    float cs[VE], sn[VE];
    uint32_t out_of_range = 0;  // a bit a pair: these stay as they are
    if (turn) {
        out_of_range = load_angles<VE>(a, c, row, cs, sn);
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
            turn_pairs<VE>(u, v, cs, sn, a.interleaved, y, w);
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
    const int32_t chunks = plan_chunks<VE>(v);
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
