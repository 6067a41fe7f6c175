// Attention over the 8-bit paged cache (lora_kv_attention), the plain kernel:
// one warp per (row, query head), one pass over the keys in groups of 32 with
// the running maximum m and sum l of the softmax,
//     m' = max(m, s_j),  l = l e^(m - m') + sum e^(s_j - m'),  o likewise,
// everything in fp32 on the CUDA cores.
#include <cuda_runtime.h>
#include <math.h>

#include "attn_device.cuh"
#include "attn_internal.h"

namespace lora {

namespace {

template <typename T, int D, int FMT>
__global__ void __launch_bounds__(128) attn_simple_kernel(const __grid_constant__ AttnView a) {
    __shared__ float sq[4][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t h = blockIdx.y * 4 + warp;
    const KvView &b = a.kv;
    const int32_t row = blockIdx.x;
    // the row's sequence (bad offsets find some sequence; read_seq checks it)
    int32_t lo = 0, hi = b.num_seqs;
    if (b.offsets) {
        while (lo < hi) {
            const int32_t mid = (lo + hi) >> 1;
            if (b.offsets[mid + 1] > row) hi = mid; else lo = mid + 1;
        }
    } else {
        lo = row;
    }
    if (lo >= b.num_seqs || h >= a.q_heads) return;
    if (b.offsets && row < b.offsets[lo]) return;
    SeqRows r = read_seq(b, lo, h == 0 && lane == 0);
    if (r.n > a.max_queries) {
        if (h == 0 && lane == 0) record_error(b.status, kDevBadSegment, static_cast<uint32_t>(lo));
        r.n = r.len = 0;
    }
    const T *q = static_cast<const T *>(a.q.p) + row * a.q.row + h * a.q.head;
    for (int d = lane; d < D; d += 32) sq[warp][d] = to_float(q[d]) * a.scale;
    __syncwarp();
    const int32_t pos = r.n > 0 ? r.len - r.n + (row - r.off) : -1;
    const int32_t end = r.n == 0 ? 0 : a.causal ? pos + 1 : r.len;
    const int32_t begin = a.window > 0 && pos - a.window + 1 > 0 ? pos - a.window + 1 : 0;
    const int32_t head = h / a.group;
    float m = -INFINITY, l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int32_t j0 = begin & ~31; j0 < end; j0 += 32) {
        const int32_t j = j0 + lane;
        float s = -INFINITY;
        int32_t page = -1;
        if (j < end) page = read_page(b, lo, j >> b.page_shift);
        const int32_t t = j & (b.page_tokens - 1);
        const int64_t at = tile_offset<D>(b, page < 0 ? 0 : page, head, t / kKvTile);
        const float vscale = page < 0 ? 0.0f : b.v_scales[static_cast<int64_t>(page) * b.heads + head];
        if (j >= begin && j < end) {
            float dot = 0.0f;
            for (int d = 0; d < D; d += 16) {
                const uint4 w = *reinterpret_cast<const uint4 *>(b.k_pages + at + d / 64 * (kKvTile * 64) +
                                                                 (t % kKvTile) * 64 + d % 64);
                float f[16];
                codes_to_float<FMT>(w.x, f);
                codes_to_float<FMT>(w.y, f + 4);
                codes_to_float<FMT>(w.z, f + 8);
                codes_to_float<FMT>(w.w, f + 12);
#pragma unroll
                for (int e = 0; e < 16; ++e) dot = fmaf(f[e], sq[warp][d + e], dot);
            }
            s = page < 0 ? 0.0f : dot * b.k_scales[static_cast<int64_t>(page) * b.heads + head];
        }
        float mx = s;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
        mx = fmaxf(mx, m);
        if (!__any_sync(0xffffffffu, j >= begin && j < end)) continue;  // (a maximum of -inf may also hide NaN)
        const float keep = expf(m - mx);
        const float p = expf(s - mx);
        float sum = p;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        l = l * keep + sum;
        m = mx;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] *= keep;
        const float pv = p * vscale;
        for (int t4 = 0; t4 < 32; t4 += 4) {
            if (j0 + t4 >= end) break;
            const int64_t at4 = __shfl_sync(0xffffffffu, at, t4);
            float p4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) p4[e] = __shfl_sync(0xffffffffu, pv, t4 + e);
            if (lane * 4 >= D) continue;
            const int32_t q4 = ((j0 + t4) % kKvTile) / 4;
            const uint4 w = *reinterpret_cast<const uint4 *>(b.v_pages + at4 + lane * 64 + q4 * 16);
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                float f[4];
                codes_to_float<FMT>(ws[d], f);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (j0 + t4 + e >= begin && j0 + t4 + e < end) o[d] = fmaf(p4[e], f[e], o[d]);
            }
        }
    }
    T *out = static_cast<T *>(a.out.p) + row * a.out.row + h * a.out.head;
    const float inv = begin < end ? 1.0f / l : 0.0f;
    if (lane * 4 < D)
        for (int e = 0; e < 4; ++e) out[lane * 4 + e] = from_float<T>(o[e] * inv);
    if (a.lse && lane == 0) a.lse[static_cast<int64_t>(row) * a.q_heads + h] = begin < end ? m + logf(l) : -INFINITY;
}

template <typename T, int D>
cudaError_t simple_typed(const AttnView &v, lora_kv_format_t fmt, cudaStream_t stream) {
    const dim3 grid(v.kv.rows, (v.q_heads + 3) / 4);
    if (fmt == LORA_KV_INT8)
        attn_simple_kernel<T, D, LORA_KV_INT8><<<grid, 128, 0, stream>>>(v);
    else
        attn_simple_kernel<T, D, LORA_KV_E4M3><<<grid, 128, 0, stream>>>(v);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

size_t attention_workspace_bytes(const AttnView &, lora_kv_format_t, int, lora_dtype_t) { return 256; }

cudaError_t launch_attention(const AttnView &v, lora_kv_format_t fmt, int head_dim, lora_dtype_t dtype,
                             cudaStream_t stream) {
    if (dtype == LORA_FP32)
        return head_dim == 64 ? simple_typed<float, 64>(v, fmt, stream) : simple_typed<float, 128>(v, fmt, stream);
    return head_dim == 64 ? simple_typed<__nv_bfloat16, 64>(v, fmt, stream)
                          : simple_typed<__nv_bfloat16, 128>(v, fmt, stream);
}

}  // namespace lora
