// Norms of queries and keys for each head with the rotary positions in the same
// pass (lora_norm_rope), and its gradient (lora_norm_rope_backward).  For a head x
// with weights W (w, or 1 + w):
//     r = 1 / sqrt(mean(x^2) + eps),  n = x r W,  y = rotate(n)
// and, with g the gradient of y,
//     h = rotate^-1(g),  dW = sum over rows and heads of h x r,
//     a = h W,  dx = r (a - x r^2 mean(a x)).
//
// Both are bound by memory: each value is read once and written once (twice read
// for the gradient), 7 and 14 flops a value.  A head is taken by a group of
// lanes, the least power of two with a chunk (attn_rope.cuh) each, which add up
// its squares by shuffles; the head's values stay in registers in between.  A
// group works on heads of q alone or of k alone, so that its weights are read
// once, and on several heads of a row, so that the angles are.
#include <cuda_runtime.h>

#include "attn_rope.cuh"

namespace lora {

namespace {

constexpr int kNormThreads = 256;     // of a block, about
constexpr int kNormMaxThreads = 512;
constexpr int kGradCtas = 2;          // of the gradient, per SM: what 128 registers a thread leave room for

// What a thread has to know of its place: lane c of a group of L, the group's
// tensor and heads h0, h0 + step, ... of it, and the row within the block.
struct Group {
    bool is_k;
    int32_t c, h0, step, heads;
    uint32_t mask;  // of the group's lanes

    __device__ __forceinline__ Group(const NormRopeView &a) {
        const int32_t L = blockDim.x, j = threadIdx.y;
        c = threadIdx.x;
        is_k = j >= a.q_groups;
        h0 = is_k ? j - a.q_groups : j;
        step = is_k ? a.k_groups : a.q_groups;
        heads = is_k ? a.rope.k_heads : a.rope.q_heads;
        const uint32_t lane = ((threadIdx.z * blockDim.y + j) * L + c) & 31u;
        mask = L == 32 ? 0xffffffffu : ((1u << L) - 1u) << (lane & ~static_cast<uint32_t>(L - 1));
    }
    __device__ __forceinline__ float sum(float x) const {
        for (int32_t o = blockDim.x >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(mask, x, o);
        return x;
    }
};

// A thread's chunks of a head, NC at most: chunk c, then c + L.
template <typename T, int NC>
struct Chunks {
    static constexpr int VE = VecTraits<T>::kElems;
    Chunk at[NC];
    bool has[NC];
    float w[NC][2][VE];  // weights

    __device__ __forceinline__ Chunks(const NormRopeView &a, const Group &g) {
        const int32_t count = a.rope.rot_dim / (2 * VE) + (a.rope.head_dim - a.rope.rot_dim) / VE;
        const void *p = g.is_k ? a.k_weight : a.q_weight;
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            const int32_t c = g.c + n * static_cast<int32_t>(blockDim.x);
            has[n] = c < count;
            at[n] = chunk_at<VE>(a.rope, has[n] ? c : 0);
            at[n].turn = at[n].turn && has[n];  // (a lane without a chunk has no angles)
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                w[n][0][e] = has[n] ? weight(a, p, at[n].d0 + e) : 0.0f;
                w[n][1][e] = at[n].turn ? weight(a, p, at[n].d1 + e) : 0.0f;
            }
        }
    }
    static __device__ __forceinline__ float weight(const NormRopeView &a, const void *p, int32_t d) {
        const float add = a.unit_offset ? 1.0f : 0.0f;
        if (!p) return 1.0f;
        return add + (a.weight_fp32 ? static_cast<const float *>(p)[d] : __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[d]));
    }
    __device__ __forceinline__ void load(const T *src, uint4 (&x)[NC][2]) const {
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            x[n][0] = x[n][1] = make_uint4(0u, 0u, 0u, 0u);
            if (has[n]) x[n][0] = *reinterpret_cast<const uint4 *>(src + at[n].d0);
            if (at[n].turn) x[n][1] = *reinterpret_cast<const uint4 *>(src + at[n].d1);
        }
    }
    __device__ __forceinline__ void store(T *dst, int n, const float (&y)[VE], const float (&w1)[VE]) const {
        if (!has[n]) return;
        *reinterpret_cast<uint4 *>(dst + at[n].d0) = pack(y);
        if (at[n].turn) *reinterpret_cast<uint4 *>(dst + at[n].d1) = pack(w1);
    }
};

template <typename T>
__device__ __forceinline__ T *head_at(const HeadsView &v, int64_t row, int32_t h) {
    return static_cast<T *>(v.p) + row * v.row + h * v.head;
}

// The chunk's pairs turned; those out of range stay as they are.
template <int VE>
__device__ __forceinline__ void turn_in_range(const float (&u)[VE], const float (&v)[VE], const float (&cs)[VE], const float (&sn)[VE],
                                              uint32_t out_of_range, bool interleaved, float (&y)[VE], float (&w)[VE]) {
    turn_pairs<VE>(u, v, cs, sn, interleaved, y, w);
    if (__builtin_expect(out_of_range != 0, 0)) {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            if (out_of_range >> (interleaved ? e / 2 : e) & 1u) y[e] = u[e];
            if (out_of_range >> (interleaved ? VE / 2 + e / 2 : e) & 1u) w[e] = v[e];
        }
    }
}

template <typename T, int NC, int HPT>
__global__ void __launch_bounds__(kNormMaxThreads) norm_rope_kernel(const __grid_constant__ NormRopeView a) {
    constexpr int VE = VecTraits<T>::kElems;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.z + threadIdx.z;
    if (row >= a.rope.rows) return;
    const Group g(a);
    const Chunks<T, NC> ch(a, g);
    const HeadsView &in = g.is_k ? a.rope.k : a.rope.q, &out = g.is_k ? a.rope.k_out : a.rope.q_out;
    float cs[NC][VE], sn[NC][VE];
    uint32_t out_of_range[NC] = {};
#pragma unroll
    for (int n = 0; n < NC; ++n)
        if (ch.at[n].turn) out_of_range[n] = load_angles<VE>(a.rope, g.c + n * blockDim.x, row, cs[n], sn[n]);
    const float inv_d = 1.0f / static_cast<float>(a.rope.head_dim);
    for (int32_t h0 = g.h0; h0 < g.heads; h0 += HPT * g.step) {
        uint4 x[HPT][NC][2];
#pragma unroll
        for (int i = 0; i < HPT; ++i) {
            const int32_t h = h0 + i * g.step;
            if (h < g.heads) ch.load(head_at<T>(in, row, h), x[i]);
        }
#pragma unroll
        for (int i = 0; i < HPT; ++i) {
            const int32_t h = h0 + i * g.step;
            if (h >= g.heads) continue;
            float u[NC][VE], v[NC][VE], squares = 0.0f;
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                unpack(x[i][n][0], u[n]);
                unpack(x[i][n][1], v[n]);
#pragma unroll
                for (int e = 0; e < VE; ++e) squares = fmaf(u[n][e], u[n][e], fmaf(v[n][e], v[n][e], squares));
            }
            const float r = rsqrtf(fmaf(g.sum(squares), inv_d, a.eps));
            T *dst = head_at<T>(out, row, h);
#pragma unroll
            for (int n = 0; n < NC; ++n) {
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    u[n][e] = u[n][e] * r * ch.w[n][0][e];
                    v[n][e] = v[n][e] * r * ch.w[n][1][e];
                }
                if (ch.at[n].turn) {
                    float y[VE], w[VE];
                    turn_in_range<VE>(u[n], v[n], cs[n], sn[n], out_of_range[n], a.rope.interleaved, y, w);
                    ch.store(dst, n, y, w);
                } else {
                    ch.store(dst, n, u[n], u[n]);
                }
            }
        }
    }
}

// Blocks take rows in turn; a thread adds up its chunks' gradients of the weights
// over all its rows and heads, a block over its groups, grad_weights_kernel over
// the blocks: every sum's order is fixed.
template <typename T, int NC, int HPT>
__global__ void __launch_bounds__(kNormMaxThreads, 1) norm_rope_backward_kernel(const __grid_constant__ NormRopeView a) {
    constexpr int VE = VecTraits<T>::kElems;
    extern __shared__ float sums[];  // [group of the block][head_dim]
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Group g(a);
    const Chunks<T, NC> ch(a, g);
    const HeadsView &in = g.is_k ? a.rope.k : a.rope.q, &out = g.is_k ? a.rope.k_out : a.rope.q_out, &grad = g.is_k ? a.dk : a.dq;
    const float inv_d = 1.0f / static_cast<float>(a.rope.head_dim);
    float dw[NC][2][VE];
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int e = 0; e < VE; ++e) dw[n][0][e] = dw[n][1][e] = 0.0f;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.z + threadIdx.z; row < a.rope.rows;
         row += static_cast<int64_t>(gridDim.x) * blockDim.z) {
        float cs[NC][VE], sn[NC][VE];
        uint32_t out_of_range[NC] = {};
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            if (!ch.at[n].turn) continue;
            out_of_range[n] = load_angles<VE>(a.rope, g.c + n * blockDim.x, row, cs[n], sn[n]);
#pragma unroll
            for (int e = 0; e < VE; ++e) sn[n][e] = -sn[n][e];
        }
        for (int32_t h0 = g.h0; h0 < g.heads; h0 += HPT * g.step) {
            uint4 x[HPT][NC][2], dy[HPT][NC][2];
#pragma unroll
            for (int i = 0; i < HPT; ++i) {
                const int32_t h = h0 + i * g.step;
                if (h >= g.heads) continue;
                ch.load(head_at<T>(in, row, h), x[i]);
                ch.load(head_at<T>(grad, row, h), dy[i]);
            }
#pragma unroll
            for (int i = 0; i < HPT; ++i) {
                const int32_t h = h0 + i * g.step;
                if (h >= g.heads) continue;
                float u[NC][VE], v[NC][VE], y[NC][VE], w[NC][VE], squares = 0.0f, dot = 0.0f;
#pragma unroll
                for (int n = 0; n < NC; ++n) {
                    unpack(x[i][n][0], u[n]);
                    unpack(x[i][n][1], v[n]);
                    unpack(dy[i][n][0], y[n]);
                    unpack(dy[i][n][1], w[n]);
                    if (ch.at[n].turn) {
                        float s[VE], t[VE];
                        turn_in_range<VE>(y[n], w[n], cs[n], sn[n], out_of_range[n], a.rope.interleaved, s, t);
#pragma unroll
                        for (int e = 0; e < VE; ++e) {
                            y[n][e] = s[e];
                            w[n][e] = t[e];
                        }
                    }
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        squares = fmaf(u[n][e], u[n][e], fmaf(v[n][e], v[n][e], squares));
                        dot = fmaf(y[n][e] * ch.w[n][0][e], u[n][e], fmaf(w[n][e] * ch.w[n][1][e], v[n][e], dot));
                    }
                }
                const float r = rsqrtf(fmaf(g.sum(squares), inv_d, a.eps));
                const float back = g.sum(dot) * inv_d * r * r;
                T *dst = head_at<T>(out, row, h);
#pragma unroll
                for (int n = 0; n < NC; ++n) {
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        dw[n][0][e] = fmaf(y[n][e], u[n][e] * r, dw[n][0][e]);
                        dw[n][1][e] = fmaf(w[n][e], v[n][e] * r, dw[n][1][e]);
                        y[n][e] = r * fmaf(-u[n][e], back, y[n][e] * ch.w[n][0][e]);
                        w[n][e] = r * fmaf(-v[n][e], back, w[n][e] * ch.w[n][1][e]);
                    }
                    ch.store(dst, n, y[n], w[n]);
                }
            }
        }
    }
    if (!a.partial) return;
    const int32_t D = a.rope.head_dim, groups = blockDim.y;
    float *mine = sums + (threadIdx.z * groups + threadIdx.y) * D;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            if (ch.has[n]) mine[ch.at[n].d0 + e] = dw[n][0][e];
            if (ch.at[n].turn) mine[ch.at[n].d1 + e] = dw[n][1][e];
        }
    }
    __syncthreads();
    const int32_t threads = blockDim.x * blockDim.y * blockDim.z;
    for (int32_t i = (threadIdx.z * blockDim.y + threadIdx.y) * blockDim.x + threadIdx.x; i < 2 * D; i += threads) {
        const int32_t d = i % D, j0 = i < D ? 0 : a.q_groups, j1 = i < D ? a.q_groups : groups;
        float s = 0.0f;
        for (int32_t z = 0; z < static_cast<int32_t>(blockDim.z); ++z)
            for (int32_t j = j0; j < j1; ++j) s += sums[(z * groups + j) * D + d];
        a.partial[static_cast<int64_t>(blockIdx.x) * 2 * D + i] = s;
    }
}

// Sums the blocks' parts: 32 of the 2 D values a block, 16 threads each.  It may
// begin while the kernel before still writes them (as attn_join_kernel).
constexpr int kSumParts = 16;
__global__ void __launch_bounds__(32 * kSumParts) grad_weights_kernel(const float *partial, int32_t blocks, int32_t D, float *dq_weight,
                                                                      float *dk_weight) {
    __shared__ float part[kSumParts][32];
    const int32_t i = blockIdx.x * 32 + threadIdx.x, p = threadIdx.y;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float s = 0.0f;
#pragma unroll 4
    for (int32_t b = p; i < 2 * D && b < blocks; b += kSumParts) s += __ldcg(partial + static_cast<int64_t>(b) * 2 * D + i);
    part[p][threadIdx.x] = s;
    __syncthreads();
    if (p > 0 || i >= 2 * D) return;
#pragma unroll
    for (int k = 1; k < kSumParts; ++k) s += part[k][threadIdx.x];
    float *dst = i < D ? dq_weight : dk_weight;
    if (dst) dst[i % D] = s;
}

struct Shape {
    dim3 block;
    int32_t chunks;
    int64_t row_tiles;
};

// Groups of L lanes; one head a group while that fills less than the machine's
// resident threads a few times over, else `several`.
template <int VE>
Shape plan(NormRopeView &v, int several) {
    Shape s;
    s.chunks = plan_chunks<VE>(v.rope);
    int32_t L = 4;
    while (L < 32 && L < s.chunks) L *= 2;
    const int32_t qh = v.rope.q_heads, kh = v.rope.k_heads, most = kNormMaxThreads / L;
    const bool many = static_cast<int64_t>(v.rope.rows) * L * (qh + kh) > 4LL * 2048 * device_sm_count();
    const int32_t each = many ? several : 1;
    v.q_groups = (qh + each - 1) / each;
    v.k_groups = (kh + each - 1) / each;
    if (v.q_groups + v.k_groups > most) {  // in proportion, a group of k's at least
        const int32_t total = v.q_groups + v.k_groups;
        v.k_groups = kh == 0 ? 0 : static_cast<int32_t>(static_cast<int64_t>(v.k_groups) * most / total);
        if (kh > 0 && v.k_groups == 0) v.k_groups = 1;
        v.q_groups = static_cast<int32_t>(static_cast<int64_t>(v.q_groups) * most / total);
        if (v.q_groups == 0) v.q_groups = 1;
        while (v.q_groups + v.k_groups > most) --(v.q_groups > v.k_groups ? v.q_groups : v.k_groups);
    }
    const int32_t threads = L * (v.q_groups + v.k_groups);
    const int32_t z = threads >= kNormThreads ? 1 : kNormThreads / threads;
    s.block = dim3(L, v.q_groups + v.k_groups, z < 64 ? z : 64);
    s.row_tiles = (static_cast<int64_t>(v.rope.rows) + s.block.z - 1) / s.block.z;
    return s;
}

template <typename T>
cudaError_t forward_typed(NormRopeView v, cudaStream_t stream) {
    constexpr int VE = VecTraits<T>::kElems;
    const Shape s = plan<VE>(v, 4);
    const unsigned grid = static_cast<unsigned>(s.row_tiles);
    const bool many = v.q_groups < v.rope.q_heads;
    auto *kernel = many ? norm_rope_kernel<T, 1, 4> : norm_rope_kernel<T, 1, 1>;
    if constexpr (sizeof(T) == 4)  // (a bf16 head has 31 chunks at most)
        if (s.chunks > 32) kernel = norm_rope_kernel<T, 2, 1>;
    kernel<<<grid, s.block, 0, stream>>>(v);
    count_launches(1);
    return cudaGetLastError();
}

template <typename T>
cudaError_t backward_typed(NormRopeView v, float *dq_weight, float *dk_weight, cudaStream_t stream) {
    constexpr int VE = VecTraits<T>::kElems;
    const Shape s = plan<VE>(v, 2);
    const int64_t most = static_cast<int64_t>(device_sm_count()) * kGradCtas;
    const int32_t grid = static_cast<int32_t>(s.row_tiles < most ? s.row_tiles : most), D = v.rope.head_dim;
    if (!dq_weight && !dk_weight) v.partial = nullptr;
    const size_t smem = v.partial ? static_cast<size_t>(s.block.y) * s.block.z * D * sizeof(float) : 0;
    auto *kernel = norm_rope_backward_kernel<T, 1, 2>;
    if constexpr (sizeof(T) == 4)
        if (s.chunks > 32) kernel = norm_rope_backward_kernel<T, 2, 1>;
    kernel<<<grid, s.block, smem, stream>>>(v);
    cudaError_t e = cudaGetLastError();
    count_launches(1);
    if (e != cudaSuccess || !v.partial) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((2 * D + 31) / 32);
    cfg.blockDim = dim3(32, kSumParts);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, grad_weights_kernel, static_cast<const float *>(v.partial), grid, D, dq_weight, dk_weight);
    count_launches(1);
    return e;
}

}  // namespace

size_t norm_rope_workspace_bytes(int head_dim) {
    return static_cast<size_t>(device_sm_count()) * kGradCtas * 2 * head_dim * sizeof(float);
}

cudaError_t launch_norm_rope(const NormRopeView &v, lora_dtype_t dtype, cudaStream_t stream) {
    return dtype == LORA_FP32 ? forward_typed<float>(v, stream) : forward_typed<__nv_bfloat16>(v, stream);
}

cudaError_t launch_norm_rope_backward(const NormRopeView &v, lora_dtype_t dtype, float *dq_weight, float *dk_weight,
                                      cudaStream_t stream) {
    return dtype == LORA_FP32 ? backward_typed<float>(v, dq_weight, dk_weight, stream)
                              : backward_typed<__nv_bfloat16>(v, dq_weight, dk_weight, stream);
}

}  // namespace lora
