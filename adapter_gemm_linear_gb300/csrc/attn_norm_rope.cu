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
#include "f32x2.cuh"

namespace lora {

namespace {

constexpr int kNormMaxThreads = 512;
constexpr int kNormThreads = 128;  // of a block, about
constexpr int kNormHeads = 4;      // of a group, where there is much work
constexpr int kGradCtas = 3;       // blocks of the gradient, per SM: what 128 registers a thread leave room for

template <typename T>
__device__ __forceinline__ void unpack2(const uint4 &q, F2 (&v)[VecTraits<T>::kElems / 2]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i) v[i] = two(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = two(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
}
template <typename T>
__device__ __forceinline__ uint4 pack2(const F2 (&v)[VecTraits<T>::kElems / 2]) {
    uint32_t w[4];
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 x = apart(v[i]);
            w[2 * i] = __float_as_uint(x.x);
            w[2 * i + 1] = __float_as_uint(x.y);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = apart(v[i]);
            const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// What a thread has to know of its place: lane c of a group of L, the group's
// tensor and heads h0, h0 + step, ... of it.
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
    __device__ __forceinline__ float sum(F2 x2) const {
        const float2 y = apart(x2);
        float x = y.x + y.y;
        for (int32_t o = blockDim.x >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(mask, x, o);
        return x;
    }
};

// A thread's chunks of a head, NC at most: chunk c, then c + L.  A chunk has two
// pieces u and v of N value pairs; one past the rotated dimensions has no v (zeros).
template <typename T, int NC>
struct Chunks {
    static constexpr int VE = VecTraits<T>::kElems, N = VE / 2;
    Chunk at[NC];
    bool has[NC];

    __device__ __forceinline__ Chunks(const NormRopeView &a, const Group &g) {
        const int32_t count = a.rope.rot_dim / (2 * VE) + (a.rope.head_dim - a.rope.rot_dim) / VE;
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            const int32_t c = g.c + n * static_cast<int32_t>(blockDim.x);
            has[n] = c < count;
            at[n] = chunk_at<VE>(a.rope, has[n] ? c : 0);
            at[n].turn = at[n].turn && has[n];  // (a lane without a chunk has no angles)
        }
    }
    // W of the chunks; 1 without a weight
    __device__ __forceinline__ void weights(const NormRopeView &a, const Group &g, F2 (&w)[NC][2][N]) const {
        const void *p = g.is_k ? a.k_weight : a.q_weight;
        const float add = a.unit_offset ? 1.0f : 0.0f;
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int32_t d = k == 0 ? at[n].d0 : at[n].d1;
#pragma unroll
                for (int i = 0; i < N; ++i) w[n][k][i] = two(1.0f, 1.0f);
                if (!p || !has[n]) continue;
                if (a.weight_fp32) {
#pragma unroll
                    for (int i = 0; i < N; i += 2) {
                        const float4 x = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + d + 2 * i));
                        w[n][k][i] = two(add + x.x, add + x.y);
                        w[n][k][i + 1] = two(add + x.z, add + x.w);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < N; i += 2) {
                        const uint2 x = __ldg(reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(p) + d + 2 * i));
                        w[n][k][i] = two(add + __uint_as_float(x.x << 16), add + __uint_as_float(x.x & 0xFFFF0000u));
                        w[n][k][i + 1] = two(add + __uint_as_float(x.y << 16), add + __uint_as_float(x.y & 0xFFFF0000u));
                    }
                }
            }
    }
    // Cosines and sines of the chunks' pairs in a row: 1 and 0 for what is not turned.
    __device__ __forceinline__ void angles(const NormRopeView &a, const Group &g, int64_t row, float (&cs)[NC][VE], float (&sn)[NC][VE]) const {
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            uint32_t still = (1u << VE) - 1u;
            if (at[n].turn) still = load_angles<VE>(a.rope, g.c + n * static_cast<int32_t>(blockDim.x), row, cs[n], sn[n]);
            if (__builtin_expect(still == 0, 1)) continue;
#pragma unroll
            for (int e = 0; e < VE; ++e)
                if (still >> e & 1u) {
                    cs[n][e] = 1.0f;
                    sn[n][e] = 0.0f;
                }
        }
    }
    __device__ __forceinline__ void load(const T *src, uint4 (&x)[NC][2]) const {
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            x[n][0] = x[n][1] = make_uint4(0u, 0u, 0u, 0u);
            if (has[n]) x[n][0] = *reinterpret_cast<const uint4 *>(src + at[n].d0);
            if (at[n].turn) x[n][1] = *reinterpret_cast<const uint4 *>(src + at[n].d1);
        }
    }
    __device__ __forceinline__ void store(T *dst, int n, const F2 (&y)[N], const F2 (&z)[N]) const {
        if (has[n]) *reinterpret_cast<uint4 *>(dst + at[n].d0) = pack2<T>(y);
        if (at[n].turn) *reinterpret_cast<uint4 *>(dst + at[n].d1) = pack2<T>(z);
    }
};

// The angle of the e-th value of piece k of a chunk (as cosines or sines).
template <int VE, bool INTER>
__device__ __forceinline__ float angle_of(const float (&x)[VE], int k, int e) { return x[INTER ? k * VE / 2 + e / 2 : e]; }

template <typename T>
__device__ __forceinline__ T *head_at(const HeadsView &v, int64_t row, int32_t h) {
    return static_cast<T *>(v.p) + row * v.row + h * v.head;
}

// y = r (x A + x' B), x' being the other value of x's pair, A = W cos and B = -W' sin
// for the first of a pair, W' sin for the second: the weights and the angles are
// multiplied once for the heads of a row.
template <typename T, int NC, int HPT, bool INTER>
__global__ void __launch_bounds__(kNormMaxThreads) norm_rope_kernel(const __grid_constant__ NormRopeView a) {
    constexpr int VE = VecTraits<T>::kElems, N = VE / 2;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.z + threadIdx.z;
    if (row >= a.rope.rows) return;
    const Group g(a);
    const Chunks<T, NC> ch(a, g);
    const HeadsView &in = g.is_k ? a.rope.k : a.rope.q, &out = g.is_k ? a.rope.k_out : a.rope.q_out;
    F2 A[NC][2][N], B[NC][2][N];
    const float inv_d = 1.0f / static_cast<float>(a.rope.head_dim);
    for (int32_t h0 = g.h0; h0 < g.heads; h0 += HPT * g.step) {
        uint4 x[HPT][NC][2];
#pragma unroll
        for (int i = 0; i < HPT; ++i) {
            const int32_t h = h0 + i * g.step;
            if (h < g.heads) ch.load(head_at<T>(in, row, h), x[i]);
        }
        if (h0 == g.h0) {  // (on their way with the first heads)
            float cs[NC][VE], sn[NC][VE];
            ch.weights(a, g, A);
            ch.angles(a, g, row, cs, sn);
#pragma unroll
            for (int n = 0; n < NC; ++n) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const F2 w[2] = {A[n][0][i], A[n][1][i]};
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const F2 c = two(angle_of<VE, INTER>(cs[n], k, 2 * i), angle_of<VE, INTER>(cs[n], k, 2 * i + 1));
                        const float s0 = angle_of<VE, INTER>(sn[n], k, 2 * i), s1 = angle_of<VE, INTER>(sn[n], k, 2 * i + 1);
                        A[n][k][i] = mul(w[k], c);
                        B[n][k][i] = INTER ? mul(swapped(w[k]), two(-s0, s1)) : mul(w[1 - k], k == 0 ? two(-s0, -s1) : two(s0, s1));
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < HPT; ++i) {
            const int32_t h = h0 + i * g.step;
            if (h >= g.heads) continue;
            F2 u[NC][N], v[NC][N], squares = two(0.0f, 0.0f);
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                unpack2<T>(x[i][n][0], u[n]);
                unpack2<T>(x[i][n][1], v[n]);
#pragma unroll
                for (int e = 0; e < N; ++e) squares = fma(u[n][e], u[n][e], fma(v[n][e], v[n][e], squares));
            }
            const float r = rsqrtf(fmaf(g.sum(squares), inv_d, a.eps));
            const F2 r2 = two(r, r);
            T *dst = head_at<T>(out, row, h);
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                F2 y[N], z[N];
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    y[e] = mul(fma(INTER ? swapped(u[n][e]) : v[n][e], B[n][0][e], mul(u[n][e], A[n][0][e])), r2);
                    z[e] = mul(fma(INTER ? swapped(v[n][e]) : u[n][e], B[n][1][e], mul(v[n][e], A[n][1][e])), r2);
                }
                ch.store(dst, n, y, z);
            }
        }
    }
}

// Blocks take rows in turn; a thread has the next head's values on their way while it
// works on one, and adds up its chunks' gradients of the weights over all its rows
// and heads, a block over its groups, grad_weights_kernel over the blocks: every
// sum's order is fixed.
template <typename T, int NC, bool INTER>
__global__ void __launch_bounds__(kNormMaxThreads, 1) norm_rope_backward_kernel(const __grid_constant__ NormRopeView a) {
    constexpr int VE = VecTraits<T>::kElems, N = VE / 2;
    extern __shared__ __align__(16) float sums[];  // [group of the block][head_dim]
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Group g(a);
    const Chunks<T, NC> ch(a, g);
    const HeadsView &in = g.is_k ? a.rope.k : a.rope.q, &out = g.is_k ? a.rope.k_out : a.rope.q_out, &grad = g.is_k ? a.dk : a.dq;
    const float inv_d = 1.0f / static_cast<float>(a.rope.head_dim);
    const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.z;
    F2 W[NC][2][N], dw[NC][2][N];
    float cs[NC][VE], sn[NC][VE];
    ch.weights(a, g, W);
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int i = 0; i < N; ++i) dw[n][0][i] = dw[n][1][i] = two(0.0f, 0.0f);
    int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.z + threadIdx.z;
    int32_t h = g.h0;
    uint4 x[NC][2], dy[NC][2];
    if (row < a.rope.rows) {
        ch.load(head_at<T>(in, row, h), x);
        ch.load(head_at<T>(grad, row, h), dy);
    }
    while (row < a.rope.rows) {
        const int64_t this_row = row;
        const int32_t this_h = h;
        F2 u[NC][N], v[NC][N], y[NC][N], z[NC][N];
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            unpack2<T>(x[n][0], u[n]);
            unpack2<T>(x[n][1], v[n]);
            unpack2<T>(dy[n][0], y[n]);
            unpack2<T>(dy[n][1], z[n]);
        }
        h += g.step;
        if (h >= g.heads) {
            h = g.h0;
            row += stride;
        }
        if (row < a.rope.rows) {
            ch.load(head_at<T>(in, row, h), x);
            ch.load(head_at<T>(grad, row, h), dy);
        }
        if (this_h == g.h0) ch.angles(a, g, this_row, cs, sn);
        F2 squares = two(0.0f, 0.0f), dot = two(0.0f, 0.0f);
        const F2 minus = two(-1.0f, -1.0f);
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
            for (int e = 0; e < N; ++e) {
                squares = fma(u[n][e], u[n][e], fma(v[n][e], v[n][e], squares));
                // y and z turned back
                const F2 y0 = y[n][e], z0 = z[n][e];
                F2 c[2], t[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    c[k] = two(angle_of<VE, INTER>(cs[n], k, 2 * e), angle_of<VE, INTER>(cs[n], k, 2 * e + 1));
                    const float s0 = angle_of<VE, INTER>(sn[n], k, 2 * e), s1 = angle_of<VE, INTER>(sn[n], k, 2 * e + 1);
                    t[k] = INTER ? two(s0, -s1) : two(s0, s1);
                }
                y[n][e] = fma(INTER ? swapped(y0) : z0, t[0], mul(y0, c[0]));
                z[n][e] = INTER ? fma(swapped(z0), t[1], mul(z0, c[1])) : fma(mul(y0, t[1]), minus, mul(z0, c[1]));
                dot = fma(mul(y[n][e], u[n][e]), W[n][0][e], fma(mul(z[n][e], v[n][e]), W[n][1][e], dot));
            }
        const float r = rsqrtf(fmaf(g.sum(squares), inv_d, a.eps));
        const float back = g.sum(dot) * inv_d * r * r;
        const F2 r2 = two(r, r), b2 = two(-back * r, -back * r);
        T *dst = head_at<T>(out, this_row, this_h);
#pragma unroll
        for (int n = 0; n < NC; ++n) {
#pragma unroll
            for (int e = 0; e < N; ++e) {
                dw[n][0][e] = fma(mul(y[n][e], u[n][e]), r2, dw[n][0][e]);
                dw[n][1][e] = fma(mul(z[n][e], v[n][e]), r2, dw[n][1][e]);
                y[n][e] = fma(u[n][e], b2, mul(mul(y[n][e], W[n][0][e]), r2));
                z[n][e] = fma(v[n][e], b2, mul(mul(z[n][e], W[n][1][e]), r2));
            }
            ch.store(dst, n, y[n], z[n]);
        }
    }
    if (!a.partial) return;
    const int32_t D = a.rope.head_dim, groups = blockDim.y;
    float *mine = sums + (threadIdx.z * groups + threadIdx.y) * D;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            if (ch.has[n]) *reinterpret_cast<F2 *>(mine + ch.at[n].d0 + 2 * e) = dw[n][0][e];
            if (ch.at[n].turn) *reinterpret_cast<F2 *>(mine + ch.at[n].d1 + 2 * e) = dw[n][1][e];
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

// Sums the blocks' parts: eight of the 2 D values a block, 64 threads each, whose loads are
// all on their way at once (with 16 threads each the kernel took 13 us).  It may begin while
// the kernel before still writes them (as attn_join_kernel).
constexpr int kSumValues = 8, kSumParts = 64;
__global__ void __launch_bounds__(kSumValues * kSumParts) grad_weights_kernel(const float *partial, int32_t blocks, int32_t D,
                                                                              float *dq_weight, float *dk_weight) {
    __shared__ float part[kSumParts][kSumValues];
    const int32_t i = blockIdx.x * kSumValues + threadIdx.x, p = threadIdx.y;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float s = 0.0f;
#pragma unroll 8
    for (int32_t b = p; b < blocks; b += kSumParts) s += __ldcg(partial + static_cast<int64_t>(b) * 2 * D + i);
    part[p][threadIdx.x] = s;
    __syncthreads();
#pragma unroll
    for (int n = kSumParts / 2; n > 0; n /= 2) {
        if (p < n) part[p][threadIdx.x] += part[p + n][threadIdx.x];
        __syncthreads();
    }
    float *dst = i < D ? dq_weight : dk_weight;
    if (p == 0 && dst) dst[i % D] = part[0][threadIdx.x];
}

struct Shape {
    dim3 block;
    int32_t chunks;
    int64_t row_tiles;
};

// Groups of L lanes; one head a group while that fills less than the machine's
// resident threads a few times over, else kNormHeads.
template <int VE>
Shape plan(NormRopeView &v) {
    Shape s;
    s.chunks = plan_chunks<VE>(v.rope);
    int32_t L = 4;
    while (L < 32 && L < s.chunks) L *= 2;
    const int32_t qh = v.rope.q_heads, kh = v.rope.k_heads, most = kNormMaxThreads / L;
    const bool many = static_cast<int64_t>(v.rope.rows) * L * (qh + kh) > 4LL * 2048 * device_sm_count();
    const int32_t each = many ? kNormHeads : 1;
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

template <typename T, bool INTER>
cudaError_t forward_typed(NormRopeView v, cudaStream_t stream) {
    constexpr int VE = VecTraits<T>::kElems;
    const Shape s = plan<VE>(v);
    const unsigned grid = static_cast<unsigned>(s.row_tiles);
    auto *kernel = v.q_groups < v.rope.q_heads ? norm_rope_kernel<T, 1, kNormHeads, INTER> : norm_rope_kernel<T, 1, 1, INTER>;
    if constexpr (sizeof(T) == 4)  // (a bf16 head has 31 chunks at most)
        if (s.chunks > 32) kernel = norm_rope_kernel<T, 2, 1, INTER>;
    kernel<<<grid, s.block, 0, stream>>>(v);
    count_launches(1);
    return cudaGetLastError();
}

template <typename T, bool INTER>
cudaError_t backward_typed(NormRopeView v, float *dq_weight, float *dk_weight, cudaStream_t stream) {
    constexpr int VE = VecTraits<T>::kElems;
    const Shape s = plan<VE>(v);
    const int64_t most = static_cast<int64_t>(device_sm_count()) * kGradCtas;
    const int32_t grid = static_cast<int32_t>(s.row_tiles < most ? s.row_tiles : most), D = v.rope.head_dim;
    if (!dq_weight && !dk_weight) v.partial = nullptr;
    const size_t smem = v.partial ? static_cast<size_t>(s.block.y) * s.block.z * D * sizeof(float) : 0;
    auto *kernel = norm_rope_backward_kernel<T, 1, INTER>;
    if constexpr (sizeof(T) == 4)
        if (s.chunks > 32) kernel = norm_rope_backward_kernel<T, 2, INTER>;
    kernel<<<grid, s.block, smem, stream>>>(v);
    cudaError_t e = cudaGetLastError();
    count_launches(1);
    if (e != cudaSuccess || !v.partial) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * D / kSumValues);  // (D is a multiple of 8)
    cfg.blockDim = dim3(kSumValues, kSumParts);
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
    if (v.rope.interleaved) return dtype == LORA_FP32 ? forward_typed<float, true>(v, stream) : forward_typed<__nv_bfloat16, true>(v, stream);
    return dtype == LORA_FP32 ? forward_typed<float, false>(v, stream) : forward_typed<__nv_bfloat16, false>(v, stream);
}

cudaError_t launch_norm_rope_backward(const NormRopeView &v, lora_dtype_t dtype, float *dq_weight, float *dk_weight,
                                      cudaStream_t stream) {
    if (v.rope.interleaved)
        return dtype == LORA_FP32 ? backward_typed<float, true>(v, dq_weight, dk_weight, stream)
                                  : backward_typed<__nv_bfloat16, true>(v, dq_weight, dk_weight, stream);
    return dtype == LORA_FP32 ? backward_typed<float, false>(v, dq_weight, dk_weight, stream)
                              : backward_typed<__nv_bfloat16, false>(v, dq_weight, dk_weight, stream);
}

}  // namespace lora
