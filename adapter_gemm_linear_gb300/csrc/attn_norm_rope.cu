// Norms of queries and keys for each head with the rotary positions in the same
// pass (lora_norm_rope), and its gradient (lora_norm_rope_backward).  For a head x
// with weights W (w, or 1 + w):
//     r = 1 / sqrt(mean(x^2) + eps),  n = x r W,  y = rotate(n)
// and, with g the gradient of y,
//     h = rotate^-1(g),  dW = sum over rows and heads of h x r,
//     a = h W,  dx = r (a - x r^2 mean(a x)).
//
// By their bytes both are bound by memory: each value is read once and written once
// (twice read for the gradient), 7 and 14 flops a value.  A head is taken by a group of
// lanes, the least power of two with a chunk (attn_rope.cuh) each, which add up
// its squares by shuffles; the head's values stay in registers in between.  A
// group works on heads of q alone or of k alone, so that its weights are read
// once, and on several heads of a row, so that the angles are.
// Measured in a graph, bf16, 8192 rows of 72 heads of 128, three axes: 52 us (5.9 TB/s of
// the 306 MB, 0.87 of a copy), the gradient 88 (5.2); of 40 heads 29.5 and 51, of 64 15.1 and 30.6,
// in fp32 (4096 rows of 128) 28.7 and 45.  The gradient waits for its own results (shuffles, reads from
// shared memory, the turn's barrier) with the 14 warps an SM that 128 registers leave in this layout of a
// head on its lanes.  One token of 64 sequences, 40 heads: 2.8 us; the gradient of 333 rows of 40 heads of 64 7.8.
#include <cuda_runtime.h>

#include <algorithm>

#include "attn_rope.cuh"
#include "attn_split.cuh"
#include "f32x2.cuh"

namespace lora {

namespace {

constexpr int kNormMaxThreads = 512, kRowThreads = 256;  // of a block, at most: for few rows, and for many
constexpr int kNormThreads = 128;                        // and about
constexpr int kNormHeads = 3;                            // of a group and turn, where there is much work
constexpr int kRowCtas = 4, kGradCtas = 4;               // blocks per SM, at most
constexpr int kStages = 2;                               // turns on their way to shared memory

// 16-byte pieces on their way, of kStages turns: threads x heads x (tensors x chunks) x 2 pieces.
__host__ __device__ constexpr size_t row_pipe_ring_bytes(int threads, int heads, int chunks) {
    return static_cast<size_t>(threads) * heads * chunks * 2 * 16 * kStages;
}

// Asynchronous copies to shared memory: through the L1 for what other threads read too.
template <int BYTES>
__device__ __forceinline__ void copy_ca(void *smem_dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(sm100::smem_u32(smem_dst)), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copy_cg(uint32_t smem_dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 load_shared(uint32_t at) {
    uint4 x;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(at) : "memory");
    return x;
}

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
// LT: L where it is known to the compiler, or 0.
template <int LT>
struct Group {
    bool is_k;
    int32_t c, h0, step, heads;
    uint32_t mask;  // of the group's lanes

    __device__ __forceinline__ Group(const NormRopeView &a) {
        const int32_t L = lanes(), j = threadIdx.y;
        c = threadIdx.x;
        is_k = j >= a.q_groups;
        h0 = is_k ? j - a.q_groups : j;
        step = is_k ? a.k_groups : a.q_groups;
        heads = is_k ? a.rope.k_heads : a.rope.q_heads;
        const uint32_t lane = ((threadIdx.z * blockDim.y + j) * L + c) & 31u;
        mask = L == 32 ? 0xffffffffu : ((1u << L) - 1u) << (lane & ~static_cast<uint32_t>(L - 1));
    }
    static __device__ __forceinline__ int32_t lanes() { return LT ? LT : static_cast<int32_t>(blockDim.x); }
    __device__ __forceinline__ float sum(F2 x2) const {
        const float2 y = apart(x2);
        float x = y.x + y.y;
        if constexpr (LT > 0) {
#pragma unroll
            for (int o = LT / 2; o > 0; o /= 2) x += __shfl_xor_sync(mask, x, o);
        } else {
            for (int32_t o = lanes() >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(mask, x, o);
        }
        return x;
    }
};

// A thread's chunks of a head, NC at most: chunk c, then c + L.  A chunk has two
// pieces u and v of N value pairs; one past the rotated dimensions has no v (zeros).
template <typename T, int NC, int LT>
struct Chunks {
    static constexpr int VE = VecTraits<T>::kElems, N = VE / 2;
    Chunk at[NC];
    bool has[NC];

    __device__ __forceinline__ Chunks(const NormRopeView &a, const Group<LT> &g) {
        const int32_t count = a.rope.rot_dim / (2 * VE) + (a.rope.head_dim - a.rope.rot_dim) / VE;
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            const int32_t c = g.c + n * Group<LT>::lanes();
            has[n] = c < count;
            at[n] = chunk_at<VE>(a.rope, has[n] ? c : 0);
            at[n].turn = at[n].turn && has[n];  // (a lane without a chunk has no angles)
        }
    }
    // W of the chunks; 1 without a weight
    __device__ __forceinline__ void weights(const NormRopeView &a, const Group<LT> &g, F2 (&w)[NC][2][N]) const {
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
    __device__ __forceinline__ void angles(const NormRopeView &a, const Group<LT> &g, int64_t row, float (&cs)[NC][VE], float (&sn)[NC][VE]) const {
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            uint32_t still = (1u << VE) - 1u;
            if (at[n].turn) still = load_angles<VE>(a.rope, g.c + n * Group<LT>::lanes(), row, cs[n], sn[n]);
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
    template <bool INTER>
    __device__ __forceinline__ void store(T *dst, int n, const F2 (&y)[N], const F2 (&z)[N]) const {
        if (INTER && at[n].turn) {  // the pieces are a sector
            const uint4 a = pack2<T>(y), b = pack2<T>(z);
            const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            sm100::store_32(dst + at[n].d0, w);
            return;
        }
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
template <int VE, int NC, bool INTER>
__device__ __forceinline__ void coefficients(const F2 (&W)[NC][2][VE / 2], const float (&cs)[NC][VE], const float (&sn)[NC][VE],
                                             F2 (&A)[NC][2][VE / 2], F2 (&B)[NC][2][VE / 2]) {
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int i = 0; i < VE / 2; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const F2 c = two(angle_of<VE, INTER>(cs[n], k, 2 * i), angle_of<VE, INTER>(cs[n], k, 2 * i + 1));
                const float s0 = angle_of<VE, INTER>(sn[n], k, 2 * i), s1 = angle_of<VE, INTER>(sn[n], k, 2 * i + 1);
                A[n][k][i] = mul(W[n][k][i], c);
                B[n][k][i] = INTER ? mul(swapped(W[n][k][i]), two(-s0, s1)) : mul(W[n][1 - k][i], k == 0 ? two(-s0, -s1) : two(s0, s1));
            }
}
template <int N, bool INTER>
__device__ __forceinline__ void turned(const F2 (&u)[N], const F2 (&v)[N], const F2 (&A)[2][N], const F2 (&B)[2][N], F2 r, F2 (&y)[N],
                                       F2 (&z)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
        y[e] = mul(fma(INTER ? swapped(u[e]) : v[e], B[0][e], mul(u[e], A[0][e])), r);
        z[e] = mul(fma(INTER ? swapped(v[e]) : u[e], B[1][e], mul(v[e], A[1][e])), r);
    }
}

// Few rows: a group has a head or a few of one row, and no more.
template <typename T, int NC, bool INTER, int LT>
__global__ void __launch_bounds__(kNormMaxThreads) norm_rope_kernel(const __grid_constant__ NormRopeView a) {
    constexpr int VE = VecTraits<T>::kElems, N = VE / 2;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.z + threadIdx.z;
    if (row >= a.rope.rows) return;
    const Group<LT> g(a);
    const Chunks<T, NC, LT> ch(a, g);
    const HeadsView &in = g.is_k ? a.rope.k : a.rope.q, &out = g.is_k ? a.rope.k_out : a.rope.q_out;
    F2 A[NC][2][N], B[NC][2][N];
    const float inv_d = 1.0f / static_cast<float>(a.rope.head_dim);
    for (int32_t h = g.h0; h < g.heads; h += g.step) {
        uint4 x[NC][2];
        ch.load(head_at<T>(in, row, h), x);
        if (h == g.h0) {  // (on their way with the first head)
            F2 W[NC][2][N];
            float cs[NC][VE], sn[NC][VE];
            ch.weights(a, g, W);
            ch.angles(a, g, row, cs, sn);
            coefficients<VE, NC, INTER>(W, cs, sn, A, B);
        }
        F2 u[NC][N], v[NC][N], squares = two(0.0f, 0.0f);
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            unpack2<T>(x[n][0], u[n]);
            unpack2<T>(x[n][1], v[n]);
#pragma unroll
            for (int e = 0; e < N; ++e) squares = fma(u[n][e], u[n][e], fma(v[n][e], v[n][e], squares));
        }
        const float r = rsqrtf(fmaf(g.sum(squares), inv_d, a.eps));
        T *dst = head_at<T>(out, row, h);
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            F2 y[N], z[N];
            turned<N, INTER>(u[n], v[n], A[n], B[n], two(r, r), y, z);
            ch.template store<INTER>(dst, n, y, z);
        }
    }
}

// Many rows: blocks take rows (blockDim.z at once) in turn, and of each a few heads a
// thread, in turns of which the next kStages are on their way to shared memory by
// asynchronous copies: a thread's own pieces of x (and dy), and the row's angles,
// which the first group's lanes fetch for all.  (With loads into registers a row's
// chain of position, angles and heads was not covered: 84 and 135 us for 8192 rows of 72
// heads of 128 and their gradient.)

template <typename T, int NC, int P, bool INTER, int LT>
struct RowPipe {
    static constexpr int VE = VecTraits<T>::kElems;
    static constexpr int kPieces = P * NC * 2;  // 16 bytes each, of a thread and head: [tensor][chunk][piece]
    // where a turn is: the thread's row and the pass over it
    struct Turn {
        int64_t row;
        int32_t pass;
    };
    const NormRopeView &a;
    const Group<LT> &g;
    const Chunks<T, NC, LT> &ch;
    // [stage][head][tensor, chunk]: the thread's first piece.  The 16 bytes of a copy lie beside each other in
    // shared memory where they do in global memory, else each half sector is a request of its own
    // and sectors are read twice (8192 rows of 72 heads 70 us instead of 52, their gradient 109 instead of 88): [piece][thread]; interleaved, where a
    // thread's two pieces are a sector, [thread][piece], in an order that keeps 8 threads off each
    // other's banks (and at a multiple of 32 bytes, so that an exclusive or finds the second).
    uint32_t ring;
    uint32_t stride;  // bytes of a piece of all threads
    float *angles;  // [stage, one more][row of the block][cosines, sines][pair]
    int32_t threads, half, pos[LORA_ROPE_MAX_AXES];
    bool fetches;       // the row's angles
    Turn now, ahead;    // the turn in work, and the one that is fetched meanwhile
    // of the head in work, and of the one that is fetched
    uint32_t at;
    int32_t h, h_ahead;
    const T *src[P];
    int64_t src_step[P];  // from a head of the thread's to its next

    __device__ __forceinline__ RowPipe(const NormRopeView &v, const Group<LT> &group, const Chunks<T, NC, LT> &c, const HeadsView (&in)[P], unsigned char *smem)
        : a(v), g(group), ch(c) {
        threads = Group<LT>::lanes() * blockDim.y * blockDim.z;
        const uint32_t tid = (threadIdx.z * blockDim.y + threadIdx.y) * Group<LT>::lanes() + threadIdx.x;
        ring = sm100::smem_u32(smem) + tid * (INTER ? 32 : 16) + (INTER ? (tid / 4 % 2) * 16 : 0);
        stride = threads * 16;
        angles = reinterpret_cast<float *>(smem + row_pipe_ring_bytes(threads, a.per_turn, P * NC));
        half = a.rope.rot_dim / 2;
        fetches = threadIdx.y == 0;
        now.row = ahead.row = static_cast<int64_t>(blockIdx.x) * blockDim.z + threadIdx.z;
        now.pass = ahead.pass = 0;
#pragma unroll
        for (int p = 0; p < P; ++p) src_step[p] = g.step * in[p].head;
    }
    __device__ __forceinline__ void next(Turn &t) const {
        if (++t.pass < a.passes) return;
        t.pass = 0;
        t.row += static_cast<int64_t>(gridDim.x) * blockDim.z;
    }
    __device__ __forceinline__ float *angle_at(int32_t stage) const { return angles + (stage * blockDim.z + threadIdx.z) * 2 * half; }

    __device__ __forceinline__ void read_positions(int64_t row) {
        if (!fetches || row >= a.rope.rows) return;
#pragma unroll
        for (int i = 0; i < LORA_ROPE_MAX_AXES; ++i)
            if (i < a.rope.num_axes) pos[i] = a.rope.positions[static_cast<int64_t>(i) * a.rope.rows + row];
    }
    __device__ __forceinline__ int32_t position(int32_t axis, int64_t row) const {  // < 0: out of range (recorded)
        int32_t p = pos[0];
#pragma unroll
        for (int i = 1; i < LORA_ROPE_MAX_AXES; ++i) p = axis == i ? pos[i] : p;
        if (p >= 0 && p < a.rope.max_pos) return p;
        record_error(a.rope.status, kDevBadBlock, static_cast<uint32_t>(row));
        return -1;
    }
    __device__ __forceinline__ void fetch_angles(int64_t row, int32_t stage) const {
        if (!fetches || row >= a.rope.rows) return;
        float *cs = angle_at(stage), *sn = cs + half;
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            if (!ch.at[n].turn) continue;
            const int32_t c = g.c + n * Group<LT>::lanes(), axis = a.rope.chunk_axis[c];
            const bool one = axis < LORA_ROPE_MAX_AXES;  // the chunk's pairs follow one axis
            int32_t p = one ? position(axis, row) : 0;
#pragma unroll 1
            for (int e = 0; e < VE; e += one ? 4 : 1) {
                const int32_t i = c * VE + e;
                if (!one) p = position(a.rope.pair_axis[i], row);
                const int64_t at = static_cast<int64_t>(max(p, 0)) * half + i;
                if (p < 0) {
                    for (int k = 0; k < (one ? 4 : 1); ++k) {
                        cs[i + k] = 1.0f;
                        sn[i + k] = 0.0f;
                    }
                } else if (one) {
                    copy_ca<16>(cs + i, a.rope.cos_table + at);
                    copy_ca<16>(sn + i, a.rope.sin_table + at);
                } else {
                    copy_ca<4>(cs + i, a.rope.cos_table + at);
                    copy_ca<4>(sn + i, a.rope.sin_table + at);
                }
            }
        }
    }
    // The heads of the turn in `stage`: at(), of them the one to work on, and the one to fetch into its place.
    __device__ __forceinline__ void first_head(const HeadsView (&in)[P], int32_t stage) {
        at = ring + stage * (a.per_turn * threads * (kPieces * 16));
        h = g.h0 + now.pass * a.per_turn * g.step;
        h_ahead = g.h0 + ahead.pass * a.per_turn * g.step;
#pragma unroll
        for (int p = 0; p < P; ++p) src[p] = head_at<T>(in[p], ahead.row, h_ahead);
    }
    __device__ __forceinline__ void next_head() {
        at += threads * (kPieces * 16);
        h += g.step;
        h_ahead += g.step;
#pragma unroll
        for (int p = 0; p < P; ++p) src[p] += src_step[p];
    }
    __device__ __forceinline__ uint32_t piece(int p, int n, int k) const {
        const uint32_t chunk = at + (p * NC + n) * 2 * stride;
        return k == 0 ? chunk : INTER ? chunk ^ 16u : chunk + stride;
    }
    __device__ __forceinline__ bool here() const { return now.row < a.rope.rows && h < g.heads; }
    __device__ __forceinline__ void fetch_head() const {
        if (ahead.row >= a.rope.rows || h_ahead >= g.heads) return;
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                if (ch.has[n]) copy_cg(piece(p, n, 0), src[p] + ch.at[n].d0);
                if (ch.at[n].turn) copy_cg(piece(p, n, 1), src[p] + ch.at[n].d1);
            }
    }
    __device__ __forceinline__ void begin(const HeadsView (&in)[P]) {
        for (int s = 0; s < kStages; ++s) {
            read_positions(ahead.row);
            fetch_angles(ahead.row, s);
            first_head(in, s);
            for (int32_t i = 0; i < a.per_turn; ++i, next_head()) fetch_head();
            asm volatile("cp.async.commit_group;" ::: "memory");
            next(ahead);
        }
        read_positions(ahead.row);
    }
    // The turn's values are there; those of the turn whose place the angles fetched next take are used up.
    __device__ __forceinline__ void ready() const {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        __syncthreads();
    }
    __device__ __forceinline__ void end_turn(int32_t t) {  // (its heads have been fetched anew by the turn itself)
        fetch_angles(ahead.row, (t + kStages) % (kStages + 1));
        asm volatile("cp.async.commit_group;" ::: "memory");
        next(now);
        next(ahead);
        read_positions(ahead.row);
    }
    __device__ __forceinline__ void take(int n, int p, F2 (&u)[VE / 2], F2 (&v)[VE / 2]) const {
        uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
        if (ch.has[n]) x = load_shared(piece(p, n, 0));
        if (ch.at[n].turn) y = load_shared(piece(p, n, 1));
        unpack2<T>(x, u);
        unpack2<T>(y, v);
    }
    __device__ __forceinline__ void take_angles(const float *from, int n, float (&cs)[VE], float (&sn)[VE]) const {
        const int32_t c = (g.c + n * Group<LT>::lanes()) * VE;
#pragma unroll
        for (int e = 0; e < VE; e += 4) {
            float4 x = make_float4(1.0f, 1.0f, 1.0f, 1.0f), y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (ch.at[n].turn) {
                x = *reinterpret_cast<const float4 *>(from + c + e);
                y = *reinterpret_cast<const float4 *>(from + half + c + e);
            }
            cs[e] = x.x; cs[e + 1] = x.y; cs[e + 2] = x.z; cs[e + 3] = x.w;
            sn[e] = y.x; sn[e + 1] = y.y; sn[e + 2] = y.z; sn[e + 3] = y.w;
        }
    }
    __device__ __forceinline__ float *after_angles() const { return angles + (kStages + 1) * blockDim.z * 2 * half; }
};

template <typename T, int NC, bool INTER, int LT>
__global__ void __launch_bounds__(kRowThreads, 2) norm_rope_rows_kernel(const __grid_constant__ NormRopeView a) {
    constexpr int VE = VecTraits<T>::kElems, N = VE / 2;
    extern __shared__ __align__(32) unsigned char smem[];
    const Group<LT> g(a);
    const Chunks<T, NC, LT> ch(a, g);
    const HeadsView in[1] = {g.is_k ? a.rope.k : a.rope.q}, &out = g.is_k ? a.rope.k_out : a.rope.q_out;
    RowPipe<T, NC, 1, INTER, LT> pipe(a, g, ch, in, smem);
    const int64_t out_step = g.step * out.head;
    const float inv_d = 1.0f / static_cast<float>(a.rope.head_dim);
    pipe.begin(in);
    F2 W[NC][2][N];
    ch.weights(a, g, W);
    for (int32_t t = 0; t < a.turns; ++t) {
        pipe.ready();
        pipe.first_head(in, t % kStages);
        F2 A[NC][2][N], B[NC][2][N];
        {
            float cs[NC][VE], sn[NC][VE];
#pragma unroll
            for (int n = 0; n < NC; ++n) pipe.take_angles(pipe.angle_at(t % (kStages + 1)), n, cs[n], sn[n]);
            coefficients<VE, NC, INTER>(W, cs, sn, A, B);
        }
        T *dst = head_at<T>(out, pipe.now.row, pipe.h);
        for (int32_t i = 0; i < a.per_turn; ++i, pipe.next_head(), dst += out_step) {
            if (!pipe.here()) {
                pipe.fetch_head();
                continue;
            }
            F2 u[NC][N], v[NC][N], squares = two(0.0f, 0.0f);
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                pipe.take(n, 0, u[n], v[n]);
#pragma unroll
                for (int e = 0; e < N; ++e) squares = fma(u[n][e], u[n][e], fma(v[n][e], v[n][e], squares));
            }
            pipe.fetch_head();
            const float r = rsqrtf(fmaf(g.sum(squares), inv_d, a.eps));
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                F2 y[N], z[N];
                turned<N, INTER>(u[n], v[n], A[n], B[n], two(r, r), y, z);
                ch.template store<INTER>(dst, n, y, z);
            }
        }
        pipe.end_turn(t);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// A thread adds up its chunks' gradients of the weights over all its rows and heads, a
// block over its groups, grad_weights_kernel over the blocks: every sum's order is fixed.
template <typename T, int NC, bool INTER, int LT>
__global__ void __launch_bounds__(kRowThreads, 2) norm_rope_backward_kernel(const __grid_constant__ NormRopeView a) {
    constexpr int VE = VecTraits<T>::kElems, N = VE / 2;
    extern __shared__ __align__(32) unsigned char smem[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Group<LT> g(a);
    const Chunks<T, NC, LT> ch(a, g);
    const HeadsView in[2] = {g.is_k ? a.rope.k : a.rope.q, g.is_k ? a.dk : a.dq}, &out = g.is_k ? a.rope.k_out : a.rope.q_out;
    RowPipe<T, NC, 2, INTER, LT> pipe(a, g, ch, in, smem);
    const int64_t out_step = g.step * out.head;
    // the weights lie in shared memory, and angles and weights are read where they are used:
    // registers are short, and with most of the L1 taken spilled ones cost a trip to the L2
    float *const weights = pipe.after_angles() + (g.is_k ? a.rope.head_dim : 0);
    if (threadIdx.z == 0 && g.h0 == 0) {
        F2 W[NC][2][N];
        ch.weights(a, g, W);
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (ch.has[n]) *reinterpret_cast<F2 *>(weights + ch.at[n].d0 + 2 * i) = W[n][0][i];
                if (ch.at[n].turn) *reinterpret_cast<F2 *>(weights + ch.at[n].d1 + 2 * i) = W[n][1][i];
            }
    }
    const float inv_d = 1.0f / static_cast<float>(a.rope.head_dim);
    pipe.begin(in);
    F2 dw[NC][2][N];
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int i = 0; i < N; ++i) dw[n][0][i] = dw[n][1][i] = two(0.0f, 0.0f);
    for (int32_t turn = 0; turn < a.turns; ++turn) {
        pipe.ready();
        pipe.first_head(in, turn % kStages);
        const float *const angles = pipe.angle_at(turn % (kStages + 1));
        T *dst = head_at<T>(out, pipe.now.row, pipe.h);
        for (int32_t i = 0; i < a.per_turn; ++i, pipe.next_head(), dst += out_step) {
            if (!pipe.here()) {
                pipe.fetch_head();
                continue;
            }
            F2 u[NC][N], v[NC][N], y[NC][N], z[NC][N];
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                pipe.take(n, 0, u[n], v[n]);
                pipe.take(n, 1, y[n], z[n]);
            }
            pipe.fetch_head();
            F2 squares = two(0.0f, 0.0f), dot = two(0.0f, 0.0f);
#pragma unroll
            for (int n = 0; n < NC; ++n)
#pragma unroll
                for (int e = 0; e < N; ++e) squares = fma(u[n][e], u[n][e], fma(v[n][e], v[n][e], squares));
            const float r = rsqrtf(fmaf(g.sum(squares), inv_d, a.eps));
            const F2 r2 = two(r, r), minus = two(-1.0f, -1.0f);
            // y and z become g turned back, h
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                float cs[VE], sn[VE];
                pipe.take_angles(angles, n, cs, sn);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const F2 y0 = y[n][e], z0 = z[n][e];
                    F2 c[2], t[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        c[k] = two(angle_of<VE, INTER>(cs, k, 2 * e), angle_of<VE, INTER>(cs, k, 2 * e + 1));
                        const float s0 = angle_of<VE, INTER>(sn, k, 2 * e), s1 = angle_of<VE, INTER>(sn, k, 2 * e + 1);
                        t[k] = INTER ? two(s0, -s1) : two(s0, s1);
                    }
                    y[n][e] = fma(INTER ? swapped(y0) : z0, t[0], mul(y0, c[0]));
                    z[n][e] = INTER ? fma(swapped(z0), t[1], mul(z0, c[1])) : fma(mul(y0, t[1]), minus, mul(z0, c[1]));
                }
            }
            // their part in the weights' gradients; then a = h W
#pragma unroll
            for (int n = 0; n < NC; ++n)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float *const w = weights + (k == 0 ? ch.at[n].d0 : ch.at[n].d1);
                    F2(&x)[N] = k == 0 ? u[n] : v[n], (&hw)[N] = k == 0 ? y[n] : z[n];
#pragma unroll
                    for (int e = 0; e < N; e += 2) {
                        const float4 W = *reinterpret_cast<const float4 *>(w + 2 * e);
                        dw[n][k][e] = fma(mul(hw[e], x[e]), r2, dw[n][k][e]);
                        dw[n][k][e + 1] = fma(mul(hw[e + 1], x[e + 1]), r2, dw[n][k][e + 1]);
                        hw[e] = mul(hw[e], two(W.x, W.y));
                        hw[e + 1] = mul(hw[e + 1], two(W.z, W.w));
                        dot = fma(hw[e], x[e], fma(hw[e + 1], x[e + 1], dot));
                    }
                }
            const float back = g.sum(dot) * inv_d * r * r;
            const F2 b2 = two(-back * r, -back * r);
#pragma unroll
            for (int n = 0; n < NC; ++n) {
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    y[n][e] = fma(u[n][e], b2, mul(y[n][e], r2));
                    z[n][e] = fma(v[n][e], b2, mul(z[n][e], r2));
                }
                ch.template store<INTER>(dst, n, y[n], z[n]);
            }
        }
        pipe.end_turn(turn);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();  // the shared memory is the sums' from here on
    float *const sums = reinterpret_cast<float *>(smem);  // [group of the block][head_dim]
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
    bool many;
};

// Groups of L lanes; one head a group where that fills less than the machine's resident
// threads a few times over, else kNormHeads, in turns (passes over a row) of as many.
template <int VE>
Shape plan(NormRopeView &v, bool in_turns, int max_threads) {
    Shape s;
    s.chunks = plan_chunks<VE>(v.rope);
    int32_t L = 4;
    while (L < 32 && L < s.chunks) L *= 2;
    const int32_t qh = v.rope.q_heads, kh = v.rope.k_heads;
    s.many = static_cast<int64_t>(v.rope.rows) * L * (qh + kh) > 4LL * 2048 * device_sm_count();
    const int32_t most = (s.many || in_turns ? max_threads : kNormMaxThreads) / L;
    const int32_t each = s.many ? kNormHeads : 1;
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
    int32_t heads = (qh + v.q_groups - 1) / v.q_groups;  // of a group, at most
    if (kh > 0) heads = std::max(heads, (kh + v.k_groups - 1) / v.k_groups);
    const int32_t limit = s.chunks > 32 ? (kNormHeads + 1) / 2 : kNormHeads;
    v.passes = (heads + limit - 1) / limit;
    v.per_turn = (heads + v.passes - 1) / v.passes;
    return s;
}

// Shared memory of a kernel that takes rows in turn, and its grid: as many blocks as fit.
struct Rows {
    int32_t grid;
    size_t smem;
};
Rows plan_rows(NormRopeView &v, const Shape &s, int pieces, int ctas) {
    Rows r;
    const int32_t threads = s.block.x * s.block.y * s.block.z;
    r.smem = row_pipe_ring_bytes(threads, v.per_turn, pieces) +
             sizeof(float) * ((kStages + 1) * s.block.z * v.rope.rot_dim + 2 * v.rope.head_dim);
    r.smem = std::max(r.smem, sizeof(float) * s.block.y * s.block.z * v.rope.head_dim);  // (the gradients' sums)
    const int32_t fit = static_cast<int32_t>(std::min<size_t>(ctas, 227 * 1024 / (r.smem + 1024)));
    const int64_t most = static_cast<int64_t>(device_sm_count()) * std::max(1, std::min(fit, 2 * kRowThreads / threads));
    r.grid = static_cast<int32_t>(std::min(s.row_tiles, most));
    v.turns = static_cast<int32_t>((s.row_tiles + r.grid - 1) / r.grid) * v.passes;
    return r;
}

// Which kernel: groups of 4, 8 and 16 lanes (heads of 64 and 128 turned whole, in either type) have
// their own, the rest (32 lanes, 0, and with two chunks a lane, 4) read their number: 40 heads
// of 64 15.4 us instead of 20, in fp32 of 128 29 instead of 31.
int lanes_kernel(const Shape &s, bool second) { return second ? 4 : s.block.x == 4 ? 1 : s.block.x == 8 ? 2 : s.block.x == 16 ? 3 : 0; }

template <typename T, bool INTER>
cudaError_t forward_typed(NormRopeView v, cudaStream_t stream) {
    constexpr int VE = VecTraits<T>::kElems;
    const Shape s = plan<VE>(v, false, kRowThreads);
    count_launches(1);
    const bool second = sizeof(T) == 4 && s.chunks > 32;  // (a bf16 head has 31 chunks at most)
    if (!s.many) {
        auto *kernel = norm_rope_kernel<T, 1, INTER, 0>;
        if constexpr (sizeof(T) == 4)
            if (second) kernel = norm_rope_kernel<T, 2, INTER, 0>;
        kernel<<<static_cast<unsigned>(s.row_tiles), s.block, 0, stream>>>(v);
        return cudaGetLastError();
    }
    static uint64_t ctx[5][128] = {};
    const Rows r = plan_rows(v, s, second ? 2 : 1, kRowCtas);
    const int which = lanes_kernel(s, second);
    auto *kernel = which == 1   ? norm_rope_rows_kernel<T, 1, INTER, 4>
                   : which == 2 ? norm_rope_rows_kernel<T, 1, INTER, 8>
                   : which == 3 ? norm_rope_rows_kernel<T, 1, INTER, 16>
                                : norm_rope_rows_kernel<T, 1, INTER, 0>;
    if constexpr (sizeof(T) == 4)
        if (second) kernel = norm_rope_rows_kernel<T, 2, INTER, 0>;
    const cudaError_t e = allow_smem(kernel, 227 * 1024, ctx[which]);
    if (e != cudaSuccess) return e;
    kernel<<<r.grid, s.block, r.smem, stream>>>(v);
    return cudaGetLastError();
}

template <typename T, bool INTER>
cudaError_t backward_typed(NormRopeView v, float *dq_weight, float *dk_weight, cudaStream_t stream) {
    constexpr int VE = VecTraits<T>::kElems;
    const Shape s = plan<VE>(v, true, kRowThreads);
    if (!dq_weight && !dk_weight) v.partial = nullptr;
    static uint64_t ctx[5][128] = {};
    const bool second = sizeof(T) == 4 && s.chunks > 32;
    const Rows r = plan_rows(v, s, second ? 4 : 2, kGradCtas);
    const int32_t grid = r.grid, D = v.rope.head_dim;
    const int which = lanes_kernel(s, second);
    auto *kernel = which == 1   ? norm_rope_backward_kernel<T, 1, INTER, 4>
                   : which == 2 ? norm_rope_backward_kernel<T, 1, INTER, 8>
                   : which == 3 ? norm_rope_backward_kernel<T, 1, INTER, 16>
                                : norm_rope_backward_kernel<T, 1, INTER, 0>;
    if constexpr (sizeof(T) == 4)
        if (second) kernel = norm_rope_backward_kernel<T, 2, INTER, 0>;
    cudaError_t e = allow_smem(kernel, 227 * 1024, ctx[which]);
    if (e != cudaSuccess) return e;
    kernel<<<grid, s.block, r.smem, stream>>>(v);
    e = cudaGetLastError();
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
