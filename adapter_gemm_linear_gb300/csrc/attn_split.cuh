// What the attention kernels that cut their keys over CTAs share: where a
// CTA's partial results go, and the kernel that joins them.
//
// The units of all items (sequence, key/value head, tile of query rows) form
// one line, of which every CTA takes an equal contiguous range.  A CTA holds
// the beginning of at most one item that goes on in the next CTA (slot 1),
// and the middle or end of at most one that began before (slot 0).
#pragma once

#include "attn_device.cuh"
#include "sm100_ptx.cuh"

namespace lora {

struct alignas(16) JoinEntry {
    int32_t last_cta;        // < 0: nothing to join
    int32_t head, off;       // key/value head, the sequence's first row
    int32_t row, rows;       // the item's first query row and its number of them
    int32_t pad[3];
};

// Floats of one partial result: [rows][D] outputs over the keys of the part
// alone, then the rows' log2 of the sum of 2^score over them.
__host__ __device__ constexpr size_t partial_floats(int rows, int D) { return static_cast<size_t>(rows) * (D + 1); }

__host__ __device__ constexpr size_t split_workspace_bytes(int ctas, int rows, int D) {
    return static_cast<size_t>(ctas) * (partial_floats(rows, D) * 2 * sizeof(float) + sizeof(JoinEntry));
}

__device__ __forceinline__ JoinEntry *join_entries(const AttnView &a, int32_t ctas, int rows, int D) {
    return reinterpret_cast<JoinEntry *>(reinterpret_cast<float *>(a.workspace) + partial_floats(rows, D) * 2 * ctas);
}

__device__ __forceinline__ float *partial_at(const AttnView &a, int32_t cta, int slot, int rows, int D) {
    return reinterpret_cast<float *>(a.workspace) + (2 * static_cast<size_t>(cta) + slot) * partial_floats(rows, D);
}

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;
// Where in f16's range the probabilities p' lie that enter the second product: a
// row's sums are (re)scaled so that the largest so far is 2^start, and again
// when one would pass 2^kGrow (below f16's largest, 65504).  What lies below
// 2^-14 has steps of 2^-24, so the largest p' are started high: a p' is off by
// 2^-25 at most, 2^-(25 + start) of the row's largest, which a long flat tail behind a
// dominant key adds up.  In the decode kernel the start costs nothing (0, 4
// and 8 within 1% of each other).  The prompt kernel waits for each rescaling of
// a row of 128: 16 prompts take 210, 213, 227 and 242 us with starts of 0,
// 4, 6 and 8, the long chunk 824, 835, 844 and 848.
constexpr float kStartDecode = 8.0f, kStartPrefill = 4.0f, kGrow = 15.9f;

// The scales of V's pages, as the exponents of the probabilities take them: in
// log2 relative to a reference vr, and within +-kSpread of it.
//     p' = 2^(s + rel - m),  o = sum p' code,  l = sum p' 2^-rel = sum 2^(s - m),  out = o vr / l
// so that neither l nor p' leaves fp32's range wherever the scales lie in theirs
// (2^-120 .. 2^121): with n keys l is between 2^-kSpread and n 2^(kGrow + kSpread).
// A page smaller than 2^-kSpread of the reference counts as that much, or as
// zero: what it is off by is 2^-kSpread of the row's largest V, below every other
// rounding here.
// The decode kernel's reference is the largest scale of an item's pages in the
// CTA, looked up beforehand.  The prompt kernel's is that of the first key tile that has
// one, until a tile's is larger than 2^kSpread of it: with d = log2 of that step, o *= 2^(lower -
// d), m -= lower, l *= 2^lower, where lower = d (o stays) unless l would then
// pass 2^kMostSum.  (In the decode kernel that change, once in the tile loop, cost
// calls of 9 to 16 query rows 5 to 14%.)
constexpr float kSpread = 40.0f;
constexpr float kSpreadFactor = 1099511627776.0f;  // 2^kSpread
constexpr float kMostSum = 60.0f;

// The `lower` above, for a row whose l is `sum`.
__device__ __forceinline__ float reference_shift(float d, float sum) {
    return fminf(fminf(d, 100.0f), fmaxf(kMostSum - log2f(sum), 0.0f));
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void store4(float *p, const float4 &v, float f) {
    *reinterpret_cast<float4 *>(p) = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float4 &v, float f) {
    __nv_bfloat162 h[2] = {__floats2bfloat162_rn(v.x * f, v.y * f), __floats2bfloat162_rn(v.z * f, v.w * f)};
    *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<uint2 *>(h);
}

// 16 bytes from global to shared memory, asynchronously; zeros if not `there`.
__device__ __forceinline__ void copy16(void *smem_dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sm100::smem_u32(smem_dst)), "l"(src), "r"(there ? 16 : 0)
                 : "memory");
}

__device__ __forceinline__ void add_scaled(float4 &v, float &L, float f, const float4 &x, float l) {
    L = fmaf(l, f, L);
    v.x = fmaf(x.x, f, v.x);
    v.y = fmaf(x.y, f, v.y);
    v.z = fmaf(x.z, f, v.z);
    v.w = fmaf(x.w, f, v.w);
}

// Joins the items that span CTAs: block x takes the item that begins in CTA x
// and goes on in the next ones, block row y some of its rows.  The partial
// results of a row go to G groups of threads in turn, which take up to eight at
// a time, so that all loads of an item in up to 8 G CTAs are in flight together:
// what bounds the kernel is their latency.  (Both kernels for one sequence of
// 2000 tokens, 32 heads on 8, each of these in 16 CTAs: 14.3 us with G = 4,
// 18.4 with 1, 16.4 with 8.)  Every sum's order is fixed.
// The kernel may begin while the one before still writes what it joins, so after
// its wait it reads through the L2 and never by the read-only path, which is
// for data that nobody writes while a kernel runs.
// The kernel also gives the rows of padding and skipped sequences their zeros,
// and records the malformed ones.
constexpr int kJoinThreads = 256;
// log2 by which the partial results' weights are lowered, so that the sum over
// them stays in range whatever V's is
constexpr float kPartialShift = 12.0f;

template <typename T, int D, int ROWS, int G>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const __grid_constant__ AttnView a, int32_t ctas,
                                                                 int32_t slot_rows) {
    constexpr int PER_ROW = D / 4, BLOCK_ROWS = kJoinThreads / (PER_ROW * G);
    const KvView &b = a.kv;
    // the malformed and padding sequences do not need the kernel before
    for (int32_t s = blockIdx.x * gridDim.y + blockIdx.y; s < b.num_seqs; s += gridDim.x * gridDim.y) {
        const SeqRows r = read_seq(b, s, threadIdx.x == 0);
        const int32_t off = b.offsets ? b.offsets[s] : s, end = b.offsets ? b.offsets[s + 1] : s + 1;
        if (r.n > a.max_queries && threadIdx.x == 0) record_error(b.status, kDevBadSegment, static_cast<uint32_t>(s));
        if (r.n > 0 && r.n <= a.max_queries) continue;
        if (off < 0 || end > b.rows) continue;
        for (int64_t i = threadIdx.x; i < static_cast<int64_t>(end - off) * a.q_heads * D; i += kJoinThreads) {
            const int64_t rh = i / D;
            const int64_t row = off + rh / a.q_heads, h = rh % a.q_heads;
            static_cast<T *>(a.out.p)[row * a.out.row + h * a.out.head + i % D] = from_float<T>(0.0f);
            if (a.lse && i % D == 0) a.lse[row * a.q_heads + h] = -INFINITY;
        }
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const JoinEntry e = join_entries(a, ctas, slot_rows, D)[blockIdx.x];
    const int32_t lane = threadIdx.x % PER_ROW, group = threadIdx.x / PER_ROW % G, r0 = threadIdx.x / (PER_ROW * G);
    const int32_t rt = blockIdx.y * BLOCK_ROWS + r0, c = lane * 4;
    if (e.last_cta < 0 || blockIdx.y * BLOCK_ROWS >= e.rows) return;
    // the group's partial results in order, of which each has weight 2^m
    constexpr int AT_ONCE = 8;
    float M = -INFINITY, L = 0.0f;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int32_t k0 = blockIdx.x + group; rt < e.rows && k0 <= e.last_cta; k0 += AT_ONCE * G) {
        float m[AT_ONCE];
        float4 x[AT_ONCE];
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            const int32_t k = k0 + i * G;
            const float *p = partial_at(a, k, k == static_cast<int32_t>(blockIdx.x) ? 1 : 0, slot_rows, D);
            m[i] = -INFINITY;
            if (k <= e.last_cta) {
                m[i] = __ldcg(p + slot_rows * D + rt);
                x[i] = __ldcg(reinterpret_cast<const float4 *>(p + rt * D + c));
            }
        }
        float mn = M;
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) mn = fmaxf(mn, m[i]);
        const float mu = mn == -INFINITY ? 0.0f : mn;
        const float f0 = ex2(M - mu);
        M = mn;
        L *= f0;
        v = make_float4(v.x * f0, v.y * f0, v.z * f0, v.w * f0);
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            if (k0 + i * G > e.last_cta) break;
            add_scaled(v, L, ex2(m[i] - mu - kPartialShift), x[i], 1.0f);
        }
    }
    if constexpr (G > 1) {
        __shared__ float4 gv[BLOCK_ROWS][G][PER_ROW];
        __shared__ float2 gml[BLOCK_ROWS][G];
        gv[r0][group][lane] = v;
        if (lane == 0) gml[r0][group] = make_float2(M, L);
        __syncthreads();
        if (group > 0) return;
#pragma unroll
        for (int i = 1; i < G; ++i) M = fmaxf(M, gml[r0][i].x);
        const float mu = M == -INFINITY ? 0.0f : M;
        const float f0 = ex2(gml[r0][0].x - mu);
        L *= f0;
        v = make_float4(v.x * f0, v.y * f0, v.z * f0, v.w * f0);
#pragma unroll
        for (int i = 1; i < G; ++i) add_scaled(v, L, ex2(gml[r0][i].x - mu), gv[r0][i][lane], gml[r0][i].y);
    }
    if (rt >= e.rows) return;
    const int32_t row = e.row + rt;
    const int32_t qi = row / a.group, qh = e.head * a.group + row % a.group;
    store4(static_cast<T *>(a.out.p) + static_cast<int64_t>(e.off + qi) * a.out.row + qh * a.out.head + c, v, 1.0f / L);
    if (a.lse && c == 0) a.lse[static_cast<int64_t>(e.off + qi) * a.q_heads + qh] = (M + kPartialShift + log2f(L)) * kLn2;
}

// Opts a kernel in to `bytes` of shared memory, once per device and context (`ctx`: what has been done).
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, uint64_t (&ctx)[128]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
    uint64_t seen = ctx[dev];
    if (first_use_in_context(&seen)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) {
            cudaGetLastError();  // reported here, not by the next launch
            return e;
        }
        ctx[dev] = seen;
    }
    return cudaSuccess;
}

// Starts the join behind the kernel that was launched last on the stream.
template <typename T, int D, int ROWS, int G>
cudaError_t launch_join(const AttnView &v, int ctas, int slot_rows, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, (ROWS * (D / 4) * G + kJoinThreads - 1) / kJoinThreads);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_join_kernel<T, D, ROWS, G>, v, static_cast<int32_t>(ctas),
                              static_cast<int32_t>(slot_rows));
}

}  // namespace lora
