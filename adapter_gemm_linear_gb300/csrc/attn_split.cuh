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
// a row of 128: 16 prompts take 210, 213, 227 and 242 us with starts of 0, 4, 6
// and 8, the long chunk 824, 835, 844 and 848, and 2048 queries on 6048 keys whose
// e4m3 scales differ by powers of two 157 and 176 with 0 and 4.
constexpr float kStartDecode = 8.0f, kStartPrefill = 4.0f, kGrow = 15.9f;

// The scales of V's pages, as the exponents of the probabilities take them: in
// log2 relative to a reference vr, the largest of an item's pages in the CTA.
//     p' = 2^(s + rel - m),  o = sum p' code,  l = sum p' 2^-rel = sum 2^(s - m),  out = o vr / l
// While rel is within [-kSpread, 0] neither l nor p' leaves fp32's range: with n
// keys l is below n 2^(kGrow + kSpread), and no p' that counts is flushed.  The
// scales themselves may be anything from 2^-120 to 2^121, and a row may see any of
// an item's pages.  Where an item's scales are further apart, l has to be taken
// from the scores alone: the prompt kernel does that in its tile loop (rel is then
// not held within anything), the decode kernel computes the item by plain_row, and
// what its tile loop gives, with rel held at -kSpread, is not used.  (With a
// reference that begins with the first page's and is changed in the tile loops where
// a later one's is too large, calls of 9 to 16 query rows took 5 to 14% longer
// and long prompts 2%; and rows that do not see the large page lost their V.)
constexpr float kSpread = 80.0f;
constexpr float kSpreadFactor = 1.2089258196146292e24f;  // 2^kSpread

// The reference for the 16-token tiles [tile0, tile1) of a sequence, by a whole
// warp, eight reads a lane in flight: 1 where no scale is above 0, and negative
// where they are too far apart.
__device__ __forceinline__ float v_reference(const KvView &b, int32_t seq, int32_t head, int32_t tile0, int32_t tile1) {
    const int shift = b.page_shift - 4;  // tiles of a page
    const int32_t p1 = (tile1 - 1) >> shift;
    float top = 0.0f, low = INFINITY;
    for (int32_t at = (tile0 >> shift) + (threadIdx.x & 31); tile0 < tile1 && at <= p1; at += 32 * 8) {
        int32_t page[8];
        float vs[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            page[k] = at + 32 * k <= p1 ? b.table[static_cast<int64_t>(seq) * b.max_pages + at + 32 * k] : -1;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            vs[k] = page[k] >= 0 && page[k] < b.num_pages ? __ldg(b.v_scales + static_cast<int64_t>(page[k]) * b.heads + head) : 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            top = fmaxf(top, vs[k]);
            low = vs[k] > 0.0f ? fminf(low, vs[k]) : low;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
    }
    if (!(top > 0.0f)) return 1.0f;
    return log2f(top) - log2f(low) <= kSpread - 1.0f ? top : -top;
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

// One query row of (sequence, key/value head) over its keys in [key0, key1), for
// items whose V scales are too far apart for the kernels' sums: a whole warp, four
// dimensions a lane, four tokens a step, in fp32 and with V relative to the largest
// scale that the row itself sees.  Writes the row's output and lse, or its
// partial result.  (Slow, some 20 us for 100 keys: 64 x 4 queries in a window of
// 1024 with one such head of eight take 780 us instead of 53.)
template <typename T, int D, int FMT>
__device__ __noinline__ void plain_row(const AttnView &a, int32_t seq, int32_t head, int32_t off, int32_t n, int32_t len,
                                       int32_t row, int32_t key0, int32_t key1, float *part, float *part_lse) {
    const KvView &b = a.kv;
    const int lane = threadIdx.x & 31, c = 4 * lane;
    const int32_t qi = row / a.group, qh = head * a.group + row % a.group, pos = len - n + qi;
    const int32_t lo = max(key0, a.window > 0 ? max(0, pos - a.window + 1) : 0), hi = min(key1, a.causal ? pos + 1 : len);
    auto page_of = [&](int32_t key) {
        const int32_t page = b.table[static_cast<int64_t>(seq) * b.max_pages + (key >> b.page_shift)];
        return page >= 0 && page < b.num_pages ? page : -1;
    };
    float q[4] = {0.0f, 0.0f, 0.0f, 0.0f}, amax = 0.0f;
    if (c < D) {
        const T *src = static_cast<const T *>(a.q.p) + static_cast<int64_t>(off + qi) * a.q.row + qh * a.q.head + c;
        for (int d = 0; d < 4; ++d) q[d] = to_float(src[d]);
    }
    for (int d = 0; d < 4; ++d) amax = fmaxf(amax, fabsf(q[d]));
    float top = 0.0f;
    for (int32_t key = (lo >> b.page_shift << b.page_shift) + (lane << b.page_shift); key < hi; key += 32 << b.page_shift) {
        const int32_t page = page_of(key);
        if (page >= 0) top = fmaxf(top, b.v_scales[static_cast<int64_t>(page) * b.heads + head]);
    }
    for (int o = 16; o > 0; o >>= 1) {
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    if (!(top > 0.0f)) top = 1.0f;
    // as the kernels do: the row's largest to [2^13, 2^14)
    int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 13;
    e = amax < INFINITY ? max(e, -126) : 0;
    const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    const float up = a.scale * kLog2e * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    for (int d = 0; d < 4; ++d) q[d] *= down;
    float M = -INFINITY, L = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int32_t k4 = lo & ~3; k4 < hi; k4 += 4) {
        const int32_t page = page_of(k4), t0 = k4 & (kKvTile - 1);
        float ks = 0.0f, vs = 0.0f, s[4], v[4][4];
        uint32_t kw[4] = {0u, 0u, 0u, 0u};
        uint4 vw = make_uint4(0u, 0u, 0u, 0u);
        if (page >= 0) {
            ks = b.k_scales[static_cast<int64_t>(page) * b.heads + head];
            vs = b.v_scales[static_cast<int64_t>(page) * b.heads + head];
            const int64_t at = tile_offset<D>(b, page, head, (k4 & (b.page_tokens - 1)) / kKvTile);
            if (c < D) {
                for (int t = 0; t < 4; ++t)
                    kw[t] = *reinterpret_cast<const uint32_t *>(b.k_pages + at + c / 64 * (kKvTile * 64) + (t0 + t) * 64 + c % 64);
                if (vs > 0.0f) vw = *reinterpret_cast<const uint4 *>(b.v_pages + at + lane * 64 + t0 * 4);
            }
        }
        float mn = M;
        for (int t = 0; t < 4; ++t) {
            float k[4];
            codes_to_float<FMT>(kw[t], k);
            float dot = q[0] * k[0] + q[1] * k[1] + (q[2] * k[2] + q[3] * k[3]);
            for (int i = 16; i > 0; i >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, i);
            s[t] = k4 + t >= lo && k4 + t < hi ? dot * (ks * up) : -INFINITY;
            mn = fmaxf(mn, s[t]);
        }
        codes_to_float<FMT>(vw.x, v[0]);
        codes_to_float<FMT>(vw.y, v[1]);
        codes_to_float<FMT>(vw.z, v[2]);
        codes_to_float<FMT>(vw.w, v[3]);
        const float mu = mn == -INFINITY ? 0.0f : mn, f = ex2(M - mu), rel = vs > 0.0f ? vs / top : 0.0f;
        float sum = 0.0f, add[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int t = 0; t < 4; ++t) {
            if (k4 + t < lo || k4 + t >= hi) continue;  // (whose codes may be NaN)
            const float w = ex2(s[t] - mu);
            sum += w;
            for (int d = 0; d < 4; ++d) add[d] = fmaf(w, v[d][t], add[d]);
        }
        M = mn;
        L = fmaf(L, f, sum);
        for (int d = 0; d < 4; ++d) o[d] = fmaf(add[d], rel, o[d] * f);
    }
    const float inv = part == nullptr || !(L == 0.0f) ? 1.0f / L : 0.0f, lse = M + log2f(L);
    const float4 y = make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
    if (c < D) {
        if (part) store4(part + c, y, top);
        else store4(static_cast<T *>(a.out.p) + static_cast<int64_t>(off + qi) * a.out.row + qh * a.out.head + c, y, top);
    }
    if (lane == 0) {
        if (part) *part_lse = lse;
        else if (a.lse) a.lse[static_cast<int64_t>(off + qi) * a.q_heads + qh] = lse * kLn2;
    }
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
// what bounds the kernel is their latency.  (Both kernels in a graph, with G = 1,
// 2, 4 and 8: one sequence of 2000 tokens, 32 heads on 8, 11.1, 10.5, 10.5 and 12.1
// us; of 4096, 64 heads on 8, 14.7, 13.0, 12.7 and 13.7; but 64 x 4 queries in a
// window of 1024, whose items span two CTAs, 42.6, 43.7, 45.7 and 49.7.)  Every
// sum's order is fixed.
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
