// Attention over the 8-bit paged cache (lora_kv_attention) for few queries a
// sequence: decode steps, checking of drafted tokens, and every fp32 call.
//
// With few query rows each key and value is used a handful of times, so the
// call is bound by reading the codes: 2 D bytes per token and key/value head.
// What the kernel does about it:
//  - One persistent CTA per SM.  The keys of all (sequence, key/value head,
//    tile of query rows) items, cut in chunks of 128 tokens, are dealt out in
//    equal contiguous ranges, so ragged lengths and few long sequences load
//    every SM alike.  An item that spans CTAs is joined by attn_join_kernel
//    from fp32 partial results (o, m, l), in a fixed order.
//  - A producer warp streams the 16-token tiles of K and V codes with bulk
//    copies into a ring of shared memory, 128 KiB deep; eight consumer warps
//    take the tiles in turn, each with its own running softmax, and are
//    merged in shared memory at an item's end.
//  - The codes become f16 in registers (exactly) and feed warp MMAs
//    (16 x 8 x 16, fp32 sums): S = q K^T with the 16 query rows as M and
//    8 tokens as N, then o += p V with the same registers of S as A operand.
//    The tiles' layout in the cache is the fragments' layout: a thread's 16
//    bytes of K are 16 dimensions of one token (four k-steps, the order of
//    the dimensions within a k-step being free as long as q follows it); its
//    16 bytes of V are four dimensions x the four tokens whose p it holds.
//  - q enters as f16 times a power of two per row (exact for bf16).  In fp32
//    calls q and p are each split in two f16 parts, hi + lo 2^-11, put in
//    rows g and g + 8 of the MMA's 16, so a thread holds both parts' sums: 22
//    significant bits at the cost of half the rows.
//  - The page's scale of V is folded into the exponent: p' = 2^(s + log2 vs -
//    m), o sums p' codes, l sums p' / vs.  p' <= 2^14 whatever the scales, so
//    f16 holds it.  m follows the maximum only when that grows by 2^14, so the
//    sums are rarely rescaled.
#include <cuda_runtime.h>
#include <math.h>

#include "attn_device.cuh"
#include "attn_internal.h"
#include "attn_split.cuh"
#include "sm100_ptx.cuh"

namespace lora {

namespace {

using namespace sm100;

constexpr int kWarps = 8;                          // consumer warps
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kChunkTiles = 8;                     // tiles of a unit of work (128 tokens)
constexpr int kMmaRows = 16;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr float kLoScale = 2048.0f;                // 2^11: the lo parts of fp32 operands

template <int D>
__host__ __device__ constexpr int slots() { return 128 * 1024 / (2 * kKvTile * D); }

template <typename T>
__host__ __device__ constexpr int tile_rows() { return sizeof(T) == 4 ? kMmaRows / 2 : kMmaRows; }  // query rows of an item

// One tile's page scales, made by the producer: K's scale, log2 and reciprocal of V's.
struct TileScales {
    float ks, vs, lv, ivs;
};

template <int D>
struct DecodeSmem {
    alignas(128) uint8_t ring[slots<D>()][2][kKvTile * D];
    float o[kWarps][kMmaRows][D + 4];  // merge: padded against bank conflicts
    float m[kWarps][kMmaRows], l[kWarps][kMmaRows];
    alignas(16) TileScales scales[slots<D>()];
    uint64_t full[slots<D>()], empty[slots<D>()];
    uint32_t issued[slots<D>()];  // tiles loaded into the slot so far
    long long warp_sum[kThreads / 32];
    long long base;  // first unit of the sequence the CTA begins in
    int32_t seq;
    int32_t dead;    // a wait ran out: nobody waits any more
};

__device__ __forceinline__ void mma_16816_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// The lo parts of two values whose f16 roundings are `hi`, times 2^11.
__device__ __forceinline__ uint32_t pack_rest(float a, float b, uint32_t hi) {
    const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    return pack_f16((a - h.x) * kLoScale, (b - h.y) * kLoScale);
}

// A sequence's work: `chunks` units for each of heads x row_tiles items, over tiles [t0, t1).
struct SeqWork {
    SeqRows r;
    int32_t t0, t1, chunks, row_tiles;
    long long units;
};

template <typename T>
__device__ __forceinline__ SeqWork seq_work(const AttnView &a, int32_t s) {
    SeqWork w;
    w.r = read_seq(a.kv, s, false);
    if (w.r.n > a.max_queries) w.r.n = 0;
    w.t0 = w.t1 = w.chunks = w.row_tiles = 0;
    if (w.r.n > 0) {
        const int32_t first = w.r.len - w.r.n;
        const int32_t begin = a.window > 0 ? max(0, first - a.window + 1) : 0;
        w.t0 = begin / kKvTile;
        w.t1 = (w.r.len + kKvTile - 1) / kKvTile;
        w.chunks = (w.t1 - w.t0 + kChunkTiles - 1) / kChunkTiles;
        w.row_tiles = (w.r.n * a.group + tile_rows<T>() - 1) / tile_rows<T>();
    }
    w.units = static_cast<long long>(w.chunks) * w.row_tiles * a.kv.heads;
    return w;
}

// One CTA's walk over its units [w, end): item by item.
template <typename T>
struct Walk {
    const AttnView &a;
    long long w, end, base;
    int32_t s;
    SeqWork work;
    // the current item
    int32_t head, row_tile, tile0, tile1;  // tiles of this CTA
    bool from_start, to_end;               // whether the item begins / ends in this CTA
    long long item_end;                    // unit after the item's last

    __device__ __forceinline__ Walk(const AttnView &v, long long w0, long long w1, int32_t seq, long long seq_base)
        : a(v), w(w0), end(w1), base(seq_base), s(seq) {
        if (w < end) work = seq_work<T>(a, s);
    }

    __device__ __forceinline__ bool next() {
        if (w >= end) return false;
        while (w >= base + work.units) {
            base += work.units;
            work = seq_work<T>(a, ++s);
        }
        const long long local = w - base;
        const long long item = local / work.chunks;
        const int32_t c = static_cast<int32_t>(local - item * work.chunks);
        head = static_cast<int32_t>(item / work.row_tiles);
        row_tile = static_cast<int32_t>(item - static_cast<long long>(head) * work.row_tiles);
        const int32_t c1 = static_cast<int32_t>(min(static_cast<long long>(work.chunks), c + (end - w)));
        tile0 = work.t0 + c * kChunkTiles;
        tile1 = min(work.t1, work.t0 + c1 * kChunkTiles);
        from_start = c == 0;
        to_end = c1 == work.chunks;
        item_end = base + (item + 1) * work.chunks;
        w += c1 - c;
        return true;
    }
};

// The query rows [row_tile * tile_rows, ...) of (sequence, key/value head): row r is query r / group of the
// sequence, query head head * group + r % group.
template <typename T, int D, int FMT>
__global__ void __launch_bounds__(kThreads, 1) attn_decode_kernel(const __grid_constant__ AttnView a) {
    extern __shared__ __align__(128) unsigned char raw[];
    DecodeSmem<D> &sm = *reinterpret_cast<DecodeSmem<D> *>(raw);
    constexpr int SLOTS = slots<D>();
    constexpr bool SPLIT = sizeof(T) == 4;  // fp32: operands in two f16 parts
    constexpr int ROWS = tile_rows<T>();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const KvView &b = a.kv;
    JoinEntry *joins = join_entries(a, gridDim.x, kMmaRows, D);

    // ---- the plan: where this CTA's range of units begins
    for (int i = threadIdx.x; i < SLOTS; i += kThreads) {
        mbar_init(&sm.full[i], 1);
        mbar_init(&sm.empty[i], 1);
        sm.issued[i] = 0;
    }
    fence_mbar_init();
    const int32_t per = (b.num_seqs + kThreads - 1) / kThreads;
    const int32_t s0 = min(b.num_seqs, static_cast<int32_t>(threadIdx.x) * per), s1 = min(b.num_seqs, s0 + per);
    long long mine = 0;
    for (int32_t s = s0; s < s1; ++s) mine += seq_work<T>(a, s).units;
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) sm.warp_sum[warp] = upto;
    if (threadIdx.x == 0) {
        sm.dead = 0;
        joins[blockIdx.x] = JoinEntry{-1, 0, 0, 0};
    }
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) upto += sm.warp_sum[w];
        total += sm.warp_sum[w];
    }
    // as many CTAs as there are units at most, so that none between two of an item is without work
    const long long ctas = min(total, static_cast<long long>(gridDim.x));
    const long long w0 = blockIdx.x < ctas ? total * blockIdx.x / ctas : 0;
    const long long w1 = blockIdx.x < ctas ? total * (blockIdx.x + 1) / ctas : 0;
    if (w0 < w1 && upto - mine <= w0 && w0 < upto) {
        long long at = upto - mine;
        int32_t s = s0;
        for (;; ++s) {
            const long long u = seq_work<T>(a, s).units;
            if (w0 < at + u) break;
            at += u;
        }
        sm.seq = s;
        sm.base = at;
    }
    __syncthreads();
    Walk<T> walk(a, w0, w1, sm.seq, sm.base);
    volatile int32_t *dead = &sm.dead;

    if (warp == kWarps) {
        // ---- producer: lane l loads tiles l, l + 32, ... of an item
        uint32_t i0 = 0;  // tiles of the items before
        while (walk.next()) {
            const int32_t count = walk.tile1 - walk.tile0;
            const int tile_shift = b.page_shift - 4;  // tiles of a page, as a shift
            int32_t page = -1;
            float ks = 0.0f, vs = 0.0f;
            auto fetch = [&](int32_t t) {
                page = read_page(b, walk.s, t >> tile_shift);
                const int64_t at = static_cast<int64_t>(page) * b.heads + walk.head;
                ks = page < 0 ? 0.0f : __ldg(b.k_scales + at);
                vs = page < 0 ? 0.0f : __ldg(b.v_scales + at);
            };
            if (lane < count) fetch(walk.tile0 + lane);
            for (int32_t j0 = 0; j0 < count; j0 += 32) {
                const int32_t j = j0 + lane;
                const int32_t t = walk.tile0 + j;
                const int32_t pg = page;
                TileScales sc;
                sc.ks = ks;
                sc.vs = vs;
                sc.lv = log2f(vs);
                sc.ivs = 1.0f / vs;
                const int64_t at = tile_offset<D>(b, pg < 0 ? 0 : pg, walk.head, t & ((1 << tile_shift) - 1));
                if (j + 32 < count) fetch(t + 32);
                // four tiles at a time, so that none waits for a slot far behind its own
                for (int q = 0; q < 8; ++q) {
                    if ((lane >> 2) != q || j >= count) continue;
                    const uint32_t i = i0 + j, slot = i % SLOTS;
                    if (!*dead && !mbar_wait_bounded(&sm.empty[slot], ((i / SLOTS) & 1u) ^ 1u, kWaitNs)) {
                        record_error(b.status, kDevTimeout, 40);
                        *dead = 1;
                    }
                    if (*dead) continue;
                    sm.scales[slot] = sc;
                    sm.issued[slot] = i / SLOTS + 1;
                    if (pg < 0) {  // a page that is not there reads as zeros
                        for (int k = 0; k < 2 * kKvTile * D / 16; ++k)
                            reinterpret_cast<uint4 *>(sm.ring[slot][0])[k] = make_uint4(0, 0, 0, 0);
                        fence_proxy_async_shared();  // before a later copy into the slot
                        mbar_arrive(&sm.full[slot]);
                    } else {
                        mbar_arrive_expect_tx(&sm.full[slot], 2 * kKvTile * D);
                        bulk_load(sm.ring[slot][0], b.k_pages + at, kKvTile * D, &sm.full[slot]);
                        bulk_load(sm.ring[slot][1], b.v_pages + at, kKvTile * D, &sm.full[slot]);
                    }
                }
                __syncwarp();
            }
            i0 += count;
        }
        // after a time-out copies may be in flight that nobody has waited for
        if (*dead) {
            __syncwarp();
            for (int k = lane; k < SLOTS; k += 32)
                if (sm.issued[k]) mbar_wait_bounded(&sm.full[k], (sm.issued[k] - 1) & 1u, kWaitNs);
        }
        return;
    }

    // ---- consumers
    const int g = lane >> 2, tig = lane & 3;
    uint32_t i0 = 0;
    bool merged = false;  // whether the merge buffer may still be read by others
    while (walk.next()) {
        const SeqRows &r = walk.work.r;
        const int32_t rows = min(ROWS, r.n * a.group - walk.row_tile * ROWS);
        // q as A fragments: row g (and g + 8), dimensions 64 h + 16 tig + 4 j + 0..3 in k-step (h, j)
        uint32_t qf[D / 16][4];
        float cr[2];             // score scale of the two rows, in log2 units
        int32_t kmin[2], kmax[2];
#pragma unroll
        for (int u = 0; u < (SPLIT ? 1 : 2); ++u) {
            const int32_t rt = g + 8 * u;
            const int32_t row = walk.row_tile * ROWS + min(rt, rows - 1);  // rows past the last repeat it
            const int32_t qi = row / a.group, qh = walk.head * a.group + row % a.group;
            const int32_t pos = r.len - r.n + qi;
            kmax[u] = a.causal ? pos + 1 : r.len;
            kmin[u] = a.window > 0 ? max(0, pos - a.window + 1) : 0;
            const T *src = static_cast<const T *>(a.q.p) + static_cast<int64_t>(r.off + qi) * a.q.row + qh * a.q.head;
            float x[D / 4];
            float amax = 0.0f;
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
#pragma unroll
                for (int e = 0; e < 16; e += VecTraits<T>::kElems)
                    VecTraits<T>::load(src + 64 * h + 16 * tig + e, x + 16 * h + e);
#pragma unroll
            for (int e = 0; e < D / 4; ++e) amax = fmaxf(amax, fabsf(x[e]));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // a power of two that brings the row's largest to [2^13, 2^14): f16 keeps
            // every value down to 2^-28 of it; not finite: left as it is
            int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 13;
            e = amax < INFINITY ? max(e, -126) : 0;
            const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
            cr[u] = a.scale * kLog2e * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const float *v = x + 4 * k;
                const uint32_t p0 = pack_f16(v[0] * down, v[1] * down), p1 = pack_f16(v[2] * down, v[3] * down);
                qf[k][u] = p0;
                qf[k][2 + u] = p1;
                if (SPLIT) {
                    qf[k][1] = pack_rest(v[0] * down, v[1] * down, p0);
                    qf[k][3] = pack_rest(v[2] * down, v[3] * down, p1);
                }
            }
        }
        if (SPLIT) {
            cr[1] = cr[0];
            kmin[1] = kmin[0];
            kmax[1] = kmax[0];
        }
        // keys that every row of the item sees: tiles within need no mask
        const int32_t pos0 = r.len - r.n + walk.row_tile * ROWS / a.group;
        const int32_t pos1 = r.len - r.n + (walk.row_tile * ROWS + rows - 1) / a.group;
        const int32_t all_hi = a.causal ? pos0 + 1 : r.len;
        const int32_t all_lo = a.window > 0 ? max(0, pos1 - a.window + 1) : 0;

        float o[D / 8][4];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
        bool seen = false;  // a tile whose V is not all zero
        float lv = 0.0f, ivs = 1.0f;

        const int32_t count = walk.tile1 - walk.tile0;
        // this warp's tiles: those whose running number is the warp's modulo kWarps
        for (int32_t j = (warp - static_cast<int32_t>(i0 % kWarps) + kWarps) % kWarps; j < count; j += kWarps) {
            const uint32_t i = i0 + j, slot = i % SLOTS;
            if (!*dead && !mbar_wait_bounded(&sm.full[slot], (i / SLOTS) & 1u, kWaitNs)) {
                record_error(b.status, kDevTimeout, 41);
                *dead = 1;
            }
            const int32_t key0 = (walk.tile0 + j) * kKvTile;
            const uint8_t *kt = sm.ring[slot][0], *vt = sm.ring[slot][1];
            const TileScales sc = sm.scales[slot];
            // S: n-tile u, column n is token 4 (n / 2) + 2 u + n % 2, so that a
            // thread's columns 2 tig, 2 tig + 1 of both are tokens 4 tig .. 4 tig + 3
            float s[2][4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                s[u][0] = s[u][1] = s[u][2] = s[u][3] = 0.0f;
                const int tok = 4 * (g >> 1) + 2 * u + (g & 1);
#pragma unroll
                for (int h = 0; h < D / 64; ++h) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(kt + h * (kKvTile * 64) + tok * 64 + tig * 16);
                    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t b0, b1;
                        codes_to_f16<FMT>(ws[k], b0, b1);
                        mma_16816_f16(s[u], qf[4 * h + k], b0, b1);
                    }
                }
            }
            // scores in log2 units, with V's scale
            if (sc.vs > 0.0f) {
                lv = sc.lv;
                ivs = sc.ivs;
                if (!seen) {  // tiles so far had V = 0 and took lv = 0: their sums move to this one's
                    seen = true;
                    m[0] += lv;
                    m[1] += lv;
                    l[0] *= ivs;
                    l[1] *= ivs;
                }
            }
            float z[2][4];  // [row][token]
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (SPLIT) {
                        z[0][2 * u + e] = fmaf(fmaf(s[u][2 + e], 1.0f / kLoScale, s[u][e]), sc.ks * cr[0], lv);
                    } else {
                        z[0][2 * u + e] = fmaf(s[u][e], sc.ks * cr[0], lv);
                        z[1][2 * u + e] = fmaf(s[u][2 + e], sc.ks * cr[1], lv);
                    }
                }
            if (key0 < all_lo || key0 + kKvTile > all_hi) {
#pragma unroll
                for (int rr = 0; rr < (SPLIT ? 1 : 2); ++rr)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int32_t key = key0 + 4 * tig + e;
                        if (key < kmin[rr] || key >= kmax[rr]) z[rr][e] = -INFINITY;
                    }
            }
            uint32_t pf[4];
            bool grow = false;
            float mx[2];
#pragma unroll
            for (int rr = 0; rr < (SPLIT ? 1 : 2); ++rr) {
                float x = fmaxf(fmaxf(z[rr][0], z[rr][1]), fmaxf(z[rr][2], z[rr][3]));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                mx[rr] = x;
                grow = grow || x > m[rr] + kGrow;  // (also from m = -inf)
            }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int rr = 0; rr < (SPLIT ? 1 : 2); ++rr) {
                    const float mn = fmaxf(m[rr], mx[rr]);
                    const float f = m[rr] == -INFINITY ? 0.0f : ex2(m[rr] - mn);
                    m[rr] = mn;
                    l[rr] *= f;
#pragma unroll
                    for (int k = 0; k < D / 8; ++k) {
                        o[k][2 * rr] *= f;
                        o[k][2 * rr + 1] *= f;
                        if (SPLIT) {
                            o[k][2] *= f;
                            o[k][3] *= f;
                        }
                    }
                }
            }
#pragma unroll
            for (int rr = 0; rr < (SPLIT ? 1 : 2); ++rr) {
                const float mu = m[rr] == -INFINITY ? 0.0f : m[rr];
                float p[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) p[e] = ex2(z[rr][e] - mu);
                l[rr] = fmaf((p[0] + p[1]) + (p[2] + p[3]), ivs, l[rr]);
                pf[rr] = pack_f16(p[0], p[1]);
                pf[2 + rr] = pack_f16(p[2], p[3]);
                if (SPLIT) {
                    pf[1] = pack_rest(p[0], p[1], pf[0]);
                    pf[3] = pack_rest(p[2], p[3], pf[2]);
                }
            }
            if (!(sc.vs > 0.0f)) pf[0] = pf[1] = pf[2] = pf[3] = 0u;  // V = 0 whatever its codes
            // codes of V past the sequence's end are whatever was there; in
            // int8 p = 0 removes them, in e4m3 they may be NaN
            const int past = FMT == LORA_KV_E4M3 ? key0 + 4 * tig + 4 - r.len : 0;
            const uint32_t keep = past <= 0 ? 0xFFFFFFFFu : past >= 4 ? 0u : 0xFFFFFFFFu >> (8 * past);
#pragma unroll
            for (int jj = 0; jj < D / 32; ++jj) {
                const uint4 w = *reinterpret_cast<const uint4 *>(vt + (g + 8 * jj) * 64 + tig * 16);
                const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t b0, b1;
                    codes_to_f16<FMT>(FMT == LORA_KV_E4M3 ? ws[k] & keep : ws[k], b0, b1);
                    mma_16816_f16(o[4 * jj + k], pf, b0, b1);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.empty[slot]);
        }
        i0 += count;

        // ---- merge the warps: row g's sums of dimensions 32 jj + 8 tig + 0..7
        if (merged) asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");  // the buffer has been read
        merged = true;
#pragma unroll
        for (int rr = 0; rr < (SPLIT ? 1 : 2); ++rr) {
            l[rr] += __shfl_xor_sync(0xffffffffu, l[rr], 1);
            l[rr] += __shfl_xor_sync(0xffffffffu, l[rr], 2);
            const int rt = g + 8 * rr;
            if (rt >= rows) continue;
            if (tig == 0) {
                sm.m[warp][rt] = m[rr];
                sm.l[warp][rt] = l[rr];
            }
#pragma unroll
            for (int jj = 0; jj < D / 32; ++jj)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float4 v;
                    const int c = 2 * rr + half;
                    v.x = o[4 * jj][c]; v.y = o[4 * jj + 1][c]; v.z = o[4 * jj + 2][c]; v.w = o[4 * jj + 3][c];
                    if (SPLIT) {
                        v.x = fmaf(o[4 * jj][2 + half], 1.0f / kLoScale, v.x);
                        v.y = fmaf(o[4 * jj + 1][2 + half], 1.0f / kLoScale, v.y);
                        v.z = fmaf(o[4 * jj + 2][2 + half], 1.0f / kLoScale, v.z);
                        v.w = fmaf(o[4 * jj + 3][2 + half], 1.0f / kLoScale, v.w);
                    }
                    *reinterpret_cast<float4 *>(&sm.o[warp][rt][32 * jj + 8 * tig + 4 * half]) = v;
                }
        }
        asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
        const bool whole = walk.from_start && walk.to_end;
        // an item that goes on in the next CTA is joined by the entry of the CTA it begins in
        float *part = partial_at(a, blockIdx.x, walk.from_start ? 1 : 0, kMmaRows, D);
        if (!whole && walk.from_start && threadIdx.x == 0) {
            const long long lastu = walk.item_end - 1;
            joins[blockIdx.x] = JoinEntry{walk.s, walk.head, walk.row_tile,
                                          static_cast<int32_t>(((lastu + 1) * ctas - 1) / total)};
        }
        constexpr int PER_ROW = kWarps * 32 / kMmaRows;  // 16 threads a row
        const int rt = threadIdx.x / PER_ROW, c0 = threadIdx.x % PER_ROW;
        if (rt < rows) {
            float M = -INFINITY, L = 0.0f, f[kWarps];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm.m[w][rt]);
            const float mu = M == -INFINITY ? 0.0f : M;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                f[w] = ex2(sm.m[w][rt] - mu);
                L = fmaf(sm.l[w][rt], f[w], L);
            }
            const float inv = 1.0f / L;
            const int32_t row = walk.row_tile * ROWS + rt;
            const int32_t qi = row / a.group, qh = walk.head * a.group + row % a.group;
            T *dst = static_cast<T *>(a.out.p) + static_cast<int64_t>(r.off + qi) * a.out.row + qh * a.out.head;
#pragma unroll
            for (int c = c0 * 4; c < D; c += PER_ROW * 4) {
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float4 x = *reinterpret_cast<const float4 *>(&sm.o[w][rt][c]);
                    v.x = fmaf(x.x, f[w], v.x);
                    v.y = fmaf(x.y, f[w], v.y);
                    v.z = fmaf(x.z, f[w], v.z);
                    v.w = fmaf(x.w, f[w], v.w);
                }
                if (whole) {
                    store4(dst + c, v, inv);
                } else {
                    *reinterpret_cast<float4 *>(part + rt * D + c) = v;
                }
            }
            if (c0 == 0) {
                if (!whole) {
                    part[kMmaRows * D + rt] = M;
                    part[kMmaRows * D + kMmaRows + rt] = L;
                } else if (a.lse) {
                    a.lse[static_cast<int64_t>(r.off + qi) * a.q_heads + qh] = (M + log2f(L)) * kLn2;
                }
            }
        }
    }
}

template <typename T, int D, int FMT>
cudaError_t decode_typed(const AttnView &v, cudaStream_t stream) {
    static uint64_t ctx[128] = {};
    constexpr int smem = static_cast<int>(sizeof(DecodeSmem<D>));
    static_assert(smem <= 227 * 1024, "the shared memory of one CTA");
    cudaError_t e = allow_smem(attn_decode_kernel<T, D, FMT>, smem, ctx);
    if (e != cudaSuccess) return e;
    const int grid = device_sm_count();
    attn_decode_kernel<T, D, FMT><<<grid, kThreads, smem, stream>>>(v);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = launch_join<T, D, tile_rows<T>()>(v, grid, kMmaRows, stream);
    count_launches(2);
    return e;
}

}  // namespace

size_t decode_workspace_bytes(int head_dim) {
    return split_workspace_bytes(device_sm_count(), kMmaRows, head_dim);
}

cudaError_t launch_attn_decode(const AttnView &v, lora_kv_format_t fmt, int head_dim, lora_dtype_t dtype,
                               cudaStream_t stream) {
    if (dtype == LORA_FP32) {
        if (head_dim == 64)
            return fmt == LORA_KV_INT8 ? decode_typed<float, 64, LORA_KV_INT8>(v, stream)
                                       : decode_typed<float, 64, LORA_KV_E4M3>(v, stream);
        return fmt == LORA_KV_INT8 ? decode_typed<float, 128, LORA_KV_INT8>(v, stream)
                                   : decode_typed<float, 128, LORA_KV_E4M3>(v, stream);
    }
    if (head_dim == 64)
        return fmt == LORA_KV_INT8 ? decode_typed<__nv_bfloat16, 64, LORA_KV_INT8>(v, stream)
                                   : decode_typed<__nv_bfloat16, 64, LORA_KV_E4M3>(v, stream);
    return fmt == LORA_KV_INT8 ? decode_typed<__nv_bfloat16, 128, LORA_KV_INT8>(v, stream)
                               : decode_typed<__nv_bfloat16, 128, LORA_KV_E4M3>(v, stream);
}

}  // namespace lora
