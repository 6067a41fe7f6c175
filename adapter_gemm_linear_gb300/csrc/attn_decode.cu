// Attention over the 8-bit paged cache (lora_kv_attention) for few queries a
// sequence: decode steps, checking of drafted tokens, and every fp32 call.
//
// With few query rows each key and value is used a handful of times, so the
// call is bound by reading the codes: 2 D bytes per token and key/value head.
// What the kernel does about it:
//  - Persistent CTAs.  The keys of all (sequence, key/value head, tile of query
//    rows) items, cut in chunks of 128 tokens, are dealt out in equal contiguous
//    ranges, so ragged lengths and few long sequences load every SM alike.  An
//    item that spans CTAs is joined by attn_join_kernel from fp32 partial
//    results (o, m, l), in a fixed order.  (Smaller pieces taken as a CTA gets
//    done, for the SMs that are slower: 326 us instead of 326 and 253 instead of
//    209 for the two large cases below, for the sake of more partial results.)
//  - A CTA's four or five consumer warps take the 16-token tiles in turn, each
//    with its own running softmax, and are merged in shared memory at an item's
//    end.  Every thread fetches the codes that it will use itself, tiles ahead,
//    by 16-byte asynchronous copies to shared memory: no barrier is between a
//    copy and its use.  (One warp
//    that fed all by bulk copies of 2 KiB was held at one copy per 85 ns and
//    SM: 3.6 TB/s with heads of 128, 1.9 with heads of 64.)  One more warp looks
//    up the tiles' pages and scales ahead of them.
//  - The codes become f16 in registers (exactly) and feed warp MMAs
//    (16 x 8 x 16, fp32 sums) with the few query rows as the narrow side:
//    S^T = K q^T with 16 tokens as M and eight rows as N, then o^T += V^T p^T
//    with 16 dimensions as M; p changes from S's layout to that of a B operand
//    by two 8 x 8 transpositions in the warp.  The tiles' layout in the cache is
//    the fragments' layout: a thread's 16 bytes of K are 16 dimensions of one
//    token (four k-steps, the order of the dimensions within a k-step being
//    free as long as q follows it); its 16 bytes of V are four dimensions x
//    the four tokens whose p it holds.  (With the rows as M, half of the MMAs
//    and exponentials of eight rows were for rows that are not there, and O
//    took twice the registers, for eight warps instead of 15: 517 us instead
//    of 388, then, for 256 sequences of 4096 tokens, 64 heads on 8.)
//  - q enters as f16 times a power of two per row (exact for bf16).  In fp32
//    calls q and p are each split in two f16 parts, hi + lo 2^-11, as two
//    column tiles of the MMA whose sums are added: 22 significant bits.
//  - The page's scale of V is folded into the exponent, relative to a reference
//    scale vr (attn_split.cuh): p' = 2^(s + log2 (vs / vr) - m), o sums p' codes,
//    l sums p' vr / vs.  p' <= 2^kGrow whatever the scales, so f16 holds it.  m
//    follows the maximum only when p' would pass that, so the sums are rarely
//    rescaled.
// Measured, with the join: 256 sequences of about 4096 tokens, 64 heads on 8 of
// 128, int8: 317 us, 5.8 TB/s (0.86 of a copy's rate; SMs that reach the memory
// less well end last).  4 sequences of 131072, e4m3: 184 us, 5.9 TB/s.  One of
// 2000, 32 heads on 8: 14.3 us (9.7 + 4.5; 10.5 in a graph), of which the reads that
// depend on one another (length, page, scale, codes) and two launches take most.
// 64 sequences of 4 new tokens in a window of 1024, heads of 64: 53 us, where the
// instructions of a tile (480 for 2 KB of codes, 43% of the issue slots) bound it,
// not the 61 MB.  16 rows a key head, 64 sequences of 4096 tokens, heads of 128: 133
// us in a graph (8 rows: 99, fp32 118; the codes take 79).  fp32 prompts take this
// kernel too, eight rows a pass over all keys: 512 tokens of 32 heads on 8, 81 us
// (bf16 30), on 4096 more 458 (55).
#include <cuda_runtime.h>
#include <math.h>

#include "attn_few.cuh"
#include "attn_internal.h"

namespace lora {

namespace {

using namespace sm100;

// Query rows of an item, with NT column tiles of eight; fp32 takes two for the parts of eight rows.
template <typename T, int NT>
__host__ __device__ constexpr int tile_rows() { return sizeof(T) == 4 ? 4 * NT : 8 * NT; }

// Several small CTAs per SM, so that while one merges its warps or begins an
// item the others' copies keep the memory busy; as many warps as the registers
// allow: three of four consumers at 128 a thread for one column tile of
// heads of 128 (and two tiles of heads of 64), two of five at 168 for two,
// four of four at 96 for one of heads of 64.
template <int D, int NT>
__host__ __device__ constexpr int consumers() { return D == 128 && NT == 2 ? 5 : 4; }
template <int D, int NT>
__host__ __device__ constexpr int ctas_per_sm() { return D == 128 ? (NT == 1 ? 3 : 2) : (NT == 1 ? 4 : 3); }

// What the looking-up warp says of a tile: where its codes are (in k_pages and
// in v_pages; < 0: not there, zeros), K's scale, V's relative to the reference vr
// (attn_split.cuh) in log2, and what takes it out again; of a V that is zero the least.
struct alignas(16) TileInfo {
    float ks, lv, ivs, vr;
    int64_t at;
    int64_t pad;
};
constexpr int64_t kNoTile = -1, kEndOfLine = -2;
constexpr int64_t kZeroV = 1;  // added to `at` (a multiple of 1024): V is zero whatever its codes

template <int D, int NT>
struct DecodeSmem {
    static constexpr int kWarps = consumers<D, NT>();
    static constexpr int kPieces = D / 32;           // 16-byte pieces a lane takes of a tile of K (and of V)
    static constexpr int kDepth = D == 128 ? 3 : NT == 1 ? 4 : 5;  // tiles a warp fetches ahead
    uint4 codes[kWarps][kDepth][2][kPieces][32];     // [.., K or V, piece, lane]
    float o[kWarps][8 * NT][D + 4];                  // merge: padded against bank conflicts
    float m[kWarps][8 * NT], l[kWarps][8 * NT];
    float vr[2];  // the reference scale of V of the item (by its parity)
    TileInfo info[kBatches][kBatch];
    uint64_t full[kBatches], empty[kBatches];
    long long warp_sum[kWarps + 1][2];
    long long base;  // first unit of the sequence the CTA begins in
    int32_t seq;
    int32_t dead;    // a wait ran out: nobody waits any more
};

// The query rows [row_tile * tile_rows, ...) of (sequence, key/value head): row r is query r / group of the
// sequence, query head head * group + r % group.
template <typename T, int D, int FMT, int NT>
__global__ void __launch_bounds__((consumers<D, NT>() + 1) * 32, ctas_per_sm<D, NT>()) attn_decode_kernel(const __grid_constant__ AttnView a) {
    extern __shared__ __align__(128) unsigned char raw[];
    DecodeSmem<D, NT> &sm = *reinterpret_cast<DecodeSmem<D, NT> *>(raw);
    using Smem = DecodeSmem<D, NT>;
    constexpr bool SPLIT = sizeof(T) == 4;  // fp32: operands in two f16 parts
    constexpr int ROWS = tile_rows<T, NT>();
    constexpr int kWarps = consumers<D, NT>(), kThreads = (kWarps + 1) * 32;
    constexpr int RT = SPLIT ? 1 : NT;  // column tiles of rows
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const KvView &b = a.kv;
    JoinEntry *joins = join_entries(a, gridDim.x, kSlotRows, D);

    // the joining kernel may come in as soon as there is room beside CTAs that
    // run or have none of the work; it waits for this one's end before it reads
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (threadIdx.x < kBatches) {
        mbar_init(&sm.full[threadIdx.x], a.test_wait_ns ? 2 : 1);
        mbar_init(&sm.empty[threadIdx.x], kWarps);
        fence_mbar_init();
    }
    if (threadIdx.x == 0) {
        sm.dead = 0;
        joins[blockIdx.x].last_cta = -1;
    }
    const Range range = plan_line<ROWS, kThreads, 0>(a, sm.warp_sum, &sm.seq, &sm.base);
    const long long total = range.total, ctas = range.ctas;
    Walk<ROWS> walk(a, range, sm.seq, sm.base);
    volatile int32_t *dead = &sm.dead;
    const uint64_t limit = a.test_wait_ns ? a.test_wait_ns : kWaitNs;

    auto wait = [&](uint64_t *bar, uint32_t parity, uint32_t site) {
        if (*dead || mbar_wait_bounded(bar, parity, limit)) return;
        record_error(b.status, kDevTimeout, site);
        *dead = 1;
    };

    if (warp == kWarps) {
        // ---- pages and scales of the CTA's tiles, 32 at a time, a lane each
        const int tile_shift = b.page_shift - 4;  // tiles of a page, as a shift
        int32_t next = 0, end = 0;  // the item's tiles that are not given out
        bool more = true;
        float vr = 1.0f, ref = 0.0f;  // of the item: the reference scale of V (v_reference) and its log2
        // (past the last tile the consumers still look for as many as they fetch ahead)
        for (int32_t n = 0, past = 0; past < kWarps * Smem::kDepth; ++n) {
            int32_t seq = -1, head = 0, t = 0;
            float own_vr = 1.0f, own_ref = 0.0f;
            for (int fill = 0; fill < kBatch;) {
                if (next == end) {
                    more = more && walk.next();
                    if (!more) {
                        past += kBatch - fill;
                        break;
                    }
                    next = walk.tile0;
                    end = walk.tile1;
                    // (the reads are hidden but for the first item's)
                    vr = v_reference(b, walk.s, walk.head, next, end);
                    ref = log2f(fabsf(vr));
                }
                const int take = min(kBatch - fill, end - next);
                if (lane >= fill && lane < fill + take) {
                    seq = walk.s;
                    head = walk.head;
                    t = next + lane - fill;
                    own_vr = vr;
                    own_ref = ref;
                }
                fill += take;
                next += take;
            }
            TileInfo x = {0.0f, -kSpread, kSpreadFactor, own_vr, kEndOfLine, 0};
            if (seq >= 0) {
                const int32_t page = read_page(b, seq, t >> tile_shift);
                x.at = kNoTile;
                if (page >= 0) {
                    x.at = tile_offset<D>(b, page, head, t & ((1 << tile_shift) - 1));
                    const int64_t sc = static_cast<int64_t>(page) * b.heads + head;
                    x.ks = __ldg(b.k_scales + sc);
                    const float vs = __ldg(b.v_scales + sc), lv = log2f(vs) - own_ref;
                    if (!(vs > 0.0f)) x.at += kZeroV;
                    else if (lv >= -kSpread) {
                        x.lv = lv;
                        x.ivs = fabsf(own_vr) / vs;
                    }
                }
            }
            __syncwarp();
            wait(&sm.empty[n % kBatches], ((n / kBatches) & 1u) ^ 1u, 40);
            // (what the consumers may still read is left alone; they see `dead` when they look for more)
            if (__any_sync(0xffffffffu, *dead)) break;
            sm.info[n % kBatches][lane] = x;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.full[n % kBatches]);
        }
        return;
    }

    // ---- consumers
    const int g = lane >> 2, tig = lane & 3;
    // S^T: rows g and g + 8 are tokens 4 (g / 2) + g % 2 and that + 2, so that
    // after the transposition a thread holds p of tokens 4 tig .. 4 tig + 3
    const int tok = 4 * (g >> 1) + (g & 1);
    auto fetch_k = [&](int64_t at, uint32_t slot) {
        const uint8_t *src = b.k_pages + (max(at, int64_t{0}) & ~kZeroV) + tok * 64 + tig * 16;
#pragma unroll
        for (int i = 0; i < Smem::kPieces; ++i)  // [64 dimensions][token or that + 2]
            if (at != kEndOfLine) copy16(&sm.codes[warp][slot][0][i][lane], src + (i >> 1) * (kKvTile * 64) + (i & 1) * 128, at >= 0);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto fetch_v = [&](int64_t at, uint32_t slot) {
        const uint8_t *src = b.v_pages + (max(at, int64_t{0}) & ~kZeroV) + g * 64 + tig * 16;
#pragma unroll
        for (int i = 0; i < Smem::kPieces; ++i)
            if (at != kEndOfLine) copy16(&sm.codes[warp][slot][1][i][lane], src + i * 512, at >= 0 && !(at & kZeroV));
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // where tile i of the CTA's line is; waits for its batch if it is the warp's first of it
    auto look = [&](uint32_t i) {
        const uint32_t n = i / kBatch;
        if (i % kBatch < kWarps) wait(&sm.full[n % kBatches], (n / kBatches) & 1u, 41);
        return *dead ? kEndOfLine : sm.info[n % kBatches][i % kBatch].at;
    };
    auto landed = [] { asm volatile("cp.async.wait_group %0;" ::"n"(2 * Smem::kDepth - 1) : "memory"); };
    for (uint32_t d = 0; d < Smem::kDepth; ++d) {
        const int64_t at = look(warp + d * kWarps);
        fetch_k(at, d);
        fetch_v(at, d);
    }
    uint32_t taken = 0;  // tiles the warp has used
    uint32_t i0 = 0;
    bool merged = false;  // whether the merge buffer may still be read by others
    uint32_t n_item = 0;
    while (walk.next()) {
        const SeqRows &r = walk.work.r;
        const int32_t rows = min(ROWS, r.n * a.group - walk.row_tile * ROWS);
        // q as B fragments: column g of tile u is row 8 u + g, dimensions 64 h +
        // 16 tig + 4 j + 0..3 in k-step (h, j)
        uint32_t qf[NT][D / 16][2];
        // of the rows 8 u + 2 tig + i that the thread's scores belong to: the
        // score scale in log2 units and the keys seen
        float cr[RT][2];
        int32_t kmin[RT][2], kmax[RT][2];
#pragma unroll
        for (int u = 0; u < RT; ++u) {
            const int32_t row = walk.row_tile * ROWS + min(8 * u + g, rows - 1);  // rows past the last repeat it
            const int32_t qi = row / a.group, qh = walk.head * a.group + row % a.group;
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
            const float up = a.scale * kLog2e * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
            const int32_t pos = r.len - r.n + qi;
            const int32_t hi = a.causal ? pos + 1 : r.len, lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {  // from the lanes of row 8 u + 2 tig + i
                cr[u][i] = __shfl_sync(0xffffffffu, up, 8 * tig + 4 * i);
                kmax[u][i] = __shfl_sync(0xffffffffu, hi, 8 * tig + 4 * i);
                kmin[u][i] = __shfl_sync(0xffffffffu, lo, 8 * tig + 4 * i);
            }
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const float *v = x + 4 * k;
                qf[u][k][0] = pack_f16(v[0] * down, v[1] * down);
                qf[u][k][1] = pack_f16(v[2] * down, v[3] * down);
                if (SPLIT) {
                    qf[NT - 1][k][0] = pack_rest(v[0] * down, v[1] * down, qf[0][k][0]);
                    qf[NT - 1][k][1] = pack_rest(v[2] * down, v[3] * down, qf[0][k][1]);
                }
            }
        }
        // keys that every row of the item sees: tiles within need no mask
        const int32_t pos0 = r.len - r.n + walk.row_tile * ROWS / a.group;
        const int32_t pos1 = r.len - r.n + (walk.row_tile * ROWS + rows - 1) / a.group;
        const int32_t all_hi = a.causal ? pos0 + 1 : r.len;
        const int32_t all_lo = a.window > 0 ? max(0, pos1 - a.window + 1) : 0;

        float o[NT][D / 16][4];  // o^T: rows d = 4 (g + 8 (k / 2)) + 2 (k % 2) and d + 1, columns 2 tig and the next
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int k = 0; k < D / 16; ++k) o[u][k][0] = o[u][k][1] = o[u][k][2] = o[u][k][3] = 0.0f;
        float m[RT][2], l[RT][2];
#pragma unroll
        for (int u = 0; u < RT; ++u)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[u][i] = -INFINITY;
                l[u][i] = 0.0f;
            }

        const int32_t count = walk.tile1 - walk.tile0;
        // this warp's tiles: those whose running number is the warp's modulo kWarps
        const int32_t j0 = (warp - static_cast<int32_t>(i0 % kWarps) + kWarps) % kWarps;
        if (j0 == 0 && lane == 0) sm.vr[n_item & 1] = sm.info[i0 / kBatch % kBatches][i0 % kBatch].vr;
        for (int32_t j = j0; j < count; j += kWarps) {
            const uint32_t i = i0 + j, slot = taken++ % Smem::kDepth;
            const int32_t key0 = (walk.tile0 + j) * kKvTile;
            const TileInfo &info = sm.info[i / kBatch % kBatches][i % kBatch];
            const float ks = info.ks, lv = info.lv, ivs = info.ivs;
            const int64_t ahead = look(i + Smem::kDepth * kWarps);
            float s[NT][4];
#pragma unroll
            for (int u = 0; u < NT; ++u) s[u][0] = s[u][1] = s[u][2] = s[u][3] = 0.0f;
            landed();
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
                const uint4 wa = sm.codes[warp][slot][0][2 * h][lane], wb = sm.codes[warp][slot][0][2 * h + 1][lane];
                const uint32_t was[4] = {wa.x, wa.y, wa.z, wa.w}, wbs[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t f[4];
                    codes_to_f16<FMT>(was[k], f[0], f[2]);
                    codes_to_f16<FMT>(wbs[k], f[1], f[3]);
#pragma unroll
                    for (int u = 0; u < NT; ++u) mma_16816_f16(s[u], f, qf[u][4 * h + k][0], qf[u][4 * h + k][1]);
                }
            }
            fetch_k(ahead, slot);
            // scores in log2 units, with V's scale
            float z[RT][4];  // [2 * token half + row]
#pragma unroll
            for (int u = 0; u < RT; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float sum = SPLIT ? fmaf(s[NT - 1][e], 1.0f / kLoScale, s[0][e]) : s[u][e];
                    z[u][e] = fmaf(sum, ks * cr[u][e & 1], lv);
                }
            const bool edge = key0 < all_lo || key0 + kKvTile > all_hi;  // some row does not see some key
            if (edge) {
#pragma unroll
                for (int u = 0; u < RT; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int32_t key = key0 + tok + (e & 2);
                        if (key < kmin[u][e & 1] || key >= kmax[u][e & 1]) z[u][e] = -INFINITY;
                    }
            }
            bool grow = false;
            float mx[RT][2];
#pragma unroll
            for (int u = 0; u < RT; ++u)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float x = fmaxf(z[u][i], z[u][i + 2]);
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                    mx[u][i] = x;
                    grow = grow || x > m[u][i] + kGrow;  // (also from m = -inf)
                }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int u = 0; u < RT; ++u)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float mn = fmaxf(m[u][i], mx[u][i] - kStartDecode);
                        const float f = m[u][i] == -INFINITY ? 0.0f : ex2(m[u][i] - mn);
                        m[u][i] = mn;
                        l[u][i] *= f;
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            o[u][k][i] *= f;
                            o[u][k][i + 2] *= f;
                            if (SPLIT) {
                                o[NT - 1][k][i] *= f;
                                o[NT - 1][k][i + 2] *= f;
                            }
                        }
                    }
            }
            uint32_t pf[NT][2];  // p^T as B fragments
#pragma unroll
            for (int u = 0; u < RT; ++u) {
                const float m0 = m[u][0] == -INFINITY ? 0.0f : m[u][0], m1 = m[u][1] == -INFINITY ? 0.0f : m[u][1];
                const float p[4] = {ex2(z[u][0] - m0), ex2(z[u][1] - m1), ex2(z[u][2] - m0), ex2(z[u][3] - m1)};
                l[u][0] = fmaf(p[0] + p[2], ivs, l[u][0]);
                l[u][1] = fmaf(p[1] + p[3], ivs, l[u][1]);
                const uint32_t h0 = pack_f16(p[0], p[1]), h1 = pack_f16(p[2], p[3]);
                pf[u][0] = transpose_8x8(h0);
                pf[u][1] = transpose_8x8(h1);
                if (SPLIT) {
                    pf[NT - 1][0] = transpose_8x8(pack_rest(p[0], p[1], h0));
                    pf[NT - 1][1] = transpose_8x8(pack_rest(p[2], p[3], h1));
                }
            }
            // codes of V past the sequence's end are whatever was there; in
            // int8 p = 0 removes them, in e4m3 they may be NaN
            const int past = FMT == LORA_KV_E4M3 ? key0 + 4 * tig + 4 - r.len : 0;
            const uint32_t keep = past <= 0 ? 0xFFFFFFFFu : past >= 4 ? 0u : 0xFFFFFFFFu >> (8 * past);
            landed();
            if (FMT == LORA_KV_E4M3 && edge) {
                // p = 0 does not keep a NaN of V from a row that does not see its
                // token: such codes become 0, and the rows that do see them get
                // the NaN from here
                uint32_t some = 0;
#pragma unroll
                for (int jj = 0; jj < D / 32; ++jj) {
                    const uint4 w = sm.codes[warp][slot][1][jj][lane];
                    some |= e4m3_nan(w.x & keep) | e4m3_nan(w.y & keep) | e4m3_nan(w.z & keep) | e4m3_nan(w.w & keep);
                }
                if (__builtin_expect(__any_sync(0xffffffffu, some != 0), 0)) {
                    uint32_t seen[RT][2];  // the tile's tokens that the row sees, a bit each
#pragma unroll
                    for (int u = 0; u < RT; ++u)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int from = min(max(kmin[u][i] - key0, 0), 16), to = min(max(kmax[u][i] - key0, 0), 16);
                            seen[u][i] = ((1u << to) - 1u) & ~((1u << from) - 1u);
                        }
#pragma unroll
                    for (int jj = 0; jj < D / 32; ++jj) {
                        const uint4 w = sm.codes[warp][slot][1][jj][lane];
                        uint32_t ws[4] = {w.x & keep, w.y & keep, w.z & keep, w.w & keep};
#pragma unroll
                        for (int q = 0; q < 4; ++q) {  // dimension q of the piece's four
                            const uint32_t nan = e4m3_nan(ws[q]);
                            uint32_t tokens = ((nan >> 7 & 1u) | (nan >> 14 & 2u) | (nan >> 21 & 4u) | (nan >> 28 & 8u)) << (4 * tig);
                            tokens |= __shfl_xor_sync(0xffffffffu, tokens, 1);
                            tokens |= __shfl_xor_sync(0xffffffffu, tokens, 2);
#pragma unroll
                            for (int u = 0; u < RT; ++u)
#pragma unroll
                                for (int i = 0; i < 2; ++i)
                                    if (tokens & seen[u][i]) o[u][2 * jj + (q >> 1)][i + 2 * (q & 1)] = __int_as_float(0x7FFFFFFF);
                            ws[q] = e4m3_without(ws[q], nan);
                        }
                        sm.codes[warp][slot][1][jj][lane] = make_uint4(ws[0], ws[1], ws[2], ws[3]);
                    }
                }
            }
#pragma unroll
            for (int jj = 0; jj < D / 32; ++jj) {
                const uint4 w = sm.codes[warp][slot][1][jj][lane];
                const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint32_t f[4];
                    codes_to_f16<FMT>(FMT == LORA_KV_E4M3 ? ws[2 * k] & keep : ws[2 * k], f[0], f[2]);
                    codes_to_f16<FMT>(FMT == LORA_KV_E4M3 ? ws[2 * k + 1] & keep : ws[2 * k + 1], f[1], f[3]);
#pragma unroll
                    for (int u = 0; u < NT; ++u) mma_16816_f16(o[u][2 * jj + k], f, pf[u][0], pf[u][1]);
                }
            }
            fetch_v(ahead, slot);
            // the warp's last tile of a batch
            if (i % kBatch >= kBatch - kWarps) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.empty[i / kBatch % kBatches]);
            }
        }
        i0 += count;

        // ---- merge the warps
        if (merged) asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");  // the buffer has been read
        merged = true;
#pragma unroll
        for (int u = 0; u < RT; ++u)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float sum = l[u][i];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                const int rt = 8 * u + 2 * tig + i;
                if (rt >= rows) continue;
                if (g == 0) {
                    sm.m[warp][rt] = m[u][i];
                    sm.l[warp][rt] = sum;
                }
#pragma unroll
                for (int jj = 0; jj < D / 32; ++jj) {
                    float4 v = make_float4(o[u][2 * jj][i], o[u][2 * jj][i + 2], o[u][2 * jj + 1][i], o[u][2 * jj + 1][i + 2]);
                    if (SPLIT) {
                        v.x = fmaf(o[NT - 1][2 * jj][i], 1.0f / kLoScale, v.x);
                        v.y = fmaf(o[NT - 1][2 * jj][i + 2], 1.0f / kLoScale, v.y);
                        v.z = fmaf(o[NT - 1][2 * jj + 1][i], 1.0f / kLoScale, v.z);
                        v.w = fmaf(o[NT - 1][2 * jj + 1][i + 2], 1.0f / kLoScale, v.w);
                    }
                    *reinterpret_cast<float4 *>(&sm.o[warp][rt][32 * jj + 4 * g]) = v;
                }
            }
        asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
        const bool whole = walk.from_start && walk.to_end;
        // an item that goes on in the next CTA is joined by the entry of the CTA it begins in
        float *part = partial_at(a, blockIdx.x, walk.from_start ? 1 : 0, kSlotRows, D);
        if (!whole && walk.from_start && threadIdx.x == 0) {
            const long long lastu = walk.item_end - 1;
            joins[blockIdx.x] = JoinEntry{static_cast<int32_t>(((lastu + 1) * ctas - 1) / total), walk.head, r.off,
                                          walk.row_tile * ROWS, rows, {}};
        }
        constexpr int PER_ROW = kWarps * 32 / ROWS;  // threads a row
        const int rt = threadIdx.x / PER_ROW, c0 = threadIdx.x % PER_ROW;
        const float scale = sm.vr[n_item & 1];
        if (__builtin_expect(scale < 0.0f, 0)) {
            for (int r0 = warp; r0 < rows; r0 += kWarps)
                plain_row<T, D, FMT>(a, walk.s, walk.head, r.off, r.n, r.len, walk.row_tile * ROWS + r0, walk.tile0 * kKvTile,
                                     min(walk.tile1 * kKvTile, r.len), whole ? nullptr : part + r0 * D, part + kSlotRows * D + r0);
        } else if (rt < rows) {
            float M = -INFINITY, L = 0.0f, f[kWarps];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm.m[w][rt]);
            const float mu = M == -INFINITY ? 0.0f : M;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                f[w] = ex2(sm.m[w][rt] - mu);
                L = fmaf(sm.l[w][rt], f[w], L);
            }
            // (a part of an item may have no key that the row sees: nothing, not 0 / 0)
            const float inv = whole || !(L == 0.0f) ? 1.0f / L : 0.0f;
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
                v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);  // (inv * scale may leave fp32's range)
                if (whole) {
                    store4(dst + c, v, scale);
                } else {
                    store4(part + rt * D + c, v, scale);
                }
            }
            if (c0 == 0) {
                const float lse = M + log2f(L);
                if (!whole) {
                    part[kSlotRows * D + rt] = lse;
                } else if (a.lse) {
                    a.lse[static_cast<int64_t>(r.off + qi) * a.q_heads + qh] = lse * kLn2;
                }
            }
        }
        ++n_item;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <typename T, int D, int FMT, int NT>
cudaError_t decode_tiles(const AttnView &v, cudaStream_t stream) {
    static uint64_t ctx[128] = {};
    constexpr int smem = static_cast<int>(sizeof(DecodeSmem<D, NT>));
    static_assert((smem + 1024) * ctas_per_sm<D, NT>() <= 228 * 1024, "the shared memory of an SM");
    cudaError_t e = allow_smem(attn_decode_kernel<T, D, FMT, NT>, smem, ctx);
    if (e != cudaSuccess) return e;
    const int grid = device_sm_count() * ctas_per_sm<D, NT>();
    attn_decode_kernel<T, D, FMT, NT><<<grid, (consumers<D, NT>() + 1) * 32, smem, stream>>>(v);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = launch_join<T, D, tile_rows<T, NT>(), 4>(v, grid, kSlotRows, stream);
    count_launches(2);
    return e;
}

template <typename T, int D, int FMT>
cudaError_t decode_typed(const AttnView &v, cudaStream_t stream) {
    if constexpr (sizeof(T) == 4) return decode_tiles<T, D, FMT, 2>(v, stream);
    // one column tile of eight rows where that is all that any sequence has
    else if (static_cast<int64_t>(v.max_queries) * v.group <= 8) return decode_tiles<T, D, FMT, 1>(v, stream);
    else return decode_tiles<T, D, FMT, 2>(v, stream);
}

}  // namespace

size_t decode_workspace_bytes(int head_dim) {
    constexpr int kMostCtas = 4;  // per SM
    return split_workspace_bytes(device_sm_count() * kMostCtas, kSlotRows, head_dim);
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
