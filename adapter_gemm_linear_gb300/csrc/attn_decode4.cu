// Attention over the 4-bit paged cache (LORA_KV_UINT4) for few queries a sequence,
// and for every fp32 call.  The line of work, the persistent CTAs, the warps' ring of
// asynchronous copies and the join are those of attn_decode.cu; what is different:
//
//  - With s and m a token's scale and least value in 64 dimensions, c its codes,
//        q.k = sum over blocks of  s (q.c) + m sum(q),
//        o   = sum_j (p_j s_j) c_j + sum_j p_j m_j,
//    so the matrix instructions take codes, and scales and least values enter in
//    fp32.  A word of codes becomes four operand registers by four ANDs and a
//    shift (attn_uint4.cuh): f16 subnormals, whose 2^-24 and 2^-20 come out of the
//    score's factor, of q (second pairs of a word by 1/16) and of the results.  In fp32
//    calls they are f16 values of code - 8 instead (one instruction more a pair): the
//    matrix instructions' sums cut off what is below their last bit, which adds up
//    where all codes are positive and most of the sum goes out again with the least
//    values (5e-5 of the result, with code - 8 3e-7).
//  - p' = p s enters as f16 times a factor fr of the row, a power of two that is
//    lowered (with the row's sums) when a p' would leave f16's range, and first set
//    so that the row's largest p' is in [2^8, 2^9); p itself is relative to a maximum
//    that is raised when a score passes it by kSlack, and fr is raised with it, so
//    that the largest p' there is stays above 2^8 (or fr is 2^60).  Both are looked
//    at lane by lane; only a raise takes shuffles.
//  - A warp takes two tiles a step, whose fixed instructions (waits, looks, the checks)
//    are shared by 32 tokens.
// As it is laid out it is bound by the warps' instructions (issue slots 56% used with three warps a
// quarter of the SM, of which each instruction waits for some before it; the ALU busy for 52%), then by
// memory, half a byte a value and 1/16 of scales.  64 query heads on 8 of 128, in a graph: one
// token of each of 256 sequences of some 4096, 1.04 GB, 199 us (5.2 TB/s; its floor is 154); of
// 64 sequences of 4097 68.7 us, with 128 query heads 109, in fp32 113.  One token of one sequence of
// 2000: 10.0.  4 queries of 64 sequences, 32 heads of 64 on 8, in a window of 1024: 30.3.
// In fp32 128 queries of 32 heads of 128 on 1024 + 128 keys 46.4, 512 on their own 97: the cache is read
// once for every eight rows.
#include <cuda_runtime.h>
#include <math.h>

#include "attn_few.cuh"
#include "attn_internal.h"
#include "attn_uint4.cuh"
#include "f32x2.cuh"

namespace lora {

namespace {

using namespace sm100;

template <typename T, int NT>
__host__ __device__ constexpr int tile_rows() { return sizeof(T) == 4 ? 4 * NT : 8 * NT; }

// Registers are given out by a quarter of the SM, so what counts is the warps of a quarter: two of
// 255 registers, three of 168 or four of 128.  Two column tiles of rows with heads of 128 need the
// 255 (16 query rows a key head, 64 sequences of 4097, 8 key heads, when this was chosen: 122 us, with
// three warps a quarter and their spills 229, with one tile a step 135; now 109); else four are better, in
// three CTAs (256 sequences then 206 us, in four of four warps 214, in two of eight 235, now 199; heads
// of 64 then 51 us, in four CTAs of five warps 56, now 46).
template <int D, int NT>
__host__ __device__ constexpr int consumers() { return D == 128 && NT == 2 ? 7 : 4; }
template <int D, int NT>
__host__ __device__ constexpr int ctas_per_sm() { return D == 128 && NT == 2 ? 1 : 3; }

constexpr int32_t kNoTile = -1, kEndOfLine = -2;  // zeros; nothing any more (a tile has 512 bytes and more: 31 bits number 1 TB)
constexpr int kLooks = 2;                         // batches looked up ahead
constexpr int kItemRing = 64;

// What the CTA has of an item.
struct Item4 {
    int32_t off, n, len;  // the sequence's queries and length; n = 0: no more items
    int32_t head, row_tile, tile0, tile1;
    int32_t last_cta;  // that it goes on to, kWhole, or kNotFirst: it began in another CTA
};
static_assert(sizeof(Item4) == 32, "two 16-byte pieces");
constexpr int32_t kWhole = -1, kNotFirst = -2;
// What beginning and ending an item costs, in units of 128 keys.  Without it CTAs that
// get many short items take twice as long as the others (4 queries of 64 sequences, heads of 64, in a
// window of 1024: 46 us).  When it was chosen one token of 256 sequences of some 4096 took 197, 199 and 201 us with 2, 3
// and 4, of some 500 46, 48 and 50; 4 queries of 256 sequences of some 700, heads of 64, 58.8, 57.0 and
// 59.5, in that window 29.1, 28.5 and 27.8.
template <int D, int NT>
__host__ __device__ constexpr int item_units() { return D == 128 && NT == 1 ? 2 : 3; }
constexpr float kSlack = 8.0f;                    // log2 by which a score may pass the row's maximum so far
constexpr int kTopExponent = 8;                   // a row's largest p' begins in [2^8, 2^9)
constexpr float kMostFactor = 1.152921504606847e18f;  // 2^60: fr of rows without a scale so far

template <int D, int NT>
struct Decode4Smem {
    static constexpr int kWarps = consumers<D, NT>();
    static constexpr int H = D / kBlockDims;
    static constexpr int TS = 2;                                    // tiles of a step
    static constexpr int kDepth = 2;                                // steps a warp fetches ahead (of 3: 72 us instead of 71, 48.4 instead of 47)
    static constexpr int kMeta = TS * 2 * H * 4;                    // 16-byte pieces of a step's scales
    uint4 codes[kWarps][kDepth][2][TS * H][32];                     // [.., K or V, (tile, block), lane]
    uint4 meta[kWarps][kDepth][kMeta];                              // [.., (tile, K or V, block, four tokens)]
    float o[kWarps][8 * NT][D + 4];                                 // merge: padded against bank conflicts
    float m[kWarps][8 * NT], l[kWarps][8 * NT];
    int2 info[kLooks][kBatch / 2];                                  // of a step: tile_index, kNoTile or kEndOfLine
    alignas(16) Item4 items[kItemRing];
    uint64_t full[kLooks], empty[kLooks], merge_full, merge_empty;
    // A batch's items are written when every warp has looked at its last step of the batch kLooks before, and
    // so has used the step kDepth of its own before that: what it may still read are the item of that
    // step and later ones, each of at least one step.
    static_assert(1 + kLooks * (kBatch / TS) + (kDepth + 1) * kWarps <= kItemRing, "items that are still read");
    long long warp_sum[kWarps + 1][2];
    long long base;  // first unit of the sequence the CTA begins in
    int32_t seq;
    int32_t dead;    // a wait ran out: nobody waits any more
};

// The query rows [row_tile * tile_rows, ...) of (sequence, key/value head): row r is query r / group of the
// sequence, query head head * group + r % group.
template <typename T, int D, int NT>
__global__ void __launch_bounds__((consumers<D, NT>() + 1) * 32, ctas_per_sm<D, NT>()) attn_decode4_kernel(const __grid_constant__ AttnView a) {
    extern __shared__ __align__(128) unsigned char raw[];
    using Smem = Decode4Smem<D, NT>;
    Smem &sm = *reinterpret_cast<Smem *>(raw);
    constexpr bool SPLIT = sizeof(T) == 4;  // fp32: operands in two f16 parts
    constexpr int ROWS = tile_rows<T, NT>();
    constexpr int kWarps = Smem::kWarps, kThreads = (kWarps + 1) * 32;
    constexpr int RT = SPLIT ? 1 : NT;  // column tiles of rows
    constexpr int H = Smem::H, TS = Smem::TS, kDepth = Smem::kDepth;
    constexpr int kSteps = kBatch / TS;  // of a batch of looked-up tiles
    // what the products with codes are units of: first and second pairs of a word
    constexpr float kUnit0 = SPLIT ? 1.0f : 1.0f / kCode0, kUnit1 = SPLIT ? 1.0f : 1.0f / kCode1;
    auto pairs = [](uint32_t w, uint32_t (&f)[4]) {
        if constexpr (SPLIT) nibbles_less<8>(w, f);
        else nibble_pairs(w, f);
    };
    // a token's scale and least value (for code 8 in fp32 calls)
    auto scale_of = [](uint32_t meta) {
        float2 x = f16_pair(meta);
        if constexpr (SPLIT) x.y = fmaf(8.0f, x.x, x.y);
        return x;
    };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const KvView &b = a.kv;
    // the joining kernel may come in as soon as there is room beside CTAs that
    // run or have none of the work; it waits for this one's end before it reads
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (threadIdx.x < kLooks) {
        mbar_init(&sm.full[threadIdx.x], a.test_wait_ns ? 2 : 1);
        mbar_init(&sm.empty[threadIdx.x], kWarps);
        fence_mbar_init();
    }
    if (threadIdx.x == 0) {
        mbar_init(&sm.merge_full, kWarps);
        mbar_init(&sm.merge_empty, kWarps);
        fence_mbar_init();
        sm.dead = 0;
        join_entries(a, gridDim.x, kSlotRows, D)[blockIdx.x].last_cta = -1;
    }
    const Range range = plan_line<ROWS, kThreads, item_units<D, NT>()>(a, sm.warp_sum, &sm.seq, &sm.base);
    volatile int32_t *dead = &sm.dead;
    const uint64_t limit = a.test_wait_ns ? a.test_wait_ns : kWaitNs;

    auto wait = [&](uint64_t *bar, uint32_t parity, uint32_t site) {
        if (*dead) return false;
        if (mbar_wait_bounded(bar, parity, limit)) return true;
        record_error(b.status, kDevTimeout, site);
        *dead = 1;
        return false;
    };

    if (warp == kWarps) {
        // ---- the CTA's items, and places of their tiles, 32 at a time, a lane each; an item's are rounded up to
        // whole steps.  (The consumers' own walks took registers that they had to spill, and 5% of their time.)
        Walk<ROWS> walk(a, range, sm.seq, sm.base);
        uint32_t item = 0;
        const int tile_shift = b.page_shift - 4;  // tiles of a page, as a shift
        int32_t next = 0, end = 0, last = 0;      // the item's tiles that are not given out: up to `last`, rounded up `end`
        bool more = true;
        // (past the last tile the consumers still look for as many as they fetch ahead)
        for (int32_t n = 0, past = 0; past < kWarps * kDepth * TS; ++n) {
            wait(&sm.empty[n % kLooks], ((n / kLooks) & 1u) ^ 1u, 45);
            // (what the consumers may still read is left alone; they see `dead` when they look for more)
            if (__any_sync(0xffffffffu, *dead)) break;
            int32_t seq = -1, head = 0, t = 0;
            for (int fill = 0; fill < kBatch;) {
                if (next == end) {
                    if (more) {
                        more = walk.next();
                        const long long last_cta = more ? (walk.item_end * range.ctas - 1) / range.total : 0;
                        if (lane == 0)
                            sm.items[item % kItemRing] =
                                !more ? Item4{}
                                      : Item4{walk.work.r.off, walk.work.r.n, walk.work.r.len, walk.head, walk.row_tile, walk.tile0, walk.tile1,
                                              !walk.from_start ? kNotFirst : walk.to_end ? kWhole : static_cast<int32_t>(last_cta)};
                        ++item;
                    }
                    if (!more) {
                        past += kBatch - fill;
                        break;
                    }
                    next = walk.tile0;
                    last = walk.tile1;
                    end = next + (last - next + TS - 1) / TS * TS;
                }
                const int take = min(kBatch - fill, end - next);
                if (lane >= fill && lane < fill + take) {
                    t = next + lane - fill;
                    seq = t < last ? walk.s : -2;
                    head = walk.head;
                }
                fill += take;
                next += take;
            }
            int32_t at = seq == -1 ? kEndOfLine : kNoTile;
            if (seq >= 0) {
                const int32_t page = read_page(b, seq, t >> tile_shift);
                if (page >= 0) at = static_cast<int32_t>(tile_index(b, page, head, t & ((1 << tile_shift) - 1)));
            }
            reinterpret_cast<int32_t *>(sm.info[n % kLooks])[lane] = at;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.full[n % kLooks]);
        }
        return;
    }

    // ---- consumers
    const int g = lane >> 2, tig = lane & 3;
    const int tok = k_token(g);  // S^T: rows g and g + 8 are tokens tok and tok + 2 of a tile
    auto fetch = [&](const int32_t (&at)[TS], uint32_t slot) {
#pragma unroll
        for (int j = 0; j < TS; ++j) {
            if (at[j] == kEndOfLine) continue;
            const int64_t byte = static_cast<int64_t>(max(at[j], 0)) * (H * kBlockBytes) + lane * 16;
#pragma unroll
            for (int h = 0; h < H; ++h) copy16(&sm.codes[warp][slot][0][j * H + h][lane], b.k_pages + byte + h * kBlockBytes, at[j] >= 0);
#pragma unroll
            for (int h = 0; h < H; ++h) copy16(&sm.codes[warp][slot][1][j * H + h][lane], b.v_pages + byte + h * kBlockBytes, at[j] >= 0);
        }
        if (lane < Smem::kMeta) {
            const int32_t tile = lane >= 8 * H ? at[1] : at[0];
            const float *from = lane / (4 * H) % 2 ? b.v_scales : b.k_scales;
            if (tile != kEndOfLine)
                copy16(&sm.meta[warp][slot][lane], from + (static_cast<int64_t>(max(tile, 0)) * (H * kKvTile) + lane % (4 * H) * 4), tile >= 0);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // where the tiles of the line's step i are; waits for their batch if it is the warp's
    // first of it, and gives the batch back after the last
    bool gone = false;
    auto look = [&](uint32_t i, int32_t (&at)[TS]) {
        const uint32_t n = i / kSteps, k = i % kSteps;
        if (k < kWarps && !wait(&sm.full[n % kLooks], (n / kLooks) & 1u, 46)) gone = true;
        const int2 x = sm.info[n % kLooks][k];
        at[0] = gone ? kEndOfLine : x.x;
        at[1] = gone ? kEndOfLine : x.y;
        if (k >= kSteps - kWarps) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.empty[n % kLooks]);
        }
    };
    auto landed = [] { asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory"); };
    for (uint32_t d = 0; d < kDepth; ++d) {
        int32_t at[TS];
        look(warp + d * kWarps, at);
        fetch(at, d);
    }
    uint32_t taken = 0;  // steps the warp has used
    uint32_t i0 = 0;     // steps of the items before
    // (the warp has looked at its next step, so the item's entry, which came with its first step's batch, is there)
    auto item = [&](uint32_t n) {
        const int4 *const entry = reinterpret_cast<const int4 *>(&sm.items[n % kItemRing]);
        const int4 e0 = entry[0], e1 = entry[1];
        return Item4{e0.x, e0.y, e0.z, e0.w, e1.x, e1.y, e1.z, e1.w};
    };
    // What the warps have written of item n joined, each thread some of a row's dimensions.
    auto finish = [&](uint32_t n) {
        wait(&sm.merge_full, n & 1u, 48);
        const Item4 it = item(n);
        const int32_t off = it.off, head = it.head, row0 = it.row_tile * ROWS, last_cta = it.last_cta;
        const int32_t rows = min(ROWS, it.n * a.group - row0);
        const bool whole = last_cta == kWhole;
        // an item that goes on in the next CTA is joined by the entry of the CTA it begins in
        float *part = partial_at(a, blockIdx.x, last_cta >= 0 ? 1 : 0, kSlotRows, D);
        if (last_cta >= 0 && threadIdx.x == 0)
            join_entries(a, gridDim.x, kSlotRows, D)[blockIdx.x] = JoinEntry{last_cta, head, off, row0, rows, {}};
        constexpr int PER_ROW = kWarps * 32 / ROWS;  // threads a row
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
            // (a part of an item may have no key that the row sees: nothing, not 0 / 0)
            const float inv = whole || !(L == 0.0f) ? 1.0f / L : 0.0f;
            const int32_t row = row0 + rt;
            const int32_t qi = row / a.group, qh = head * a.group + row % a.group;
            T *dst = static_cast<T *>(a.out.p) + static_cast<int64_t>(off + qi) * a.out.row + qh * a.out.head;
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
                if (whole) store4(dst + c, v, inv);
                else store4(part + rt * D + c, v, inv);
            }
            if (c0 == 0) {
                const float lse = M + log2f(L);
                if (!whole) {
                    part[kSlotRows * D + rt] = lse;
                } else if (a.lse) {
                    a.lse[static_cast<int64_t>(off + qi) * a.q_heads + qh] = lse * kLn2;
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.merge_empty);
    };
    constexpr int VE = VecTraits<T>::kElems;
    for (uint32_t ni = 0;; ++ni) {
        if (__any_sync(0xffffffffu, *dead)) break;
        const Item4 it = item(ni);
        if (it.n == 0) {
            if (ni > 0) finish(ni - 1);
            break;
        }
        const int32_t rows = min(ROWS, it.n * a.group - it.row_tile * ROWS);
        // The lane's part of the queries (dimensions 64 h + 16 tig + 0..15 of row 8 u + g; rows past the last repeat
        // it), on their way while the item before is finished, for which the other warps have had time to
        // write theirs
        uint4 q_raw[RT][H][16 / VE];
#pragma unroll
        for (int u = 0; u < RT; ++u) {
            const int32_t row = it.row_tile * ROWS + min(8 * u + g, rows - 1);
            const int32_t qi = row / a.group, qh = it.head * a.group + row % a.group;
            const T *src = static_cast<const T *>(a.q.p) + static_cast<int64_t>(it.off + qi) * a.q.row + qh * a.q.head;
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int e = 0; e < 16 / VE; ++e) q_raw[u][h][e] = *reinterpret_cast<const uint4 *>(src + 64 * h + 16 * tig + e * VE);
        }
        if (ni > 0) finish(ni - 1);
        const int32_t key_end = min(it.tile1 * kKvTile, it.len);
        // q as B fragments: column g of tile u is row 8 u + g, dimensions 64 h + 16 tig +
        // 4 j + 0..3 in k-step (h, j), the last two by kUnit0 / kUnit1
        uint32_t qf[NT][D / 16][2];
        // of the rows 8 u + 2 tig + i that the thread's scores belong to: the score
        // scale in log2 units over kUnit0, the blocks' sums of q times kUnit0, and the keys seen
        // (pairs: of rows 2 tig and the next)
        F2 cr[RT], qs[RT][H];
        int32_t kmin[RT][2], kmax[RT][2];
#pragma unroll
        for (int u = 0; u < RT; ++u) {
            const int32_t row = it.row_tile * ROWS + min(8 * u + g, rows - 1);
            const int32_t qi = row / a.group;
            float x[D / 4];
            float amax = 0.0f;
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int e = 0; e < 16 / VE; ++e) VecTraits<T>::load(reinterpret_cast<const T *>(&q_raw[u][h][e]), x + 16 * h + e * VE);
#pragma unroll
            for (int e = 0; e < D / 4; ++e) amax = fmaxf(amax, fabsf(x[e]));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // a power of two that brings the row's largest to [2^13, 2^14): f16 keeps
            // every value down to 2^-24 of it; not finite: left as it is
            int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 13;
            e = amax < INFINITY ? max(e, -126) : 0;
            const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
            const float up = fminf(a.scale * kLog2e * __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * (1.0f / kUnit0), 3e38f);
            const int32_t pos = it.len - it.n + qi;
            const int32_t hi = min(a.causal ? pos + 1 : it.len, key_end), lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
            float sum[H];
#pragma unroll
            for (int h = 0; h < H; ++h) {
                sum[h] = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) sum[h] += x[16 * h + i] * down;
                sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
                sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
                sum[h] *= kUnit0;
            }
            // from the lanes of rows 8 u + 2 tig and the next
            auto of_rows = [&](float x) { return two(__shfl_sync(0xffffffffu, x, 8 * tig), __shfl_sync(0xffffffffu, x, 8 * tig + 4)); };
            cr[u] = of_rows(up);
#pragma unroll
            for (int h = 0; h < H; ++h) qs[u][h] = of_rows(sum[h]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                kmax[u][i] = __shfl_sync(0xffffffffu, hi, 8 * tig + 4 * i);
                kmin[u][i] = __shfl_sync(0xffffffffu, lo, 8 * tig + 4 * i);
            }
            const float down2 = down * (kUnit0 / kUnit1);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const float *v = x + 4 * k;
                qf[u][k][0] = pack_f16(v[0] * down, v[1] * down);
                qf[u][k][1] = pack_f16(v[2] * down2, v[3] * down2);
                if (SPLIT) {
                    qf[NT - 1][k][0] = pack_rest(v[0] * down, v[1] * down, qf[0][k][0]);
                    qf[NT - 1][k][1] = pack_rest(v[2] * down2, v[3] * down2, qf[0][k][1]);
                }
            }
        }
        // keys that every row of the item sees: steps within need no mask
        const int32_t pos0 = it.len - it.n + it.row_tile * ROWS / a.group;
        const int32_t pos1 = it.len - it.n + (it.row_tile * ROWS + rows - 1) / a.group;
        const int32_t all_hi = min(a.causal ? pos0 + 1 : it.len, key_end);
        const int32_t all_lo = a.window > 0 ? max(0, pos1 - a.window + 1) : 0;

        // o^T, in units of kUnit0 / fr (rows d = 4 (g + 8 (k / 2)) + 2 (k % 2)) and kUnit1 / fr
        // (d + 1), columns 2 tig and the next; om: what the least values add, in 1 / fr
        float o[NT][D / 16][4];
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int k = 0; k < D / 16; ++k) o[u][k][0] = o[u][k][1] = o[u][k][2] = o[u][k][3] = 0.0f;
        float m[RT][2];
        F2 less[RT], l[RT], fr[RT], om[RT][H];  // less: -m, 0 for -inf
#pragma unroll
        for (int u = 0; u < RT; ++u) {
            m[u][0] = m[u][1] = -INFINITY;
            less[u] = l[u] = two(0.0f, 0.0f);
            fr[u] = two(kMostFactor, kMostFactor);
#pragma unroll
            for (int h = 0; h < H; ++h) om[u][h] = two(0.0f, 0.0f);
        }
        auto rescale = [&](int u, F2 f) {  // the rows' o and om
#pragma unroll
            for (int h = 0; h < H; ++h) om[u][h] = mul(om[u][h], f);
            const float2 x = apart(f);
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    o[u][k][e] *= e & 1 ? x.y : x.x;
                    if (SPLIT) o[NT - 1][k][e] *= e & 1 ? x.y : x.x;
                }
        };

        const int32_t steps = (it.tile1 - it.tile0 + TS - 1) / TS;
        // this warp's steps: those whose running number is the warp's modulo kWarps
        const int32_t j0 = (warp - static_cast<int32_t>(i0 % kWarps) + kWarps) % kWarps;
        for (int32_t st = j0; st < steps; st += kWarps) {
            const uint32_t slot = taken++ % kDepth;
            const int32_t key0 = (it.tile0 + st * TS) * kKvTile;
            landed();
            __syncwarp();  // every lane's copies of scales
            // scale and least value of token tok + 2 t, of K (v = 0) or V
            const uint32_t *meta = reinterpret_cast<const uint32_t *>(sm.meta[warp][slot]) + tok;
            auto meta_of = [&](int v, int j, int t, int h) { return meta[(j * 2 * H + v * H + h) * kKvTile + 2 * t]; };
            float s[TS][H][NT][4];
#pragma unroll
            for (int j = 0; j < TS; ++j)
#pragma unroll
                for (int h = 0; h < H; ++h) {
#pragma unroll
                    for (int u = 0; u < NT; ++u) s[j][h][u][0] = s[j][h][u][1] = s[j][h][u][2] = s[j][h][u][3] = 0.0f;
                    const uint4 w = sm.codes[warp][slot][0][j * H + h][lane];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t x[4], y[4];
                        pairs(k == 0 ? w.x : w.y, x);
                        pairs(k == 0 ? w.z : w.w, y);
                        const uint32_t f0[4] = {x[0], y[0], x[1], y[1]}, f1[4] = {x[2], y[2], x[3], y[3]};
#pragma unroll
                        for (int u = 0; u < NT; ++u) {
                            mma_16816_f16(s[j][h][u], f0, qf[u][4 * h + 2 * k][0], qf[u][4 * h + 2 * k][1]);
                            mma_16816_f16(s[j][h][u], f1, qf[u][4 * h + 2 * k + 1][0], qf[u][4 * h + 2 * k + 1][1]);
                        }
                    }
                }
            // scores in log2 units
            F2 z[TS][RT][2];  // [token half]
#pragma unroll
            for (int j = 0; j < TS; ++j)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        const float2 ks = scale_of(meta_of(0, j, t, h));
                        const F2 scale = two(ks.x, ks.x), least = two(ks.y, ks.y);
#pragma unroll
                        for (int u = 0; u < RT; ++u) {
                            F2 dot = two(s[j][h][u][2 * t], s[j][h][u][2 * t + 1]);
                            if (SPLIT)
                                dot = fma(two(s[j][h][NT - 1][2 * t], s[j][h][NT - 1][2 * t + 1]), two(1.0f / kLoScale, 1.0f / kLoScale), dot);
                            z[j][u][t] = fma(scale, dot, h == 0 ? mul(least, qs[u][0]) : fma(least, qs[u][h], z[j][u][t]));
                        }
                    }
#pragma unroll
                    for (int u = 0; u < RT; ++u) z[j][u][t] = mul(z[j][u][t], cr[u]);
                }
            uint32_t vmeta[TS][2][H];
#pragma unroll
            for (int j = 0; j < TS; ++j)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int h = 0; h < H; ++h) vmeta[j][t][h] = meta_of(1, j, t, h);
            if (key0 < all_lo || key0 + TS * kKvTile > all_hi) {  // some row does not see some key
#pragma unroll
                for (int j = 0; j < TS; ++j) {
#pragma unroll
                    for (int u = 0; u < RT; ++u)
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const int32_t key = key0 + j * kKvTile + tok + 2 * t;
                            float2 x = apart(z[j][u][t]);
                            if (key < kmin[u][0] || key >= kmax[u][0]) x.x = -INFINITY;
                            if (key < kmin[u][1] || key >= kmax[u][1]) x.y = -INFINITY;
                            z[j][u][t] = two(x.x, x.y);
                        }
                    // Scales and least values of V may be NaN or infinite, and 0 * NaN is not 0: past the sequence's
                    // end they are whatever was there, and of other keys they are for the rows that see them, whose om
                    // becomes NaN
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const int32_t key = key0 + j * kKvTile + tok + 2 * t;
#pragma unroll
                        for (int h = 0; h < H; ++h) {
                            const bool number = (((vmeta[j][t][h] & 0x7FFF7FFFu) + 0x04000400u) & 0x80008000u) == 0;  // both
                            if (!number && key < key_end) {
#pragma unroll
                                for (int u = 0; u < RT; ++u)
                                    om[u][h] = add(om[u][h], two(key >= kmin[u][0] && key < kmax[u][0] ? NAN : 0.0f,
                                                                 key >= kmin[u][1] && key < kmax[u][1] ? NAN : 0.0f));
                            }
                            if (!number || key >= key_end) vmeta[j][t][h] = 0;
                        }
                    }
                }
            }
            float2 top[RT];  // the lane's largest scores
            bool grow = false;
#pragma unroll
            for (int u = 0; u < RT; ++u) {
                top[u] = make_float2(-INFINITY, -INFINITY);
#pragma unroll
                for (int j = 0; j < TS; ++j)
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const float2 x = apart(z[j][u][t]);
                        top[u] = make_float2(fmaxf(top[u].x, x.x), fmaxf(top[u].y, x.y));
                    }
                grow = grow || top[u].x > m[u][0] + kSlack || top[u].y > m[u][1] + kSlack;  // (also from m = -inf)
            }
            auto probabilities = [&] {  // and l
#pragma unroll
                for (int u = 0; u < RT; ++u)
#pragma unroll
                    for (int j = 0; j < TS; ++j)
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const float2 x = apart(add(z[j][u][t], less[u]));
                            z[j][u][t] = two(ex2(x.x), ex2(x.y));
                            l[u] = add(l[u], z[j][u][t]);
                        }
            };
            // p' = p s fr, rows side by side: [.., token half]
            uint32_t ph[TS][H][NT][2];
            auto scaled = [&] {
                uint32_t over = 0;  // the largest of the hi parts: infinite where fr is too large
#pragma unroll
                for (int j = 0; j < TS; ++j)
#pragma unroll
                    for (int h = 0; h < H; ++h)
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const float vs = f16_pair(vmeta[j][t][h]).x;
#pragma unroll
                            for (int u = 0; u < RT; ++u) {
                                const float2 x = apart(mul(mul(z[j][u][t], fr[u]), two(vs, vs)));
                                const uint32_t hi = pack_f16(x.x, x.y);
                                ph[j][h][u][t] = hi;
                                if (SPLIT) ph[j][h][NT - 1][t] = pack_rest(x.x, x.y, hi);
                                const __half2 most = __hmax2(*reinterpret_cast<const __half2 *>(&over), *reinterpret_cast<const __half2 *>(&hi));
                                over = *reinterpret_cast<const uint32_t *>(&most);
                            }
                        }
                return ((over + 0x04000400u) & 0x80008000u) != 0;  // (7C00 in either half)
            };
            // fr anew, `most` at most; f: what m's change makes of the row's sums
            auto fit = [&](int u, float2 f, float2 most) {
                float2 largest = make_float2(0.0f, 0.0f);  // of p s
#pragma unroll
                for (int j = 0; j < TS; ++j)
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int h = 0; h < H; ++h) {
                            const float2 x = apart(z[j][u][t]);
                            const float vs = f16_pair(vmeta[j][t][h]).x;
                            const float2 ps = make_float2(x.x * vs, x.y * vs);  // (infinite ones are for their own dimensions)
                            largest = make_float2(ps.x < INFINITY ? fmaxf(largest.x, ps.x) : largest.x, ps.y < INFINITY ? fmaxf(largest.y, ps.y) : largest.y);
                        }
                float now[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float x = i ? largest.y : largest.x;
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                    // 2^(8 - exponent of the largest), where that is less
                    const int e = static_cast<int>(__float_as_uint(x) >> 23) - 127;
                    now[i] = fminf(__uint_as_float(static_cast<uint32_t>(127 + min(max(kTopExponent - e, -60), 60)) << 23), i ? most.y : most.x);
                }
                const float2 was = apart(fr[u]);
                rescale(u, two(f.x * (now[0] / was.x), f.y * (now[1] / was.y)));
                fr[u] = two(now[0], now[1]);
            };
            if (__any_sync(0xffffffffu, grow)) {
                // A row's fr may be raised with its m, by the next power of two, so that it goes by what the keys
                // weigh now: with the fr of large scales that have lost their weight later p' would sink to f16's
                // least steps.  Rows that do not pass m by kSlack keep it.
                float2 f[RT], most[RT];
#pragma unroll
                for (int u = 0; u < RT; ++u) {
                    const float2 was = apart(fr[u]);
                    float fi[2], mi[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float old = m[u][i];
                        float mx = fmaxf(old, i ? top[u].y : top[u].x);
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                        if (!(mx > old + kSlack)) mx = old;
                        m[u][i] = mx;
                        const float more = old == -INFINITY ? 0.0f : mx - old;
                        fi[i] = old == -INFINITY ? 0.0f : ex2(-more);
                        const uint32_t up = static_cast<uint32_t>(127 + static_cast<int>(ceilf(fminf(more, 120.0f)))) << 23;
                        mi[i] = fminf((i ? was.y : was.x) * __uint_as_float(up), kMostFactor);
                    }
                    less[u] = two(m[u][0] == -INFINITY ? 0.0f : -m[u][0], m[u][1] == -INFINITY ? 0.0f : -m[u][1]);
                    f[u] = make_float2(fi[0], fi[1]);
                    most[u] = make_float2(mi[0], mi[1]);
                    l[u] = mul(l[u], two(fi[0], fi[1]));
                }
                probabilities();
#pragma unroll
                for (int u = 0; u < RT; ++u) fit(u, f[u], most[u]);
                scaled();
            } else {
                probabilities();
                if (__any_sync(0xffffffffu, scaled())) {
#pragma unroll
                    for (int u = 0; u < RT; ++u) fit(u, make_float2(1.0f, 1.0f), apart(fr[u]));
                    scaled();
                }
            }
#pragma unroll
            for (int j = 0; j < TS; ++j)
#pragma unroll
                for (int u = 0; u < RT; ++u)
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int h = 0; h < H; ++h) {
                            const float vm = scale_of(vmeta[j][t][h]).y;
                            om[u][h] = fma(mul(z[j][u][t], fr[u]), two(vm, vm), om[u][h]);
                        }
#pragma unroll
            for (int j = 0; j < TS; ++j)
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    uint32_t pf[NT][2];  // p'^T as B fragments
#pragma unroll
                    for (int u = 0; u < NT; ++u) {
                        pf[u][0] = transpose_8x8(ph[j][h][u][0]);
                        pf[u][1] = transpose_8x8(ph[j][h][u][1]);
                    }
                    const uint4 w = sm.codes[warp][slot][1][j * H + h][lane];
                    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t f[4];
                        pairs(ws[k], f);
#pragma unroll
                        for (int u = 0; u < NT; ++u) mma_16816_f16(o[u][4 * h + k], f, pf[u][0], pf[u][1]);
                    }
                }
            __syncwarp();  // every lane has read the scales
            int32_t ahead[TS];
            look(i0 + st + kDepth * kWarps, ahead);
            fetch(ahead, slot);
        }
        i0 += steps;

        // ---- the warp's part, for the merge
        wait(&sm.merge_empty, (ni & 1u) ^ 1u, 47);  // the buffer has been read
#pragma unroll
        for (int u = 0; u < RT; ++u)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                auto over_lanes = [](float x) {
                    x += __shfl_xor_sync(0xffffffffu, x, 4);
                    x += __shfl_xor_sync(0xffffffffu, x, 8);
                    return x + __shfl_xor_sync(0xffffffffu, x, 16);
                };
                auto row_of = [&](F2 x) { return i ? apart(x).y : apart(x).x; };
                const float sum = over_lanes(row_of(l[u])), un = 1.0f / row_of(fr[u]);
                float least[H];
#pragma unroll
                for (int h = 0; h < H; ++h) least[h] = over_lanes(row_of(om[u][h]));
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
                    const float add = least[jj / 2];
                    *reinterpret_cast<float4 *>(&sm.o[warp][rt][32 * jj + 4 * g]) =
                        make_float4(fmaf(v.x, 1.0f / kUnit0, add) * un, fmaf(v.y, 1.0f / kUnit1, add) * un,
                                    fmaf(v.z, 1.0f / kUnit0, add) * un, fmaf(v.w, 1.0f / kUnit1, add) * un);
                }
            }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.merge_full);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <typename T, int D, int NT>
cudaError_t decode4_tiles(const AttnView &v, cudaStream_t stream) {
    static uint64_t ctx[128] = {};
    constexpr int smem = static_cast<int>(sizeof(Decode4Smem<D, NT>));
    static_assert((smem + 1024) * ctas_per_sm<D, NT>() <= 228 * 1024, "the shared memory of an SM");
    cudaError_t e = allow_smem(attn_decode4_kernel<T, D, NT>, smem, ctx);
    if (e != cudaSuccess) return e;
    const int grid = device_sm_count() * ctas_per_sm<D, NT>();
    attn_decode4_kernel<T, D, NT><<<grid, (consumers<D, NT>() + 1) * 32, smem, stream>>>(v);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = launch_join<T, D, tile_rows<T, NT>(), 4>(v, grid, kSlotRows, stream);
    count_launches(2);
    return e;
}

template <typename T, int D>
cudaError_t decode4_typed(const AttnView &v, cudaStream_t stream) {
    if constexpr (sizeof(T) == 4) return decode4_tiles<T, D, 2>(v, stream);
    // one column tile of eight rows where that is all that any sequence has
    else if (static_cast<int64_t>(v.max_queries) * v.group <= 8) return decode4_tiles<T, D, 1>(v, stream);
    else return decode4_tiles<T, D, 2>(v, stream);
}

}  // namespace

cudaError_t launch_attn_decode4(const AttnView &v, int head_dim, lora_dtype_t dtype, cudaStream_t stream) {
    if (dtype == LORA_FP32) return head_dim == 64 ? decode4_typed<float, 64>(v, stream) : decode4_typed<float, 128>(v, stream);
    return head_dim == 64 ? decode4_typed<__nv_bfloat16, 64>(v, stream) : decode4_typed<__nv_bfloat16, 128>(v, stream);
}

}  // namespace lora
