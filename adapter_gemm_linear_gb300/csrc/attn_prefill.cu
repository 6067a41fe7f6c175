// Attention over the 8-bit paged cache (lora_kv_attention) for many queries a
// sequence, in bf16: prompts and chunks of prompts, on the tcgen05 tensor
// cores.
//
// With hundreds of query rows per key the call is bound by the two matrix
// products, 4 D flops per (query, head, key).  Rows are the queries of all
// query heads that share a key/value head (row r: query r / group, head r %
// group), so one load and conversion of a key serves group times as many rows.
// One persistent CTA per SM works on items of 256 rows, as two tiles A and B
// of 128, over tiles of 128 keys:
//
//   S_X = Q_X K^T     (M = 128 rows, N = 128 keys, both from shared memory)
//   P_X = 2^(S_X c + log2 vs - m)      one thread per row, registers
//   O_X += P_X V      (A = P from Tensor Memory, N = D)
//
//  - warps 0-3 and 4-7: the softmax of A and B, thread = row, no shuffles;
//    while one tile's softmax runs, the other tile's products run.
//  - warps 8-11 turn the codes, and the queries, into f16 tiles in shared memory
//    (exactly), in the 128-byte-swizzled K-major layout of tcgen05.mma: K as
//    [keys][dims], V as [dims][keys], which the cache's layout of V gives
//    without a transposition.  Two stages each; the next tile's codes are on their way
//    to shared memory meanwhile by 16-byte asynchronous copies, each thread's
//    its own (loads into registers took half as long again: with 225 KB of
//    shared memory taken, what is left of the L1 holds too few in flight;
//    and 32 bulk copies of 2 KB a tile take the copy engine 2 us).
//  - warp 12 issues the products; warp 13 hands out the items, and warp 14
//    looks up the pages and scales of the key tiles, four tiles ahead.
//  - q is f16 times a power of two per row (exact for bf16), P is f16 (11
//    bits) with the page's scale of V in its exponent (attn_split.cuh); a
//    row's sums are rescaled only when a p' would leave f16.
//  - Tensor Memory: S_A, S_B (128 columns each, P over the first 64), O_A, O_B.
// The key tiles of all items form one line that the CTAs share equally
// (attn_split.cuh), so causal and ragged work is level to one tile.
// Measured, with the join: 2048 queries x 34816 keys, 32 heads on 8 of 128, int8:
// 795 us in a graph (830-843 one by one), 1.43 PFLOP/s (0.74 of the measured bf16
// product): 1.75 us for a key tile whose products take 1.1.  The tensor pipes are
// busy for 51% of the time and 52% of the issue slots are used, so neither bounds
// it alone, but the roles' waits for one another.  With 32 query rows, a quarter
// of tile A and none of B, a key tile takes as long (64 x 4 queries of 64 heads on 8
// on 4096 keys: 187 us, whose codes take 79): it is the converting warps or A's
// own chain that the others wait for.  16 causal prompts, 8192 tokens, 64 heads on 8:
// 212-217 us (207 in a graph), 0.56 PFLOP/s of what the mask leaves: an item has
// some four key tiles there, and costs about four more (its queries' conversion, the
// masked tile, the results' way out); pipes 31%, issue slots 50%.
#include <cuda_runtime.h>
#include <math.h>

#include "attn_device.cuh"
#include "attn_internal.h"
#include "attn_split.cuh"
#include "attn_sums.h"
#include "attn_uint4.cuh"
#include "sm100_ptx.cuh"

namespace lora {

namespace {

using namespace sm100;

constexpr int kRows = 256;       // query rows of an item
constexpr int kHalf = 128;       // and of one MMA tile
constexpr int kKeys = 128;       // keys of a tile
constexpr int kSubs = kKeys / kKvTile;
constexpr int kPreThreads = 512;
constexpr int kItemRing = 4;
constexpr int kItemReaders = 8 + 1 + 1;  // warps that read an item's entry
constexpr int kTileRing = 4;             // key tiles looked up ahead
// What beginning and ending an item costs, in key tiles: an item has so many
// units of the line more than key tiles, in front.  (Short prompts have items
// of one tile; without this the CTAs that got them took twice as long.)
constexpr int kItemUnits = 4;
constexpr long long kWaitClocks = 4000000000ll;  // about 2 s: far beyond any legitimate wait

struct Item {
    int32_t seq, head, row_tile, last_cta;
    int32_t off, n, len;
    int32_t tile0, tile1;  // key tiles of this CTA; tile1 < 0: no more items
    int32_t flags;
    float vr;  // v_reference of the key tiles
};
constexpr int kFromStart = 1, kToEnd = 2;

// A key tile of the CTA's line: where its 16-key pieces are, and their scales.
struct KeyTile {
    // Of each piece K's scale, and V's relative to the reference vr (attn_split.cuh)
    // in log2, and what takes it out again; of a V that is zero the least.
    float4 scales[kSubs];
    // (of the 4-bit cache 1, 0 and 1)
    int64_t at[kSubs];    // offset in k_pages (of the 4-bit cache its tile_index); < 0: past the end or not there, zeros
    int64_t at_v[kSubs];  // and in v_pages
    int32_t key0, len;    // first key, the sequence's length; key0 < 0: no more tiles
    int32_t off, n, head, row_tile;  // of an item's first tile: its queries (n = 0 in its other tiles)
    float vr;      // the item's v_reference
    int32_t edge;  // some row of the item does not see some key
};
static_assert(sizeof(KeyTile) % 16 == 0, "scales are read as 16-byte pieces");

// The codes on their way: 16-byte pieces of the converting threads, of K and of V, each read by
// the thread that fetched it.
template <int D, int FMT>
struct Codes {
    uint4 codes[2][2 * D / 32][128];
};
// Of the 4-bit cache half as many, and in the other half: its scales, by the tile's parity
// (of a warp's two 16-key pieces K's and V's, [64 dimensions][key](scale, least) in f16),
// and sixteen more columns of K and of Q_A and Q_B (32 bytes a row, 32-byte swizzle).
template <int D>
struct Codes<D, LORA_KV_UINT4> {
    static constexpr int H = D / kBlockDims;
    uint4 codes[2][D / 32][128];
    uint32_t meta[2][4][2 * 2 * H * kKvTile];  // [parity][warp]
    alignas(1024) uint8_t kx[kKeys * 32];
    uint8_t qx[2][kHalf * 32];
};

template <int D, int FMT>
struct PrefillSmem : Codes<D, FMT> {
    alignas(1024) uint8_t q[2][kHalf * D * 2];
    uint8_t k[2][kKeys * D * 2];
    uint8_t v[2][kKeys * D * 2];
    alignas(16) KeyTile tiles[kTileRing];
    int8_t q_exponent[2][2 * kHalf];  // of an item's rows, by the item's parity: q is 2^this times what is in q
    Item items[kItemRing];
    uint64_t item_full[kItemRing], item_empty[kItemRing], tile_full[kTileRing], tile_empty[kTileRing];
    uint64_t q_full[2], q_empty[2], k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_ready[2][2], half_done[2], o_done[2], drain;
    long long warp_sum[kPreThreads / 32];
    long long base;
    int32_t seq;
    int32_t nan_item[kItemRing];      // number (from 1) of the last item with a NaN (4 bits: or infinity) hidden in V, by number
    int32_t head0, row_tile0, skip0;  // where the CTA's line begins
    uint32_t tmem;
    int32_t dead;
};

// ---------------------------------------------------------------- PTX

// One lane of the (converged) warp, known to be one to the compiler.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

// D (+)= A B^T, A: f16 in Tensor Memory (two per column), B: shared memory, fp32 sums.
__device__ __forceinline__ void mma_f16_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
        "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// 16 columns of the thread's TMEM lane (for the rare rescaling, where registers are short).
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Instruction descriptor of kind::f16 with f16 A and B, fp32 D, both K-major.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N) {
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Two fp32 values at once.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Wait for a phase of an mbarrier, bounded by the SM's clock (cheaper to read
// than the global timer), or until another wait has run out (`dead`).
__device__ __forceinline__ bool wait_clocks(uint64_t *bar, uint32_t parity, long long limit, const volatile int32_t *dead) {
    const long long t0 = clock64();
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 8; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (*dead || clock64() - t0 > limit) return false;
    }
}

// ---------------------------------------------------------------- the line of work

// A sequence's row tiles: tile i covers rows [256 i, 256 i + 256) of n *
// group.  (The host refuses calls with 2^31 rows * group or more.)
struct RowTiles {
    int32_t first, len, rows, group, count, window, causal;

    __device__ __forceinline__ RowTiles(const AttnView &a, const SeqRows &r)
        : first(r.len - r.n), len(r.len), rows(r.n * a.group), group(a.group), count((rows + kRows - 1) / kRows),
          window(a.window), causal(a.causal) {}

    // key tiles [lo, hi) that the queries of row tile i see
    __device__ __forceinline__ int32_t hi(int32_t i) const {
        const int32_t last = min(i * kRows + kRows - 1, rows - 1);
        const int32_t end = causal ? first + last / group + 1 : len;
        return static_cast<int32_t>((static_cast<uint32_t>(end) + kKeys - 1) / kKeys);
    }
    __device__ __forceinline__ int32_t lo(int32_t i) const {
        if (window <= 0) return 0;
        return max(0, first + i * kRows / group - window + 1) / kKeys;
    }
    // units of the row tiles before i: kItemUnits and hi - lo each.  256 = 2 * 128, so hi(i) =
    // floor((2 i + floor((255 + group (first + 128)) / 128)) / group) for every
    // tile but the last, and lo(i) = max(0, floor((2 i + floor(group (first -
    // window + 1) / 128)) / group)).
    __device__ __forceinline__ long long before(int32_t i) const {
        long long sum;
        if (causal) {
            const long long c = (kRows - 1 + static_cast<long long>(group) * (first + kKeys)) >> 7;
            sum = sum_of_floors(min(i, count - 1), group, static_cast<uint32_t>(c));
            if (i == count) sum += hi(count - 1);
        } else {
            sum = static_cast<long long>(i) * hi(0);
        }
        if (window > 0) {
            const long long x = static_cast<long long>(group) * (first - window + 1);
            const int32_t e = static_cast<int32_t>(x >> 7);  // floor, of negative numbers too
            const int32_t i0 = e >= 0 ? 0 : (1 - e) / 2;
            if (i > i0) sum -= sum_of_floors(i - i0, group, 2 * i0 + e);
        }
        return sum + static_cast<long long>(i) * kItemUnits;
    }
};

__device__ __forceinline__ SeqRows prefill_seq(const AttnView &a, int32_t s) {
    SeqRows r = read_seq(a.kv, s, false);
    if (r.n > a.max_queries) r.n = 0;
    return r;
}

__device__ __forceinline__ long long seq_units(const AttnView &a, int32_t s) {
    const SeqRows r = prefill_seq(a, s);
    if (r.n == 0) return 0;
    const RowTiles t(a, r);
    return t.before(t.count) * a.kv.heads;
}

// ---------------------------------------------------------------- the products
//
// Tensor Memory columns: S_A 0, S_B 128 (P over their first 64), O_A 256, O_B 384.

template <int D, int FMT>
__device__ __forceinline__ void issue_scores(PrefillSmem<D, FMT> &sm, uint32_t X, uint32_t stage) {
    const uint64_t q = desc_kmajor_sw128(smem_u32(sm.q[0])) + X * (sizeof(sm.q[0]) >> 4);
    const uint64_t k = desc_kmajor_sw128(smem_u32(sm.k[0])) + stage * (sizeof(sm.k[0]) >> 4);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        const uint32_t at = (i / 4) * (kHalf * 128 >> 4) + (i % 4) * 2;
        mma_bf16_f32(X * 128, q + at, k + at, idesc_f16_f32(kHalf, kKeys), i > 0);
    }
}

// Of the 4-bit cache: K's value s code + m = (code - 8) s_a + (code - 8) s_b + (m + 8 s), s_a
// the upper seven bits of s, but not above 8128, and s_b the rest, so that both products
// are f16 values exactly (s is 8733 at most, where least and largest value are f16's):
// two tiles.  The last term is one column for all dimensions of a block, against the
// sum of q over them, which has two f16 parts: m twice, and 4 s twice against twice that.  There is
// room for one stage of the two tiles; each is given back and filled anew by itself
// (barriers 0 and 1 of k_full and k_empty), so that the first of the next keys is there
// when the last product with the second of these ends (2048 queries on 34816 keys 1137 us
// instead of 1189 when that was chosen).
template <int D>
__device__ __forceinline__ void issue_scores_part(PrefillSmem<D, LORA_KV_UINT4> &sm, uint32_t X, uint32_t part) {
    const uint64_t q = desc_kmajor_sw128(smem_u32(sm.q[0])) + X * (sizeof(sm.q[0]) >> 4);
    const uint64_t k = desc_kmajor_sw128(smem_u32(sm.k[0])) + part * (sizeof(sm.k[0]) >> 4);
    if (part == 0) {
        const uint64_t qx = desc_kmajor_sw32(smem_u32(sm.qx[0])) + X * (sizeof(sm.qx[0]) >> 4);
        mma_bf16_f32(X * 128, qx, desc_kmajor_sw32(smem_u32(sm.kx)), idesc_f16_f32(kHalf, kKeys), 0);
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        const uint32_t at = (i / 4) * (kHalf * 128 >> 4) + (i % 4) * 2;
        mma_bf16_f32(X * 128, q + at, k + at, idesc_f16_f32(kHalf, kKeys), 1);
    }
}

// Half h of the keys.
template <int D, int FMT>
__device__ __forceinline__ void issue_values(PrefillSmem<D, FMT> &sm, uint32_t X, uint32_t stage, uint32_t h, bool accumulate) {
    const uint64_t v = desc_kmajor_sw128(smem_u32(sm.v[0])) + stage * (sizeof(sm.v[0]) >> 4) + h * (D * 128 >> 4);
#pragma unroll
    for (int i = 0; i < kKeys / 32; ++i)
        mma_f16_ts(256 + X * 128, X * 128 + h * 32 + i * 8, v + i * 2, idesc_f16_f32(kHalf, D), i > 0 || accumulate);
}

// Of dimensions [d0, d0 + 32): a bit for each in which V is NaN at a key that
// the row sees, [kmin, kmax), in one of the tiles [tile0, tile1) that not
// every row sees whole.  (In those NaN codes are taken as 0 by the product,
// as p = 0 would not keep them from the rows that do not see the key.)  Of the
// 4-bit cache: values that are no f16 numbers, by their scale and least value.
template <int D, int FMT>
__device__ __noinline__ uint32_t nan_dims(const KvView &b, int32_t seq, int32_t head, int32_t tile0, int32_t tile1, int32_t all_lo,
                                          int32_t all_hi, int32_t kmin, int32_t kmax, int32_t d0) {
    uint32_t mask = 0;
    for (int32_t k = tile0 * kKeys; k < tile1 * kKeys; k += kKvTile) {
        const int32_t key0 = k & ~(kKeys - 1);
        if ((key0 >= all_lo && key0 + kKeys <= all_hi) || k >= kmax || k + kKvTile <= kmin) continue;
        const int32_t page = b.table[static_cast<int64_t>(seq) * b.max_pages + (k >> b.page_shift)];
        if (page < 0 || page >= b.num_pages) continue;
        if (FMT == LORA_KV_UINT4) {
            const uint32_t *scales = reinterpret_cast<const uint32_t *>(b.v_scales) +
                                     (tile_index(b, page, head, (k & (b.page_tokens - 1)) / kKvTile) * (D / kBlockDims) + d0 / kBlockDims) * kKvTile;
            for (int t = max(0, kmin - k); t < min(kKvTile, kmax - k); ++t)
                if (!are_numbers(scales[t])) mask = ~0u;
            continue;
        }
        if (!(b.v_scales[static_cast<int64_t>(page) * b.heads + head] > 0.0f)) continue;
        const uint32_t *v = reinterpret_cast<const uint32_t *>(
            b.v_pages + tile_offset<D>(b, page, head, (k & (b.page_tokens - 1)) / kKvTile));
        for (int q = 0; q < 4; ++q) {
            uint32_t seen = 0;
            for (int t = 0; t < 4; ++t)
                if (k + 4 * q + t >= kmin && k + 4 * q + t < kmax) seen |= 0x80u << (8 * t);
            for (int d = 0; seen && d < 32; ++d)
                if (e4m3_nan(v[((d0 + d) / 4 * 4 + q) * 4 + d % 4]) & seen) mask |= 1u << d;
        }
    }
    return mask;
}

// ---------------------------------------------------------------- kernel

// PARTS (4-bit cache): K in two parts, exactly; else its values rounded to f16.
template <int D, int FMT, bool PARTS>
__global__ void __launch_bounds__(kPreThreads, 1) attn_prefill_kernel(const __grid_constant__ AttnView a) {
    extern __shared__ __align__(1024) unsigned char raw[];
    PrefillSmem<D, FMT> &sm = *reinterpret_cast<PrefillSmem<D, FMT> *>(raw);
    constexpr bool U4 = FMT == LORA_KV_UINT4;
    static_assert(U4 || !PARTS, "parts of 4-bit values");
    constexpr int H = D / kBlockDims;
    constexpr uint32_t kRowAtom = kHalf * 128;    // bytes of one atom of 128 rows
    constexpr uint32_t kVAtom = D * 128;          // bytes of 64 keys of V
    // (the same for the warp, which the compiler cannot know of threadIdx.x / 32:
    // the roles below may then use uniform registers)
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const KvView &b = a.kv;
    JoinEntry *joins = join_entries(a, gridDim.x, kRows, D);
    // where a wait ran out (0: none did); then nobody waits any more, no entry of
    // the rings is written again, and every role ends when it looks for more
    volatile int32_t *dead = &sm.dead;
    const long long limit = a.test_wait_ns ? 2 * static_cast<long long>(a.test_wait_ns) : kWaitClocks;  // (2 GHz)

    auto wait = [&](uint64_t *bar, uint32_t parity, int32_t site) {  // whether the phase is complete
        if (mbar_try_wait(bar, parity) || wait_clocks(bar, parity, limit, dead)) return true;
        if (!*dead) *dead = site;
        return false;
    };
    auto all = [](bool yes) { return __all_sync(0xffffffffu, yes) != 0; };
    auto any_dead = [&] { return __any_sync(0xffffffffu, *dead != 0) != 0; };  // the same for the whole warp

    // the joining kernel may come in as soon as there is room beside CTAs that
    // run or have none of the work; it waits for this one's end before it reads
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- set-up and plan
    if (threadIdx.x == 0) {
        for (int i = 0; i < kItemRing; ++i) {
            mbar_init(&sm.item_full[i], 1);
            mbar_init(&sm.item_empty[i], kItemReaders);
        }
        for (int i = 0; i < kTileRing; ++i) {
            mbar_init(&sm.tile_full[i], 1);
            mbar_init(&sm.tile_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.q_full[i], 4);
            mbar_init(&sm.q_empty[i], 1);
            mbar_init(&sm.k_full[i], 4);
            mbar_init(&sm.k_empty[i], 1);
            mbar_init(&sm.v_full[i], a.test_wait_ns ? 5 : 4);
            mbar_init(&sm.v_empty[i], 1);
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.p_ready[i][0], 4);
            mbar_init(&sm.p_ready[i][1], 4);
            mbar_init(&sm.half_done[i], 1);
            mbar_init(&sm.o_done[i], 1);
        }
        mbar_init(&sm.drain, 1);
        fence_mbar_init();
        sm.dead = 0;
        for (int i = 0; i < kItemRing; ++i) sm.nan_item[i] = 0;
        joins[blockIdx.x].last_cta = -1;
    }
    if (warp == 12) {
        tmem_alloc(&sm.tmem, 512);
        tmem_relinquish();
    }
    const int32_t per = (b.num_seqs + kPreThreads - 1) / kPreThreads;
    const int32_t s0 = min(b.num_seqs, static_cast<int32_t>(threadIdx.x) * per), s1 = min(b.num_seqs, s0 + per);
    long long mine = 0;
    for (int32_t s = s0; s < s1; ++s) mine += seq_units(a, s);
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) sm.warp_sum[warp] = upto;
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < kPreThreads / 32; ++w) {
        if (w < warp) upto += sm.warp_sum[w];
        total += sm.warp_sum[w];
    }
    const long long ctas = min(total, static_cast<long long>(gridDim.x));
    const long long w0 = blockIdx.x < ctas ? total * blockIdx.x / ctas : 0;
    const long long w1 = blockIdx.x < ctas ? total * (blockIdx.x + 1) / ctas : 0;
    if (w0 < w1 && upto - mine <= w0 && w0 < upto) {
        long long at = upto - mine;
        int32_t s = s0;
        for (;; ++s) {
            const long long u = seq_units(a, s);
            if (w0 < at + u) break;
            at += u;
        }
        sm.seq = s;
        sm.base = at;
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = sm.tmem;
    if (w0 < w1) {  // the first item: the row tile i with before(i) <= u < before(i + 1)
        const RowTiles t(a, prefill_seq(a, sm.seq));
        const long long units = t.before(t.count), local = w0 - sm.base;
        const int32_t head = static_cast<int32_t>(local / units);
        const long long u = local - head * units;
        for (int32_t i = threadIdx.x; i < t.count; i += kPreThreads) {
            const long long at = t.before(i);
            if (at <= u && u < at + kItemUnits + t.hi(i) - t.lo(i)) {
                sm.head0 = head;
                sm.row_tile0 = i;
                sm.skip0 = static_cast<int32_t>(u - at);
            }
        }
    }
    __syncthreads();

    if (warp < 8) {
        // ================================================ softmax of tile X
        const int X = warp >> 2;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // the warp's TMEM lanes
        const uint32_t ts = tmem + lanes + X * 128, to = tmem + lanes + 256 + X * 128;
        const int rt = X * kHalf + (warp & 3) * 32 + lane;             // the thread's row of the item
        uint32_t n_item = 0, n_tile = 0, n_own = 0, n_part = 0;        // items, key tiles; those of X
        auto get_item = [&](Item &it) {
            const uint32_t e = n_item % kItemRing;
            wait(&sm.item_full[e], (n_item / kItemRing) & 1u, 50);
            it = sm.items[e];
            if (any_dead()) it.tile1 = -1;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.item_empty[e]);
            ++n_item;
        };
        auto takes_part = [&](const Item &it) {  // tile B may be empty
            return it.tile1 >= 0 && (X == 0 || it.n * a.group - it.row_tile * kRows > kHalf);
        };

        Item it;
        get_item(it);
        while (it.tile1 >= 0) {
            if (!takes_part(it)) {
                n_tile += it.tile1 - it.tile0;
                get_item(it);
                continue;
            }
            const int32_t rows = min(kRows, it.n * a.group - it.row_tile * kRows);
            const int32_t row = it.row_tile * kRows + min(rt, rows - 1);
            const int32_t qi = row / a.group, qh = it.head * a.group + row % a.group;
            const int32_t pos = it.len - it.n + qi;
            const int32_t kmax = a.causal ? pos + 1 : it.len;
            const int32_t kmin = a.window > 0 ? max(0, pos - a.window + 1) : 0;
            // keys that every row of the item sees
            const int32_t all_hi = a.causal ? it.len - it.n + it.row_tile * kRows / a.group + 1 : it.len;
            const int32_t all_lo = a.window > 0 ? it.len - it.n + (it.row_tile * kRows + rows - 1) / a.group - a.window + 1 : 0;
            float m = -INFINITY, l = 0.0f, cr = 0.0f, vr = 1.0f;
            float top = -INFINITY;  // where vr < 0: l is the sum of 2^(s - top), top the largest score
            for (int32_t t = it.tile0; t < it.tile1; ++t, ++n_tile, ++n_own) {
                wait(&sm.tile_full[n_tile % kTileRing], (n_tile / kTileRing) & 1u, 55);
                wait(&sm.s_full[X], n_own & 1u, 51 + X);
                __syncwarp();  // (lanes may leave a wait apart; what follows is for the whole warp at once)
                tc_fence_after_sync();
                const KeyTile &tile = sm.tiles[n_tile % kTileRing];
                if (t == it.tile0) {
                    cr = a.scale * kLog2e * __uint_as_float(static_cast<uint32_t>(127 + sm.q_exponent[(n_item - 1) & 1u][rt]) << 23);
                    vr = tile.vr;
                }
                const int32_t key0 = t * kKeys;
                if (__builtin_expect(key0 < all_lo || key0 + kKeys > all_hi, 0)) {
                    // keys that the row does not see: -inf, in place
#pragma unroll 1
                    for (int i = 0; i < kKeys; i += 16) {
                        uint32_t x[16];
                        tmem_ld_32x32b_x16(ts + i, x);
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (key0 + i + e < kmin || key0 + i + e >= kmax) x[e] = 0xFF800000u;
                        tmem_st_32x32b_x16(ts + i, x);
                    }
                    tmem_st_wait();
                }
                if (__builtin_expect(vr < 0.0f, 0)) {
                    // V's scales are so far apart that the probabilities with them
                    // in their exponents do not give l: from the scores alone
#pragma unroll 1
                    for (int i = 0; i < kSubs; ++i) {
                        uint32_t x[16];
                        tmem_ld_32x32b_x16(ts + 16 * i, x);
                        const float f = fmaxf(tile.scales[i].x * cr, 1e-37f);
                        float most = top, sum = 0.0f;
#pragma unroll
                        for (int e = 0; e < 16; ++e) most = fmaxf(most, __uint_as_float(x[e]) * f);
                        const float from = most == -INFINITY ? 0.0f : most;
#pragma unroll
                        for (int e = 0; e < 16; ++e) sum += ex2(fmaf(__uint_as_float(x[e]), f, -from));
                        l = fmaf(l, ex2(top - from), sum);
                        top = most;
                    }
                }
                // Two halves of 64 keys, one after the other, each with the row's
                // maximum so far: the product with the first half's V runs while
                // the second is in work.  (A loop, and no more than half of S in
                // registers: the four roles' code and registers have to stay
                // small, for warps that waited for instructions, and spills, had
                // been the largest losses.)
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    uint32_t s[2][32];
                    tmem_ld_32x32b_x32(ts + 64 * h, s[0]);
                    tmem_ld_32x32b_x32(ts + 64 * h + 32, s[1]);
                    tmem_ld_wait(s[0]);
                    tmem_ld_wait(s[1]);
                    // the maximum, in log2 units and with V's scale (a factor of
                    // 0 would make NaN of what is masked)
                    float mx = -INFINITY, c[4], d[4];
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const float2 sc = *reinterpret_cast<const float2 *>(&tile.scales[4 * h + v]);
                        const uint32_t *p = &s[v >> 1][(v & 1) * 16];
                        float x = max3(__uint_as_float(p[0]), __uint_as_float(p[1]), __uint_as_float(p[2]));
                        float y = max3(__uint_as_float(p[3]), __uint_as_float(p[4]), __uint_as_float(p[5]));
#pragma unroll
                        for (int e = 6; e < 14; e += 4) {
                            x = max3(x, __uint_as_float(p[e]), __uint_as_float(p[e + 1]));
                            y = max3(y, __uint_as_float(p[e + 2]), __uint_as_float(p[e + 3]));
                        }
                        x = max3(x, __uint_as_float(p[14]), __uint_as_float(p[15]));
                        c[v] = fmaxf(sc.x * cr, 1e-37f);
                        d[v] = sc.y;
                        mx = fmaxf(mx, fmaf(fmaxf(x, y), c[v], d[v]));
                    }
                    const bool grow = mx > m + kGrow;
                    if (__builtin_expect(__any_sync(0xffffffffu, grow), 0)) {
                        const float mn = grow ? mx - kStartPrefill : m;
                        const float f = !grow ? 1.0f : m == -INFINITY ? 0.0f : ex2(m - mn);
                        m = mn;
                        if (vr > 0.0f) l *= f;
                        if (t > it.tile0 || h > 0) {
                            // the products so far are complete: of earlier tiles since
                            // s_full, of this one's first half when half_done says so
                            if (h > 0) {
                                wait(&sm.half_done[X], n_own & 1u, 57);
                                __syncwarp();
                                tc_fence_after_sync();
                            }
#pragma unroll 1
                            for (int i = 0; i < D / 16; ++i) {
                                uint32_t o[16];
                                tmem_ld_32x32b_x16(to + 16 * i, o);
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tmem_st_32x32b_x16(to + 16 * i, o);
                            }
                        }
                    }
                    const float mu = m == -INFINITY ? 0.0f : m;
                    uint32_t pk[32];
                    // (first the half's own sum: l, which may be far larger than each
                    // of the terms of a long tail, is rounded once for 64 keys)
                    float half = 0.0f;
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const uint64_t c2 = pack2(c[v], c[v]), d2 = pack2(d[v] - mu, d[v] - mu);
                        const uint32_t *p = &s[v >> 1][(v & 1) * 16];
                        uint64_t sum = 0;
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            float x, y;
                            unpack2(fma2(pack2(__uint_as_float(p[e]), __uint_as_float(p[e + 1])), c2, d2), x, y);
                            x = ex2(x);
                            y = ex2(y);
                            sum = e == 0 ? pack2(x, y) : add2(sum, pack2(x, y));
                            pk[8 * v + e / 2] = pack_h2(x, y);
                        }
                        float x, y;
                        unpack2(sum, x, y);
                        half = fmaf(x + y, tile.scales[4 * h + v].z, half);
                    }
                    l += half;
                    tmem_st_32x32b_x32(ts + 32 * h, pk);
                    tmem_st_wait();
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.p_ready[X][h]);
                }
            }
            wait(&sm.o_done[X], n_part & 1u, 53 + X);
            __syncwarp();
            ++n_part;
            tc_fence_after_sync();
            const bool whole = (it.flags & (kFromStart | kToEnd)) == (kFromStart | kToEnd);
            float *part = partial_at(a, blockIdx.x, it.flags & kFromStart ? 1 : 0, kRows, D);
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.out.p) + static_cast<int64_t>(it.off + qi) * a.out.row + qh * a.out.head;
            // (a part of an item may have no key that the row sees: nothing, not 0 / 0)
            float inv = whole || !(l == 0.0f) ? 1.0f / l : 0.0f, lse = m + log2f(l);
            if (__builtin_expect(vr < 0.0f, 0)) {
                // out = o 2^(m - top) |vr| / l, the power in two halves; m <= top, as no V is above vr
                const float half = top == -INFINITY ? 0.0f : ex2(0.5f * (m - top));
                lse = top + log2f(l);
                inv *= half;
                vr *= -half;
            }
            const bool hidden = FMT != LORA_KV_INT8 && *static_cast<volatile int32_t *>(&sm.nan_item[n_item % kItemRing]) == static_cast<int32_t>(n_item);
#pragma unroll 1
            for (int i = 0; i < D / 32; ++i) {
                uint32_t o[32];
                tmem_ld_32x32b_x32(to + 32 * i, o);
                tmem_ld_wait(o);
                if (rt < rows) {
                    if (FMT != LORA_KV_INT8 && __builtin_expect(hidden, 0)) {
                        const uint32_t nan = nan_dims<D, FMT>(b, it.seq, it.head, it.tile0, it.tile1, all_lo, all_hi, kmin, kmax, 32 * i);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (nan >> e & 1u) o[e] = 0x7FFFFFFFu;
                    }
                    // (one after the other: 1 / l times vr may leave fp32's normal range)
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * inv * vr);
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 32; e += 16) {
                            uint32_t h[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const __nv_bfloat162 two = __floats2bfloat162_rn(__uint_as_float(o[e + 2 * k]), __uint_as_float(o[e + 2 * k + 1]));
                                h[k] = *reinterpret_cast<const uint32_t *>(&two);
                            }
                            store_32(dst + 32 * i + e, h);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            const uint32_t w[8] = {o[e], o[e + 1], o[e + 2], o[e + 3], o[e + 4], o[e + 5], o[e + 6], o[e + 7]};
                            store_32(part + rt * D + 32 * i + e, w);
                        }
                    }
                }
                __syncwarp();  // before the next load, which takes the whole warp
            }
            tc_fence_before_sync();
            if (rt < rows) {
                if (!whole) {
                    part[kRows * D + rt] = lse;
                } else if (a.lse) {
                    a.lse[static_cast<int64_t>(it.off + qi) * a.q_heads + qh] = lse * kLn2;
                }
            }
            if (!whole && (it.flags & kFromStart) && threadIdx.x == 0)
                joins[blockIdx.x] = JoinEntry{it.last_cta, it.head, it.off, it.row_tile * kRows, rows, {}};
            get_item(it);
        }
    } else if (warp < 12) {
        // ================================================ codes to f16 tiles
        const int wq = warp - 8;  // the warp's 32 keys of a tile
        constexpr int NL = U4 ? D / 32 : 2 * D / 32;  // 16-byte pieces a lane holds of K (or V)
        uint32_t n_tile = 0;
        const int cc = lane & 3, dpar = (lane >> 2) & 1, dq = lane >> 3;
        // of one tile: its first key, the length, and where the warp's two 16-key pieces are
        struct Tile {
            int32_t key0, len;
            int64_t at[2], at_v;  // (of V the thread's own)
            int32_t off, n, head, row_tile, edge;
        };
        Tile cur, nxt;
        auto look = [&](Tile &x, uint32_t n) {
            const uint32_t e = n % kTileRing;
            x.key0 = all(wait(&sm.tile_full[e], (n / kTileRing) & 1u, 60)) ? sm.tiles[e].key0 : -1;
            x.len = sm.tiles[e].len;
            x.at[0] = sm.tiles[e].at[2 * wq];
            x.at[1] = sm.tiles[e].at[2 * wq + 1];
            x.at_v = sm.tiles[e].at_v[2 * wq + (cc >> 1)];
            x.n = sm.tiles[e].n;
            x.off = sm.tiles[e].off;
            x.head = sm.tiles[e].head;
            x.row_tile = sm.tiles[e].row_tile;
            x.edge = sm.tiles[e].edge;
        };
        uint4 *kc = &sm.codes[0][0][wq * 32 + lane], *vc = &sm.codes[1][0][wq * 32 + lane];
        // the thread's piece i of a tile; zeros where there is no page
        auto fetch_k = [&](const Tile &x, int i) {
            const int64_t at = i < NL / 2 ? x.at[0] : x.at[1];
            if constexpr (U4) copy16(kc + 128 * i, b.k_pages + (max(at, int64_t{0}) * H + i % H) * kBlockBytes + lane * 16, at >= 0);
            else copy16(kc + 128 * i, b.k_pages + max(at, int64_t{0}) + 16 * (lane + 32 * (i % (NL / 2))), at >= 0);
        };
        auto fetch_v = [&](const Tile &x, int i) {
            if constexpr (U4)  // tokens 8 cc .. 8 cc + 7 of the warp's, four a piece
                copy16(vc + 128 * i, b.v_pages + (max(x.at_v, int64_t{0}) * H + (i >> 1)) * kBlockBytes + (lane >> 2) * 64 + (cc & 1) * 32 + (i & 1) * 16,
                       x.at_v >= 0);
            else copy16(vc + 128 * i, b.v_pages + max(x.at_v, int64_t{0}) + (dq * 2 + dpar) * 64 + (cc & 1) * 32 + (i >> 1) * 512 + (i & 1) * 16,
                   x.at_v >= 0);
        };
        // The 4-bit cache's scales of the warp's keys, of tile n (lanes read what others fetched).
        auto fetch_scales = [&](const Tile &x, uint32_t n) {
            if constexpr (U4) {
                if (lane >= 16 * H) return;
                const int64_t at = lane < 8 * H ? x.at[0] : x.at[1];
                const float *from = lane / (4 * H) % 2 ? b.v_scales : b.k_scales;
                copy16(&sm.meta[n & 1][wq][lane * 4], from + (max(at, int64_t{0}) * (H * kKvTile) + lane % (4 * H) * 4), at >= 0);
            }
        };
        auto fetched = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };
        // Where the thread's pieces go (all but constants).  K: piece i is of key
        // 32 wq + 16 (i / (NL / 2)) + 8 (i % 2) + lane / 4, so the row's place
        // in the swizzle is lane / 4; 16 dimensions, two 16-byte chunks.  V: of
        // dimensions 4 d4 .. 4 d4 + 3, d4 = 8 k + 2 dq + dpar, 8 keys.
        const int kr = lane >> 2, kp = lane & 3;
        const uint32_t k_at = (wq * 32 + kr) * 128, k_c0 = ((2 * kp) ^ kr) << 4, k_c1 = ((2 * kp + 1) ^ kr) << 4;
        const uint32_t v_at = (wq >> 1) * kVAtom + (8 * dq + 4 * dpar) * 128, v_c = ((wq & 1) * 4 + cc) ^ (4 * dpar);
        auto landed = [] { asm volatile("cp.async.wait_group 1;" ::: "memory"); };  // all groups but the newest
        // Row r of the sixteen more columns: eight values, and zeros.
        auto extra = [&](uint8_t *tile, int r, const uint32_t (&w)[4]) {
            uint4 *const at = reinterpret_cast<uint4 *>(tile + r * 32);
            at[r >> 2 & 1] = make_uint4(w[0], w[1], w[2], w[3]);
            at[~r >> 2 & 1] = make_uint4(0u, 0u, 0u, 0u);
        };
        // An item's Q_A and Q_B, the warp's 32 rows of each: copied to their
        // places as bf16, several rows at a time and 16 bytes a lane ...
        uint32_t n_q = 0, n_qb = 0;
        auto q_tiles = [&](const Tile &t) { return t.n * a.group - t.row_tile * kRows > kHalf ? 2 : 1; };
        auto q_place = [&](int X, int r, int piece) {
            return reinterpret_cast<uint4 *>(sm.q[X] + (wq * 32 + r) * 128 + (piece / 8) * kRowAtom + (((piece ^ r) & 7) << 4));
        };
        auto fetch_q = [&](const Tile &t, int X) {
            constexpr int LANES = D / 8;         // lanes of a row
            constexpr int AT_ONCE = 32 / LANES;  // rows of a copy
            constexpr int TURN = 8 / AT_ONCE;    // copies after which the swizzle repeats
            const int piece = lane % LANES, sub = lane / LANES;
            const int32_t row = t.row_tile * kRows + X * kHalf + wq * 32 + lane, qi = row / a.group;  // the lane's row
            const long long mine = row < t.n * a.group
                ? (static_cast<int64_t>(t.off + qi) * a.q.row + static_cast<int64_t>(t.head * a.group + row - qi * a.group) * a.q.head) * 2
                : -1;  // past the last: zeros
            uint8_t *dst = sm.q[X] + (wq * 32 + sub) * 128 + (piece / 8) * kRowAtom;
            const uint32_t swizzle = ((piece ^ sub) & 7) << 4;
            wait(&sm.q_empty[X], ((X ? n_qb : n_q) & 1u) ^ 1u, 65);
#pragma unroll 1
            for (int r = sub; r < 32; r += 8, dst += 1024) {
#pragma unroll
                for (int i = 0; i < TURN; ++i) {
                    const long long at = __shfl_sync(0xffffffffu, mine, r + i * AT_ONCE);
                    copy16(dst + i * AT_ONCE * 128 + (swizzle ^ (i * AT_ONCE << 4)), static_cast<const uint8_t *>(a.q.p) + max(at, 0ll) + piece * 16, at >= 0);
                }
            }
            fetched();
        };
        // ... and turned in place into f16 times a power of two per row (its
        // largest value in [2^13, 2^14); with K in parts [2^7, 2^8), so that the sums
        // of 64 are f16 values too), a row a lane.
        auto convert_q = [&](int X) {
            __syncwarp();  // every lane's copies
            float amax = 0.0f;
#pragma unroll 4
            for (int i = 0; i < D / 8; ++i) {
                const uint4 x = *q_place(X, lane, i);
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    amax = max3(amax, fabsf(__uint_as_float(w[k] << 16)), fabsf(__uint_as_float(w[k] & 0xFFFF0000u)));
            }
            int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127 - (PARTS ? 7 : 13);
            e = amax < INFINITY ? max(e, -126) : 0;
            const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
            sm.q_exponent[n_q & 1u][X * kHalf + wq * 32 + lane] = static_cast<int8_t>(e);
            float sum = 0.0f;
            uint32_t sums[4] = {0u, 0u, 0u, 0u};  // of 64 dimensions, in two parts, and twice that
#pragma unroll 2
            for (int i = 0; i < D / 8; ++i) {
                uint4 *at = q_place(X, lane, i);
                const uint4 x = *at;
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                uint32_t h[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float x0 = __uint_as_float(w[k] << 16) * down, x1 = __uint_as_float(w[k] & 0xFFFF0000u) * down;
                    h[k] = pack_h2(x0, x1);
                    sum += x0 + x1;
                }
                *at = make_uint4(h[0], h[1], h[2], h[3]);
                if constexpr (PARTS) {
                    if (i % 8 == 7) {
                        const float hi = __half2float(__float2half_rn(sum));
                        sums[2 * (i / 8)] = pack_h2(hi, sum - hi);
                        sums[2 * (i / 8) + 1] = pack_h2(2.0f * hi, 2.0f * (sum - hi));
                        sum = 0.0f;
                    }
                }
            }
            if constexpr (PARTS) extra(sm.qx[X], wq * 32 + lane, sums);
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.q_full[X]);
        };
        look(cur, 0);
        for (int i = 0; cur.key0 >= 0 && i < NL; ++i) fetch_k(cur, i);
        if (cur.key0 >= 0) fetch_scales(cur, 0);
        fetched();
        for (int i = 0; cur.key0 >= 0 && i < NL; ++i) fetch_v(cur, i);
        fetched();
        while (cur.key0 >= 0) {
            const uint32_t stage = n_tile & 1u, ph = (n_tile >> 1) & 1u;
            look(nxt, n_tile + 1);
            const bool more = nxt.key0 >= 0;
            // K: row = key, 16 dimensions of one key a piece
            if (!PARTS) wait(&sm.k_empty[stage], ph ^ 1u, 61);
            landed();
            uint8_t *kdst = sm.k[stage] + k_at;
            if constexpr (U4) {
                __syncwarp();  // every lane's copies
                if (more) fetch_scales(nxt, n_tile + 1);
                const uint32_t *const sc = sm.meta[n_tile & 1][wq];
                uint4 c[NL];
#pragma unroll
                for (int i = 0; i < NL; ++i) {
                    c[i] = kc[128 * i];
                    if (more) fetch_k(nxt, i);
                }
                // a piece: 16 dimensions of keys `tok` and tok + 2 of 16; values, or (code - 8) times the upper
                // (part 0) or lower bits of the scale
                const int tok = k_token(kr);
                const int x7 = tok & 7;
                auto convert_k = [&](int part) {
                    uint8_t *const row = sm.k[PARTS ? part : stage] + (wq * 32 + tok) * 128;
#pragma unroll
                    for (int i = 0; i < NL; ++i) {
                        const uint32_t words[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
                        uint8_t *const dst = row + (i / H) * (kKvTile * 128) + i % H * kRowAtom;
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const uint32_t y = sc[(i / H * 2 * H + i % H) * kKvTile + tok + 2 * t], s2 = __byte_perm(y, y, 0x1010);
                            const uint32_t sa = at_most(s2 & 0xFFF0FFF0u, 0x6FF06FF0u), by = part == 0 ? sa : less(s2, sa), m2 = __byte_perm(y, y, 0x3232);
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                uint32_t f[4];
                                nibbles_less<PARTS ? 8 : 0>(words[2 * t + k], f);
#pragma unroll
                                for (int e = 0; e < 4; ++e) f[e] = PARTS ? times(f[e], by) : times_and(f[e], s2, m2);
                                *reinterpret_cast<uint4 *>(dst + t * 256 + (((2 * kp + k) ^ (x7 + 2 * t)) << 4)) =
                                    make_uint4(f[0], f[1], f[2], f[3]);
                            }
                        }
                    }
                };
                if constexpr (PARTS) {
                    wait(&sm.k_empty[0], stage ^ 1u, 61);
                    uint32_t w[4] = {0u, 0u, 0u, 0u};  // a key a lane: least values, and 4 scales
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        const uint32_t y = sc[(lane / kKvTile * 2 * H + h) * kKvTile + lane % kKvTile];
                        w[2 * h] = __byte_perm(y, y, 0x3232);
                        w[2 * h + 1] = times(__byte_perm(y, y, 0x1010), 0x44004400u);
                    }
                    extra(sm.kx, wq * 32 + lane, w);
                }
                convert_k(0);
                if constexpr (PARTS) {
                    fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.k_full[0]);
                    wait(&sm.k_empty[1], stage ^ 1u, 63);
                    convert_k(1);
                }
            } else {
#pragma unroll 2
            for (int i = 0; i < NL; ++i) {
                const uint4 r = kc[128 * i];
                if (more) fetch_k(nxt, i);
                uint8_t *dst = kdst + (i / (NL / 2)) * (kKvTile * 128) + (i % 2) * 1024 + (i % (NL / 2)) / 2 * kRowAtom;
                uint32_t w[8];
                codes_to_f16<FMT>(r.x, w[0], w[1]);
                codes_to_f16<FMT>(r.y, w[2], w[3]);
                codes_to_f16<FMT>(r.z, w[4], w[5]);
                codes_to_f16<FMT>(r.w, w[6], w[7]);
                *reinterpret_cast<uint4 *>(dst + k_c0) = make_uint4(w[0], w[1], w[2], w[3]);
                *reinterpret_cast<uint4 *>(dst + k_c1) = make_uint4(w[4], w[5], w[6], w[7]);
            }
            }
            fetched();
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.k_full[PARTS ? 1 : stage]);
            const bool first = cur.n > 0;  // tile of an item: its queries, on their way while V is converted
            if (first) fetch_q(cur, 0);
            // V: row = dimension, 8 keys a piece; keys past the end are zeros
            // (their codes may be anything, and 0 * NaN is not 0)
            wait(&sm.v_empty[stage], ph ^ 1u, 62);
            if (first) asm volatile("cp.async.wait_group 2;" ::: "memory");
            else landed();
            if constexpr (U4) {
                // keys past the end: scale and least value 0 (what is there may be NaN)
                const int have = cur.len - (cur.key0 + wq * 32 + cc * 8);
                const uint32_t *const sc = sm.meta[n_tile & 1][wq];
                if (cur.edge) {
                    // what is no number at keys that not every row sees: taken out, and noted for the item (nan_dims)
                    const uint32_t item = n_q + (first ? 1u : 0u);
                    bool some = false;
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        uint32_t *const w = &sm.meta[n_tile & 1][wq][(lane / kKvTile * 2 * H + H + h) * kKvTile + lane % kKvTile];
                        if (cur.key0 + wq * 32 + lane < cur.len && !are_numbers(*w)) {
                            *w = 0u;
                            some = true;
                        }
                    }
                    if (some) sm.nan_item[item % kItemRing] = static_cast<int32_t>(item);
                    __syncwarp();
                }
#pragma unroll 1
                for (int h = 0; h < H; ++h) {
                    const uint4 *y = reinterpret_cast<const uint4 *>(sc + ((cc >> 1) * 2 * H + H + h) * kKvTile + (cc & 1) * 8);
                    const uint4 ya = y[0], yb = y[1];
                    uint32_t s2[4] = {__byte_perm(ya.x, ya.y, 0x5410), __byte_perm(ya.z, ya.w, 0x5410), __byte_perm(yb.x, yb.y, 0x5410),
                                      __byte_perm(yb.z, yb.w, 0x5410)};
                    uint32_t m2[4] = {__byte_perm(ya.x, ya.y, 0x7632), __byte_perm(ya.z, ya.w, 0x7632), __byte_perm(yb.x, yb.y, 0x7632),
                                      __byte_perm(yb.z, yb.w, 0x7632)};
                    if (__builtin_expect(have < 8, 0)) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t there = (2 * k < have ? 0xFFFFu : 0u) | (2 * k + 1 < have ? 0xFFFF0000u : 0u);
                            s2[k] &= there;
                            m2[k] &= there;
                        }
                    }
                    const uint4 ra = vc[128 * (2 * h)], rb = vc[128 * (2 * h + 1)];
                    if (more) {
                        fetch_v(nxt, 2 * h);
                        fetch_v(nxt, 2 * h + 1);
                    }
                    const uint32_t wa[4] = {ra.x, ra.y, ra.z, ra.w}, wb[4] = {rb.x, rb.y, rb.z, rb.w};
                    uint8_t *const to = sm.v[stage] + (wq >> 1) * kVAtom + h * (kBlockDims * 128);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t fa[4], fb[4];
                        nibbles_less<0>(wa[j], fa);
                        nibbles_less<0>(wb[j], fb);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {  // dimensions d and d + 1: of keys 0, 1 and 2, 3
                            const int d = 4 * kr + 32 * (j >> 1) + 2 * (j & 1) + k;
                            *reinterpret_cast<uint4 *>(to + d * 128 + ((((wq & 1) * 4 + cc) ^ (d & 7)) << 4)) =
                                make_uint4(times_and(fa[k], s2[0], m2[0]), times_and(fa[2 + k], s2[1], m2[1]), times_and(fb[k], s2[2], m2[2]),
                                           times_and(fb[2 + k], s2[3], m2[3]));
                        }
                    }
                }
            } else {
            uint32_t keep[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int past = cur.key0 + wq * 32 + cc * 8 + 4 * i + 4 - cur.len;
                keep[i] = past <= 0 ? 0xFFFFFFFFu : past >= 4 ? 0u : 0xFFFFFFFFu >> (8 * past);
            }
            if (FMT == LORA_KV_E4M3 && cur.edge) {
                // NaN of keys that not every row sees: taken out, and noted for the item (nan_dims)
                bool some = false;
#pragma unroll 1
                for (int i = 0; i < NL; ++i) {
                    const uint4 r = vc[128 * i];
                    uint32_t w[4] = {r.x, r.y, r.z, r.w}, any = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t nan = e4m3_nan(w[e] & ((i & 1) ? keep[1] : keep[0]));
                        any |= nan;
                        w[e] = e4m3_without(w[e], nan);
                    }
                    if (any) {
                        vc[128 * i] = make_uint4(w[0], w[1], w[2], w[3]);
                        some = true;
                    }
                }
                const uint32_t item = n_q + (first ? 1u : 0u);
                if (some) sm.nan_item[item % kItemRing] = static_cast<int32_t>(item);
            }
            uint8_t *vdst = sm.v[stage] + v_at;
#pragma unroll 1
            for (int k = 0; k < NL / 2; ++k, vdst += 4096) {
                const uint4 ra = vc[128 * (2 * k)], rb = vc[128 * (2 * k + 1)];
                if (more) {
                    fetch_v(nxt, 2 * k);
                    fetch_v(nxt, 2 * k + 1);
                }
                const uint32_t wa[4] = {ra.x, ra.y, ra.z, ra.w}, wb[4] = {rb.x, rb.y, rb.z, rb.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t w[4];
                    codes_to_f16<FMT>(wa[e] & keep[0], w[0], w[1]);
                    codes_to_f16<FMT>(wb[e] & keep[1], w[2], w[3]);
                    *reinterpret_cast<uint4 *>(vdst + e * 128 + ((v_c ^ e) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            }
            fetched();
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.v_full[stage]);
            if (first) {
                const bool both = q_tiles(cur) > 1;
                if (both) fetch_q(cur, 1);
                else fetched();
                asm volatile("cp.async.wait_group 2;" ::: "memory");
                convert_q(0);
                if (both) {
                    asm volatile("cp.async.wait_group 0;" ::: "memory");
                    convert_q(1);
                    ++n_qb;
                }
                ++n_q;
            }
            cur = nxt;
            ++n_tile;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        if (warp == 12) {
            // ============================================ the products
            auto commit = [](uint64_t *bar) {
                if (elect_one()) mma_commit(bar);
                __syncwarp();
            };
            uint32_t n_item = 0, n_tile = 0, n_b = 0, n_qb = 0;
            // (Tensor Memory begins at column 0: the CTA has all of it)
            // (of key tile n, which the first of them waits for; the last gives K back)
            auto scores = [&](uint32_t X, uint32_t n, bool first, bool last) {
                if constexpr (PARTS) {
#pragma unroll 1
                    for (uint32_t part = 0; part < 2; ++part) {
                        if (first) wait(&sm.k_full[part], n & 1u, 72);
                        tc_fence_after_sync();
                        if (elect_one()) {
                            issue_scores_part(sm, X, part);
                            if (part == 1) mma_commit(&sm.s_full[X]);
                            if (last) mma_commit(&sm.k_empty[part]);
                        }
                        __syncwarp();
                    }
                } else {
                    if (elect_one()) {
                        issue_scores(sm, X, n & 1u);
                        mma_commit(&sm.s_full[X]);
                    }
                    __syncwarp();
                }
            };
            while (true) {
                const uint32_t e = n_item % kItemRing;
                wait(&sm.item_full[e], (n_item / kItemRing) & 1u, 70);
                const int32_t nt = sm.items[e].tile1 - sm.items[e].tile0, stop = sm.items[e].tile1 < 0;
                const uint32_t nx = sm.items[e].n * a.group - sm.items[e].row_tile * kRows > kHalf ? 2 : 1;  // tile B may be empty
                __syncwarp();
                if (elect_one()) mbar_arrive(&sm.item_empty[e]);
                if (any_dead() || stop) break;
                if (!PARTS) wait(&sm.k_full[n_tile & 1u], (n_tile >> 1) & 1u, 72);
#pragma unroll 1
                for (uint32_t X = 0; X < nx; ++X) {
                    wait(&sm.q_full[X], (X ? n_qb : n_item) & 1u, 71);
                    tc_fence_after_sync();
                    scores(X, n_tile, X == 0, X + 1 == nx);
                    if (nt == 1) commit(&sm.q_empty[X]);
                }
                ++n_item;
                n_qb += nx - 1;
                if (!PARTS) commit(&sm.k_empty[n_tile & 1u]);
#pragma unroll 1
                for (int32_t j = 0; j < nt; ++j, ++n_tile) {
                    const uint32_t st = n_tile & 1u, ph = (n_tile >> 1) & 1u;
                    const uint32_t st1 = (n_tile + 1) & 1u, ph1 = ((n_tile + 1) >> 1) & 1u;
                    const bool more = j + 1 < nt;
                    if (!all(wait(&sm.v_full[st], ph, 74))) break;  // no products of what may not be there
#pragma unroll 1
                    for (uint32_t X = 0; X < nx; ++X) {
#pragma unroll 1
                        for (uint32_t h = 0; h < 2; ++h) {
                            wait(&sm.p_ready[X][h], (X ? n_b : n_tile) & 1u, 75);
                            tc_fence_after_sync();
                            if (elect_one()) {
                                issue_values(sm, X, st, h, j > 0 || h > 0);
                                if (h == 0) mma_commit(&sm.half_done[X]);
                            }
                            __syncwarp();
                        }
                        if (more) {
                            if (!PARTS && X == 0) wait(&sm.k_full[st1], ph1, 76);
                            tc_fence_after_sync();
                            scores(X, n_tile + 1, X == 0, X + 1 == nx);
                            if (j + 2 == nt) commit(&sm.q_empty[X]);
                        } else {
                            commit(&sm.o_done[X]);
                        }
                    }
                    n_b += nx - 1;
                    commit(&sm.v_empty[st]);
                    commit(&sm.tile_empty[n_tile % kTileRing]);  // (the softmax has read its scales)
                    if (!PARTS && more) commit(&sm.k_empty[st1]);
                }
            }
            // nothing of this thread's may be in flight when Tensor Memory is freed
            commit(&sm.drain);
            const int32_t alone = 0;
            wait_clocks(&sm.drain, 0, kWaitClocks, &alone);
        } else if (warp == 13) {
            // ============================================ the items
            uint32_t n_item = 0;
            auto publish = [&](const Item &it) {
                const uint32_t e = n_item % kItemRing;
                wait(&sm.item_empty[e], ((n_item / kItemRing) & 1u) ^ 1u, 80);
                if (!any_dead() && lane == 0) {
                    sm.items[e] = it;
                    mbar_arrive(&sm.item_full[e]);
                }
                __syncwarp();
                ++n_item;
            };
            Item it;
            if (w0 < w1) {
                it.seq = sm.seq;
                it.head = sm.head0;
                it.row_tile = sm.row_tile0;
                int32_t skip = sm.skip0;  // units of the first item that belong to the CTA before
                SeqRows r = prefill_seq(a, it.seq);
                int32_t count = RowTiles(a, r).count;
                long long w = w0;
                while (true) {
                    const RowTiles t(a, r);
                    const int32_t lo = t.lo(it.row_tile), hi = t.hi(it.row_tile), units = kItemUnits + hi - lo;
                    const int32_t take = static_cast<int32_t>(min(static_cast<long long>(units - skip), w1 - w));
                    it.off = r.off;
                    it.n = r.n;
                    it.len = r.len;
                    it.tile0 = lo + max(skip - kItemUnits, 0);
                    it.tile1 = lo + skip + take - kItemUnits;
                    it.flags = (it.tile0 == lo ? kFromStart : 0) | (it.tile1 == hi ? kToEnd : 0);
                    it.last_cta = static_cast<int32_t>(((w + (units - skip)) * ctas - 1) / total);
                    if (it.tile1 > it.tile0) {
                        // (items ahead of their use: its reads are hidden but for the first item's)
                        it.vr = FMT == LORA_KV_UINT4
                                    ? 1.0f  // (its values come whole)
                                    : v_reference(b, it.seq, it.head, it.tile0 * kSubs, min(it.tile1 * kSubs, (it.len + kKvTile - 1) / kKvTile));
                        publish(it);
                    }
                    w += take;
                    if (any_dead() || w >= w1) break;
                    skip = 0;
                    if (++it.row_tile == count) {
                        it.row_tile = 0;
                        if (++it.head == b.heads) {
                            it.head = 0;
                            do r = prefill_seq(a, ++it.seq); while (r.n == 0);
                            count = RowTiles(a, r).count;
                        }
                    }
                }
            }
            it.tile0 = 0;
            it.tile1 = -1;
            it.vr = 1.0f;
            publish(it);
        }
        if (warp == 14) {
            // ============================================ pages and scales of the key tiles
            uint32_t n_item = 0, n_tile = 0;
            const int sub = lane & 7;
            while (true) {
                const uint32_t e = n_item % kItemRing;
                wait(&sm.item_full[e], (n_item / kItemRing) & 1u, 90);
                const int32_t seq = sm.items[e].seq, head = sm.items[e].head, len = sm.items[e].len;
                if (any_dead()) break;
                const int32_t tile0 = sm.items[e].tile0, tile1 = sm.items[e].tile1;
                const float vr = sm.items[e].vr;
                const int32_t off = sm.items[e].off, n = sm.items[e].n, row_tile = sm.items[e].row_tile;
                // keys that every row of the item sees
                const int32_t all_hi = a.causal ? len - n + row_tile * kRows / a.group + 1 : len;
                const int32_t last_row = min((row_tile + 1) * kRows, n * a.group) - 1;
                const int32_t all_lo = a.window > 0 ? len - n + last_row / a.group - a.window + 1 : 0;
                // and the first that some row sees (pages that lie before it may be gone)
                const int32_t some_lo = a.window > 0 ? len - n + row_tile * kRows / a.group - a.window + 1 : 0;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.item_empty[e]);
                ++n_item;
                // four tiles at a time: lane = (tile, piece)
                const float ref = log2f(fabsf(vr));
                for (int32_t t0 = tile0; t0 < max(tile1, tile0 + 1); t0 += 4) {
                    const int32_t t = t0 + (lane >> 3), key = t * kKeys + sub * kKvTile;
                    int64_t at = -1;
                    float ks = 0.0f, vs = 0.0f;
                    if (t < tile1 && key < len && key + kKvTile > some_lo) {
                        const int32_t page = read_page(b, seq, key >> b.page_shift);
                        if (page >= 0 && FMT == LORA_KV_UINT4) {
                            at = tile_index(b, page, head, (key & (b.page_tokens - 1)) / kKvTile);
                        } else if (page >= 0) {
                            at = tile_offset<D>(b, page, head, (key & (b.page_tokens - 1)) / kKvTile);
                            ks = __ldg(b.k_scales + static_cast<int64_t>(page) * b.heads + head);
                            vs = __ldg(b.v_scales + static_cast<int64_t>(page) * b.heads + head);
                        }
                    }
                    __syncwarp();
                    // (with scales too far apart l is not taken from these: iv = 0)
                    const float rel = vs > 0.0f ? log2f(vs) - ref : -INFINITY;
                    const float lv = fmaxf(rel, vr < 0.0f ? -400.0f : -kSpread);
                    const float iv = vr < 0.0f ? 0.0f : rel >= -kSpread ? vr / vs : kSpreadFactor;
                    for (int q = 0; q < 4 && t0 + q < max(tile1, tile0 + 1); ++q) {
                        const uint32_t r = n_tile % kTileRing;
                        wait(&sm.tile_empty[r], ((n_tile / kTileRing) & 1u) ^ 1u, 91);
                        if (any_dead()) break;
                        if ((lane >> 3) == q) {
                            sm.tiles[r].scales[sub] = FMT == LORA_KV_UINT4 ? make_float4(1.0f, 0.0f, 1.0f, 0.0f) : make_float4(ks, lv, iv, 0.0f);
                            sm.tiles[r].at[sub] = at;
                            sm.tiles[r].at_v[sub] = FMT == LORA_KV_UINT4 || vs > 0.0f ? at : -1;
                            if (sub == 0) {
                                sm.tiles[r].key0 = tile1 < 0 ? -1 : t * kKeys;
                                sm.tiles[r].len = len;
                                sm.tiles[r].off = off;
                                sm.tiles[r].n = t == tile0 ? n : 0;
                                sm.tiles[r].head = head;
                                sm.tiles[r].row_tile = row_tile;
                                sm.tiles[r].edge = t * kKeys < all_lo || t * kKeys + kKeys > all_hi;
                                sm.tiles[r].vr = vr;
                            }
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sm.tile_full[r]);
                        ++n_tile;
                    }
                }
                if (tile1 < 0) break;
            }
        }
        __syncwarp();
    }
    tc_fence_before_sync();
    __syncthreads();
    if (threadIdx.x == 0 && *dead) record_error(b.status, kDevTimeout, static_cast<uint32_t>(*dead));
    if (warp == 12) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, int FMT, bool PARTS = false>
cudaError_t prefill_typed(const AttnView &v, cudaStream_t stream) {
    static uint64_t ctx[128] = {};
    // more than half of an SM's shared memory even for D = 64: a CTA takes all of its Tensor Memory
    constexpr int smem = static_cast<int>(sizeof(PrefillSmem<D, FMT>) > 128 * 1024 ? sizeof(PrefillSmem<D, FMT>) : 128 * 1024);
    static_assert(smem <= 227 * 1024, "the shared memory of one CTA");
    cudaError_t e = allow_smem(attn_prefill_kernel<D, FMT, PARTS>, smem, ctx);
    if (e != cudaSuccess) return e;
    const int grid = device_sm_count();
    attn_prefill_kernel<D, FMT, PARTS><<<grid, kPreThreads, smem, stream>>>(v);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = launch_join<__nv_bfloat16, D, kRows, 1>(v, grid, kRows, stream);
    count_launches(2);
    return e;
}

}  // namespace

size_t prefill_workspace_bytes(int head_dim) { return split_workspace_bytes(device_sm_count(), kRows, head_dim); }

cudaError_t launch_attn_prefill(const AttnView &v, lora_kv_format_t fmt, int head_dim, cudaStream_t stream) {
    if (fmt == LORA_KV_UINT4) {
        // The scores' rounding shows in lse, which is fp32 (off by 1e-6 with K rounded), not in a
        // bf16 result beside its own rounding (1.76e-3 from the exact one, 1.67e-3 with K in parts), where
        // keys lie around 0; at 10 times their spread from it 2.4e-3, at 100 times 1.2e-2 (in parts 1.7e-3
        // both), which callers are told.  In parts 2048 queries of 34816 keys (32 heads of 128, 8 of the
        // cache) take 1180 us instead of 912.
        if (v.lse)
            return head_dim == 64 ? prefill_typed<64, LORA_KV_UINT4, true>(v, stream) : prefill_typed<128, LORA_KV_UINT4, true>(v, stream);
        return head_dim == 64 ? prefill_typed<64, LORA_KV_UINT4>(v, stream) : prefill_typed<128, LORA_KV_UINT4>(v, stream);
    }
    if (head_dim == 64)
        return fmt == LORA_KV_INT8 ? prefill_typed<64, LORA_KV_INT8>(v, stream) : prefill_typed<64, LORA_KV_E4M3>(v, stream);
    return fmt == LORA_KV_INT8 ? prefill_typed<128, LORA_KV_INT8>(v, stream) : prefill_typed<128, LORA_KV_E4M3>(v, stream);
}

}  // namespace lora
