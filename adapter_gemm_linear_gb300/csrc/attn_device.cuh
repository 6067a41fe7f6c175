// Device helpers of the cache and attention kernels: which rows a sequence
// has, where a token's codes are, and the conversions of the two formats.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "attn_internal.h"
#include "lora_device.cuh"

namespace lora {

// One sequence's rows [off, off + n) and its length; position of row off + i: len - n + i.
struct SeqRows {
    int32_t off, n, len;
};

// Reads sequence s; n = 0 where it has no rows, is padding (length 0) or is
// malformed (recorded when `report`).
__device__ __forceinline__ SeqRows read_seq(const KvView &b, int32_t s, bool report) {
    SeqRows r;
    r.len = b.seq_lens[s];
    r.off = b.offsets ? b.offsets[s] : s;
    const int32_t end = b.offsets ? b.offsets[s + 1] : s + 1;
    r.n = end - r.off;
    if (r.off < 0 || r.n < 0 || end > b.rows || (r.len > 0 && r.n > r.len)) {
        if (report) record_error(b.status, kDevBadSegment, static_cast<uint32_t>(s));
        r.off = r.n = r.len = 0;
    }
    if (r.len < 0 || r.len > (1 << 30) || r.len > static_cast<int64_t>(b.max_pages) * b.page_tokens) {
        if (report) record_error(b.status, kDevBadBlock, static_cast<uint32_t>(s));
        r.n = r.len = 0;
    }
    if (r.len == 0) r.n = 0;
    return r;
}

// Page of a sequence's token block, or -1 (recorded) where the table's entry is out of range.
__device__ __forceinline__ int32_t read_page(const KvView &b, int32_t s, int32_t slot) {
    const int32_t p = b.table[static_cast<int64_t>(s) * b.max_pages + slot];
    if (p >= 0 && p < b.num_pages) return p;
    record_error(b.status, kDevBadBlock, static_cast<uint32_t>(s));
    return -1;
}

// Element offset of 16-token tile g of (page, head): the tiles of K and V have the same size.
template <int D>
__device__ __forceinline__ int64_t tile_offset(const KvView &b, int32_t page, int32_t head, int32_t g) {
    return ((static_cast<int64_t>(page) * b.heads + head) * (b.page_tokens / kKvTile) + g) * (kKvTile * D);
}

// The first index in [0, n) at which a non-decreasing `above(index)` holds (n
// if none), by a whole warp: 32 questions at a time.
template <typename F>
__device__ __forceinline__ int32_t warp_search(int32_t n, F above) {
    const int lane = threadIdx.x & 31;
    int32_t lo = 0;
    while (n > 0) {
        const int32_t step = (n + 31) >> 5;
        const int32_t end = min(static_cast<int32_t>(lane + 1) * step, n);  // of the lane's part
        const uint32_t yes = __ballot_sync(0xffffffffu, lane * step < n && above(lo + end - 1));
        if (yes == 0) return lo + n;
        const int first = __ffs(yes) - 1;
        lo += first * step;
        n = step == 1 ? 0 : min(step, n - first * step);
    }
    return lo;
}

// The new rows of a batch cut where the token position is a multiple of 2^shift
// (a page, or a tile of 16): unit u < num_seqs is the first, possibly partial,
// piece of sequence u; unit num_seqs + w holds the pieces that begin within
// rows [w * 2^shift, (w + 1) * 2^shift), at most one per sequence.  f(s, r, lo,
// hi) gets the sequence, its rows, and the token positions [lo, hi) of a piece;
// whole warps call it, and all of a block's with the same unit take the same
// steps.  (f stands here once, as its code, run once by each warp, takes longer
// to fetch than to execute.)
template <typename F>
__device__ __forceinline__ void for_pieces(const KvView &b, int32_t unit, int shift, bool report, F f) {
    const int lane = threadIdx.x & 31;
    const int32_t size = 1 << shift;
    const bool head = unit < b.num_seqs;
    const int64_t w0 = static_cast<int64_t>(unit - b.num_seqs) << shift;
    // the first sequence whose rows end past w0 (offsets do not decrease; if
    // they do, the pieces found are some of the valid ones, and the unit of
    // the bad sequence records it)
    int32_t s0 = head ? unit : warp_search(b.num_seqs, [&](int32_t m) { return b.offsets[m + 1] > w0; });
    const int32_t s_end = head ? unit + 1 : b.num_seqs;
    for (; s0 < s_end; s0 += 32) {
        // a sequence a lane
        const int32_t s = s0 + lane;
        SeqRows r = {0, 0, 0};
        int64_t lo = 0;
        bool has = false, past = false;
        if (s < s_end) {
            past = !head && b.offsets[s] >= w0 + size;
            if (!past) r = read_seq(b, s, report && head);
            if (r.n > 0) {
                const int32_t first = r.len - r.n;  // position of row off
                lo = first;
                if (!head) {  // the least boundary past the first row's position with its row at w0 or later
                    const int64_t from = max(static_cast<int64_t>(first) + 1, first + (w0 - r.off));
                    lo = ((from + size - 1) >> shift) << shift;
                }
                has = lo < r.len && (head || r.off + (lo - first) < w0 + size);
            }
        }
        for (uint32_t left = __ballot_sync(0xffffffffu, has); left; left &= left - 1) {
            const int from = __ffs(left) - 1;
            SeqRows x;
            x.off = __shfl_sync(0xffffffffu, r.off, from);
            x.n = __shfl_sync(0xffffffffu, r.n, from);
            x.len = __shfl_sync(0xffffffffu, r.len, from);
            const int32_t p = __shfl_sync(0xffffffffu, static_cast<int32_t>(lo), from);
            f(s0 + from, x, p, static_cast<int32_t>(min(static_cast<int64_t>(x.len), ((static_cast<int64_t>(p) >> shift) + 1) << shift)));
        }
        if (__any_sync(0xffffffffu, past)) break;
    }
}

// ---------------------------------------------------------------- formats

// Two e4m3 codes (low byte first) to two f16, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(two));
    return r;
}

// The bytes of four e4m3 codes that are NaN: their top bits.
__device__ __forceinline__ uint32_t e4m3_nan(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// The same codes with 0 for NaN, where `nan` says so.
__device__ __forceinline__ uint32_t e4m3_without(uint32_t w, uint32_t nan) { return w & ~((nan >> 7) * 0xFFu); }

// Four codes to four f16 values (exactly), in order: lo holds codes 0 and 1.
// An int8 code c is (c + 128) + 1024 as an f16 whose low byte is c ^ 0x80,
// less 1152.
template <int FMT>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if (FMT == LORA_KV_INT8) {
        w ^= 0x80808080u;
        const uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
        const __half2 k = __half2half2(__ushort_as_half(0x6480));  // 1152
        const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&a), k);
        const __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&b), k);
        lo = *reinterpret_cast<const uint32_t *>(&x);
        hi = *reinterpret_cast<const uint32_t *>(&y);
    } else {
        lo = e4m3x2_to_f16x2(w & 0xFFFFu);
        hi = e4m3x2_to_f16x2(w >> 16);
    }
}

template <int FMT>
__device__ __forceinline__ void codes_to_float(uint32_t w, float *v) {
    uint32_t lo, hi;
    codes_to_f16<FMT>(w, lo, hi);
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
}

}  // namespace lora
