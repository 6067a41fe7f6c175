// What the attention kernels for few queries a sequence share (attn_decode.cu,
// attn_decode4.cu): the warp's matrix instructions, and a CTA's walk over its part
// of the line of work.
#pragma once

#include <cuda_fp16.h>

#include "attn_device.cuh"
#include "attn_split.cuh"

namespace lora {

constexpr int kChunkTiles = 8;                     // tiles of a unit of work (128 tokens)
constexpr int kSlotRows = 16;                      // rows a partial result has place for
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr float kLoScale = 2048.0f;                // 2^11: the lo parts of fp32 operands
constexpr int kBatch = 32, kBatches = 8;  // tiles looked up at once, and ahead

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

// An 8 x 8 matrix of f16 (a thread: row lane / 4, columns 2 (lane % 4) and the next) transposed.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// A sequence's work: `items` items (heads x row_tiles) of `chunks` units each, over tiles [t0, t1).
struct SeqWork {
    SeqRows r;
    int32_t t0, t1, chunks, row_tiles;
    long long items;
};

template <int ROWS>
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
        w.row_tiles = (w.r.n * a.group + ROWS - 1) / ROWS;
    }
    w.items = static_cast<long long>(w.row_tiles) * a.kv.heads;
    return w;
}

// The units that a CTA takes of the line: [w0, w1) of `total`, which `ctas` CTAs share.
// Every item has `extra` units more than chunks, in front: what beginning and ending it costs.
struct Range {
    long long w0, w1, total, ctas;
    int32_t extra;
};

// One CTA's walk over its units: item by item, those of which it has chunks.
template <int ROWS>
struct Walk {
    const AttnView &a;
    long long w, end, base;
    int32_t s, extra;
    SeqWork work;
    // the current item
    int32_t head, row_tile, tile0, tile1;  // tiles of this CTA
    bool from_start, to_end;               // whether the item begins / ends in this CTA
    long long item_end;                    // unit after the item's last

    __device__ __forceinline__ Walk(const AttnView &v, const Range &range, int32_t seq, long long seq_base)
        : a(v), w(range.w0), end(range.w1), base(seq_base), s(seq), extra(range.extra) {
        if (w < end) work = seq_work<ROWS>(a, s);
    }

    __device__ __forceinline__ bool next() {
        while (w < end) {
            while (w >= base + work.items * (work.chunks + extra)) {
                base += work.items * (work.chunks + extra);
                work = seq_work<ROWS>(a, ++s);
            }
            const int32_t units = work.chunks + extra;
            const long long local = w - base;
            const long long item = local / units;
            const int32_t u = static_cast<int32_t>(local - item * units);
            head = static_cast<int32_t>(item / work.row_tiles);
            row_tile = static_cast<int32_t>(item - static_cast<long long>(head) * work.row_tiles);
            const int32_t u1 = static_cast<int32_t>(min(static_cast<long long>(units), u + (end - w)));
            const int32_t c = max(u - extra, 0);
            tile0 = work.t0 + c * kChunkTiles;
            tile1 = min(work.t1, work.t0 + (u1 - extra) * kChunkTiles);
            from_start = c == 0;
            to_end = u1 == units;
            item_end = base + (item + 1) * units;
            w += u1 - u;
            if (u1 > extra) return true;
        }
        return false;
    }
};

// The plan: where this CTA's range begins, by all of its threads (two barriers; what
// they wrote to shared memory before is there for all after).  `seq` and `base` (shared
// memory) become the sequence that it begins in and that sequence's first unit.  Items
// have EXTRA more units where there are more chunks than CTAs.
template <int ROWS, int THREADS, int EXTRA>
__device__ __forceinline__ Range plan_line(const AttnView &a, long long (*warp_sum)[2], int32_t *seq, long long *base) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t per = (a.kv.num_seqs + THREADS - 1) / THREADS;
    const int32_t s0 = min(a.kv.num_seqs, static_cast<int32_t>(threadIdx.x) * per), s1 = min(a.kv.num_seqs, s0 + per);
    long long chunks = 0, items = 0;
    for (int32_t s = s0; s < s1; ++s) {
        const SeqWork w = seq_work<ROWS>(a, s);
        chunks += w.items * w.chunks;
        items += w.items;
    }
    long long c_upto = chunks, i_upto = items;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long c = __shfl_up_sync(0xffffffffu, c_upto, o), i = EXTRA ? __shfl_up_sync(0xffffffffu, i_upto, o) : 0;
        if (lane >= o) {
            c_upto += c;
            i_upto += i;
        }
    }
    if (lane == 31) {
        warp_sum[warp][0] = c_upto;
        warp_sum[warp][1] = i_upto;
    }
    __syncthreads();
    long long c_total = 0, i_total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) {
            c_upto += warp_sum[w][0];
            i_upto += warp_sum[w][1];
        }
        c_total += warp_sum[w][0];
        i_total += warp_sum[w][1];
    }
    Range r;
    r.extra = EXTRA && c_total > static_cast<long long>(gridDim.x) ? EXTRA : 0;
    r.total = c_total + r.extra * i_total;
    const long long upto = c_upto + r.extra * i_upto, mine = chunks + r.extra * items;
    // as many CTAs as there are units at most, so that none between two of an item is without work
    r.ctas = min(r.total, static_cast<long long>(gridDim.x));
    r.w0 = blockIdx.x < r.ctas ? r.total * blockIdx.x / r.ctas : 0;
    r.w1 = blockIdx.x < r.ctas ? r.total * (blockIdx.x + 1) / r.ctas : 0;
    if (r.w0 < r.w1 && upto - mine <= r.w0 && r.w0 < upto) {
        long long at = upto - mine;
        int32_t s = s0;
        for (;; ++s) {
            const SeqWork w = seq_work<ROWS>(a, s);
            const long long u = w.items * (w.chunks + r.extra);
            if (r.w0 < at + u) break;
            at += u;
        }
        *seq = s;
        *base = at;
    }
    __syncthreads();
    return r;
}

}  // namespace lora
