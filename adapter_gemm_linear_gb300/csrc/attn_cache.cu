// The 8-bit paged key/value cache: rows quantised into it (lora_kv_append)
// and read back (lora_kv_gather).
//
// Both are bound by memory: append reads a value once in its dtype and writes
// one byte, gather the other way round; a handful of operations a value.
//
// Append: one warp takes one 16-token tile of one (page, head) of K or V; the
// warps of a page share the page's largest magnitude through shared memory, and
// hold their rows as they were read until the scale is known (with heads of 128
// in 80 registers some of them in local memory: 140 bytes a thread in bf16, 500 in
// fp32).  Codes that are
// there already are only touched where the page's scale grows (or, in V's
// tiles, where they share a 16-byte piece with a new token).
// What bounds it is the chain of dependent reads (the sequence, its page, the
// rows), which as many warps as possible have to cover, and the instructions: 23
// a value and lane, of which an int8 code's rounding takes two fused
// multiply-adds, and magnitudes are compared two at a time.  8192 tokens of 8
// heads of 128 take 22 us (50 MB; 11.9 million instructions, 10 us of issue
// slots, 55% of them used), one token of each of 256 sequences 15.5 (50%).  With
// 128 registers a thread instead of 80: 24 and 16.4; with the rows read twice by
// rolled code that rounds with conversion instructions: 31.5 and 18.4.  In fp32, in
// a graph with the reading back, 54 us for 31.
#include <cuda_runtime.h>

#include "attn_device.cuh"
#include "attn_internal.h"

namespace lora {

namespace {

constexpr float kMinScale = 7.52316385e-37f;  // 2^-120: its reciprocal is finite

__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a < __int_as_float(0x7F800000) ? a : 0.0f;  // infinities and NaN do not count
}

// The least scale that holds magnitudes up to a.
template <int FMT>
__device__ __forceinline__ float scale_for(float a) {
    if (!(a > 0.0f)) return 0.0f;
    if (FMT == LORA_KV_INT8) return fmaxf(__fdiv_rn(a, 127.0f), kMinScale);
    // the least 2^e with a <= 448 * 2^e: a = m * 2^x, m in [1, 2), and 448 = 1.75 * 2^8
    const uint32_t bits = __float_as_uint(fmaxf(a, 448.0f * kMinScale));
    const int x = static_cast<int>(bits >> 23) - 127;
    const int e = x - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// s0 times the least power of two that makes it `least` at least (both normal, s0 below it).
__device__ __forceinline__ float doubled_to(float s0, float least) {
    const uint32_t a = __float_as_uint(s0), b = __float_as_uint(least);
    const float s = __uint_as_float((a & 0x7FFFFFu) | (b & 0x7F800000u));  // with the exponent of `least`
    return s < least ? 2.0f * s : s;
}

// Adding it rounds a float below 2^22 to an integer (ties to even), whose low
// byte is the sum's: one add where a rounding and a conversion instruction
// would take eight times as long each.
constexpr float kRound = 12582912.0f;  // 1.5 * 2^23

// The low bytes of four floats, in order.
__device__ __forceinline__ uint32_t low_bytes(const float (&t)[4]) {
    const uint32_t a = __byte_perm(__float_as_uint(t[0]), __float_as_uint(t[1]), 0x0040);
    const uint32_t b = __byte_perm(__float_as_uint(t[2]), __float_as_uint(t[3]), 0x0040);
    return __byte_perm(a, b, 0x5410);
}

__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Four values to int8 codes by the quotients themselves; NaN becomes 0.
__device__ __noinline__ uint32_t int8_codes_near(float4 x, float s) {
    float t[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float q = __fdiv_rn(t[i], s);
        t[i] = kRound + (q == q ? fminf(fmaxf(rintf(q), -127.0f), 127.0f) : 0.0f);
    }
    return low_bytes(t);
}

// Four values to four codes, low byte first; inv = 1/s, rounded.
template <int FMT>
__device__ __forceinline__ uint32_t encode4(const float (&x)[4], float s, float inv) {
    if (!(s > 0.0f)) return 0u;
    if (FMT == LORA_KV_INT8) {
        // x * inv is within 3e-5 of x / s for quotients up to 128, so the two
        // round alike unless the product lies nearer than that to a half; there
        // (and where x is not finite) the quotients decide
        float t[4];
        bool sure = true;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            t[i] = fmaf(x[i], inv, kRound);
            sure = sure && fabsf(fmaf(x[i], inv, kRound - t[i])) < 0.4999f;
        }
        if (!sure) return int8_codes_near(make_float4(x[0], x[1], x[2], x[3]), s);
        return low_bytes(t);
    }
    return e4m3_pair(x[0] * inv, x[1] * inv) | (e4m3_pair(x[2] * inv, x[3] * inv) << 16);
}

// Four older codes at a grown scale: code * ratio, rounded to a code.
template <int FMT>
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
    float v[4];
    codes_to_float<FMT>(w, v);
    if (FMT == LORA_KV_INT8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __fadd_rn(__fmul_rn(v[i], ratio), kRound);
        return low_bytes(v);
    }
    return e4m3_pair(v[0] * ratio, v[1] * ratio) | (e4m3_pair(v[2] * ratio, v[3] * ratio) << 16);
}

// A lane's piece as it was read: [four groups][four values].
template <typename T>
struct Raw;

template <>
struct Raw<__nv_bfloat16> {
    uint32_t w[4][2];
    __device__ __forceinline__ void load_row(int k, const __nv_bfloat16 *p) {
        const uint2 x = __ldg(reinterpret_cast<const uint2 *>(p));
        w[k][0] = x.x; w[k][1] = x.y;
    }
    __device__ __forceinline__ void load_all(const __nv_bfloat16 *p) {
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(p) + k / 2);
            w[k][0] = x.x; w[k][1] = x.y; w[k + 1][0] = x.z; w[k + 1][1] = x.w;
        }
    }
    __device__ __forceinline__ void clear(int k) { w[k][0] = w[k][1] = 0u; }
    __device__ __forceinline__ float value(int k, int e) const {
        return __uint_as_float(e & 1 ? w[k][e >> 1] & 0xFFFF0000u : w[k][e >> 1] << 16);
    }
    // the largest magnitude, infinities among them; NaN does not count
    __device__ __forceinline__ float largest() const {
        __nv_bfloat162 m = __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w[0][0]));
#pragma unroll
        for (int i = 1; i < 8; ++i) m = __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i >> 1][i & 1])));
        return fmaxf(__low2float(m), __high2float(m));
    }
};

template <>
struct Raw<float> {
    float4 w[4];
    __device__ __forceinline__ void load_row(int k, const float *p) { w[k] = __ldg(reinterpret_cast<const float4 *>(p)); }
    __device__ __forceinline__ void load_all(const float *p) {
#pragma unroll
        for (int k = 0; k < 4; ++k) load_row(k, p + 4 * k);
    }
    __device__ __forceinline__ void clear(int k) { w[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
    __device__ __forceinline__ float value(int k, int e) const { return e == 0 ? w[k].x : e == 1 ? w[k].y : e == 2 ? w[k].z : w[k].w; }
    __device__ __forceinline__ float largest() const {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(value(i >> 2, i & 3)));
        return m;
    }
};

// One page of one head, K or V: new tokens [lo, hi) (positions).  `tile` is the
// warp's 16-token tile of the page.  All threads of the page's warps call it
// together.  A lane's 16-byte piece of codes is 16 dimensions of a token (K),
// or four dimensions of a token quad (V), the lanes' pieces in memory order.
template <typename T, int D, int FMT, bool IS_V>
__device__ __forceinline__ void append_page(const KvView &b, const HeadsView &x, const SeqRows &r, int32_t page, int32_t head,
                                            int32_t lo, int32_t hi, int32_t tile, float *unit_amax, int32_t unit_warps,
                                            int lane) {
    constexpr int PIECES = kKvTile * D / 16 / 32;  // of a lane
    constexpr int TOKENS = IS_V ? 4 : 1;           // of a piece
    uint8_t *pages = IS_V ? b.v_pages : b.k_pages;
    float *scale_at = (IS_V ? b.v_scales : b.k_scales) + static_cast<int64_t>(page) * b.heads + head;
    uint4 *out = reinterpret_cast<uint4 *>(pages + tile_offset<D>(b, page, head, tile)) + lane;
    const int32_t p0 = lo & ~(b.page_tokens - 1);  // position of the page's first token
    const int32_t t0 = p0 + tile * kKvTile;        // and of the tile's
    const float old_s = lo > p0 ? *scale_at : 0.0f;
    // of position p: row r.off + p - (r.len - r.n)
    const T *src = static_cast<const T *>(x.p) + head * x.head + static_cast<int64_t>(r.off - (r.len - r.n)) * x.row;
    // the values of piece i, zero where the token is not new: groups of four
    // along the dimensions, of one token (K) or one of each of four (V)
    auto token = [&](int i) { return IS_V ? (lane & 3) * 4 : ((lane + 32 * i) >> 2) % kKvTile; };
    auto dim = [&](int i) { return IS_V ? ((lane + 32 * i) >> 2) * 4 : ((lane + 32 * i) >> 6) * 64 + (lane & 3) * 16; };
    auto load = [&](int i, Raw<T> &v) {
        const int32_t pos = t0 + token(i);
        const T *at = src + static_cast<int64_t>(pos) * x.row + dim(i);
#pragma unroll
        for (int k = 0; k < 4; ++k) v.clear(k);
        if (IS_V) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (pos + k >= lo && pos + k < hi) v.load_row(k, at + k * x.row);
        } else if (pos >= lo && pos < hi) {
            v.load_all(at);
        }
    };
    // tokens of piece i that are there already
    auto older_of = [&](int i) { return min(max(lo - (t0 + token(i)), 0), TOKENS); };
    Raw<T> v[PIECES];
    uint4 was[IS_V ? PIECES : 1];  // the codes beside which new ones go
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        if (IS_V && lo > t0) {
            const int32_t older = older_of(i);
            if (older > 0 && older < TOKENS) was[i] = out[32 * i];
        }
        load(i, v[i]);
    }
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) amax = fmaxf(amax, v[i].largest());
    if (__any_sync(0xffffffffu, amax == INFINITY)) {  // again, without the infinities
        amax = 0.0f;
#pragma unroll 1
        for (int i = 0; i < PIECES; ++i) {
            Raw<T> y;
            load(i, y);
#pragma unroll
            for (int e = 0; e < 16; ++e) amax = fmaxf(amax, finite_abs(y.value(e >> 2, e & 3)));
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (amax == 0.0f && t0 < hi && lo < t0 + kKvTile) {
        // new tokens without a finite value but zeros: an infinity or a NaN
        // among them needs a code, and so a scale, the least one (by way of the
        // least float, which leaves the scale alone wherever the page's other
        // tiles have a finite value)
        bool some = false;
#pragma unroll 1
        for (int i = 0; i < PIECES; ++i) {
            Raw<T> y;
            load(i, y);
#pragma unroll
            for (int e = 0; e < 16; ++e) some = some || !(fabsf(y.value(e >> 2, e & 3)) < INFINITY);
        }
        if (__any_sync(0xffffffffu, some)) amax = __uint_as_float(1u);
    }
    if (unit_warps > 1) {
        if (lane == 0) unit_amax[tile] = amax;
        __syncthreads();
        for (int32_t w = 0; w < unit_warps; ++w) amax = fmaxf(amax, unit_amax[w]);
        __syncthreads();
    }
    const float least = scale_for<FMT>(amax);
    float s = fmaxf(old_s, least);
    if (FMT == LORA_KV_INT8 && b.growth == LORA_KV_GROW_DOUBLING && old_s > 0.0f && least > old_s) s = doubled_to(old_s, least);
    const float inv = s > 0.0f ? __fdiv_rn(1.0f, s) : 0.0f;
    const float ratio = s > 0.0f ? __fdiv_rn(old_s, s) : 0.0f;
    __syncwarp();  // every lane has read the old scale
    if (tile == 0 && lane == 0) *scale_at = s;
    const bool grown = s != old_s;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const int32_t older = older_of(i);
        if (t0 + token(i) >= hi || older == TOKENS) continue;
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float y[4];  // V: four tokens side by side
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = IS_V ? v[i].value(e, k) : v[i].value(k, e);
            w[k] = encode4<FMT>(y, s, inv);
        }
        if (IS_V && older > 0) {
            const uint32_t ow[4] = {was[i].x, was[i].y, was[i].z, was[i].w};
            const uint32_t keep = (1u << (8 * older)) - 1u;
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = ((grown ? rescale4<FMT>(ow[k], ratio) : ow[k]) & keep) | (w[k] & ~keep);
        }
        out[32 * i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (grown && lo > t0) {  // the pieces of older tokens alone
#pragma unroll 1
        for (int i = 0; i < PIECES; ++i) {
            if (older_of(i) < TOKENS) continue;
            uint4 *at = out + 32 * i;
            const uint4 y = *at;
            *at = make_uint4(rescale4<FMT>(y.x, ratio), rescale4<FMT>(y.y, ratio), rescale4<FMT>(y.z, ratio),
                             rescale4<FMT>(y.w, ratio));
        }
    }
}

// Block: (warps of one page) x (pages, as many (head, K or V) of the same
// piece as fit four warps, eight for pages of 128).  grid.x: pieces of the
// new rows; grid.y: groups of (K or V, head).
template <typename T, int D, int FMT>
__global__ void __launch_bounds__(256, 3) kv_append_kernel(const __grid_constant__ KvView b,
                                                        const __grid_constant__ HeadsView k,
                                                        const __grid_constant__ HeadsView v) {
    __shared__ float amax[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t unit_warps = b.page_tokens / kKvTile;
    const int32_t per_block = static_cast<int32_t>(blockDim.x >> 5) / unit_warps;
    const int32_t u = warp / unit_warps, tile = warp % unit_warps;
    const int32_t hv = blockIdx.y * per_block + u;  // K heads, then V heads
    // threads past the last head stay for the block's barriers, without a page
    const bool has_head = hv < 2 * b.heads;
    const int32_t head = hv < b.heads ? hv : hv - b.heads;
    for_pieces(b, blockIdx.x, b.page_shift, blockIdx.y == 0 && threadIdx.x < 32,
               [&](int32_t s, const SeqRows &r, int32_t lo, int32_t hi) {
                   const int32_t page = read_page(b, s, lo >> b.page_shift);
                   if (page < 0) return;  // the same for every thread of the block
                   if (!has_head) {
                       if (unit_warps > 1) {
                           __syncthreads();
                           __syncthreads();
                       }
                       return;
                   }
                   float *const unit_amax = amax + u * unit_warps;
                   if (hv < b.heads) append_page<T, D, FMT, false>(b, k, r, page, head, lo, hi, tile, unit_amax, unit_warps, lane);
                   else append_page<T, D, FMT, true>(b, v, r, page, head, lo, hi, tile, unit_amax, unit_warps, lane);
               });
}

// ---------------------------------------------------------------- gather

__device__ __forceinline__ void store8(float *p, const float *v) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float *v) {
    __nv_bfloat162 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<uint4 *>(h);
}

// One warp per (16-token tile, head, K or V).  grid.x: pieces of the rows cut
// at multiples of 16 tokens; grid.y: groups of four (K or V, head).  Bound by
// memory: 262144 tokens of 8 heads of 128 as bf16, 1.6 GB, take 251 us (6.4 TB/s,
// 0.95 of a copy's rate); some 1000 tokens 5.1 us, the reads that depend on one
// another.  Eight blocks an SM, which bounds the registers, hide those.
template <typename T, int D, int FMT>
__global__ void __launch_bounds__(128, 8) kv_gather_kernel(const __grid_constant__ KvView b,
                                                        const __grid_constant__ HeadsView k,
                                                        const __grid_constant__ HeadsView v) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t hv = blockIdx.y * 4 + warp;
    if (hv >= 2 * b.heads) return;
    const bool is_v = hv >= b.heads;
    const int32_t head = is_v ? hv - b.heads : hv;
    const HeadsView &x = is_v ? v : k;
    for_pieces(b, blockIdx.x, 4, blockIdx.y == 0 && threadIdx.x < 32,
               [&](int32_t s, const SeqRows &r, int32_t lo, int32_t hi) {
        const int32_t page = read_page(b, s, lo >> b.page_shift);
        const int32_t t0 = lo & ~(kKvTile - 1);
        const int32_t tile = (t0 & (b.page_tokens - 1)) / kKvTile;
        const int64_t at = page < 0 ? 0 : tile_offset<D>(b, page, head, tile);
        const uint8_t *in = (is_v ? b.v_pages : b.k_pages) + at;
        const float scale = page < 0 ? 0.0f : (is_v ? b.v_scales : b.k_scales)[static_cast<int64_t>(page) * b.heads + head];
        T *dst = static_cast<T *>(x.p) + static_cast<int64_t>(r.off - (r.len - r.n)) * x.row + head * x.head;
        if (!is_v) {
            constexpr int N = kKvTile * D / 16 / 32;
            uint4 w[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int32_t c = lane + i * 32, t = c / (D / 16), d = c % (D / 16) * 16;
                w[i] = *reinterpret_cast<const uint4 *>(in + d / 64 * (kKvTile * 64) + t * 64 + d % 64);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int32_t c = lane + i * 32, t = c / (D / 16), d = c % (D / 16) * 16;
                const int32_t pos = t0 + t;
                if (pos < lo || pos >= hi) continue;
                float f[16];
                codes_to_float<FMT>(w[i].x, f);
                codes_to_float<FMT>(w[i].y, f + 4);
                codes_to_float<FMT>(w[i].z, f + 8);
                codes_to_float<FMT>(w[i].w, f + 12);
#pragma unroll
                for (int e = 0; e < 16; ++e) f[e] = page < 0 ? 0.0f : f[e] * scale;
                T *o = dst + static_cast<int64_t>(pos) * x.row + d;
                store8(o, f);
                store8(o + 8, f + 8);
            }
        } else {
            // lane = (8 dimensions, token quad): two 16-byte pieces, four tokens of 8 values
            uint4 w[D / 64][2];
#pragma unroll
            for (int i = 0; i < D / 64; ++i)
#pragma unroll
                for (int half = 0; half < 2; ++half)
                    w[i][half] = *reinterpret_cast<const uint4 *>(in + ((lane >> 2) * 2 + i * 16 + half) * 64 + (lane & 3) * 16);
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                float f[8][4];  // [dimension][token]
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    codes_to_float<FMT>(w[i][half].x, f[half * 4]);
                    codes_to_float<FMT>(w[i][half].y, f[half * 4 + 1]);
                    codes_to_float<FMT>(w[i][half].z, f[half * 4 + 2]);
                    codes_to_float<FMT>(w[i][half].w, f[half * 4 + 3]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int32_t pos = t0 + (lane & 3) * 4 + j;
                    if (pos < lo || pos >= hi) continue;
                    float o[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = page < 0 ? 0.0f : f[e][j] * scale;
                    store8(dst + static_cast<int64_t>(pos) * x.row + (lane >> 2) * 8 + i * 64, o);
                }
            }
        }
    });
}

// grid.x of the pieces of 2^shift tokens (for_pieces)
int64_t pieces(const KvView &v, int shift) {
    if (!v.offsets) return v.num_seqs;
    return static_cast<int64_t>(v.num_seqs) + ((static_cast<int64_t>(v.rows) + (1 << shift) - 1) >> shift);
}

template <typename T, int D, int FMT>
cudaError_t append_typed(const KvView &b, const HeadsView &k, const HeadsView &v, cudaStream_t stream) {
    const int unit_warps = b.page_tokens / kKvTile;
    const int warps = unit_warps > 4 ? unit_warps : 4;
    const int per_block = warps / unit_warps;
    const dim3 grid(static_cast<unsigned>(pieces(b, b.page_shift)), (2 * b.heads + per_block - 1) / per_block);
    kv_append_kernel<T, D, FMT><<<grid, warps * 32, 0, stream>>>(b, k, v);
    count_launches(1);
    return cudaGetLastError();
}

template <typename T, int D, int FMT>
cudaError_t gather_typed(const KvView &b, const HeadsView &k, const HeadsView &v, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(pieces(b, 4)), (2 * b.heads + 3) / 4);
    kv_gather_kernel<T, D, FMT><<<grid, 128, 0, stream>>>(b, k, v);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

#define LORA_KV_DISPATCH(FN)                                                                              \
    if (dtype == LORA_FP32) {                                                                             \
        if (head_dim == 64)                                                                               \
            return fmt == LORA_KV_INT8 ? FN<float, 64, LORA_KV_INT8>(b, k, v, stream)                     \
                                       : FN<float, 64, LORA_KV_E4M3>(b, k, v, stream);                    \
        return fmt == LORA_KV_INT8 ? FN<float, 128, LORA_KV_INT8>(b, k, v, stream)                        \
                                   : FN<float, 128, LORA_KV_E4M3>(b, k, v, stream);                       \
    }                                                                                                     \
    if (head_dim == 64)                                                                                   \
        return fmt == LORA_KV_INT8 ? FN<__nv_bfloat16, 64, LORA_KV_INT8>(b, k, v, stream)                 \
                                   : FN<__nv_bfloat16, 64, LORA_KV_E4M3>(b, k, v, stream);                \
    return fmt == LORA_KV_INT8 ? FN<__nv_bfloat16, 128, LORA_KV_INT8>(b, k, v, stream)                    \
                               : FN<__nv_bfloat16, 128, LORA_KV_E4M3>(b, k, v, stream);

cudaError_t launch_kv_append(const KvView &b, lora_kv_format_t fmt, int head_dim, lora_dtype_t dtype,
                             const HeadsView &k, const HeadsView &v, cudaStream_t stream) {
    LORA_KV_DISPATCH(append_typed)
}

cudaError_t launch_kv_gather(const KvView &b, lora_kv_format_t fmt, int head_dim, lora_dtype_t dtype,
                             const HeadsView &k, const HeadsView &v, cudaStream_t stream) {
    LORA_KV_DISPATCH(gather_typed)
}

}  // namespace lora
