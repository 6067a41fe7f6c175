// The 8-bit paged key/value cache: rows quantised into it (lora_kv_append)
// and read back (lora_kv_gather).
//
// Both are bound by memory: append reads a value once in its dtype and writes
// one byte, gather the other way round; a handful of operations a value.
//
// Append: one warp takes one 16-token tile of one (page, head) of K or V; the
// warps of a page share the page's largest magnitude through shared memory.
// The rows are read twice, for the magnitude and for the codes, the second
// time from the L1.  The code is kept short and rolled: a warp runs it once,
// and with everything unrolled and held in registers fetching instructions
// took most of 65 us for 8192 tokens of 8 heads (now TIMEAPPEND).  Codes that
// are there already are only touched where the page's scale grows (or, in
// V's tiles, where they share a 16-byte piece with a new token).
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

// x / s rounded to the nearest code, as int8 bits.  x * inv (inv = 1/s
// rounded) is within 3e-5 of x / s for quotients up to 128, so the two round
// alike unless the product lies nearer than that to a half; there the
// quotient itself decides.
__device__ __forceinline__ int32_t int8_code(float x, float s, float inv) {
    const float y = x * inv;
    if (!(y == y)) return 0;
    float r = rintf(y);
    if (fabsf(fabsf(y - r) - 0.5f) < 1e-4f) r = rintf(__fdiv_rn(x, s));
    return static_cast<int32_t>(fminf(fmaxf(r, -127.0f), 127.0f));
}

__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Four values to four codes, low byte first.
template <int FMT>
__device__ __forceinline__ uint32_t encode4(const float *x, float s, float inv) {
    if (!(s > 0.0f)) return 0u;
    if (FMT == LORA_KV_INT8) {
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) w |= (static_cast<uint32_t>(int8_code(x[i], s, inv)) & 0xFFu) << (8 * i);
        return w;
    }
    return e4m3_pair(x[0] * inv, x[1] * inv) | (e4m3_pair(x[2] * inv, x[3] * inv) << 16);
}

// Four older codes at a grown scale: code * ratio, rounded to a code.
template <int FMT>
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
    float v[4];
    codes_to_float<FMT>(w, v);
    if (FMT == LORA_KV_INT8) {
        uint32_t r = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r |= (static_cast<uint32_t>(static_cast<int32_t>(rintf(v[i] * ratio))) & 0xFFu) << (8 * i);
        return r;
    }
    return e4m3_pair(v[0] * ratio, v[1] * ratio) | (e4m3_pair(v[2] * ratio, v[3] * ratio) << 16);
}

// Four values.
__device__ __forceinline__ void load4(const __nv_bfloat16 *p, float *v) {
    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(p));
    v[0] = __uint_as_float(w.x << 16);
    v[1] = __uint_as_float(w.x & 0xFFFF0000u);
    v[2] = __uint_as_float(w.y << 16);
    v[3] = __uint_as_float(w.y & 0xFFFF0000u);
}
__device__ __forceinline__ void load4(const float *p, float *v) {
    const float4 w = __ldg(reinterpret_cast<const float4 *>(p));
    v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
}

// One page of one head, K or V: new tokens [lo, hi) (positions).  `tile` is the
// warp's 16-token tile of the page.  All threads of the page's warps call it
// together.  A lane's 16-byte piece of codes is 16 dimensions of a token (K),
// or four dimensions of a token quad (V), the lanes' pieces in memory order.
template <typename T, int D, int FMT>
__device__ __forceinline__ void append_page(const KvView &b, const HeadsView &x, bool is_v, const SeqRows &r, int32_t page,
                                            int32_t head, int32_t lo, int32_t hi, int32_t tile, float *unit_amax,
                                            int32_t unit_warps, int lane) {
    constexpr int PIECES = kKvTile * D / 16 / 32;  // of a lane
    uint8_t *pages = is_v ? b.v_pages : b.k_pages;
    float *scale_at = (is_v ? b.v_scales : b.k_scales) + static_cast<int64_t>(page) * b.heads + head;
    const int32_t p0 = lo & ~(b.page_tokens - 1);  // position of the page's first token
    const int32_t t0 = p0 + tile * kKvTile;        // and of the tile's
    const float old_s = lo > p0 ? *scale_at : 0.0f;
    // of position p: row r.off + p - (r.len - r.n)
    const T *src = static_cast<const T *>(x.p) + head * x.head + static_cast<int64_t>(r.off - (r.len - r.n)) * x.row;
    // the values of piece i, zero where the token is not new: groups of four
    // along the dimensions, of one token (K) or one of each of four (V)
    auto token = [&](int i) { return is_v ? (lane & 3) * 4 : ((lane + 32 * i) >> 2) % kKvTile; };
    auto dim = [&](int i) { return is_v ? ((lane + 32 * i) >> 2) * 4 : ((lane + 32 * i) >> 6) * 64 + (lane & 3) * 16; };
    auto load = [&](int i, float (&v)[4][4]) {
        const int32_t pos = t0 + token(i), d = dim(i);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int32_t p = is_v ? pos + k : pos;
            v[k][0] = v[k][1] = v[k][2] = v[k][3] = 0.0f;
            if (p >= lo && p < hi) load4(src + static_cast<int64_t>(p) * x.row + d + (is_v ? 0 : 4 * k), v[k]);
        }
    };
    float amax = 0.0f;
#pragma unroll 2
    for (int i = 0; i < PIECES; ++i) {
        float v[4][4];
        load(i, v);
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) amax = fmaxf(amax, finite_abs(v[k][e]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (unit_warps > 1) {
        if (lane == 0) unit_amax[tile] = amax;
        __syncthreads();
        for (int32_t w = 0; w < unit_warps; ++w) amax = fmaxf(amax, unit_amax[w]);
        __syncthreads();
    }
    const float s = fmaxf(old_s, scale_for<FMT>(amax));
    const float inv = s > 0.0f ? __fdiv_rn(1.0f, s) : 0.0f;
    const float ratio = s > 0.0f ? __fdiv_rn(old_s, s) : 0.0f;
    __syncwarp();  // every lane has read the old scale
    if (tile == 0 && lane == 0) *scale_at = s;
    const bool grown = s != old_s;
    uint4 *out = reinterpret_cast<uint4 *>(pages + tile_offset<D>(b, page, head, tile));
#pragma unroll 1
    for (int i = 0; i < PIECES; ++i) {
        const int32_t pos = t0 + token(i), tokens = is_v ? 4 : 1;
        const int32_t older = min(max(lo - pos, 0), tokens);  // of the piece's tokens
        if (pos >= hi || (older == tokens && !grown)) continue;
        float v[4][4];
        load(i, v);
        if (is_v) {  // codes of four tokens side by side
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int e = 0; e < k; ++e) {
                    const float t = v[k][e];
                    v[k][e] = v[e][k];
                    v[e][k] = t;
                }
        }
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = encode4<FMT>(v[k], s, inv);
        uint4 *at = out + lane + 32 * i;
        if (older > 0) {
            const uint4 was = *at;
            const uint32_t ow[4] = {was.x, was.y, was.z, was.w};
            const uint32_t keep = older == tokens ? 0xFFFFFFFFu : (1u << (8 * older)) - 1u;
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = ((grown ? rescale4<FMT>(ow[k], ratio) : ow[k]) & keep) | (w[k] & ~keep);
        }
        *at = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Block: (warps of one page) x (pages, as many (head, K or V) of the same
// piece as fit four warps, eight for pages of 128).  grid.x: pieces of the
// new rows; grid.y: groups of (K or V, head).
template <typename T, int D, int FMT>
__global__ void __launch_bounds__(256) kv_append_kernel(const __grid_constant__ KvView b,
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
                   append_page<T, D, FMT>(b, hv < b.heads ? k : v, hv >= b.heads, r, page, head, lo, hi, tile,
                                          amax + u * unit_warps, unit_warps, lane);
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
// at multiples of 16 tokens; grid.y: groups of four (K or V, head).
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
