// The 4-bit paged key/value cache (LORA_KV_UINT4): rows quantised into it
// (lora_kv_append) and read back (lora_kv_gather).
//
// Each 64 dimensions of a token and head have a scale s and a least value m of
// their own, value = s code + m, so a token is written without a look at the
// page's older ones; and a token's share of each 16-byte piece is whole bytes, so
// that nothing is read before it is written.  One warp takes one 16-token tile of
// one head, K or V, its lanes the pieces (attn_uint4.cuh).
// Both are bound by memory in principle (a value read in its dtype, half a byte and
// 1/16 byte of scales written, or the other way round).
#include <cuda_runtime.h>

#include "attn_uint4.cuh"

namespace lora {

namespace {

constexpr float kLargest = 32768.0f;   // magnitudes held
constexpr float kRound = 12582912.0f;  // 1.5 * 2^23: adding it rounds a float below 2^22 to an integer, ties to even

// N values as they are read, in fp32.
template <int N>
__device__ __forceinline__ void load_values(const __nv_bfloat16 *p, float *v) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        uint2 x;
        if (N >= 8) {
            if (i % 8) continue;
            const uint4 y = __ldg(reinterpret_cast<const uint4 *>(p + i));
            const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[i + 2 * k] = __uint_as_float(w[k] << 16);
                v[i + 2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
            }
        } else {
            x = __ldg(reinterpret_cast<const uint2 *>(p + i));
            v[i] = __uint_as_float(x.x << 16); v[i + 1] = __uint_as_float(x.x & 0xFFFF0000u);
            v[i + 2] = __uint_as_float(x.y << 16); v[i + 3] = __uint_as_float(x.y & 0xFFFF0000u);
        }
    }
}
template <int N>
__device__ __forceinline__ void load_values(const float *p, float *v) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const float4 x = __ldg(reinterpret_cast<const float4 *>(p + i));
        v[i] = x.x; v[i + 1] = x.y; v[i + 2] = x.z; v[i + 3] = x.w;
    }
}

// Least and largest of N values (+inf and -inf where none counts): NaN is turned into
// 0, what is beyond kLargest cut; infinities stay, and do not count.
template <int N>
__device__ __forceinline__ void bounds(float *v, float &lo, float &hi) {
    uint32_t most = 0;
    lo = INFINITY;
    hi = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        most = max(most, __float_as_uint(v[i]) & 0x7FFFFFFFu);
        lo = fminf(lo, v[i]);
        hi = fmaxf(hi, v[i]);
    }
    if (__builtin_expect(most > __float_as_uint(kLargest), 0)) {
        lo = INFINITY;
        hi = -INFINITY;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (!(v[i] == v[i])) v[i] = 0.0f;
            if (fabsf(v[i]) == INFINITY) continue;
            v[i] = fminf(fmaxf(v[i], -kLargest), kLargest);
            lo = fminf(lo, v[i]);
            hi = fmaxf(hi, v[i]);
        }
    }
}

struct Scale {
    __half2 stored;  // (scale, least)
    float s, m, inv;

    __device__ __forceinline__ Scale(float lo, float hi) {
        if (!(lo <= hi)) lo = hi = 0.0f;  // no finite value
        stored = __halves2half2(__float2half_rn((hi - lo) * (1.0f / 15.0f)), __float2half_rn(lo));
        s = __low2float(stored);
        m = __high2float(stored);
        inv = s > 0.0f ? __fdiv_rn(1.0f, s) : 0.0f;
    }
    // A value's code, as the low bits of a float that is kRound + code.
    __device__ __forceinline__ uint32_t code(float x) const {
        const float d = x - m;
        // d * inv is within 2e-6 of d / s where it is below 15, so both round
        // alike unless it lies nearer than that to a half: there the quotient decides
        float t = fminf(fmaxf(d * inv, 0.0f), 15.0f);
        float r = t + kRound;
        if (__builtin_expect(fabsf(t - (r - kRound)) > 0.4999f, 0)) r = fminf(fmaxf(rintf(__fdiv_rn(d, s)), 0.0f), 15.0f) + kRound;
        return s > 0.0f ? __float_as_uint(r) : __float_as_uint(kRound);
    }
};

// Codes into nibbles: sums of (kRound + code) << shift, less what the kRound make.
struct Word {
    uint32_t sum = 0, less = 0;
    __device__ __forceinline__ void add(uint32_t code, int nibble) {
        sum += code << (4 * nibble);
        less += __float_as_uint(kRound) << (4 * nibble);
    }
    __device__ __forceinline__ uint32_t bits() const { return sum - less; }
};

// A warp's tile of K: new tokens [lo, hi) (positions) of the tile that begins at t0.
template <typename T, int D>
__device__ __forceinline__ void append_k(const T *src, int64_t row, uint8_t *codes, __half2 *scales, int32_t t0, int32_t lo, int32_t hi,
                                         int lane) {
    const int g = lane >> 2, q = lane & 3;
#pragma unroll
    for (int h = 0; h < D / kBlockDims; ++h) {
        uint32_t w[2][2];
        bool fresh[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int t = k_token(g) + 2 * k;
            const int32_t pos = t0 + t;
            fresh[k] = pos >= lo && pos < hi;
            float v[16], a, z;
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = 0.0f;
            if (fresh[k]) load_values<16>(src + static_cast<int64_t>(pos) * row + h * kBlockDims + 16 * q, v);
            bounds<16>(v, a, z);
#pragma unroll
            for (int o = 1; o < 4; o *= 2) {
                a = fminf(a, __shfl_xor_sync(0xffffffffu, a, o));
                z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, o));
            }
            const Scale s(a, z);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                Word x;
#pragma unroll
                for (int e = 0; e < 8; ++e) x.add(s.code(v[8 * j + e]), (e >> 1) + 4 * (e & 1));
                w[k][j] = x.bits();
            }
            if (q == 0 && fresh[k]) scales[h * kKvTile + t] = s.stored;
        }
        uint4 *at = reinterpret_cast<uint4 *>(codes + h * kBlockBytes) + lane;
        if (fresh[0] && fresh[1]) *at = make_uint4(w[0][0], w[0][1], w[1][0], w[1][1]);
        else if (fresh[0]) reinterpret_cast<uint2 *>(at)[0] = make_uint2(w[0][0], w[0][1]);
        else if (fresh[1]) reinterpret_cast<uint2 *>(at)[1] = make_uint2(w[1][0], w[1][1]);
    }
}

template <typename T, int D>
__device__ __forceinline__ void append_v(const T *src, int64_t row, uint8_t *codes, __half2 *scales, int32_t t0, int32_t lo, int32_t hi,
                                         int lane) {
    const int g = lane >> 2, q = lane & 3;
    const int32_t first = t0 + 4 * q;
#pragma unroll
    for (int h = 0; h < D / kBlockDims; ++h) {
        Word w[4];
        __half2 stored[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const bool fresh = first + t >= lo && first + t < hi;
            float v[8], a, z;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0.0f;
            const T *p = src + static_cast<int64_t>(first + t) * row + h * kBlockDims + 4 * g;
            if (fresh) {
                load_values<4>(p, v);
                load_values<4>(p + 32, v + 4);
            }
            bounds<8>(v, a, z);
#pragma unroll
            for (int o = 4; o < 32; o *= 2) {
                a = fminf(a, __shfl_xor_sync(0xffffffffu, a, o));
                z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, o));
            }
            const Scale s(a, z);
            stored[t] = s.stored;
            constexpr int kByte[4] = {0, 2, 1, 3};
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e >> 1].add(s.code(v[e]), 2 * kByte[t] + (e & 1));
        }
        uint8_t *at = codes + h * kBlockBytes + lane * 16;
        __half2 *sc = scales + h * kKvTile + 4 * q;
        if (first >= lo && first + 4 <= hi) {
            *reinterpret_cast<uint4 *>(at) = make_uint4(w[0].bits(), w[1].bits(), w[2].bits(), w[3].bits());
            if (g == 0) *reinterpret_cast<uint4 *>(sc) = *reinterpret_cast<const uint4 *>(stored);
        } else {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                if (first + t < lo || first + t >= hi) continue;
                const int byte = t == 1 ? 2 : t == 2 ? 1 : t;
#pragma unroll
                for (int j = 0; j < 4; ++j) at[4 * j + byte] = static_cast<uint8_t>(w[j].bits() >> (8 * byte));
                if (g == 0) sc[t] = stored[t];
            }
        }
    }
}

// grid.x: pieces of the rows cut at multiples of 16 tokens; grid.y: groups of four (K or V, head).
template <typename T, int D>
__global__ void __launch_bounds__(128) kv_append4_kernel(const __grid_constant__ KvView b, const __grid_constant__ HeadsView k,
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
        if (page < 0) return;
        const int32_t t0 = lo & ~(kKvTile - 1);
        const int64_t tile = tile_index(b, page, head, (t0 & (b.page_tokens - 1)) / kKvTile);
        uint8_t *codes = (is_v ? b.v_pages : b.k_pages) + tile * (D / kBlockDims * kBlockBytes);
        __half2 *scales = reinterpret_cast<__half2 *>(is_v ? b.v_scales : b.k_scales) + tile * (D / kBlockDims * kKvTile);
        // of position p: row r.off + p - (r.len - r.n)
        const T *src = static_cast<const T *>(x.p) + head * x.head + static_cast<int64_t>(r.off - (r.len - r.n)) * x.row;
        if (is_v) append_v<T, D>(src, x.row, codes, scales, t0, lo, hi, lane);
        else append_k<T, D>(src, x.row, codes, scales, t0, lo, hi, lane);
    });
}

// ---------------------------------------------------------------- gather

template <int N>
__device__ __forceinline__ void store_values(float *p, const float *v) {
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<float4 *>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}
template <int N>
__device__ __forceinline__ void store_values(__nv_bfloat16 *p, const float *v) {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    if constexpr (N >= 8) {
#pragma unroll
        for (int i = 0; i < N / 2; i += 4) reinterpret_cast<uint4 *>(p)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    } else {
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(128, 8) kv_gather4_kernel(const __grid_constant__ KvView b, const __grid_constant__ HeadsView k,
                                                            const __grid_constant__ HeadsView v) {
    constexpr int H = D / kBlockDims;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int32_t hv = blockIdx.y * 4 + warp;
    if (hv >= 2 * b.heads) return;
    const bool is_v = hv >= b.heads;
    const int32_t head = is_v ? hv - b.heads : hv;
    const HeadsView &x = is_v ? v : k;
    for_pieces(b, blockIdx.x, 4, blockIdx.y == 0 && threadIdx.x < 32,
               [&](int32_t s, const SeqRows &r, int32_t lo, int32_t hi) {
        const int32_t page = read_page(b, s, lo >> b.page_shift);
        const int32_t t0 = lo & ~(kKvTile - 1);
        const int64_t tile = page < 0 ? 0 : tile_index(b, page, head, (t0 & (b.page_tokens - 1)) / kKvTile);
        const uint4 *codes = reinterpret_cast<const uint4 *>((is_v ? b.v_pages : b.k_pages) + tile * (H * kBlockBytes)) + lane;
        const __half2 *scales = reinterpret_cast<const __half2 *>(is_v ? b.v_scales : b.k_scales) + tile * (H * kKvTile);
        T *dst = static_cast<T *>(x.p) + static_cast<int64_t>(r.off - (r.len - r.n)) * x.row + head * x.head;
        uint4 c[H];
        float2 sc[H][4];  // of K's two tokens, or V's four
#pragma unroll
        for (int h = 0; h < H; ++h) {
            c[h] = codes[h * 32];
            if (is_v) {
                const uint4 y = *reinterpret_cast<const uint4 *>(scales + h * kKvTile + 4 * q);
                sc[h][0] = f16_pair(y.x); sc[h][1] = f16_pair(y.y); sc[h][2] = f16_pair(y.z); sc[h][3] = f16_pair(y.w);
            } else {
                sc[h][0] = __half22float2(scales[h * kKvTile + k_token(g)]);
                sc[h][1] = __half22float2(scales[h * kKvTile + k_token(g) + 2]);
            }
        }
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const uint32_t w[4] = {c[h].x, c[h].y, c[h].z, c[h].w};
            // (a table entry out of range reads as zeros)
            auto value = [&](float code, float unit, const float2 &s) { return page < 0 ? 0.0f : fmaf(code, s.x * unit, s.y); };
            if (!is_v) {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int32_t pos = t0 + k_token(g) + 2 * t;
                    float o[16];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t f[4];
                        nibble_pairs(w[2 * t + j], f);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 y = f16_pair(f[i]);
                            o[8 * j + 2 * i] = value(y.x, i & 1 ? kCode1 : kCode0, sc[h][t]);
                            o[8 * j + 2 * i + 1] = value(y.y, i & 1 ? kCode1 : kCode0, sc[h][t]);
                        }
                    }
                    if (pos >= lo && pos < hi) store_values<16>(dst + static_cast<int64_t>(pos) * x.row + h * kBlockDims + 16 * q, o);
                }
            } else {
                float o[4][2][4];  // [token][half of the 64][dimension]
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t f[4];
                    nibble_pairs(w[j], f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {  // tokens 2 (i / 2) and the next, dimension i % 2 of the word
                        const float2 y = f16_pair(f[i]);
                        const int t = i & 2, d = 2 * (j & 1) + (i & 1);
                        o[t][j >> 1][d] = value(y.x, i & 1 ? kCode1 : kCode0, sc[h][t]);
                        o[t + 1][j >> 1][d] = value(y.y, i & 1 ? kCode1 : kCode0, sc[h][t + 1]);
                    }
                }
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const int32_t pos = t0 + 4 * q + t;
                    if (pos < lo || pos >= hi) continue;
                    T *to = dst + static_cast<int64_t>(pos) * x.row + h * kBlockDims + 4 * g;
                    store_values<4>(to, o[t][0]);
                    store_values<4>(to + 32, o[t][1]);
                }
            }
        }
    });
}

dim3 pieces_grid(const KvView &b) {
    const int64_t n = !b.offsets ? b.num_seqs : static_cast<int64_t>(b.num_seqs) + (static_cast<int64_t>(b.rows) + kKvTile - 1) / kKvTile;
    return dim3(static_cast<unsigned>(n), (2 * b.heads + 3) / 4);
}

}  // namespace

cudaError_t launch_kv_append4(const KvView &b, int head_dim, lora_dtype_t dtype, const HeadsView &k, const HeadsView &v,
                              cudaStream_t stream) {
    auto *kernel = dtype == LORA_FP32 ? (head_dim == 64 ? kv_append4_kernel<float, 64> : kv_append4_kernel<float, 128>)
                                      : (head_dim == 64 ? kv_append4_kernel<__nv_bfloat16, 64> : kv_append4_kernel<__nv_bfloat16, 128>);
    kernel<<<pieces_grid(b), 128, 0, stream>>>(b, k, v);
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_kv_gather4(const KvView &b, int head_dim, lora_dtype_t dtype, const HeadsView &k, const HeadsView &v,
                              cudaStream_t stream) {
    auto *kernel = dtype == LORA_FP32 ? (head_dim == 64 ? kv_gather4_kernel<float, 64> : kv_gather4_kernel<float, 128>)
                                      : (head_dim == 64 ? kv_gather4_kernel<__nv_bfloat16, 64> : kv_gather4_kernel<__nv_bfloat16, 128>);
    kernel<<<pieces_grid(b), 128, 0, stream>>>(b, k, v);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace lora
