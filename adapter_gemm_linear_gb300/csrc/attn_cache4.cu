// The 4-bit paged key/value cache (LORA_KV_UINT4): rows quantised into it
// (lora_kv_append) and read back (lora_kv_gather).
//
// Each 64 dimensions of a token and head have a scale s and a least value m of
// their own, value = s code + m, so a token is written without a look at the
// page's older ones; and a token's share of each 16-byte piece is whole bytes, so
// that nothing is read before it is written.  One warp takes one 16-token tile of
// one head, K or V, its lanes the pieces (attn_uint4.cuh).
// By their bytes both are bound by memory (a value read in its dtype, half a byte and 1/16
// byte of scales written, or the other way round).  Measured, 8 heads of 128, bf16: 262144 tokens
// read back in 214 us (6.4 TB/s, 0.95 of a copy); 8192 tokens of 16 prompts written in 18.4 and read
// back in 12 (24.6 together in a graph), one of each of 256 sequences in 9.4 and 8.5 (12.0).
// (These one by one under a profiler, from a cold L2; in a graph, segments of 512, 14.6 and 9.0, in fp32 18.6
// and 14.0; a token of 256 sequences 6.0 and 4.3, in fp32 6.7 and 4.8; 65536 tokens of 64 sequences 116 and
// 57, in fp32 141 and 99.)  Of the
// write 60% of the issue slots are used, by 25 warps an SM: 22 instructions for a value and
// lane; the rest is reads that wait for each other (sequence, page, row).
#include <cuda_runtime.h>

#include "attn_uint4.cuh"
#include "f32x2.cuh"
#include "sm100_ptx.cuh"

namespace lora {

namespace {

constexpr float kLargest = 32768.0f;   // magnitudes held
constexpr float kRound = 12582912.0f;  // 1.5 * 2^23: adding it rounds a float below 2^22 to an integer, ties to even

// Least and largest of values, NaN if one of them is.
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// N values as they are read.
template <typename T, int N>
struct Raw {
    static constexpr int kWords = N * static_cast<int>(sizeof(T)) / 4;
    uint32_t w[kWords];

    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < kWords; i += 4) {
            const uint4 y = __ldg(reinterpret_cast<const uint4 *>(p) + i / 4);
            w[i] = y.x; w[i + 1] = y.y; w[i + 2] = y.z; w[i + 3] = y.w;
        }
    }
    // as pairs in fp32, and the least and the largest of them (NaN if one of them is)
    __device__ __forceinline__ void values(F2 (&v)[N / 2], float &lo, float &hi) const {
        if constexpr (sizeof(T) == 2) {
            __nv_bfloat162 l, h;
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162 *>(&w[i]);
                l = i == 0 ? x : __hmin2_nan(l, x);
                h = i == 0 ? x : __hmax2_nan(h, x);
                v[i] = two(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
            }
            lo = min_nan(__low2float(l), __high2float(l));
            hi = max_nan(__low2float(h), __high2float(h));
        } else {
            lo = hi = __uint_as_float(w[0]);
#pragma unroll
            for (int i = 1; i < kWords; ++i) {
                lo = min_nan(lo, __uint_as_float(w[i]));
                hi = max_nan(hi, __uint_as_float(w[i]));
            }
#pragma unroll
            for (int i = 0; i < N / 2; ++i) v[i] = two(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        }
    }
};

// Values of which some are not finite or beyond kLargest: NaN turned into 0, finite ones
// cut, and the least and largest of the finite (+inf and -inf if there is none).
__device__ __noinline__ void clean(float *v, int n, float *bounds) {
    float lo = INFINITY, hi = -INFINITY;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        float x = v[i];
        if (!(x == x)) x = 0.0f;
        if (fabsf(x) < INFINITY) {
            x = fminf(fmaxf(x, -kLargest), kLargest);
            lo = fminf(lo, x);
            hi = fmaxf(hi, x);
        }
        v[i] = x;
    }
    bounds[0] = lo;
    bounds[1] = hi;
}
// Codes by the quotients themselves, cut to [0, 15].
__device__ __noinline__ void codes_cut(float *v, int n, float s, float m) {
#pragma unroll 1
    for (int i = 0; i < n; ++i) v[i] = s > 0.0f ? fminf(fmaxf(rintf(__fdiv_rn(v[i] - m, s)), 0.0f), 15.0f) : 0.0f;
}
template <int N>
__device__ __forceinline__ void to_array(const F2 (&v)[N], float (&x)[2 * N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float2 y = apart(v[i]);
        x[2 * i] = y.x;
        x[2 * i + 1] = y.y;
    }
}
template <int N>
__device__ __forceinline__ void from_array(F2 (&v)[N], const float (&x)[2 * N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = two(x[2 * i], x[2 * i + 1]);
}

// Whether that was so.
template <int N>
__device__ __forceinline__ bool bounds_of(F2 (&v)[N], float &lo, float &hi) {
    const bool some = !(lo >= -kLargest && hi <= kLargest);
    if (__builtin_expect(some, 0)) {
        float x[2 * N], b[2];
        to_array(v, x);
        clean(x, 2 * N, b);
        from_array(v, x);
        lo = b[0];
        hi = b[1];
    }
    return some;
}

struct Scale {
    __half2 stored;  // (scale, least)
    float s, m, inv;
    bool plain;      // every code is within [0, 15] without being cut to it

    // from the least and largest of all 64
    __device__ __forceinline__ Scale(float lo, float hi) {
        if (!(lo <= hi)) lo = hi = 0.0f;  // no finite value
        stored = __halves2half2(__float2half_rn((hi - lo) * (1.0f / 15.0f)), __float2half_rn(lo));
        s = __low2float(stored);
        m = __high2float(stored);
        inv = s > 0.0f ? __frcp_rn(s) : 0.0f;
        plain = s == 0.0f || ((lo - m) * inv > -0.49f && (hi - m) * inv < 15.49f);
    }
    // The codes of the lane's values, negative.  (x - m) / s is rounded as a division rounds
    // it: with inv = 1 / s correctly rounded, t = d inv and r = d - t s by one fused
    // multiply-add, t + r inv is the correctly rounded quotient (Markstein).  Values that are
    // not finite or not within the codes' range (`odd`) take the divisions themselves.
    template <int N>
    __device__ __forceinline__ void codes(const F2 (&v)[N], bool odd, F2 (&q)[N]) const {
        const F2 less = two(-m, -m), i2 = two(inv, inv), s2 = two(-s, -s), round = two(kRound, kRound), minus = two(-1.0f, -1.0f);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const F2 d = add(v[i], less), t = mul(d, i2);
            q[i] = fma(add(fma(fma(t, s2, d), i2, t), round), minus, round);
        }
        if (__builtin_expect(odd || !plain, 0)) {
            float x[2 * N];
            to_array(v, x);
            codes_cut(x, 2 * N, s, m);
            from_array(q, x);
#pragma unroll
            for (int i = 0; i < N; ++i) q[i] = mul(q[i], minus);
        }
    }
};

constexpr float kBits = 8388608.0f;  // 2^23: the low bits of a float that is this and an integer are the integer's

// A warp's tile: new tokens [lo, hi) (positions) of the tile that begins at t0.  A lane takes
// 16 dimensions of a token a turn, of K and of V; V's codes change places in shared
// memory (`stage`, 512 bytes of the warp's own), or go out byte by byte where the tile is
// not written whole.  (In a loop, with the next turn's values on their way: the code of a
// warp that has one token to write takes longer to fetch than to run; unrolled, 23 us for a
// token of 256 sequences.)
template <typename T, int D>
__device__ __forceinline__ void append_tile(const T *src, int64_t row, uint8_t *codes, __half2 *scales, int32_t t0, int32_t lo, int32_t hi,
                                            bool is_v, uint8_t *stage, int lane) {
    const int g = lane >> 2, q = lane & 3;
    constexpr int kTurns = 2 * (D / kBlockDims);
    const bool whole = lo <= t0 && hi >= t0 + kKvTile;
    auto token = [&](int i) { return k_token(g) + 2 * (i & 1); };
    auto is_fresh = [&](int i) { return t0 + token(i) >= lo && t0 + token(i) < hi; };
    auto read = [&](int i, Raw<T, 16> &x) {
        x.zero();
        if (is_fresh(i)) x.load(src + static_cast<int64_t>(t0 + token(i)) * row + (i >> 1) * kBlockDims + 16 * q);
    };
    Raw<T, 16> next;
    read(0, next);
#pragma unroll 1
    for (int i = 0; i < kTurns; ++i) {
        const Raw<T, 16> x = next;
        if (i + 1 < kTurns) read(i + 1, next);
        const bool fresh = is_fresh(i);
        if (!__any_sync(0xffffffffu, fresh)) continue;
        F2 v[8], c[8];
        float a, z;
        x.values(v, a, z);
        const bool odd = bounds_of(v, a, z);
#pragma unroll
        for (int o = 1; o < 4; o *= 2) {
            a = fminf(a, __shfl_xor_sync(0xffffffffu, a, o));
            z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, o));
        }
        const Scale s(a, z);
        s.codes(v, odd, c);
        const int h = i >> 1;
        uint8_t *const block = codes + h * kBlockBytes;
        if (q == 0 && fresh) scales[h * kKvTile + token(i)] = s.stored;
        if (!is_v) {
            // a word's even dimensions make its low half, the odd ones its high half
            uint32_t w[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                F2 sum = fma(c[4 * k], two(-1.0f, -1.0f), two(kBits, kBits));
                sum = fma(c[4 * k + 1], two(-16.0f, -16.0f), sum);
                sum = fma(c[4 * k + 2], two(-256.0f, -256.0f), sum);
                sum = fma(c[4 * k + 3], two(-4096.0f, -4096.0f), sum);
                const float2 y = apart(sum);
                w[k] = __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x5410);
            }
            if (fresh) reinterpret_cast<uint2 *>(block)[2 * lane + (i & 1)] = make_uint2(w[0], w[1]);
        } else {
            // the byte of token t and dimensions 2 p, 2 p + 1 (p of 32): piece 4 (p % 16 / 2) + t / 4, word 2 (p /
            // 16) + p % 2, byte 0, 2, 1, 3 by t % 4; here p = 8 q + k
            const int t = token(i), at = (q & 1) * 256 + (t >> 2) * 16 + (q >> 1) * 8 + (t & 1) * 2 + (t >> 1 & 1);
            if (whole && !(i & 1)) __syncwarp();  // the block before has been read
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float2 y = apart(c[k]);
                const uint8_t b = static_cast<uint8_t>(__float_as_uint(fmaf(y.y, -16.0f, kBits - y.x)));
                uint8_t *const to = (whole ? stage : block) + at + (k >> 1) * 64 + (k & 1) * 4;
                if (fresh) *to = b;
            }
            if (whole && (i & 1)) {
                __syncwarp();
                reinterpret_cast<uint4 *>(block)[lane] = reinterpret_cast<const uint4 *>(stage)[lane];
            }
        }
    }
}

// grid.x: pieces of the rows cut at multiples of 16 tokens; grid.y: groups of four (K or V, head).
template <typename T, int D>
__global__ void __launch_bounds__(128, 7) kv_append4_kernel(const __grid_constant__ KvView b, const __grid_constant__ HeadsView k,
                                                         const __grid_constant__ HeadsView v) {
    __shared__ __align__(16) uint8_t stage[4][kBlockBytes];
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
        append_tile<T, D>(src, x.row, codes, scales, t0, lo, hi, is_v, stage[warp], lane);
    });
}

// ---------------------------------------------------------------- gather

// N values, 32 bytes at a time where there are so many (a K lane's piece of a row is a sector, or two).
template <int N>
__device__ __forceinline__ void store_values(float *p, const F2 (&v)[N / 2]) {
    uint32_t w[N];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const float2 x = apart(v[i]);
        w[2 * i] = __float_as_uint(x.x);
        w[2 * i + 1] = __float_as_uint(x.y);
    }
    if constexpr (N >= 8) {
#pragma unroll
        for (int i = 0; i < N; i += 8) sm100::store_32(p + i, *reinterpret_cast<const uint32_t(*)[8]>(w + i));
    } else {
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}
template <int N>
__device__ __forceinline__ void store_values(__nv_bfloat16 *p, const F2 (&v)[N / 2]) {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const float2 x = apart(v[i]);
        const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    if constexpr (N >= 16) {
#pragma unroll
        for (int i = 0; i < N / 2; i += 8) sm100::store_32(p + 2 * i, *reinterpret_cast<const uint32_t(*)[8]>(w + i));
    } else {
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    }
}

// A warp takes a tile of heads hv, hv + 4 gridDim.y, ... of the 2 heads (K's, then V's): the
// more of them, the fewer times the tile's place is looked up.
template <typename T, int D>
__global__ void __launch_bounds__(128, 8) kv_gather4_kernel(const __grid_constant__ KvView b, const __grid_constant__ HeadsView k,
                                                            const __grid_constant__ HeadsView v) {
    constexpr int H = D / kBlockDims;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    for_pieces(b, blockIdx.x, 4, blockIdx.y == 0 && threadIdx.x < 32,
               [&](int32_t s, const SeqRows &r, int32_t lo, int32_t hi) {
        const int32_t page = read_page(b, s, lo >> b.page_shift);
        const int32_t t0 = lo & ~(kKvTile - 1);
        const int64_t row0 = r.off - (r.len - r.n);  // of position 0
#pragma unroll 1
        for (int32_t hv = blockIdx.y * 4 + warp; hv < 2 * b.heads; hv += 4 * gridDim.y) {
            const bool is_v = hv >= b.heads;
            const int32_t head = is_v ? hv - b.heads : hv;
            const HeadsView &x = is_v ? v : k;
            const int64_t tile = page < 0 ? 0 : tile_index(b, page, head, (t0 & (b.page_tokens - 1)) / kKvTile);
            const uint4 *codes = reinterpret_cast<const uint4 *>((is_v ? b.v_pages : b.k_pages) + tile * (H * kBlockBytes)) + lane;
            const uint32_t *scales = reinterpret_cast<const uint32_t *>(is_v ? b.v_scales : b.k_scales) + tile * (H * kKvTile);
            T *dst = static_cast<T *>(x.p) + row0 * x.row + head * x.head;
            uint4 c[H];
            uint32_t sc[H][4];  // of K's two tokens, or V's four
#pragma unroll
            for (int h = 0; h < H; ++h) {
                c[h] = codes[h * 32];
                if (is_v) {
                    const uint4 y = *reinterpret_cast<const uint4 *>(scales + h * kKvTile + 4 * q);
                    sc[h][0] = y.x; sc[h][1] = y.y; sc[h][2] = y.z; sc[h][3] = y.w;
                } else {
                    sc[h][0] = scales[h * kKvTile + k_token(g)];
                    sc[h][1] = scales[h * kKvTile + k_token(g) + 2];
                }
                if (page < 0) sc[h][0] = sc[h][1] = sc[h][2] = sc[h][3] = 0u;  // (a table entry out of range reads as zeros)
            }
            if (!is_v) {
#pragma unroll
                for (int h = 0; h < H; ++h)
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const int32_t pos = t0 + k_token(g) + 2 * t;
                        const float2 y = f16_pair(sc[h][t]);
                        const F2 s0 = two(y.x * kCode0, y.x * kCode0), s1 = two(y.x * kCode1, y.x * kCode1), m = two(y.y, y.y);
                        F2 o[8];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            uint32_t f[4];
                            nibble_pairs(t == 0 ? (j == 0 ? c[h].x : c[h].y) : (j == 0 ? c[h].z : c[h].w), f);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float2 code = f16_pair(f[i]);
                                o[4 * j + i] = fma(two(code.x, code.y), i & 1 ? s1 : s0, m);
                            }
                        }
                        if (pos >= lo && pos < hi) store_values<16>(dst + pos * x.row + h * kBlockDims + 16 * q, o);
                    }
            } else {
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const uint32_t w[4] = {c[h].x, c[h].y, c[h].z, c[h].w};
#pragma unroll
                    for (int t = 0; t < 4; t += 2) {  // tokens t and t + 1 side by side
                        const float2 ya = f16_pair(sc[h][t]), yb = f16_pair(sc[h][t + 1]);
                        const F2 s0 = two(ya.x * kCode0, yb.x * kCode0), s1 = two(ya.x * kCode1, yb.x * kCode1), m = two(ya.y, yb.y);
                        F2 z[4][2];  // [word][dimension of it]
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t y = t == 0 ? w[j] : w[j] >> 8;
                            const float2 a = f16_pair(y & kNibbles0), e = f16_pair(y & kNibbles1);
                            z[j][0] = fma(two(a.x, a.y), s0, m);
                            z[j][1] = fma(two(e.x, e.y), s1, m);
                        }
                        const int32_t pos = t0 + 4 * q + t;
                        T *to = dst + pos * x.row + h * kBlockDims + 4 * g;
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            if (pos + u < lo || pos + u >= hi) continue;
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                F2 o[2];
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    const float2 a = apart(z[2 * half + j][0]), e = apart(z[2 * half + j][1]);
                                    o[j] = two(u ? a.y : a.x, u ? e.y : e.x);
                                }
                                store_values<4>(to + u * x.row + 32 * half, o);
                            }
                        }
                    }
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
    // one turn a warp while that is less than the machine has room for four times over
    dim3 grid = pieces_grid(b);
    const unsigned enough = static_cast<unsigned>(device_sm_count()) * 8 * 4;
    while (grid.y > 1 && static_cast<uint64_t>(grid.x) * ((grid.y + 1) / 2) >= enough) grid.y = (grid.y + 1) / 2;
    kernel<<<grid, 128, 0, stream>>>(b, k, v);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace lora
