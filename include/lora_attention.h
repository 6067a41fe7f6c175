/*
 * lora_attention.h — C ABI of what stands between the adapted q/k/v
 * projections (lora.h) and the adapted o projection: rotary positions, with
 * norms of queries and keys or without, a paged key/value cache of 8 or 4 bits,
 * and attention over it.
 *
 * The conventions of lora.h hold for every entry point: plain C, the caller
 * owns all device memory, work is ordered on `stream`, device pointers are
 * 16-byte aligned (arrays of lengths, offsets, positions and page numbers 4-byte
 * aligned), errors found on the host leave all state unchanged, and
 * errors found by kernels are recorded in the status word that
 * lora_get_device_status() reads.  No call allocates device memory, waits
 * for the device or reads device memory from the host, so every call can be
 * captured in a CUDA graph (after one call outside a capture).
 * "Dtype" is LORA_BF16 or LORA_FP32 throughout; sums, softmax statistics and
 * scales are fp32.
 */
#ifndef LORA_ATTENTION_H
#define LORA_ATTENTION_H

#include "lora.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------- */
/* Rotary positions                                                        */
/* ---------------------------------------------------------------------- */

#define LORA_ROPE_MAX_AXES 4
#define LORA_ROPE_MAX_PAIRS 256

/* Rows of heads: element (row, head, d) at ptr[row*row_stride + head*head_stride + d]. */
typedef struct lora_heads {
    void *ptr;            /* device; 16-byte aligned */
    int64_t row_stride;   /* elements; 16-byte multiples */
    int64_t head_stride;  /* elements; 16-byte multiples */
} lora_heads_t;

/*
 * Rotary positions on the first rot_dim dimensions of every head of q and k:
 * pair i (of rot_dim/2) is turned by the angle whose cosine and sine stand in
 * row p of the tables, p = positions[axis(i)][row]:
 *
 *     y1 = x1 cos[p][i] - x2 sin[p][i],   y2 = x2 cos[p][i] + x1 sin[p][i]
 *
 * (x1, x2) are dimensions (i, i + rot_dim/2), or (2i, 2i + 1) if
 * `interleaved`.  With one axis this is the ordinary rotary embedding of
 * text; with several (time, height, width of image and video tokens) every
 * pair follows one axis.  `inverse` turns the other way, which undoes the
 * call and is also its gradient.  Dimensions past rot_dim are copied.  An
 * output may be its own input (same pointer and strides); other overlaps are
 * not allowed.  Arithmetic in fp32, one rounding to the dtype.
 * Errors: INVALID_ARG, ALIGNMENT, DTYPE, UNSUPPORTED (head_dim over 1024),
 * CUDA.  A position outside
 * [0, max_pos) leaves its pairs unturned and is recorded (DEVICE_INDEX,
 * detail = row).
 */
typedef struct lora_rope_args {
    lora_dtype_t dtype;
    int32_t rows;             /* >= 0; 0 is a no-op */
    int32_t head_dim;         /* multiple of 8, up to 1024 */
    int32_t rot_dim;          /* multiple of 16, 16 .. min(head_dim, 2*LORA_ROPE_MAX_PAIRS) */
    int32_t num_q_heads;      /* >= 1 */
    int32_t num_k_heads;      /* >= 0; 0: q only */
    lora_heads_t q, q_out;
    lora_heads_t k, k_out;
    const float *cos_table;   /* device [max_pos][rot_dim/2] */
    const float *sin_table;
    int32_t max_pos;
    int32_t num_axes;         /* 1 .. LORA_ROPE_MAX_AXES */
    const int32_t *positions; /* device [num_axes][rows]; 4-byte aligned */
    const uint8_t *pair_axis; /* HOST [rot_dim/2], each < num_axes; NULL: every pair follows axis 0 */
    int32_t interleaved;
    int32_t inverse;
} lora_rope_args_t;

lora_status_t lora_rope(const lora_rope_args_t *args, void *stream);

/*
 * Norms of q and k for each head, and the rotary positions, in one pass: with W =
 * w, or 1 + w if unit_offset, a head x of head_dim = D values becomes
 *
 *     n_d = x_d W_d / sqrt(sum_d x_d^2 / D + eps),   y = n turned as by lora_rope
 *
 * (dimensions past rot_dim are normalised, not turned).  Each value is read and
 * written once.  Arithmetic in fp32, squares and their sum included, one
 * rounding to the dtype at the end.  A head with an infinity or NaN becomes NaN or 0, no
 * other head is touched by it.  A weight of NULL stands for W = 1.
 * An output may be its own input (same pointer and strides); other overlaps are
 * not allowed.  Errors: as lora_rope, and UNSUPPORTED for head_dim over 256 or
 * `inverse`; a position out of range leaves its pairs unturned (normalised).
 */
typedef struct lora_norm_rope_args {
    lora_rope_args_t rope;    /* its `inverse` is 0 */
    const void *q_weight;     /* device [head_dim] of weight_dtype, or NULL */
    const void *k_weight;
    lora_dtype_t weight_dtype;
    int32_t unit_offset;
    float eps;                /* > 0, finite */
} lora_norm_rope_args_t;

lora_status_t lora_norm_rope(const lora_norm_rope_args_t *args, void *stream);

/*
 * The gradient of that call.  args as given to it, with q and k its inputs, and
 * q_out and k_out where their gradients go; dq and dk: the gradients of its outputs.
 * With h = dy turned back, r = 1 / sqrt(mean(x^2) + eps) and a = h W:
 *
 *     dx = r (a - x r^2 mean(a x)),   dw = sum over rows and heads of h x r
 *
 * in fp32; dx is rounded once to the dtype, dw is fp32, its sums' order fixed by
 * the sizes and the device's number of SMs.  A gradient may take the place of dy, or of
 * the input (same pointer and strides).  With rows = 0 the weights' gradients are set to 0.
 */
typedef struct lora_norm_rope_grads {
    lora_heads_t dq, dk;      /* like q and k */
    float *dq_weight;         /* device [head_dim], 4-byte aligned; NULL: not wanted */
    float *dk_weight;
    void *workspace;          /* device, >= lora_norm_rope_backward_workspace_bytes, if a weight's gradient is wanted */
    size_t workspace_bytes;
} lora_norm_rope_grads_t;

/* Scratch bytes on the current device; it keeps nothing between calls.  0 if the arguments are invalid. */
size_t lora_norm_rope_backward_workspace_bytes(const lora_norm_rope_args_t *args);

lora_status_t lora_norm_rope_backward(const lora_norm_rope_args_t *args, const lora_norm_rope_grads_t *grads, void *stream);

/* ---------------------------------------------------------------------- */
/* The paged key/value cache, of 8 or 4 bits                                */
/* ---------------------------------------------------------------------- */

typedef enum lora_kv_format {
    LORA_KV_INT8 = 0, /* int8 in [-127, 127], scale = largest magnitude / 127 */
    LORA_KV_E4M3 = 1, /* 8-bit floating point (4 exponent, 3 mantissa bits), power-of-two scale */
    LORA_KV_UINT4 = 4 /* 4 bits, 0 to 15, with an f16 scale and least value for each 64 dimensions of a token */
} lora_kv_format_t;

/* How an int8 page's scale grows when a later token does not fit (e4m3 scales are powers of two either way). */
typedef enum lora_kv_growth {
    LORA_KV_GROW_LEAST = 0,   /* to the least that holds it: the finest steps for pages written at once */
    LORA_KV_GROW_DOUBLING = 1 /* by the least power of two that holds it: for pages filled token by token */
} lora_kv_growth_t;

/*
 * One layer's cache.  A page holds page_tokens consecutive tokens of one
 * sequence; a value is code * scale, with one fp32 scale per page and head,
 * for K and for V: k_scales[page*num_heads + head].  The codes of one page
 * and head are contiguous, in tiles of 16 tokens (LORA_BLOCK_ROWS):
 *
 *   k_pages [num_pages][num_heads][page_tokens/16][head_dim/64][16 tokens][64 dims]
 *   v_pages [num_pages][num_heads][page_tokens/16][head_dim/4][4 token quads][4 dims][4 tokens]
 *
 * so that one 16-byte load of a K tile is a piece of a token's row, one of a
 * V tile four tokens of four dimensions: what a thread of the attention
 * kernels' matrix instructions takes of each, without a transposition.
 *
 * LORA_KV_UINT4: a value is code * scale + least, with an f16 scale and least
 * value for each 64 dimensions of a token and head (0.5625 bytes a value):
 *
 *   k_pages, v_pages    uint8 [num_pages][num_heads][page_tokens/16][head_dim/64][32 pieces][16]
 *   k_scales, v_scales  f16 [num_pages][num_heads][page_tokens/16][head_dim/64][16 tokens][scale, least]
 *
 * K: piece 4g + q holds dimensions 16q .. 16q + 15 of token t = 4(g/2) + g%2 of the
 * tile (its first 8 bytes) and of token t + 2; each four bytes eight dimensions: 0 and 2,
 * 4 and 6, 1 and 3, 5 and 7, the first in the low half of the byte.  V: piece 4g + q holds
 * tokens 4q .. 4q + 3; its j-th four bytes dimension d = 4g + 32(j/2) + 2(j%2) in the low
 * halves and d + 1 in the high ones, of tokens 4q, 4q + 2, 4q + 1, 4q + 3.  Scales are
 * not negative, and values within f16's range (an append's are within 2^15, about);
 * what tokens that are not written yet have may be anything.
 */
typedef struct lora_kv_cache {
    lora_kv_format_t format;
    int32_t num_pages;    /* >= 1 */
    int32_t num_heads;    /* key/value heads, >= 1 */
    int32_t head_dim;     /* 64 or 128 */
    int32_t page_tokens;  /* 16, 32, 64 or 128 */
    int32_t growth;       /* a lora_kv_growth_t; LORA_KV_UINT4 has no use for it */
    void *k_pages, *v_pages;    /* device; lora_kv_codes_bytes each */
    void *k_scales, *v_scales;  /* device; float [num_pages][num_heads], or as above */
} lora_kv_cache_t;

/* Device bytes of an 8-bit cache's k_pages (and of v_pages); 0 on bad input. */
size_t lora_kv_pages_bytes(int32_t num_pages, int32_t num_heads, int32_t head_dim, int32_t page_tokens);

/* Device bytes of k_pages and of k_scales (and as many for v) in any format; 0 on bad input. */
size_t lora_kv_codes_bytes(lora_kv_format_t format, int32_t num_pages, int32_t num_heads, int32_t head_dim, int32_t page_tokens);
size_t lora_kv_scales_bytes(lora_kv_format_t format, int32_t num_pages, int32_t num_heads, int32_t head_dim, int32_t page_tokens);

/*
 * Which rows of a call belong to which sequence: rows offsets[s] up to
 * offsets[s+1] are the LAST tokens of sequence s, whose cache holds (or, for
 * an append, will hold) seq_lens[s] tokens: with n = offsets[s+1] -
 * offsets[s] rows, row offsets[s] + i is the token at position
 * seq_lens[s] - n + i.  Token t lies in page block_table[s][t / page_tokens].
 * A sequence of length 0 is padding (its rows stand for no token); one
 * without rows is passed over.  Recorded by the kernels, the sequence then
 * skipped: offsets not within [0, rows] or decreasing, more rows than
 * tokens (SEGMENTS, detail = s); a length below 0, past max_pages pages or
 * past 2^30 (DEVICE_INDEX, detail = s).  A table entry outside [0, num_pages) that is
 * needed is recorded (DEVICE_INDEX, detail = s); its tokens are not written,
 * and read as zeros.
 */
typedef struct lora_kv_batch {
    int32_t num_seqs;           /* >= 0 */
    int32_t rows;               /* rows of the call's tensors, >= 0 */
    const int32_t *seq_lens;    /* device [num_seqs] */
    const int32_t *offsets;     /* device [num_seqs + 1]; NULL: one row each (rows == num_seqs) */
    const int32_t *block_table; /* device [num_seqs][max_pages]; entries past a sequence's end are not read */
    int32_t max_pages;          /* >= 1 */
} lora_kv_batch_t;

/*
 * Write the rows' keys and values into the cache, quantised.  For each page
 * and head that new tokens fall into, with a the largest finite |x| of the
 * call's new values there and s0 the page's scale (0 if the page's first
 * token is new):
 *   int8:  s = max(s0, a / 127), a / 127 taken as 2^-120 at least if a > 0;
 *          code = x / s rounded to nearest even, within [-127, 127];
 *          older codes of the page become code * (s0 / s), rounded so too.
 *          With LORA_KV_GROW_DOUBLING and s0 > 0, s = s0 * 2^k with the least
 *          such k >= 0 that gives s >= a / 127.
 *   e4m3:  s = max(s0, the least power of two with a <= 448 s, 2^-120 at
 *          least if a > 0); code = x / s rounded to nearest even; older codes
 *          are rescaled by s0 / s, exactly unless they fall below the
 *          format's least normal.
 * All of it in fp32.  Every growth of an int8 page's scale rounds its older
 * codes once more: after g growths a value may be off by (g + 1) / 2 steps of
 * the page's scale, and where the magnitudes of a page grow little by little g may
 * be as large as its number of tokens (128 tokens that grow by 0.5% each: 42 of
 * 127 steps).  With LORA_KV_GROW_DOUBLING the roundings halve each other: it is
 * off by less than one step, of a scale less than twice the least.  e4m3 codes
 * are rescaled exactly.  Infinities take the largest code, NaN code 0 in int8
 * and NaN in e4m3; neither moves the scale of its neighbours, but where the
 * call's new values have no finite one but zeros, an infinity or NaN among them
 * counts as the least a > 0 (s is 2^-120 at least), so that it has a code.  A
 * page with no value but zeros has scale 0.  Pages are not shared: no two
 * sequences of a call may write the same page.
 *   uint4: for each 64 dimensions of a token and head, with NaN counted as 0,
 *          finite values cut to [-2^15, 2^15], and lo, hi the least and the largest
 *          finite one (0, 0 if there is none):
 *          least = lo and scale = (hi - lo) * fp32(1/15), each rounded to f16 (nearest even);
 *          code = (x - least) / scale rounded to nearest even, within [0, 15]; infinities
 *          take the end codes; with scale 0 every code is 0.
 *          In fp32 but for the two roundings.  Older tokens are not touched.
 * k, v: the rows' [num_heads][head_dim] in `dtype`.
 * Errors: INVALID_ARG, ALIGNMENT, DTYPE, UNSUPPORTED (head_dim, page_tokens
 * or format), CUDA.
 */
lora_status_t lora_kv_append(const lora_kv_cache_t *cache, const lora_kv_batch_t *batch, lora_dtype_t dtype,
                             const lora_heads_t *k, const lora_heads_t *v, void *stream);

/*
 * Read the rows' keys and values back: code * scale (+ least), rounded once to
 * `dtype`.  With n = seq_lens a sequence is read whole.  Rows of padding or
 * skipped sequences are not written.  Errors: as lora_kv_append.
 */
lora_status_t lora_kv_gather(const lora_kv_cache_t *cache, const lora_kv_batch_t *batch, lora_dtype_t dtype,
                             const lora_heads_t *k, const lora_heads_t *v, void *stream);

/*
 * Softmax attention of the rows' queries over their sequences' cached keys
 * and values (which must hold the rows' own tokens already: append first).
 * The query at position p of a sequence of L tokens sees the keys j with
 * j < L, j <= p if causal, and j > p - window if window > 0:
 *
 *     out = sum_j softmax_j(scale q . k_j) v_j,   lse = log sum_j exp(scale q . k_j)
 *
 * Query head h reads key/value head h / (num_q_heads / num_heads).  A query
 * that sees no key (padding, skipped sequences) has out = 0 and lse = -inf.
 * A NaN in the cache reaches the queries that see its token, and no others; of
 * LORA_KV_UINT4 so does a scale or least value that is infinite or NaN, of V in its 64
 * dimensions (which become NaN or infinite).
 * Rows outside every sequence are not written.  Pages that no row of a sequence sees
 * (before its window) are not needed: their table entries may name no page.
 * max_queries bounds the rows of one sequence (it and max_pages choose the kernel); a
 * sequence with more rows is recorded (SEGMENTS) and skipped.
 * Precision: products with the codes exact, fp32 sums.  A probability p_j
 * enters the second product, times its page's scale of V, with 11 significant
 * bits for bf16 calls and 22 for fp32 ones, but not with less than a fixed
 * step: with P the row's largest p_j * (page's scale of V), each is off by at
 * most 2^-29 P (bf16), 2^-33 P (bf16, where the call takes the kernel for few
 * queries) or 2^-44 P (fp32) beyond that.  Over n keys this adds up to n 2^-29 P times
 * the largest code, which stays below bf16's own rounding of the largest values
 * up to a million keys.  Values that a query does not see have no part in this.
 * (Pages whose V scales differ by more than 2^79 within a sequence and head cost
 * time: twice as much for prompts, some ten times for few queries.)
 * LORA_KV_UINT4: in every fp32 call, and where a bf16 call takes the kernel for few
 * queries, codes enter the products exactly, scales and least values in fp32: each p_j
 * times the token's scale has 22 and 11 bits, and is off by at most 2^-44 and 2^-33 of
 * the row's largest such product beyond that (and by 2^-96 and 2^-85 of the sum of all p_j).
 * (fp32 calls take a value as scale (code - 8) and least + 8 scale.)  Where a bf16 call takes the one for many,
 * V's values enter rounded to f16 (11 bits), and a p_j is off by at most 2^-29 of the
 * row's largest beyond its 11 bits; K's values enter exactly if lse is given, else rounded
 * to f16, which moves scores by up to 2^-12 scale sum |q k|.  Where a token's 64 values lie around
 * 0 (a least value of up to some 15 scales) that is less than 1% of K's own step, and `out` with and
 * without lse differs by less than bf16's rounding of it; keys far from 0 in all dimensions are another
 * matter (near 100 and varying by 1: `out` off by 1.2% in the root mean square): give lse for those.
 * Errors: INVALID_ARG, ALIGNMENT, DTYPE, UNSUPPORTED (num_q_heads /
 * num_heads over 64; num_q_heads not a multiple; rows * num_q_heads of 2^31
 * or more), WORKSPACE, CUDA.
 */
typedef struct lora_kv_attention_args {
    lora_dtype_t dtype;      /* of q and out */
    int32_t num_q_heads;     /* a multiple of the cache's num_heads */
    lora_heads_t q, out;     /* the rows' [num_q_heads][head_dim] */
    float *lse;              /* NULL, or device [rows][num_q_heads], natural logarithm */
    float scale;             /* > 0, finite */
    int32_t causal;
    int32_t window;          /* >= 0; 0: no window */
    int32_t max_queries;     /* >= 1 */
    void *workspace;         /* device, >= lora_kv_attention_workspace_bytes; keeps nothing between calls */
    size_t workspace_bytes;
} lora_kv_attention_args_t;

/* Scratch bytes of a call with these arguments on the current device (256 at least), 0 if they are invalid. */
size_t lora_kv_attention_workspace_bytes(const lora_kv_cache_t *cache, const lora_kv_batch_t *batch,
                                         const lora_kv_attention_args_t *args);

lora_status_t lora_kv_attention(const lora_kv_cache_t *cache, const lora_kv_batch_t *batch,
                                const lora_kv_attention_args_t *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_ATTENTION_H */
