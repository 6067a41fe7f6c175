/*
 * lora_attention.h — C ABI of what stands between the adapted q/k/v
 * projections (lora.h) and the adapted o projection: rotary positions, an
 * 8-bit paged key/value cache, and attention over it.
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

/* ---------------------------------------------------------------------- */
/* The 8-bit paged key/value cache                                         */
/* ---------------------------------------------------------------------- */

typedef enum lora_kv_format {
    LORA_KV_INT8 = 0, /* int8 in [-127, 127], scale = largest magnitude / 127 */
    LORA_KV_E4M3 = 1  /* 8-bit floating point (4 exponent, 3 mantissa bits), power-of-two scale */
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
 */
typedef struct lora_kv_cache {
    lora_kv_format_t format;
    int32_t num_pages;    /* >= 1 */
    int32_t num_heads;    /* key/value heads, >= 1 */
    int32_t head_dim;     /* 64 or 128 */
    int32_t page_tokens;  /* 16, 32, 64 or 128 */
    int32_t growth;       /* a lora_kv_growth_t */
    void *k_pages, *v_pages;    /* device; num_pages*num_heads*page_tokens*head_dim bytes each */
    float *k_scales, *v_scales; /* device [num_pages][num_heads] */
} lora_kv_cache_t;

/* Device bytes of k_pages (and of v_pages); 0 on bad input. */
size_t lora_kv_pages_bytes(int32_t num_pages, int32_t num_heads, int32_t head_dim, int32_t page_tokens);

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
 * k, v: the rows' [num_heads][head_dim] in `dtype`.
 * Errors: INVALID_ARG, ALIGNMENT, DTYPE, UNSUPPORTED (head_dim, page_tokens
 * or format), CUDA.
 */
lora_status_t lora_kv_append(const lora_kv_cache_t *cache, const lora_kv_batch_t *batch, lora_dtype_t dtype,
                             const lora_heads_t *k, const lora_heads_t *v, void *stream);

/*
 * Read the rows' keys and values back: code * scale, rounded once to
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
 * A NaN in the cache reaches the queries that see its token, and no others.
 * Rows outside every sequence are not written.
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
