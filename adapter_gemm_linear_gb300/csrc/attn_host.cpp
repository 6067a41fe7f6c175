// Host side of lora_attention.h: argument validation and dispatch.  No entry
// point here allocates device memory or waits for the device.
#include <algorithm>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "attn_internal.h"

namespace {

constexpr int32_t kMaxKvHeads = 4096;  // keeps every grid dimension in range
constexpr int32_t kMaxNormDim = 256;   // of a head that lora_norm_rope normalises: two chunks a lane at most

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

cudaStream_t as_stream(void *s) { return reinterpret_cast<cudaStream_t>(s); }

lora_status_t fail(cudaError_t e) {
    lora::set_last_cuda_error(static_cast<int32_t>(e));
    return LORA_ERR_CUDA;
}

// Rows of heads of `dtype`, `dim` elements each.
lora_status_t check_heads(const lora_heads_t *h, lora_dtype_t dtype, int32_t rows, lora::HeadsView *out) {
    if (!h) return LORA_ERR_INVALID_ARG;
    const int64_t ve = dtype == LORA_FP32 ? 4 : 8;
    if (h->row_stride < 0 || h->head_stride < 0) return LORA_ERR_INVALID_ARG;
    if (rows > 0) {
        if (!h->ptr) return LORA_ERR_INVALID_ARG;
        if (!aligned(h->ptr, 16)) return LORA_ERR_ALIGNMENT;
    }
    if (h->row_stride % ve || h->head_stride % ve) return LORA_ERR_ALIGNMENT;
    *out = lora::HeadsView{h->ptr, h->row_stride, h->head_stride};
    return LORA_OK;
}

lora_status_t check_cache(const lora_kv_cache_t *c) {
    if (!c) return LORA_ERR_INVALID_ARG;
    if (c->format != LORA_KV_INT8 && c->format != LORA_KV_E4M3 && c->format != LORA_KV_UINT4) return LORA_ERR_UNSUPPORTED;
    if (c->num_pages <= 0 || c->num_heads <= 0) return LORA_ERR_INVALID_ARG;
    if (c->num_heads > kMaxKvHeads) return LORA_ERR_UNSUPPORTED;
    if (c->head_dim != 64 && c->head_dim != 128) return LORA_ERR_UNSUPPORTED;
    if (c->page_tokens != 16 && c->page_tokens != 32 && c->page_tokens != 64 && c->page_tokens != 128)
        return LORA_ERR_UNSUPPORTED;
    if (c->growth != LORA_KV_GROW_LEAST && c->growth != LORA_KV_GROW_DOUBLING) return LORA_ERR_UNSUPPORTED;
    if (!c->k_pages || !c->v_pages || !c->k_scales || !c->v_scales) return LORA_ERR_INVALID_ARG;
    if (!aligned(c->k_pages, 16) || !aligned(c->v_pages, 16) || !aligned(c->k_scales, 16) || !aligned(c->v_scales, 16))
        return LORA_ERR_ALIGNMENT;
    return LORA_OK;
}

lora_status_t check_batch(const lora_kv_cache_t *c, const lora_kv_batch_t *b, lora::KvView *v) {
    lora_status_t s = check_cache(c);
    if (s != LORA_OK) return s;
    if (!b) return LORA_ERR_INVALID_ARG;
    if (b->num_seqs < 0 || b->rows < 0 || b->max_pages <= 0) return LORA_ERR_INVALID_ARG;
    if (!b->offsets && b->rows != b->num_seqs) return LORA_ERR_INVALID_ARG;
    if (b->num_seqs > 0 && b->rows > 0) {
        if (!b->seq_lens || !b->block_table) return LORA_ERR_INVALID_ARG;
        if (!aligned(b->seq_lens, 4) || !aligned(b->offsets, 4) || !aligned(b->block_table, 4))
            return LORA_ERR_ALIGNMENT;
    }
    v->k_pages = static_cast<uint8_t *>(c->k_pages);
    v->v_pages = static_cast<uint8_t *>(c->v_pages);
    v->k_scales = static_cast<float *>(c->k_scales);
    v->v_scales = static_cast<float *>(c->v_scales);
    v->seq_lens = b->seq_lens;
    v->offsets = b->offsets;
    v->table = b->block_table;
    v->num_pages = c->num_pages;
    v->heads = c->num_heads;
    v->page_tokens = c->page_tokens;
    v->page_shift = c->page_tokens == 16 ? 4 : c->page_tokens == 32 ? 5 : c->page_tokens == 64 ? 6 : 7;
    v->num_seqs = b->num_seqs;
    v->rows = b->rows;
    v->max_pages = b->max_pages;
    v->growth = c->growth;
    v->status = nullptr;
    return LORA_OK;
}

bool valid_dtype(lora_dtype_t t) { return t == LORA_BF16 || t == LORA_FP32; }

lora_status_t check_rope(const lora_rope_args_t *a, lora::RopeView *out) {
    if (!a) return LORA_ERR_INVALID_ARG;
    if (!valid_dtype(a->dtype)) return LORA_ERR_DTYPE;
    if (a->rows < 0 || a->head_dim <= 0 || a->num_q_heads <= 0 || a->num_k_heads < 0 || a->max_pos <= 0)
        return LORA_ERR_INVALID_ARG;
    if (a->num_axes < 1 || a->num_axes > LORA_ROPE_MAX_AXES) return LORA_ERR_INVALID_ARG;
    if (a->rot_dim < 16 || a->rot_dim > a->head_dim || a->rot_dim > 2 * LORA_ROPE_MAX_PAIRS)
        return LORA_ERR_INVALID_ARG;
    if (a->head_dim % 8 || a->rot_dim % 16) return LORA_ERR_ALIGNMENT;
    if (a->head_dim > 1024) return LORA_ERR_UNSUPPORTED;
    lora::RopeView &v = *out;
    lora_status_t s = check_heads(&a->q, a->dtype, a->rows, &v.q);
    if (s == LORA_OK) s = check_heads(&a->q_out, a->dtype, a->rows, &v.q_out);
    if (s == LORA_OK) s = check_heads(&a->k, a->dtype, a->num_k_heads ? a->rows : 0, &v.k);
    if (s == LORA_OK) s = check_heads(&a->k_out, a->dtype, a->num_k_heads ? a->rows : 0, &v.k_out);
    if (s != LORA_OK) return s;
    if (a->rows > 0) {
        if (!a->cos_table || !a->sin_table || !a->positions) return LORA_ERR_INVALID_ARG;
        if (!aligned(a->cos_table, 16) || !aligned(a->sin_table, 16) || !aligned(a->positions, 4))
            return LORA_ERR_ALIGNMENT;
    }
    memset(v.pair_axis, 0, sizeof(v.pair_axis));
    for (int32_t i = 0; a->pair_axis && i < a->rot_dim / 2; ++i) {
        if (a->pair_axis[i] >= a->num_axes) return LORA_ERR_INVALID_ARG;
        v.pair_axis[i] = a->pair_axis[i];
    }
    v.cos_table = a->cos_table;
    v.sin_table = a->sin_table;
    v.positions = a->positions;
    v.rows = a->rows;
    v.head_dim = a->head_dim;
    v.rot_dim = a->rot_dim;
    v.q_heads = a->num_q_heads;
    v.k_heads = a->num_k_heads;
    v.max_pos = a->max_pos;
    v.num_axes = a->num_axes;
    v.interleaved = a->interleaved != 0;
    v.inverse = a->inverse != 0;
    v.status = nullptr;
    return LORA_OK;
}

lora_status_t check_norm_rope(const lora_norm_rope_args_t *a, lora::NormRopeView *v) {
    if (!a) return LORA_ERR_INVALID_ARG;
    const lora_status_t s = check_rope(&a->rope, &v->rope);
    if (s != LORA_OK) return s;
    if (a->rope.inverse) return LORA_ERR_UNSUPPORTED;
    if (a->rope.head_dim > kMaxNormDim) return LORA_ERR_UNSUPPORTED;
    if (!valid_dtype(a->weight_dtype)) return LORA_ERR_DTYPE;
    if (!(a->eps > 0.0f) || !isfinite(a->eps)) return LORA_ERR_INVALID_ARG;
    if (!aligned(a->q_weight, 16) || !aligned(a->k_weight, 16)) return LORA_ERR_ALIGNMENT;
    v->dq = v->dk = lora::HeadsView{nullptr, 0, 0};
    v->q_weight = a->q_weight;
    v->k_weight = a->k_weight;
    v->partial = nullptr;
    v->eps = a->eps;
    v->weight_fp32 = a->weight_dtype == LORA_FP32;
    v->unit_offset = a->unit_offset != 0;
    v->q_groups = v->k_groups = 0;
    return LORA_OK;
}

lora_status_t check_attention(const lora_kv_cache_t *c, const lora_kv_batch_t *b, const lora_kv_attention_args_t *a,
                              lora::AttnView *v) {
    lora_status_t s = check_batch(c, b, &v->kv);
    if (s != LORA_OK) return s;
    if (!a) return LORA_ERR_INVALID_ARG;
    if (!valid_dtype(a->dtype)) return LORA_ERR_DTYPE;
    if (a->num_q_heads <= 0 || a->window < 0 || a->max_queries <= 0) return LORA_ERR_INVALID_ARG;
    if (!(a->scale > 0.0f) || !isfinite(a->scale)) return LORA_ERR_INVALID_ARG;
    if (a->num_q_heads % c->num_heads || a->num_q_heads / c->num_heads > lora::kMaxGroup)
        return LORA_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(b->rows) * a->num_q_heads > INT32_MAX) return LORA_ERR_UNSUPPORTED;
    s = check_heads(&a->q, a->dtype, b->rows, &v->q);
    if (s == LORA_OK) s = check_heads(&a->out, a->dtype, b->rows, &v->out);
    if (s != LORA_OK) return s;
    if (a->lse && !aligned(a->lse, 4)) return LORA_ERR_ALIGNMENT;
    v->lse = a->lse;
    v->q_heads = a->num_q_heads;
    v->group = a->num_q_heads / c->num_heads;
    v->scale = a->scale;
    v->causal = a->causal != 0;
    v->window = a->window;
    v->max_queries = a->max_queries;
    v->workspace = static_cast<unsigned char *>(a->workspace);
    v->test_wait_ns = 0;
    return LORA_OK;
}

// Which kernel: that of attn_decode.cu works on up to 16 query rows (queries x
// heads that share a key/value head) at a time, the tensor-core kernel of
// attn_prefill.cu on 256, and is faster as soon as the first would take more
// than one pass: 64 sequences of 4096 tokens, 8 heads of 128, with 16 rows
// 133 against 186 us, with 32 rows 244 against 187 us (in a graph, as what
// follows).  But it takes some 20 us to get going, so where the tables have no
// room for more than eight of the first's units of work an SM (16 rows x 128
// keys), those are done sooner: 128 queries of 32 heads on 8 on their own keys
// (512 units) 13.6 against 20.9 us, 64 on 1064 (1152 units) 25.1 against 25.0, 178
// x 2 heads on 7673 (1440 units) 28.5 against 28.8, 4 x 128 queries (2048 units)
// 43.5 against 22.0.  (What the tables have room for is all that the host knows of
// the lengths: a wider table of the same sequences may take the other kernel.)
// The 4-bit cache's kernels (attn_decode4.cu in place of the first) take the same rule: 64
// sequences of 4097, 8 heads of 128, with 16 rows 109 against 207 us, with 32 203 against 208; 64
// queries of 32 heads on 1064 keys (1152 units) 22.3 against 24.5, 4 x 128 queries
// (2048 units) 47.7 against 25.2.  Its heads of 64 take two passes of the first: with 32 rows 121
// against 162, with 48 175 against 163.
bool many_queries(const lora::AttnView &v, const lora_kv_cache_t *c, lora_dtype_t dtype) {
    const int64_t rows = static_cast<int64_t>(v.max_queries) * v.group;  // of a sequence, at most
    if (dtype != LORA_BF16 || rows <= (c->format == LORA_KV_UINT4 && c->head_dim == 64 ? 32 : 16)) return false;
    const double row_tiles = std::min(static_cast<double>(v.kv.num_seqs) * static_cast<double>((rows + 15) / 16),
                                      static_cast<double>(v.kv.rows) * v.group / 16 + v.kv.num_seqs);
    const double chunks = (static_cast<double>(v.kv.max_pages) * v.kv.page_tokens + 127) / 128;
    return row_tiles * v.kv.heads * chunks > 8.0 * lora::device_sm_count();
}

size_t workspace_bytes(const lora::AttnView &v, const lora_kv_cache_t *c, lora_dtype_t dtype) {
    return many_queries(v, c, dtype) ? lora::prefill_workspace_bytes(c->head_dim) : lora::decode_workspace_bytes(c->head_dim);
}

}  // namespace

extern "C" {

lora_status_t lora_rope(const lora_rope_args_t *a, void *stream) {
    lora::RopeView v;
    const lora_status_t s = check_rope(a, &v);
    if (s != LORA_OK || a->rows == 0) return s;
    cudaError_t e = lora::device_status_ptr(&v.status);
    if (e == cudaSuccess) e = lora::launch_rope(v, a->dtype, as_stream(stream));
    return e == cudaSuccess ? LORA_OK : fail(e);
}

lora_status_t lora_norm_rope(const lora_norm_rope_args_t *a, void *stream) {
    lora::NormRopeView v;
    const lora_status_t s = check_norm_rope(a, &v);
    if (s != LORA_OK || a->rope.rows == 0) return s;
    cudaError_t e = lora::device_status_ptr(&v.rope.status);
    if (e == cudaSuccess) e = lora::launch_norm_rope(v, a->rope.dtype, as_stream(stream));
    return e == cudaSuccess ? LORA_OK : fail(e);
}

size_t lora_norm_rope_backward_workspace_bytes(const lora_norm_rope_args_t *a) {
    lora::NormRopeView v;
    return check_norm_rope(a, &v) == LORA_OK ? lora::norm_rope_workspace_bytes(a->rope.head_dim) : 0;
}

lora_status_t lora_norm_rope_backward(const lora_norm_rope_args_t *a, const lora_norm_rope_grads_t *g, void *stream) {
    lora::NormRopeView v;
    lora_status_t s = check_norm_rope(a, &v);
    if (s != LORA_OK) return s;
    if (!g) return LORA_ERR_INVALID_ARG;
    s = check_heads(&g->dq, a->rope.dtype, a->rope.rows, &v.dq);
    if (s == LORA_OK) s = check_heads(&g->dk, a->rope.dtype, a->rope.num_k_heads ? a->rope.rows : 0, &v.dk);
    if (s != LORA_OK) return s;
    if (!aligned(g->dq_weight, 4) || !aligned(g->dk_weight, 4)) return LORA_ERR_ALIGNMENT;
    cudaStream_t st = as_stream(stream);
    if (a->rope.rows == 0) {  // sums of nothing
        const size_t bytes = sizeof(float) * a->rope.head_dim;
        cudaError_t e = g->dq_weight ? cudaMemsetAsync(g->dq_weight, 0, bytes, st) : cudaSuccess;
        if (e == cudaSuccess && g->dk_weight) e = cudaMemsetAsync(g->dk_weight, 0, bytes, st);
        return e == cudaSuccess ? LORA_OK : fail(e);
    }
    if (g->dq_weight || g->dk_weight) {
        if (!g->workspace || g->workspace_bytes < lora::norm_rope_workspace_bytes(a->rope.head_dim)) return LORA_ERR_WORKSPACE;
        if (!aligned(g->workspace, 16)) return LORA_ERR_ALIGNMENT;
        v.partial = static_cast<float *>(g->workspace);
    }
    cudaError_t e = lora::device_status_ptr(&v.rope.status);
    if (e == cudaSuccess) e = lora::launch_norm_rope_backward(v, a->rope.dtype, g->dq_weight, g->dk_weight, st);
    return e == cudaSuccess ? LORA_OK : fail(e);
}

size_t lora_kv_pages_bytes(int32_t num_pages, int32_t num_heads, int32_t head_dim, int32_t page_tokens) {
    if (num_pages <= 0 || num_heads <= 0 || head_dim <= 0 || page_tokens <= 0) return 0;
    return static_cast<size_t>(num_pages) * num_heads * head_dim * page_tokens;
}

size_t lora_kv_codes_bytes(lora_kv_format_t format, int32_t num_pages, int32_t num_heads, int32_t head_dim, int32_t page_tokens) {
    const size_t n = lora_kv_pages_bytes(num_pages, num_heads, head_dim, page_tokens);
    return format == LORA_KV_UINT4 ? n / 2 : format == LORA_KV_INT8 || format == LORA_KV_E4M3 ? n : 0;
}

size_t lora_kv_scales_bytes(lora_kv_format_t format, int32_t num_pages, int32_t num_heads, int32_t head_dim, int32_t page_tokens) {
    const size_t n = lora_kv_codes_bytes(format, num_pages, num_heads, head_dim, page_tokens);
    if (n == 0) return 0;
    return format == LORA_KV_UINT4 ? n / 8 : static_cast<size_t>(num_pages) * num_heads * sizeof(float);
}

static lora_status_t rows_call(bool append, const lora_kv_cache_t *cache, const lora_kv_batch_t *batch,
                               lora_dtype_t dtype, const lora_heads_t *k, const lora_heads_t *v, void *stream) {
    lora::KvView view;
    lora_status_t s = check_batch(cache, batch, &view);
    if (s != LORA_OK) return s;
    if (!valid_dtype(dtype)) return LORA_ERR_DTYPE;
    lora::HeadsView kh, vh;
    s = check_heads(k, dtype, batch->rows, &kh);
    if (s == LORA_OK) s = check_heads(v, dtype, batch->rows, &vh);
    if (s != LORA_OK) return s;
    if (batch->rows == 0 || batch->num_seqs == 0) return LORA_OK;
    cudaError_t e = lora::device_status_ptr(&view.status);
    if (e == cudaSuccess && cache->format == LORA_KV_UINT4)
        e = (append ? lora::launch_kv_append4 : lora::launch_kv_gather4)(view, cache->head_dim, dtype, kh, vh, as_stream(stream));
    else if (e == cudaSuccess)
        e = (append ? lora::launch_kv_append : lora::launch_kv_gather)(view, cache->format, cache->head_dim, dtype, kh,
                                                                       vh, as_stream(stream));
    return e == cudaSuccess ? LORA_OK : fail(e);
}

lora_status_t lora_kv_append(const lora_kv_cache_t *cache, const lora_kv_batch_t *batch, lora_dtype_t dtype,
                             const lora_heads_t *k, const lora_heads_t *v, void *stream) {
    return rows_call(true, cache, batch, dtype, k, v, stream);
}

lora_status_t lora_kv_gather(const lora_kv_cache_t *cache, const lora_kv_batch_t *batch, lora_dtype_t dtype,
                             const lora_heads_t *k, const lora_heads_t *v, void *stream) {
    return rows_call(false, cache, batch, dtype, k, v, stream);
}

size_t lora_kv_attention_workspace_bytes(const lora_kv_cache_t *cache, const lora_kv_batch_t *batch,
                                         const lora_kv_attention_args_t *args) {
    lora::AttnView v;
    if (check_attention(cache, batch, args, &v) != LORA_OK) return 0;
    return workspace_bytes(v, cache, args->dtype);
}

lora_status_t lora_kv_attention(const lora_kv_cache_t *cache, const lora_kv_batch_t *batch,
                                const lora_kv_attention_args_t *args, void *stream) {
    lora::AttnView v;
    lora_status_t s = check_attention(cache, batch, args, &v);
    if (s != LORA_OK) return s;
    if (batch->rows == 0 || batch->num_seqs == 0) return LORA_OK;
    const size_t need = workspace_bytes(v, cache, args->dtype);
    if (!v.workspace || args->workspace_bytes < need) return LORA_ERR_WORKSPACE;
    if (!aligned(v.workspace, 16)) return LORA_ERR_ALIGNMENT;
    cudaError_t e = lora::device_status_ptr(&v.kv.status);
    v.test_wait_ns = lora::take_test_wait_limit();
    if (e == cudaSuccess)
        e = many_queries(v, cache, args->dtype)
                ? lora::launch_attn_prefill(v, cache->format, cache->head_dim, as_stream(stream))
            : cache->format == LORA_KV_UINT4
                ? lora::launch_attn_decode4(v, cache->head_dim, args->dtype, as_stream(stream))
                : lora::launch_attn_decode(v, cache->format, cache->head_dim, args->dtype, as_stream(stream));
    return e == cudaSuccess ? LORA_OK : fail(e);
}

}  // extern "C"
