// Shared between the host side and the kernels of lora_attention.h.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "lora_attention.h"
#include "lora_internal.h"

namespace lora {

constexpr int kKvTile = LORA_BLOCK_ROWS;  // tokens of one tile of codes
constexpr int kMaxGroup = 64;             // query heads that share a key/value head

// Kernel view of a cache and of the call's rows.
struct KvView {
    uint8_t *k_pages, *v_pages;
    float *k_scales, *v_scales;
    const int32_t *seq_lens, *offsets, *table;
    int32_t num_pages, heads, page_tokens, page_shift;  // page_tokens = 1 << page_shift
    int32_t num_seqs, rows, max_pages;
    int32_t growth;  // lora_kv_growth_t
    unsigned long long *status;
};

struct HeadsView {
    void *p;
    int64_t row, head;  // strides in elements
};

struct RopeView {
    HeadsView q, q_out, k, k_out;
    const float *cos_table, *sin_table;
    const int32_t *positions;
    unsigned long long *status;
    int32_t rows, head_dim, rot_dim, q_heads, k_heads, max_pos, num_axes;
    int32_t interleaved, inverse;
    uint8_t pair_axis[LORA_ROPE_MAX_PAIRS];
    uint8_t chunk_axis[LORA_ROPE_MAX_PAIRS / 4];  // of a thread's pairs, or LORA_ROPE_MAX_AXES where they differ
};

struct AttnView {
    KvView kv;
    HeadsView q, out;
    float *lse;
    int32_t q_heads, group;     // group = q_heads / kv.heads
    float scale;
    int32_t causal, window, max_queries;
    unsigned char *workspace;
    // lora_test_arm_wait_timeout: 0, or the time limit of this call's waits, of
    // which some then expect one arrival more than there is
    uint64_t test_wait_ns;
};

cudaError_t launch_rope(const RopeView &v, lora_dtype_t dtype, cudaStream_t stream);
cudaError_t launch_kv_append(const KvView &v, lora_kv_format_t fmt, int head_dim, lora_dtype_t dtype,
                             const HeadsView &k, const HeadsView &val, cudaStream_t stream);
cudaError_t launch_kv_gather(const KvView &v, lora_kv_format_t fmt, int head_dim, lora_dtype_t dtype,
                             const HeadsView &k, const HeadsView &val, cudaStream_t stream);
// Few query rows a sequence, and every fp32 call (attn_decode.cu).
size_t decode_workspace_bytes(int head_dim);
cudaError_t launch_attn_decode(const AttnView &v, lora_kv_format_t fmt, int head_dim, lora_dtype_t dtype,
                               cudaStream_t stream);

// Many query rows a sequence, bf16 (attn_prefill.cu).
size_t prefill_workspace_bytes(int head_dim);
cudaError_t launch_attn_prefill(const AttnView &v, lora_kv_format_t fmt, int head_dim, cudaStream_t stream);

}  // namespace lora
