// step.cuh -- what stands around the attention of a step: the norm and rotary position of queries and
// keys (alone, and on the way into a pool), attention under a mask, and token scores.  Launch declarations.
#pragma once

#include "attn.cuh"

namespace acache {

// Rows of queries, keys and values on their way to their outputs (kRotate: k to k_out; else k and v to
// the pool's slots).  Strides count elements.  q or (kRotate) k may be null.
enum RotateMode { kRotate = 0, kRotateStore = 1, kRotateStoreQ8 = 2 };
struct RotateCall {
    AttnArgs a;
    const acache_rope* rope;                // null: no rotation
    int64_t rows;
    const int32_t *positions, *write_slot;
    const void *q, *k, *v, *q_weight, *k_weight;
    int64_t q_stride, k_stride, v_stride;
    float eps;
    void *q_out, *k_out;
    int64_t q_out_stride, k_out_stride;
    void *k_cache, *v_cache;
    uint8_t* kv_scale;
    int64_t num_slots, private_begin;
    int32_t* dev_status;
    cudaStream_t stream;
};
int launch_rotate(const RotateCall& c, RotateMode mode);

// Attention under a mask.  q_start / kv_start: ragged batches (then n_q and T_len bound the
// per-request counts and q holds total_q rows), else null.
struct MaskedAttn {
    AttnArgs a;
    acache_mask mask;
    int B, n_q, T_len, total_q;
    const int32_t *q_start, *kv_start;
    const void* q;
    const int32_t* read_slot;
    const void *k_cache, *v_cache;
    int64_t num_slots;
    void* out;
    int32_t* dev_status;
    cudaStream_t stream;
};
int launch_masked_simt(const MaskedAttn& c);
// True when the tcgen05 kernel covers the call: bf16, a positive scale, at most 128 heads to a group, a pool with a row.
bool masked_tc_supported(const MaskedAttn& c);
int launch_masked_tc(const MaskedAttn& c);
// ... and the one for few rows per (request, KV head): at most 32 (queries x heads of a group).
bool masked_decode_supported(const MaskedAttn& c);
int launch_masked_decode(const MaskedAttn& c);

struct ScoreCall {
    int dtype;
    int64_t rows;
    int vocab;
    const void* logits;
    int64_t row_stride;
    float temperature;
    const int32_t* tokens;
    float *token_logprob, *entropy;
    int k;
    int32_t* top_tokens;
    float* top_logprob;
    int32_t* dev_status;
    cudaStream_t stream;
};
int launch_token_scores(const ScoreCall& c);

}  // namespace acache
