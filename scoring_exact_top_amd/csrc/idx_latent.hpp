// Latent attention: host entry points implemented in idx_latent.hip (absorbed
// form, over listed slots or paged sequences) and idx_expanded.hip.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "idx_topk.h"

namespace idxk {

constexpr int kLatent = IDX_TOPK_LATENT;
constexpr int kRope = IDX_TOPK_ROPE;
constexpr int kLatRow = kLatent + kRope;  // numbers of a latent row
constexpr int kNope = IDX_TOPK_NOPE;
constexpr int kValue = IDX_TOPK_VALUE;
constexpr int kMaxHeads = IDX_TOPK_MAX_ATTN_HEADS;

size_t latent_selected_workspace_bytes(int32_t T, int32_t H, int32_t K);
int latent_selected(const void* q, int64_t q_token, int64_t q_head, const void* cache, int64_t num_slots,
                    const int32_t* slots, int32_t K, int32_t T, int32_t H, float scale, int32_t dtype, void* out,
                    float* lse, void* workspace, size_t workspace_bytes, hipStream_t stream);

size_t latent_paged_workspace_bytes(int32_t B, int32_t S, int32_t H, int32_t max_pages);
int latent_paged(const void* q, int64_t q_seq, int64_t q_token, int64_t q_head, const void* cache,
                 int32_t num_pages, const int32_t* page_table, int32_t max_pages, const int32_t* seq_lens, int32_t B,
                 int32_t S, int32_t H, float scale, int32_t dtype, void* out, float* lse, void* workspace,
                 size_t workspace_bytes, hipStream_t stream);

size_t latent_expanded_workspace_bytes(int32_t Tq, int32_t B, int32_t max_q, int32_t max_k, int32_t H);
int latent_expanded(const void* q, int64_t q_token, int64_t q_head, const void* kv, int64_t kv_token,
                    int64_t kv_head, const void* k_rope, int64_t rope_token, const int32_t* cu_q,
                    const int32_t* cu_k, int32_t B, int32_t Tq, int32_t Tk, int32_t max_q, int32_t max_k, int32_t H,
                    float scale, int32_t causal, int32_t dtype, void* out, float* lse, void* workspace,
                    size_t workspace_bytes, hipStream_t stream);

}  // namespace idxk
