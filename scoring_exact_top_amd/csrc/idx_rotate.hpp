// Norm and rotation of heads, and the append that norms and rotates on the way: host entry
// points implemented in idx_rotate.hip.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "idx_topk.h"

namespace idxk {

int norm_rotate(const void* x, int64_t x_token, int64_t x_head, int32_t norm, const void* weight, const void* bias, float eps,
                const int32_t* positions, const float* table, int32_t table_rows, int32_t rope_at, int32_t interleaved,
                int32_t T, int32_t H, int32_t D, int32_t dtype, void* out, int64_t out_token, int64_t out_head,
                uint8_t* codes, float* scales, hipStream_t stream);

int cache_append_rotary(const void* latents, int64_t latent_token, int32_t latent_norm, const void* latent_weight,
                        float latent_eps, int32_t latent_interleaved, const void* index_keys, int64_t key_token,
                        int32_t key_norm, const void* key_weight, const void* key_bias, float key_eps, int32_t key_rope_at,
                        int32_t key_interleaved, const int32_t* slots, const int32_t* positions, const float* table,
                        int32_t table_rows, int32_t T, int32_t dtype, void* latent_cache, uint8_t* k_cache, float* k_scale,
                        int64_t num_slots, void* latents_out, hipStream_t stream);

}  // namespace idxk
