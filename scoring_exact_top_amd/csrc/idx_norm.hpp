// Norm to e4m3 and cache append: host entry points implemented in idx_norm.hip.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "idx_topk.h"

namespace idxk {

int norm_quant(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride, const void* weight,
               float eps, int32_t rows, int32_t width, int32_t group, int32_t dtype, uint8_t* codes, float* scales,
               void* residual_out, hipStream_t stream);

int cache_append(const void* latents, int64_t latent_token, const void* index_keys, int64_t key_token,
                 const int32_t* slots, int32_t T, int32_t dtype, void* latent_cache, uint8_t* k_cache, float* k_scale,
                 int64_t num_slots, hipStream_t stream);

}  // namespace idxk
