// Matrix product of e4m3 operands with block scales: host entry points implemented in
// idx_matmul.hip.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "idx_topk.h"

namespace idxk {

int matmul_e4m3(const uint8_t* x, int64_t x_row, const float* x_scale, int32_t x_group, const uint8_t* w,
                const float* w_scale, int32_t M, int32_t N, int32_t K, int32_t dtype, void* out, int64_t out_row,
                hipStream_t stream);

}  // namespace idxk
