// Root-mean-square norm with the residual's addition to e4m3 codes and scales, and the append
// of new tokens to the caches (gfx950).  Both are bound by memory: every input is read once and
// every output written once.
#include "idx_common.hpp"
#include "idx_latent.hpp"
#include "idx_norm.hpp"

namespace idxk {

constexpr float kE4m3Max = 448.f;
constexpr int kGroup = 128;
constexpr int kMaxWidth = 16384;

struct NormArgs {
  const void* x;
  int64_t x_stride;
  const void* residual;
  int64_t residual_stride;
  const void* weight;
  float eps;
  int32_t rows, width, group;
  uint8_t* codes;
  float* scales;
  void* residual_out;
};

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) x += __shfl_xor(x, d, 64);
  return x;
}
__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) x = fmaxf(x, __shfl_xor(x, d, 64));
  return x;
}

// One row a workgroup, element by element, h computed again in each pass:
// any width, stride and alignment.
template <class E>
__global__ __launch_bounds__(256) void k_norm_any(NormArgs A) {
  __shared__ float s_red[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t row = blockIdx.x;
  const E* x = static_cast<const E*>(A.x) + row * A.x_stride;
  const E* res = A.residual ? static_cast<const E*>(A.residual) + row * A.residual_stride : nullptr;
  const E* w = static_cast<const E*>(A.weight);
  const auto hidden = [&](int i) { return res ? (float)x[i] + (float)res[i] : (float)x[i]; };
  float ss = 0.f;
  for (int i = tid; i < A.width; i += 256) {
    const float v = hidden(i);
    ss = fmaf(v, v, ss);
  }
  ss = wave_sum(ss);
  if (lane == 0) s_red[wave] = ss;
  __syncthreads();
  ss = (s_red[0] + s_red[1]) + (s_red[2] + s_red[3]);
  __syncthreads();
  const float rstd = 1.f / sqrtf(ss / (float)A.width + A.eps);
  const auto value = [&](int i) { return hidden(i) * rstd * (w ? (float)w[i] : 1.f); };
  const int step = A.group ? A.group : A.width;
  for (int g0 = 0, g = 0; g0 < A.width; g0 += step, ++g) {
    float top = 0.f;
    for (int i = g0 + tid; i < g0 + step; i += 256) top = fmaxf(top, fabsf(value(i)));
    top = wave_max(top);
    if (lane == 0) s_red[wave] = top;
    __syncthreads();
    top = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
    __syncthreads();
    const float scale = top > 0.f ? top / kE4m3Max : 1.f;
    for (int i = g0 + tid; i < g0 + step; i += 256) {
      A.codes[row * A.width + i] = (uint8_t)e4m3x2_enc(value(i) / scale, 0.f);
    }
    if (tid == 0) A.scales[row * (A.width / step) + g] = scale;
  }
  if (A.residual_out) {
    // last: it may be x or residual itself, and each thread rewrites what only it read since the barrier
    E* out = static_cast<E*>(A.residual_out) + row * A.width;
    __syncthreads();
    for (int i = tid; i < A.width; i += 256) out[i] = (E)hidden(i);
  }
}

struct AppendArgs {
  const char* latents;
  int64_t latent_token;
  const char* keys;
  int64_t key_token;
  const int32_t* slots;
  int32_t T;
  char* latent_cache;
  uint8_t* k_cache;
  float* k_scale;
  int64_t num_slots;
};

// One wave a token: 72 16-byte chunks of the latent row, two numbers of the
// index key a lane.
template <class E>
__global__ __launch_bounds__(256) void k_append(AppendArgs A) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= A.T) return;
  const int64_t slot = A.slots[t];
  if (slot < 0 || slot >= A.num_slots) return;
  if (A.latent_cache) {
    const uint4* src = reinterpret_cast<const uint4*>(A.latents + t * A.latent_token * 2);
    uint4* dst = reinterpret_cast<uint4*>(A.latent_cache + slot * (kLatRow * 2));
    dst[lane] = src[lane];
    if (lane < 8) dst[64 + lane] = src[64 + lane];
  }
  if (A.k_cache) {
    const E* k = reinterpret_cast<const E*>(A.keys) + t * A.key_token + 2 * lane;
    const float a = (float)k[0], b = (float)k[1];
    const float top = wave_max(fmaxf(fabsf(a), fabsf(b)));
    const float scale = top > 0.f ? top / kE4m3Max : 1.f;
    reinterpret_cast<uint16_t*>(A.k_cache + slot * kD)[lane] = (uint16_t)e4m3x2_enc(a / scale, b / scale);
    if (lane == 0) A.k_scale[slot] = scale;
  }
}

// ------------------------------------------------------------------ host

static inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

int norm_quant(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride, const void* weight,
               float eps, int32_t rows, int32_t width, int32_t group, int32_t dtype, uint8_t* codes, float* scales,
               void* residual_out, hipStream_t stream) {
  if (rows < 0 || width < 1 || width > kMaxWidth || x_stride < 0 || residual_stride < 0 || !(eps >= 0.f) || !(eps < INFINITY))
    return IDX_EINVAL;
  if (dtype != IDX_TOPK_BF16 && dtype != IDX_TOPK_F16) return IDX_EINVAL;
  if (group != 0 && group != kGroup) return IDX_EUNSUPPORTED;
  if (group != 0 && width % group != 0) return IDX_EINVAL;
  if (rows == 0) return IDX_OK;
  if (!x || !codes || !scales) return IDX_EINVAL;
  if (((uintptr_t)x | (uintptr_t)residual | (uintptr_t)weight | (uintptr_t)residual_out) & 1u) return IDX_EINVAL;
  if ((uintptr_t)scales & 3u) return IDX_EINVAL;
  if (rows > 1 && residual_out && ((residual_out == x && x_stride != width) || (residual_out == residual && residual_stride != width)))
    return IDX_EINVAL;
  const NormArgs A{x, x_stride, residual, residual_stride, weight, eps, rows, width, group, codes, scales, residual_out};
  if (dtype == IDX_TOPK_BF16) k_norm_any<__bf16><<<dim3(rows), dim3(256), 0, stream>>>(A);
  else k_norm_any<_Float16><<<dim3(rows), dim3(256), 0, stream>>>(A);
  return hipGetLastError() == hipSuccess ? IDX_OK : IDX_EHIP;
}

int cache_append(const void* latents, int64_t latent_token, const void* index_keys, int64_t key_token,
                 const int32_t* slots, int32_t T, int32_t dtype, void* latent_cache, uint8_t* k_cache, float* k_scale,
                 int64_t num_slots, hipStream_t stream) {
  if (T < 0 || num_slots < 0 || latent_token < 0 || (latent_token & 7) || key_token < 0 || (key_token & 7)) return IDX_EINVAL;
  if (dtype != IDX_TOPK_BF16 && dtype != IDX_TOPK_F16) return IDX_EINVAL;
  if ((!latents) != (!latent_cache) || (!index_keys) != (!k_cache) || (!k_cache) != (!k_scale)) return IDX_EINVAL;
  if (T == 0 || num_slots == 0 || (!latents && !index_keys)) return IDX_OK;
  if (!slots || !aligned16(latents) || !aligned16(latent_cache) || !aligned16(index_keys) || !aligned16(k_cache) ||
      ((uintptr_t)k_scale & 3u))
    return IDX_EINVAL;
  const AppendArgs A{static_cast<const char*>(latents), latent_token, static_cast<const char*>(index_keys), key_token,
                     slots, T, static_cast<char*>(latent_cache), k_cache, k_scale, num_slots};
  const dim3 grid((uint32_t)(((int64_t)T + 3) / 4));
  if (dtype == IDX_TOPK_BF16) k_append<__bf16><<<grid, dim3(256), 0, stream>>>(A);
  else k_append<_Float16><<<grid, dim3(256), 0, stream>>>(A);
  return hipGetLastError() == hipSuccess ? IDX_OK : IDX_EHIP;
}

}  // namespace idxk
