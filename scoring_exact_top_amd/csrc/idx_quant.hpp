// Building blocks of the kernels that read rows of 16-bit numbers and write e4m3 codes with
// scales (gfx950): maxima that keep NaN, the scale and the quotient, loads at any alignment,
// grids of any size.
#pragma once
#include "idx_common.hpp"

namespace idxk {

constexpr float kE4m3Max = 448.f;

// Largest magnitudes are taken over the bits of |y| as integers: these order
// finite numbers as the numbers do, infinity above them and every NaN above
// that, so that a maximum keeps what fmaxf would drop.
__device__ __forceinline__ uint32_t magnitude(float y) { return __float_as_uint(y) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) x = max(x, (uint32_t)__shfl_xor((int)x, d, 64));
  return x;
}
__device__ __forceinline__ bool finite(uint32_t top) { return top < 0x7f800000u; }

// The scale of a group whose largest magnitude is top: 1 for an all-zero group
// (and for one so small that its scale would round to 0), and for one with a NaN
// or an infinity, whose codes are all NaN.
__device__ __forceinline__ float scale_of(uint32_t top) {
  const float s = __uint_as_float(top) / kE4m3Max;
  return finite(top) && s > 0.f ? s : 1.f;
}
constexpr uint32_t kNanCodes = 0x7f7f7f7fu;

// value / scale, rounded to FP32 once, with one division a group: the product
// with the reciprocal is corrected by its own remainder, which an FMA gives
// exactly (r = v - q s; q + r / s).  The product alone falls on the other side of
// a tie between codes for one in 2000 of 16-bit keys.  `up` lifts small scales
// so that neither the reciprocal nor the remainder leaves FP32 (a power of two: exact).
struct Scaler {
  float up, s, inv;
  __device__ __forceinline__ explicit Scaler(float scale)
      : up(scale < 0x1p-64f ? 0x1p96f : 1.f), s(scale * up), inv(1.f / s) {}
  __device__ __forceinline__ float operator()(float v) const {
    const float q = v * up * inv;
    return fmaf(fmaf(-q, s, v * up), inv, q);
  }
};

// Eight numbers at p, or the n there are and zeros.  kAny: at any address (the memory pipeline takes
// unaligned 16-byte accesses); else all eight, on 16 bytes.
template <bool kAny, class E>
__device__ __forceinline__ auto load8(const E* p, int n) {
  typedef E v8 __attribute__((ext_vector_type(8)));
  typedef E v8u __attribute__((ext_vector_type(8), aligned(2)));
  if (!kAny) return *reinterpret_cast<const v8*>(p);
  if (n >= 8) return (v8)*reinterpret_cast<const v8u*>(p);
  v8 v = {};
#pragma unroll
  for (int j = 0; j < 7; ++j)
    if (j < n) v[j] = p[j];
  return v;
}

// A launch dimension takes fewer than 2^32 threads (a larger one wraps, without an
// error): workgroups of 256 beyond 2^22 go on in the second dimension.
constexpr int64_t kGridX = 1 << 22;
__device__ __forceinline__ int64_t workgroup() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }
static inline dim3 grid_of(int64_t groups) {
  return groups <= kGridX ? dim3((uint32_t)groups) : dim3((uint32_t)kGridX, (uint32_t)((groups + kGridX - 1) / kGridX));
}

}  // namespace idxk
