// Root-mean-square norm with the residual's addition to e4m3 codes and scales, and the append
// of new tokens to the caches (gfx950).  Both are bound by memory: every input is read once and
// every output written once.  Measured: 8192 rows of 5120 with the residual 55.2 us, 5.3 TB/s;
// 30000 appended tokens 16.1 us, 5.0 TB/s (a large copy reaches 4.7); 1024 rows of 128 take 3 us on
// the card, and the host sets the call's 7.3.
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
static dim3 grid_of(int64_t groups) {
  return groups <= kGridX ? dim3((uint32_t)groups) : dim3((uint32_t)kGridX, (uint32_t)((groups + kGridX - 1) / kGridX));
}

// Rows in chunks of 8 numbers, one load each: TPR threads a row (16, 64
// or 256), NC chunks a thread, h kept in registers between the passes, so
// that every byte is moved once.  A group of 128 columns is 16 neighbouring
// chunks: its maximum needs four exchanges within 16 lanes.  kAny: rows of any
// width (the last chunk may be short: zeros change neither sum nor maximum) and alignment.
template <class E, int TPR, int NC, bool kAny>
__global__ __launch_bounds__(256) void k_norm_rows(NormArgs A) {
  typedef E v8 __attribute__((ext_vector_type(8)));
  typedef E v8u __attribute__((ext_vector_type(8), aligned(2)));
  typedef uint32_t u2u __attribute__((ext_vector_type(2), aligned(1)));
  __shared__ float s_sum[4];
  __shared__ uint32_t s_top[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t row = workgroup() * (256 / TPR) + tid / TPR;
  const int at = tid % TPR;  // this thread's first chunk
  const int chunks = (A.width + 7) >> 3;
  const bool live = row < A.rows;
  const E* x = static_cast<const E*>(A.x) + row * A.x_stride;
  const E* res = A.residual ? static_cast<const E*>(A.residual) + row * A.residual_stride : nullptr;
  const E* w = static_cast<const E*>(A.weight);

  float h[NC][8];
  {
    v8 xv[NC], rv[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = at + c * TPR;
      const bool in = live && i < chunks;
      xv[c] = in ? load8<kAny>(x + 8 * i, A.width - 8 * i) : v8{};
      rv[c] = in && res ? load8<kAny>(res + 8 * i, A.width - 8 * i) : v8{};
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) h[c][j] = res ? (float)xv[c][j] + (float)rv[c][j] : (float)xv[c][j];
  }
  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    float t = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) t = fmaf(h[c][j], h[c][j], t);
    ss += t;
  }
#pragma unroll
  for (int d = 1; d < (TPR < 64 ? TPR : 64); d <<= 1) ss += __shfl_xor(ss, d, 64);
  if (TPR == 256) {
    if (lane == 0) s_sum[wave] = ss;
    __syncthreads();
    ss = (s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]);
  }
  if (A.residual_out) {
    E* out = static_cast<E*>(A.residual_out) + row * A.width;  // it may be x or residual itself: what this thread read
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = at + c * TPR;
      v8 v;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = (E)h[c][j];
      if (!live || i >= chunks) continue;
      if (!kAny) *reinterpret_cast<v8*>(out + 8 * i) = v;
      else if (8 * i + 8 <= A.width) *reinterpret_cast<v8u*>(out + 8 * i) = v;
      else
#pragma unroll
        for (int j = 0; j < 7; ++j)
          if (8 * i + j < A.width) out[8 * i + j] = v[j];
    }
  }
  const float ms = ss / (float)A.width + A.eps;
  float rstd = ms < INFINITY ? 1.f / sqrtf(ms) : NAN;  // a NaN or an infinity in the row, or its squares left FP32
  if (ms == 0.f) {  // no eps: zeros stay zeros, and numbers whose squares are lost have no norm here
    rstd = 1.f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) h[c][j] = h[c][j] == 0.f ? 0.f : INFINITY;
  }
  uint32_t top[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int i = at + c * TPR;
    v8 wv = {};
    if (w && i < chunks) wv = load8<kAny>(w + 8 * i, A.width - 8 * i);
    top[c] = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      h[c][j] = h[c][j] * rstd * (w ? (float)wv[j] : 1.f);
      top[c] = max(top[c], magnitude(h[c][j]));
    }
  }
  if (A.group) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) top[c] = max(top[c], (uint32_t)__shfl_xor((int)top[c], d, 64));
  } else {
    uint32_t t = top[0];
#pragma unroll
    for (int c = 1; c < NC; ++c) t = max(t, top[c]);
#pragma unroll
    for (int d = 1; d < (TPR < 64 ? TPR : 64); d <<= 1) t = max(t, (uint32_t)__shfl_xor((int)t, d, 64));
    if (TPR == 256) {
      if (lane == 0) s_top[wave] = t;
      __syncthreads();
      t = max(max(s_top[0], s_top[1]), max(s_top[2], s_top[3]));
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) top[c] = t;
  }
  if (!live) return;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int i = at + c * TPR;
    if (i >= chunks) break;
    const float scale = scale_of(top[c]);
    const Scaler to(scale);
    uint2 v;
    v.x = e4m3x2_enc(to(h[c][0]), to(h[c][1])) | e4m3x2_enc(to(h[c][2]), to(h[c][3])) << 16;
    v.y = e4m3x2_enc(to(h[c][4]), to(h[c][5])) | e4m3x2_enc(to(h[c][6]), to(h[c][7])) << 16;
    if (!finite(top[c])) v.x = v.y = kNanCodes;
    uint8_t* codes = A.codes + row * A.width + 8 * i;
    if (!kAny) *reinterpret_cast<uint2*>(codes) = v;
    else if (8 * i + 8 <= A.width) *reinterpret_cast<u2u*>(codes) = u2u{v.x, v.y};
    else
#pragma unroll
      for (int j = 0; j < 7; ++j)
        if (8 * i + j < A.width) codes[j] = (uint8_t)((j < 4 ? v.x : v.y) >> 8 * (j & 3));
    if (A.group) {
      if ((i & 15) == 0) A.scales[row * (A.width / kGroup) + (i >> 4)] = scale;
    } else if (i == 0) {
      A.scales[row] = scale;
    }
  }
}

// Threads a row: the fewest whose registers hold it, so that short rows share a workgroup.
template <class E, bool kAny>
static void launch_rows(const NormArgs& A, hipStream_t stream) {
  const int chunks = (A.width + 7) >> 3;
  const auto grid = [&](int tpr) { return grid_of(((int64_t)A.rows * tpr + 255) / 256); };
  if (chunks <= 16) k_norm_rows<E, 16, 1, kAny><<<grid(16), dim3(256), 0, stream>>>(A);
  else if (chunks <= 64) k_norm_rows<E, 64, 1, kAny><<<grid(64), dim3(256), 0, stream>>>(A);
  else if (chunks <= 128) k_norm_rows<E, 64, 2, kAny><<<grid(64), dim3(256), 0, stream>>>(A);
  else if (chunks <= 256) k_norm_rows<E, 256, 1, kAny><<<grid(256), dim3(256), 0, stream>>>(A);
  else if (chunks <= 512) k_norm_rows<E, 256, 2, kAny><<<grid(256), dim3(256), 0, stream>>>(A);
  else if (chunks <= 768) k_norm_rows<E, 256, 3, kAny><<<grid(256), dim3(256), 0, stream>>>(A);
  else if (chunks <= 1024) k_norm_rows<E, 256, 4, kAny><<<grid(256), dim3(256), 0, stream>>>(A);
  else k_norm_rows<E, 256, 8, kAny><<<grid(256), dim3(256), 0, stream>>>(A);
}

// Rows of whole chunks on 16 bytes need no tests: 52.6 us against 55.2 through the general form for 8192
// rows of 5120 with the residual, 11.3 against 12.1 for 8192 of 1024 (8 bytes off: 55.7 and 11.9).
template <class E>
static void launch_norm(const NormArgs& A, hipStream_t stream) {
  const bool whole = (A.width & 7) == 0 && (((uintptr_t)A.x | (uintptr_t)A.residual | (uintptr_t)A.weight |
                     (uintptr_t)A.residual_out) & 15u) == 0 && ((uintptr_t)A.codes & 7u) == 0 &&
                     (A.rows == 1 || (A.x_stride & 7) == 0) && (!A.residual || A.rows == 1 || (A.residual_stride & 7) == 0);
  if (whole) launch_rows<E, false>(A, stream);
  else launch_rows<E, true>(A, stream);
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
  const int64_t t = workgroup() * 4 + (threadIdx.x >> 6);
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
    const uint32_t top = wave_max(max(magnitude(a), magnitude(b)));
    const float scale = scale_of(top);
    const Scaler to(scale);
    reinterpret_cast<uint16_t*>(A.k_cache + slot * kD)[lane] = (uint16_t)(finite(top) ? e4m3x2_enc(to(a), to(b)) : kNanCodes);
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
  if (dtype == IDX_TOPK_BF16) launch_norm<__bf16>(A, stream);
  else launch_norm<_Float16>(A, stream);
  return hipGetLastError() == hipSuccess ? IDX_OK : IDX_EHIP;
}

int cache_append(const void* latents, int64_t latent_token, const void* index_keys, int64_t key_token,
                 const int32_t* slots, int32_t T, int32_t dtype, void* latent_cache, uint8_t* k_cache, float* k_scale,
                 int64_t num_slots, hipStream_t stream) {
  if (T < 0 || num_slots < 0 || latent_token < 0 || (latent_token & 7) || key_token < 0 || (key_token & 7)) return IDX_EINVAL;
  if (dtype != IDX_TOPK_BF16 && dtype != IDX_TOPK_F16) return IDX_EINVAL;
  if (T == 0 || num_slots == 0) return IDX_OK;  // empty tensors have no address
  if ((!latents) != (!latent_cache) || (!index_keys) != (!k_cache) || (!k_cache) != (!k_scale)) return IDX_EINVAL;
  if (!latents && !index_keys) return IDX_OK;
  if (!slots || !aligned16(latents) || !aligned16(latent_cache) || !aligned16(index_keys) || !aligned16(k_cache) ||
      (((uintptr_t)k_scale | (uintptr_t)slots) & 3u))
    return IDX_EINVAL;
  const AppendArgs A{static_cast<const char*>(latents), latent_token, static_cast<const char*>(index_keys), key_token,
                     slots, T, static_cast<char*>(latent_cache), k_cache, k_scale, num_slots};
  const dim3 grid = grid_of(((int64_t)T + 3) / 4);
  if (dtype == IDX_TOPK_BF16) k_append<__bf16><<<grid, dim3(256), 0, stream>>>(A);
  else k_append<_Float16><<<grid, dim3(256), 0, stream>>>(A);
  return hipGetLastError() == hipSuccess ? IDX_OK : IDX_EHIP;
}

}  // namespace idxk
