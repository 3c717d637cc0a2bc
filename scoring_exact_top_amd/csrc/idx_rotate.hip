// Norm of each head with the rotation of 64 of its numbers by the token's position, to 16 bits
// or to e4m3 codes, and the append of new tokens whose latent rows and index keys are normed and
// rotated on the way (gfx950).  Both are bound by memory: every number is read once and written
// once, the norm and the rotation are done in registers.
//
//   y = x                                              (no norm)
//   y = x / sqrt(mean(x^2) + eps) * weight + bias      (root mean square)
//   y = (x - mean) / sqrt(mean((x - mean)^2) + eps) * weight + bias   (layer)
//
// and numbers a = y[i], b = y[j] of a pair become a cos - b sin and b cos + a sin with the
// angle of the pair's index at the token's position: i, j = 2p, 2p + 1 of the rotary part
// (interleaved) or p, p + 32 (halves).  The angles' cosines and sines come from a table in
// FP32, which the caller computes in 64 bits: in FP32 the angle itself would be off by 2^-8 at
// position 65536.
//
// Measured (a call in a loop, the kernel alone in brackets):
//   4096 tokens x 64 heads of 128 to codes    23.8 us (25.8)  103 MB at 4.3 TB/s
//   3001 tokens x 40 heads of 128, normed     15.7 us (16.7)  62 MB at 4.0 TB/s
//   16 tokens x 128 heads of 192               7.4 us (3.4)   the host's work for a launch
//   append of 30000 tokens, rows returned     25.5 us (26.0)  123 MB at 4.8 TB/s
//   append of 16 tokens                       10.5 us (3.4)   the host's work for a launch
#include "idx_attn.hpp"
#include "idx_latent.hpp"
#include "idx_quant.hpp"
#include "idx_rotate.hpp"

namespace idxk {

constexpr int kRopeChunks = kRope / 8;  // a rotary part's chunks of 8 numbers
constexpr int kMaxHead = 1024;          // numbers of a head at most
constexpr int64_t kManyRows = 1 << 14;  // heads a lane group takes four of

struct RotArgs {
  const void* x;
  int64_t x_token, x_head;
  const void *weight, *bias;
  float eps;
  int32_t norm;
  const int32_t* positions;
  const float* table;
  int32_t table_rows, rope_at, interleaved;
  int32_t T, H, D;
  float inv_d;
  int64_t units;  // groups of lanes with heads of one token each
  void* out;
  int64_t out_token, out_head;
  uint8_t* codes;
  float* scales;
};

// The value of the lane that `CTRL` names: l ^ 1 and l ^ 2 (quad permutations), 7 - l of 8 and 15 - l of 16.
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kMirror8 = 0x141, kMirror16 = 0x140;
template <int CTRL>
__device__ __forceinline__ uint32_t lane_move(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, true);
}
// Sum and largest over N = 8, 16 or 64 neighbouring lanes, the same bits in all of them.
template <int N>
__device__ __forceinline__ float sum_lanes(float x) {
  const auto f = [](uint32_t u) { return __uint_as_float(u); };
  x += f(lane_move<kXor1>(__float_as_uint(x)));
  x += f(lane_move<kXor2>(__float_as_uint(x)));
  x += f(lane_move<kMirror8>(__float_as_uint(x)));
  if (N >= 16) x += f(lane_move<kMirror16>(__float_as_uint(x)));
  return N == 64 ? sum_quarters(x) : x;
}
template <int N>
__device__ __forceinline__ uint32_t max_lanes(uint32_t x) {
  x = max(x, lane_move<kXor1>(x));
  x = max(x, lane_move<kXor2>(x));
  x = max(x, lane_move<kMirror8>(x));
  if (N >= 16) x = max(x, lane_move<kMirror16>(x));
  if (N == 64) {
    const auto h = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    x = max(h[0], h[1]);
    const auto q = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    x = max(q[0], q[1]);
  }
  return x;
}

// sum / n rounded once, from 1 / n: the product, corrected by its own remainder.  A row of one number has that number as its
// mean then (n of it sum exactly, 16-bit numbers and n up to 1024), and no spread; the product alone may be a step
// beside it for an n that is no power of two, which without eps, or with large numbers, is all that is normed.
__device__ __forceinline__ float mean_of(float sum, float n, float inv_n) {
  const float q = sum * inv_n;
  return fmaf(fmaf(-q, n, sum), inv_n, q);
}

// A row's norm: y = (x 2^shift - mean) * (rstd * weight) + bias, the row's numbers scaled already where it is made.
struct Norm {
  float mean, rstd;
  int shift;
  // The instruction is within one unit of the last place and takes no subnormal numbers.  Below them is only a row without
  // spread, where rstd does not count and must not be infinite.
  __device__ __forceinline__ Norm(float mean, float ms, int shift = 0)
      : mean(mean), rstd(ms < INFINITY ? (ms >= 0x1p-126f ? __builtin_amdgcn_rsqf(ms) : 1.f) : NAN), shift(shift) {}
  __device__ __forceinline__ float operator()(float x, float w, float b) const { return fmaf(x - mean, rstd * w, b); }
};

// Mean (0 without `layer`) and sum of squares of a row of d numbers (inv_d = 1 / d), NC x W of them in each of L lanes,
// of which those count whose first index `there` takes (the others are zero).
template <int L, int NC, int W, class F>
__device__ __forceinline__ void moments(const float (&h)[NC][W], const F& there, bool layer, float d, float inv_d, float& mean, float& squares) {
  float sum = 0.f;
  mean = 0.f;
  if (layer) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < W; ++j) sum += h[c][j];
    mean = mean_of(sum_lanes<L>(sum), d, inv_d);
  }
  sum = 0.f;
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const float x = there(c) ? h[c][j] - mean : 0.f;
      sum = fmaf(x, x, sum);
    }
  squares = sum_lanes<L>(sum);
}

// The norm of a row.  bfloat16's numbers go from 2^-133 to 2^128, and so their squares leave FP32 on both sides: where
// the mean square is so small that FP32 may have lost numbers of it (the smallest square to keep all bits is 2^-126), or has
// passed its end, the row is scaled by the power of two that brings its largest number, or the root of eps, to about 1.
// NaN for a row with a NaN or an infinity.
template <int L, int NC, int W, class F>
__device__ __forceinline__ Norm norm_of(float (&h)[NC][W], const F& there, bool layer, float d, float inv_d, float eps) {
  float mean, squares;
  moments<L>(h, there, layer, d, inv_d, mean, squares);
  const float ms = fmaf(squares, inv_d, eps);
  if (ms > 0x1p-100f && ms < INFINITY) return Norm(mean, ms);
  uint32_t top = 0;
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int j = 0; j < W; ++j) top = max(top, magnitude(h[c][j]));
  top = max_lanes<L>(top);
  if (!finite(top)) return Norm(0.f, NAN);
  const int of_row = __builtin_amdgcn_frexp_expf(__uint_as_float(top)), of_eps = (__builtin_amdgcn_frexp_expf(eps) + 1) >> 1;
  const int shift = top == 0 ? (eps > 0.f ? -of_eps : 0) : -(eps > 0.f ? max(of_row, of_eps) : of_row);
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int j = 0; j < W; ++j) h[c][j] = __builtin_amdgcn_ldexpf(h[c][j], shift);
  moments<L>(h, there, layer, d, inv_d, mean, squares);
  return Norm(mean, fmaf(squares, inv_d, __builtin_amdgcn_ldexpf(eps, 2 * shift)), shift);
}

// Rows (a head of a token) in chunks of 8 numbers, one 16-byte load each: LPR lanes a row, NC
// chunks a lane, HP heads of one token one after another, which share position and angles.  At
// most one of a lane's chunks lies in the rotary part, which is 8 chunks long.  Where its pairs are
// halves, the chunk that holds the partners is 4 chunks away, in another lane or another
// register: it is loaded a second time (from the cache) and normed as well, which is cheaper than
// an exchange at any offset.  All lanes of a row are in one wave and have read it before one
// writes, so that out may be x.
template <class E, int LPR, int NC, int HP, bool QUANT>
__global__ __launch_bounds__(256) void k_norm_rotate(RotArgs A) {
  typedef E v8 __attribute__((ext_vector_type(8)));
  const int tid = threadIdx.x, at = tid % LPR;
  const int64_t unit = workgroup() * (256 / LPR) + tid / LPR;
  const uint32_t per = ((uint32_t)A.H + (HP - 1)) / HP;  // units of a token
  const bool in = unit < A.units;
  const uint32_t t = in ? (uint32_t)unit / per : 0, head0 = in ? (uint32_t)unit % per * HP : 0;
  const int chunks = A.D >> 3, r0 = A.rope_at >> 3;
  const int pos = in ? A.positions[t] : -1;
  const E* x = static_cast<const E*>(A.x) + (int64_t)t * A.x_token + (int64_t)head0 * A.x_head;
  const E *w = static_cast<const E*>(A.weight), *b = static_cast<const E*>(A.bias);

  const int turn = at >= r0 ? at : at + (r0 - at + LPR - 1) / LPR * LPR;  // this lane's chunk of the rotary part
  const int ci = turn - r0;
  const bool turns = in && ci < kRopeChunks;
  const bool halves = !A.interleaved;
  const int other = turn + (ci < 4 ? 4 : -4);

  v8 xv[HP][NC], pv[HP];
#pragma unroll
  for (int k = 0; k < HP; ++k) {
    const bool there = in && (int)head0 + k < A.H;
    const E* xk = x + k * A.x_head;
#pragma unroll
    for (int c = 0; c < NC; ++c) xv[k][c] = there && at + c * LPR < chunks ? *reinterpret_cast<const v8*>(xk + 8 * (at + c * LPR)) : v8{};
    pv[k] = there && turns && halves ? *reinterpret_cast<const v8*>(xk + 8 * other) : v8{};
  }
  const bool live = pos >= 0 && pos < A.table_rows;
  // halves: the chunk's 8 angles, interleaved: its 4; a lane that does not turn has angle 0
  float cs[8], sn[8];
  {
    const float* angle = A.table + (int64_t)(live ? pos : 0) * kRope + (turns ? (halves ? 8 * (ci & 3) : 4 * ci) : 0);
    const bool need = turns && live;
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f), one = make_float4(1.f, 1.f, 1.f, 1.f);
    float4 c0 = one, c1 = one, s0 = zero, s1 = zero;
    if (need) {
      c0 = *reinterpret_cast<const float4*>(angle);
      s0 = *reinterpret_cast<const float4*>(angle + kRope / 2);
      if (halves) {
        c1 = *reinterpret_cast<const float4*>(angle + 4);
        s1 = *reinterpret_cast<const float4*>(angle + kRope / 2 + 4);
      }
    }
    const float sign = halves && ci < 4 ? -1.f : 1.f;  // a cos - b sin, b cos + a sin
    cs[0] = c0.x; cs[1] = c0.y; cs[2] = c0.z; cs[3] = c0.w; cs[4] = c1.x; cs[5] = c1.y; cs[6] = c1.z; cs[7] = c1.w;
    sn[0] = s0.x * sign; sn[1] = s0.y * sign; sn[2] = s0.z * sign; sn[3] = s0.w * sign;
    sn[4] = s1.x * sign; sn[5] = s1.y * sign; sn[6] = s1.z * sign; sn[7] = s1.w * sign;
  }
  const v8 ones = {(E)1.f, (E)1.f, (E)1.f, (E)1.f, (E)1.f, (E)1.f, (E)1.f, (E)1.f};
  v8 wv[NC], bv[NC], pw = ones, pb = {};  // weight and bias of this lane's chunks and of its partners
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int i = at + c * LPR;
    wv[c] = w && i < chunks ? *reinterpret_cast<const v8*>(w + 8 * i) : ones;
    bv[c] = b && i < chunks ? *reinterpret_cast<const v8*>(b + 8 * i) : v8{};
  }
  if (w && turns && halves) pw = *reinterpret_cast<const v8*>(w + 8 * other);
  if (b && turns && halves) pb = *reinterpret_cast<const v8*>(b + 8 * other);
#pragma unroll
  for (int k = 0; k < HP; ++k) {
    float h[NC][8], p[8];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) h[c][j] = (float)xv[k][c][j];
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = (float)pv[k][j];
    if (A.norm != IDX_TOPK_NORM_NONE) {
      const Norm norm = norm_of<LPR>(h, [&](int c) { return at + c * LPR < chunks; }, A.norm == IDX_TOPK_NORM_LAYER, (float)A.D, A.inv_d, A.eps);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int i = at + c * LPR;
#pragma unroll
        for (int j = 0; j < 8; ++j) h[c][j] = i < chunks ? norm(h[c][j], (float)wv[c][j], (float)bv[c][j]) : 0.f;
      }
      if (turns && halves) {
        if (norm.shift != 0)
#pragma unroll
          for (int j = 0; j < 8; ++j) p[j] = __builtin_amdgcn_ldexpf(p[j], norm.shift);
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = norm(p[j], (float)pw[j], (float)pb[j]);
      }
    }
    if (turns) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if (NC > 1 && at + c * LPR != turn) continue;
        if (halves) {
#pragma unroll
          for (int j = 0; j < 8; ++j) h[c][j] = fmaf(h[c][j], cs[j], p[j] * sn[j]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float u = h[c][2 * j], v = h[c][2 * j + 1];
            h[c][2 * j] = fmaf(u, cs[j], -(v * sn[j]));
            h[c][2 * j + 1] = fmaf(v, cs[j], u * sn[j]);
          }
        }
      }
    }
    uint32_t top = 0;
    if (QUANT) {
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, magnitude(h[c][j]));
      top = max_lanes<LPR>(top);
    }
    if (!live || (int)head0 + k >= A.H) continue;
    const int64_t row = (int64_t)t * A.H + head0 + k;
    const float scale = scale_of(top);
    const Scaler to(scale);
    E* out = static_cast<E*>(A.out) + (int64_t)t * A.out_token + (int64_t)(head0 + k) * A.out_head;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = at + c * LPR;
      if (i >= chunks) break;
      if (QUANT) {
        uint2 v;
        v.x = e4m3x2_enc(to(h[c][0]), to(h[c][1])) | e4m3x2_enc(to(h[c][2]), to(h[c][3])) << 16;
        v.y = e4m3x2_enc(to(h[c][4]), to(h[c][5])) | e4m3x2_enc(to(h[c][6]), to(h[c][7])) << 16;
        if (!finite(top)) v.x = v.y = kNanCodes;
        *reinterpret_cast<uint2*>(A.codes + row * A.D + 8 * i) = v;
        if (i == 0) A.scales[row] = scale;
      } else {
        v8 v;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = (E)h[c][j];
        *reinterpret_cast<v8*>(out + 8 * i) = v;
      }
    }
  }
}

// Lanes a row and chunks a lane: the fewest idle lanes among shapes that keep a row in 16 lanes.  Four
// heads a lane where there are enough rows to fill the chip so (2^14 rows: one wave a SIMD).
template <class E, bool QUANT>
static void launch_rotate(RotArgs A, hipStream_t stream) {
  const int chunks = A.D >> 3;
  const bool many = (int64_t)A.T * A.H >= kManyRows && A.H >= 4;
  A.units = A.T * (many && chunks <= 24 ? ((int64_t)A.H + 3) / 4 : (int64_t)A.H);
  const auto grid = [&](int lpr) { return grid_of((A.units * lpr + 255) / 256); };
  if (chunks <= 8) {
    if (many) k_norm_rotate<E, 8, 1, 4, QUANT><<<grid(8), dim3(256), 0, stream>>>(A);
    else k_norm_rotate<E, 8, 1, 1, QUANT><<<grid(8), dim3(256), 0, stream>>>(A);
  } else if (chunks <= 16) {
    if (many) k_norm_rotate<E, 16, 1, 4, QUANT><<<grid(16), dim3(256), 0, stream>>>(A);
    else k_norm_rotate<E, 16, 1, 1, QUANT><<<grid(16), dim3(256), 0, stream>>>(A);
  } else if (chunks <= 24) {
    if (many) k_norm_rotate<E, 8, 3, 4, QUANT><<<grid(8), dim3(256), 0, stream>>>(A);
    else k_norm_rotate<E, 8, 3, 1, QUANT><<<grid(8), dim3(256), 0, stream>>>(A);
  } else if (chunks <= 32) k_norm_rotate<E, 16, 2, 1, QUANT><<<grid(16), dim3(256), 0, stream>>>(A);
  else if (chunks <= 48) k_norm_rotate<E, 16, 3, 1, QUANT><<<grid(16), dim3(256), 0, stream>>>(A);
  else if (chunks <= 80) k_norm_rotate<E, 16, 5, 1, QUANT><<<grid(16), dim3(256), 0, stream>>>(A);
  else k_norm_rotate<E, 16, 8, 1, QUANT><<<grid(16), dim3(256), 0, stream>>>(A);
}

struct AppendRotArgs {
  const char* latents;
  int64_t latent_token;
  const void* latent_weight;
  float latent_eps;
  int32_t latent_norm, latent_interleaved;
  const char* keys;
  int64_t key_token;
  const void *key_weight, *key_bias;
  float key_eps;
  int32_t key_norm, key_rope_at, key_interleaved;
  const int32_t *slots, *positions;
  const float* table;
  int32_t table_rows, T;
  char* latent_cache;
  uint8_t* k_cache;
  float* k_scale;
  int64_t num_slots;
  char* latents_out;
};

// One wave a token: a lane holds 8 of the 512 latent numbers, the first 8 lanes 8 rotary ones too,
// and every lane two neighbouring numbers of the index key, whose rotary part is 32 lanes long.
template <class E>
__global__ __launch_bounds__(256) void k_append_rotary(AppendRotArgs A) {
  typedef E v8 __attribute__((ext_vector_type(8)));
  typedef E v2 __attribute__((ext_vector_type(2)));
  const int lane = threadIdx.x & 63;
  const int64_t t = workgroup() * 4 + (threadIdx.x >> 6);
  if (t >= A.T) return;
  const int64_t slot = A.slots[t];
  const int pos = A.positions[t];
  // the token's numbers are asked for before its slot and position are looked at
  v8 xv = {}, rv = {}, pv = {}, wv = {};
  v2 kv = {}, kw = {}, kb = {};
  if (A.latent_cache) {
    const E* x = reinterpret_cast<const E*>(A.latents) + t * A.latent_token;
    xv = *reinterpret_cast<const v8*>(x + 8 * lane);
    if (lane < kRopeChunks) {
      rv = *reinterpret_cast<const v8*>(x + kLatent + 8 * lane);
      if (!A.latent_interleaved) pv = *reinterpret_cast<const v8*>(x + kLatent + 8 * (lane ^ 4));
    }
    if (A.latent_weight) wv = *reinterpret_cast<const v8*>(static_cast<const E*>(A.latent_weight) + 8 * lane);
  }
  if (A.k_cache) {
    kv = *reinterpret_cast<const v2*>(reinterpret_cast<const E*>(A.keys) + t * A.key_token + 2 * lane);
    if (A.key_weight) kw = *reinterpret_cast<const v2*>(static_cast<const E*>(A.key_weight) + 2 * lane);
    if (A.key_bias) kb = *reinterpret_cast<const v2*>(static_cast<const E*>(A.key_bias) + 2 * lane);
  }
  if (slot < 0 || slot >= A.num_slots || pos < 0 || pos >= A.table_rows) return;
  const float* angle = A.table + (int64_t)pos * kRope;
  if (A.latent_cache) {
    v8* const dst = reinterpret_cast<v8*>(A.latent_cache + slot * (kLatRow * 2));
    v8* const out = A.latents_out ? reinterpret_cast<v8*>(A.latents_out + t * (kLatRow * 2)) : nullptr;
    if (lane < kRopeChunks) {
      const int first = A.latent_interleaved ? 4 * lane : 8 * (lane & 3);
      const float4 c0 = *reinterpret_cast<const float4*>(angle + first), s0 = *reinterpret_cast<const float4*>(angle + kRope / 2 + first);
      v8 y;
      if (A.latent_interleaved) {
        const float cs[4] = {c0.x, c0.y, c0.z, c0.w}, sn[4] = {s0.x, s0.y, s0.z, s0.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float u = (float)rv[2 * j], v = (float)rv[2 * j + 1];
          y[2 * j] = (E)fmaf(u, cs[j], -(v * sn[j]));
          y[2 * j + 1] = (E)fmaf(v, cs[j], u * sn[j]);
        }
      } else {
        const float4 c1 = *reinterpret_cast<const float4*>(angle + first + 4), s1 = *reinterpret_cast<const float4*>(angle + kRope / 2 + first + 4);
        const float cs[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w}, sn[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float v = (float)pv[j] * sn[j];
          y[j] = (E)fmaf((float)rv[j], cs[j], lane < 4 ? -v : v);
        }
      }
      dst[64 + lane] = y;
      if (out) out[64 + lane] = y;
    }
    if (A.latent_norm != IDX_TOPK_NORM_NONE) {
      float h[1][8];
#pragma unroll
      for (int j = 0; j < 8; ++j) h[0][j] = (float)xv[j];
      const Norm norm = norm_of<64>(h, [](int) { return true; }, false, kLatent, 1.f / kLatent, A.latent_eps);
#pragma unroll
      for (int j = 0; j < 8; ++j) xv[j] = (E)norm(h[0][j], A.latent_weight ? (float)wv[j] : 1.f, 0.f);
    }
    dst[lane] = xv;
    if (out) out[lane] = xv;
  }
  if (A.k_cache) {
    float a = (float)kv[0], b = (float)kv[1];
    if (A.key_norm != IDX_TOPK_NORM_NONE) {
      float h[1][2] = {{a, b}};
      const Norm norm = norm_of<64>(h, [](int) { return true; }, A.key_norm == IDX_TOPK_NORM_LAYER, kD, 1.f / kD, A.key_eps);
      a = norm(h[0][0], A.key_weight ? (float)kw[0] : 1.f, (float)kb[0]);
      b = norm(h[0][1], A.key_weight ? (float)kw[1] : 1.f, (float)kb[1]);
    }
    const int c = lane - A.key_rope_at / 2;  // this lane's two numbers of the rotary part
    const bool turns = c >= 0 && c < kRope / 2;
    if (A.key_interleaved) {
      const float cs = turns ? angle[c] : 1.f, sn = turns ? angle[kRope / 2 + c] : 0.f;
      const float u = a, v = b;
      a = turns ? fmaf(u, cs, -(v * sn)) : a;
      b = turns ? fmaf(v, cs, u * sn) : b;
    } else {
      const int other = lane + (c < 16 ? 16 : -16);  // inside the wave wherever this lane turns
      const float pa = __shfl(a, other & 63, 64), pb = __shfl(b, other & 63, 64);
      if (turns) {
        const float2 cs = *reinterpret_cast<const float2*>(angle + 2 * (c & 15)), sn = *reinterpret_cast<const float2*>(angle + kRope / 2 + 2 * (c & 15));
        a = fmaf(a, cs.x, c < 16 ? -(pa * sn.x) : pa * sn.x);
        b = fmaf(b, cs.y, c < 16 ? -(pb * sn.y) : pb * sn.y);
      }
    }
    const uint32_t top = max_lanes<64>(max(magnitude(a), magnitude(b)));
    const float scale = scale_of(top);
    const Scaler to(scale);
    reinterpret_cast<uint16_t*>(A.k_cache + slot * kD)[lane] = (uint16_t)(finite(top) ? e4m3x2_enc(to(a), to(b)) : kNanCodes);
    if (lane == 0) A.k_scale[slot] = scale;
  }
}

// ------------------------------------------------------------------ host

static inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
static inline bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
static inline bool bad_stride(int64_t s) { return s < 0 || (s & 7) != 0; }

// A norm and what comes with it: weight and bias only where there is a norm, eps finite and not negative.
static bool bad_norm(int32_t norm, const void* weight, const void* bias, float eps) {
  if (norm != IDX_TOPK_NORM_NONE && norm != IDX_TOPK_NORM_RMS && norm != IDX_TOPK_NORM_LAYER) return true;
  if (norm == IDX_TOPK_NORM_NONE) return weight || bias;
  return !(eps >= 0.f) || !(eps < INFINITY) || !aligned16(weight) || !aligned16(bias);
}

int norm_rotate(const void* x, int64_t x_token, int64_t x_head, int32_t norm, const void* weight, const void* bias, float eps,
                const int32_t* positions, const float* table, int32_t table_rows, int32_t rope_at, int32_t interleaved,
                int32_t T, int32_t H, int32_t D, int32_t dtype, void* out, int64_t out_token, int64_t out_head,
                uint8_t* codes, float* scales, hipStream_t stream) {
  if (T < 0 || H < 1 || D < kRope || D > kMaxHead || (D & 7) || rope_at < 0 || (rope_at & 7) || rope_at > D - kRope || table_rows < 0)
    return IDX_EINVAL;
  if (dtype != IDX_TOPK_BF16 && dtype != IDX_TOPK_F16) return IDX_EINVAL;
  if (bad_norm(norm, weight, bias, eps) || bad_stride(x_token) || bad_stride(x_head)) return IDX_EINVAL;
  if ((!out) == (!codes) && T > 0) return IDX_EINVAL;
  if ((!codes) != (!scales)) return IDX_EINVAL;
  if (out && (bad_stride(out_token) || bad_stride(out_head) || (T > 1 && out_token < D) || (H > 1 && out_head < D))) return IDX_EINVAL;
  if ((int64_t)T * H > 0x7fffffffLL) return IDX_EUNSUPPORTED;
  if (T == 0 || table_rows == 0) return IDX_OK;  // empty tensors have no address
  if (!x || !positions || !table || !aligned16(x) || !aligned16(out) || !aligned16(codes) || !aligned16(table) || !aligned4(positions) ||
      !aligned4(scales))
    return IDX_EINVAL;
  const bool apart = (T > 1 && x_token != out_token) || (H > 1 && x_head != out_head);
  if (out == x && apart) return IDX_EINVAL;
  const RotArgs A{x, x_token, x_head, weight, bias, eps, norm, positions, table, table_rows, rope_at, interleaved ? 1 : 0,
                  T, H, D, 1.f / (float)D, 0, out, out_token, out_head, codes, scales};
  if (dtype == IDX_TOPK_BF16) {
    if (codes) launch_rotate<__bf16, true>(A, stream);
    else launch_rotate<__bf16, false>(A, stream);
  } else {
    if (codes) launch_rotate<_Float16, true>(A, stream);
    else launch_rotate<_Float16, false>(A, stream);
  }
  return hipGetLastError() == hipSuccess ? IDX_OK : IDX_EHIP;
}

int cache_append_rotary(const void* latents, int64_t latent_token, int32_t latent_norm, const void* latent_weight,
                        float latent_eps, int32_t latent_interleaved, const void* index_keys, int64_t key_token,
                        int32_t key_norm, const void* key_weight, const void* key_bias, float key_eps, int32_t key_rope_at,
                        int32_t key_interleaved, const int32_t* slots, const int32_t* positions, const float* table,
                        int32_t table_rows, int32_t T, int32_t dtype, void* latent_cache, uint8_t* k_cache, float* k_scale,
                        int64_t num_slots, void* latents_out, hipStream_t stream) {
  if (T < 0 || num_slots < 0 || table_rows < 0 || bad_stride(latent_token) || bad_stride(key_token)) return IDX_EINVAL;
  if (dtype != IDX_TOPK_BF16 && dtype != IDX_TOPK_F16) return IDX_EINVAL;
  if (latent_norm == IDX_TOPK_NORM_LAYER || bad_norm(latent_norm, latent_weight, nullptr, latent_eps) ||
      bad_norm(key_norm, key_weight, key_bias, key_eps))
    return IDX_EINVAL;
  if (key_rope_at < 0 || (key_rope_at & 7) || key_rope_at > kD - kRope) return IDX_EINVAL;
  if (T == 0 || num_slots == 0 || table_rows == 0) return IDX_OK;  // empty tensors have no address
  if ((!latents) != (!latent_cache) || (!index_keys) != (!k_cache) || (!k_cache) != (!k_scale) || (latents_out && !latents)) return IDX_EINVAL;
  if (!latents && !index_keys) return IDX_OK;
  if (!slots || !positions || !table || !aligned16(latents) || !aligned16(latent_cache) || !aligned16(index_keys) || !aligned16(k_cache) ||
      !aligned16(latents_out) || !aligned16(table) || !aligned4(k_scale) || !aligned4(slots) || !aligned4(positions))
    return IDX_EINVAL;
  if (latents_out && latents_out == latents && T > 1 && latent_token != kLatRow) return IDX_EINVAL;
  const AppendRotArgs A{static_cast<const char*>(latents), latent_token, latent_weight, latent_eps, latent_norm, latent_interleaved ? 1 : 0,
                        static_cast<const char*>(index_keys), key_token, key_weight, key_bias, key_eps, key_norm, key_rope_at,
                        key_interleaved ? 1 : 0, slots, positions, table, table_rows, T, static_cast<char*>(latent_cache), k_cache,
                        k_scale, num_slots, static_cast<char*>(latents_out)};
  const dim3 grid = grid_of(((int64_t)T + 3) / 4);
  if (dtype == IDX_TOPK_BF16) k_append_rotary<__bf16><<<grid, dim3(256), 0, stream>>>(A);
  else k_append_rotary<_Float16><<<grid, dim3(256), 0, stream>>>(A);
  return hipGetLastError() == hipSuccess ? IDX_OK : IDX_EHIP;
}

}  // namespace idxk
