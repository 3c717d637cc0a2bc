// Building blocks of the attention kernels (gfx950).
//
// Attention of a row (one query vector) over keys i with logits
// x_i = scale * q.k_i is o = sum_i exp(x_i) v_i / sum_i exp(x_i), computed in
// one pass over the keys with a running reference m (any m at which nothing
// overflows gives the same quotient):
//
//   p_i = 2^(x_i log2(e) - m),  l = sum p_i,  o' = sum p_i v_i,
//   o = o' / l,  log(sum exp) = (m + log2 l) ln 2,
//
// and o', l are multiplied by 2^(m_old - m_new) where m moves.
//
// Both products have the keys (or the values' columns) as the rows of A and the
// attention rows as the columns of B.  In the expanded form a wave owns 32 rows
// and they are v_mfma_f32_32x32x16 (in the absorbed form 16 rows and
// v_mfma_f32_16x16x32, laid out as k_latent says):
//
//   logits^T [32 keys x 32 rows] = K [32 x d] . Q^T [d x 32]
//   o'^T     [32 columns x 32 rows] += V^T [32 x keys] . P^T [keys x 32]
//
// In a 32x32 result, lane l = 32h + c holds column c, and its register r holds
// row (r & 3) + 8 (r >> 2) + 4h.  So every lane holds one attention row's
// statistics (c), its maximum and sum need one exchange between the two wave
// halves, and o' is rescaled by a factor that is the lane's own.  The B
// operand of the second product wants 8 keys of a row in each lane: with key
// (j & 3) + 8 (j >> 2) + 4h of a 16-key step as the operand's k index 8h + j
// they are exactly the 8 logits that the lane holds, in order, so P goes from
// one product to the next without leaving its registers; the A operand then
// takes the keys in that order too, 4 at a time through the transposing
// ds_read_b64_tr_b16 (a 16-lane group reads 4 keys x 16 columns row by row
// and each lane receives one column's 4 keys).
//
// P is rounded to the inputs' 16-bit type for the matrix core: its relative
// rounding error (2^-8 at most for bfloat16, 2^-11 for half) is that of the output's
// own rounding.  Half has that precision from 2^-14 on only; below, p is off by up
// to 2^-25, and under a key that dominates a row thousands of small p may all be
// rounded the same way.  So half's reference stands some octaves under the maximum
// and p runs up to 2^15: with lift L, l is at least 2^L, and n keys together move the
// output by at most n 2^-(25 + L) of the largest value.  Logits, maxima, sums and o'
// stay in FP32; l sums the FP32 p.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace idxk {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef float w4f __attribute__((ext_vector_type(4)));

struct TBf16 {
  // A reference that never moves stands 32 octaves above the first maximum, so that logits may climb
  // by 64 with p <= 2^32: o' then stays inside FP32 for values up to 2^(127 - 32) / n keys, and
  // values down to 2^-70 keep all their bits.
  static constexpr float kHeadroom = 32.f;  // octaves that p may pass 1 by
  static __device__ __forceinline__ float first_lift(int) { return -32.f; }
  static constexpr float kLift = 0.f;       // a moved reference is that many octaves below the maximum
  static constexpr float kFullLift = 0.f;   // ... one at the true maximum
  typedef __bf16 elem;
  typedef __bf16 v8 __attribute__((ext_vector_type(8)));
  typedef __bf16 v4 __attribute__((ext_vector_type(4)));
  static __device__ __forceinline__ elem out(float x) { return (elem)x; }
  static __device__ __forceinline__ v16f mfma(v8 a, v8 b, v16f c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ w4f mfma16(v8 a, v8 b, w4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};

struct TF16 {
  static constexpr float kHeadroom = 15.f;  // half ends below 2^16
  // A reference that never moves, over 32 * tiles keys: lifted only as they need it for an error of at
  // most 2^-13 (none up to 4096 keys, 8 octaves for a million), since each octave is one less to climb.
  static __device__ __forceinline__ float first_lift(int tiles) {
    return (float)min(8, max(0, 25 - __builtin_clz(max(tiles, 2) - 1)));
  }
  static constexpr float kLift = 7.f;       // n 2^-32: 2^-13 of the largest value at half a million keys
  static constexpr float kFullLift = 15.f;
  typedef _Float16 elem;
  typedef _Float16 v8 __attribute__((ext_vector_type(8)));
  typedef _Float16 v4 __attribute__((ext_vector_type(4)));
  // The rounded weights' sum may pass l by a factor of 1 + 2^-11, and with it an average of values at the
  // end of half's range that end.  Infinities among the values stay what they are.
  static __device__ __forceinline__ elem out(float x) {
    return (elem)(fabsf(x) < INFINITY ? __builtin_amdgcn_fmed3f(x, -65504.f, 65504.f) : x);
  }
  static __device__ __forceinline__ v16f mfma(v8 a, v8 b, v16f c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ w4f mfma16(v8 a, v8 b, w4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// o' and l are rescaled only where a row's maximum passes its reference by
// this many octaves beyond the lift: p stays below 2^8 (half: 2^15), inside the
// type, and rescaling o' (all its registers) becomes rare.  The quotient is the same.
constexpr float kRescaleOctaves = 8.f;

template <class V>
__device__ __forceinline__ V lds_read(const char* p) {
  return *reinterpret_cast<const V*>(p);
}

// 4 keys (rows of LDS) of one value column: see above.
template <class T>
__device__ __forceinline__ typename T::v4 lds_read_tr(const char* p) {
  typedef short v4s __attribute__((ext_vector_type(4)));
  const v4s r = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) v4s*)(__attribute__((address_space(3))) char*)p);
  typename T::v4 o;
  __builtin_memcpy(&o, &r, sizeof o);
  return o;
}

template <class T>
__device__ __forceinline__ typename T::v8 cat(typename T::v4 a, typename T::v4 b) {
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// The value of the other half of the wave (lane l ^ 32): the swap exchanges
// the upper half of one register with the lower half of another.
__device__ __forceinline__ float other_half(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}

// Maximum over a lane and the lane l ^ 32.
__device__ __forceinline__ float max_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Maximum and sum over the lanes l, l ^ 16, l ^ 32 and l ^ 48.
__device__ __forceinline__ float max_quarters(float x) {
  x = max_halves(x);
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_quarters(float x) {
  const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(h[0]) + __uint_as_float(h[1]);
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Key of a 32-key tile whose logit is in register r of wave half h.
__device__ __forceinline__ constexpr int key_of(int r, int h) { return (r & 3) + 8 * (r >> 2) + 4 * h; }

// A row's statistics: m in octaves (-inf before the first live key), l.
struct RowStat {
  float m, l;
};

// The largest logit of each row in a tile (FP32, unscaled; -inf where masked)
// in octaves, c = scale * log2(e) > 0.  All 64 lanes take part.
__device__ __forceinline__ float tile_max(const v16f& x, float c) {
  float mx = x[0];
#pragma unroll
  for (int r = 1; r < 16; ++r) mx = fmaxf(mx, x[r]);
  return max_halves(mx) * c;
}

// Whether some row of the wave has to move its reference for a tile of
// maximum mx (the first live keys move it from -inf).
template <class T>
__device__ __forceinline__ bool must_move(const RowStat& st, float mx) {
  return __any(mx > st.m + (T::kLift + kRescaleOctaves));
}

// Moves the references to cover mx; returns the factor of o'.
template <class T>
__device__ __forceinline__ float move_reference(RowStat& st, float mx) {
  const float m = fmaxf(st.m, mx - T::kLift);
  const float alpha = st.m == m ? 1.f : __builtin_amdgcn_exp2f(st.m - m);  // 0 where m was -inf
  st.m = m;
  st.l *= alpha;
  return alpha;
}

// A tile's logits to p, in place.
__device__ __forceinline__ void softmax_tile(v16f& x, RowStat& st, float c) {
  const float m = st.m == -INFINITY ? 0.f : st.m;  // a row without a live key yet: p = 0
  float l[4] = {};
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    x[r] = __builtin_amdgcn_exp2f(fmaf(x[r], c, -m));
    l[r & 3] += x[r];
  }
  st.l += (l[0] + l[1]) + (l[2] + l[3]);  // this half's keys; the halves are added at the end
}

// p of the 16-key step s (0 or 1) of a tile as the second product's B operand.
template <class T>
__device__ __forceinline__ typename T::v8 p_operand(const v16f& p, int s) {
  typename T::v8 o;
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = (typename T::elem)p[8 * s + j];
  return o;
}

// log(sum exp).  m is a logit and a whole number of octaves, which l's exponent takes back without rounding.
__device__ __forceinline__ float row_lse(float m, float l) {
  const float e = (float)__builtin_amdgcn_frexp_expf(l);
  return l > 0.f ? (m + e + __builtin_amdgcn_logf(__builtin_amdgcn_frexp_mantf(l))) * kLn2 : (l == 0.f ? -INFINITY : l);
}

// 64 lanes x 16 bytes from src + off (a lane's) to 1 KiB of LDS in lane order,
// without registers.  The compiler does not see the write: the tile waits
// below order it.  Nor does it see a memory instruction here, so the five wait
// states that one needs after a vector instruction has written its scalar
// address (v_readlane) are in the text: the s_mov and four of the s_nop.  m0 is
// named as overwritten, so that no value that the compiler sets up there for an
// instruction of its own is taken to outlive these (it is warned of as a register
// that the compiler reserves, which is what is wanted).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma_row(const char* src, int off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(src) : "m0");
}
__device__ __forceinline__ void dma_lanes(const char* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(src) : "m0");
}
#pragma clang diagnostic pop
// All but the last N of this wave's loads to LDS are done.
template <int N>
__device__ __forceinline__ void dma_wait() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// Every wave is here, and has its LDS reads back.
__device__ __forceinline__ void tile_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

}  // namespace idxk
