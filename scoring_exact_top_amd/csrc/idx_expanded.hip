// Latent attention, expanded form (gfx950): causal attention over packed prompts with per-head
// keys (128 numbers, and 64 rotary numbers that all heads share) and values (128 numbers).
// A (query, key, head) costs 2*(192+128) operations; a workgroup takes 128 query tokens of one
// head of one prompt, 32 a wave, and its waves share each 32-key tile in LDS.  idx_attn.hpp has
// the arithmetic.
#include "idx_attn.hpp"
#include "idx_latent.hpp"

namespace idxk {

constexpr int kXTile = 32;                 // keys of a tile
constexpr int kXWaves = 4;
constexpr int kXRows = 32 * kXWaves;       // query tokens of a workgroup
constexpr int kXWidth = kNope + kRope;
constexpr int kXSteps = kXWidth / 16, kXNopeSteps = kNope / 16;
constexpr int kXCols = kValue / 32;
constexpr int kXKey = 0, kXRope = kXTile * kNope * 2, kXVal = kXRope + kXTile * kRope * 2;
constexpr int kXBytes = kXVal + kXTile * kValue * 2;

struct ExpArgs {
  const char* q;
  int64_t q_token, q_head;
  const char* kv;
  int64_t kv_token, kv_head;
  const char* rope;
  int64_t rope_token;
  const int32_t *cu_q, *cu_k;
  int32_t Tq, Tk, H, causal;
  float c;
  char* out;
  float* lse;
};

__device__ const uint4 kXZero[16] = {};

// As in the absorbed form: chunk c of a row of 16 (8) chunks stands at c ^ swz.
__device__ __forceinline__ int row_swz(int r) { return ((r & 3) << 2) | ((r >> 2) & 3); }
__device__ __forceinline__ int rot_swz(int r) { return (r >> 1) & 7; }

__device__ __forceinline__ void xdma16(const char* src, char* dst) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                   (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}

template <class T>
__global__ __launch_bounds__(64 * kXWaves) void k_expanded(ExpArgs A) {
  __shared__ __attribute__((aligned(1024))) char s_tile[kXBytes];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 5, col = lane & 31, head = blockIdx.x, b = blockIdx.z;
  const int q0 = A.cu_q[b], q1 = A.cu_q[b + 1], k0 = A.cu_k[b], k1 = A.cu_k[b + 1];
  if (q0 < 0 || q1 < q0 || q1 > A.Tq || k0 < 0 || k1 < k0 || k1 > A.Tk) return;
  const int Lq = q1 - q0, Lk = k1 - k0;
  const int first = blockIdx.y * kXRows;
  if (first >= Lq) return;
  const int row = first + wave * 32 + col;
  const bool have = row < Lq;
  const int limit = A.causal ? row + 1 + Lk - Lq : Lk;  // the row sees keys below
  const int last_row = min(first + kXRows, Lq) - 1;
  const int end = A.causal ? max(0, last_row + 1 + Lk - Lq) : Lk;

  typename T::v8 q[kXSteps];
  const typename T::elem* qp = reinterpret_cast<const typename T::elem*>(A.q) + (int64_t)(q0 + row) * A.q_token +
                               head * A.q_head + 8 * h;
#pragma unroll
  for (int s = 0; s < kXSteps; ++s) {
    if (have) q[s] = *reinterpret_cast<const typename T::v8*>(qp + 16 * s);
    else q[s] = typename T::v8{};
  }
  v16f o[kXCols];
#pragma unroll
  for (int d = 0; d < kXCols; ++d) o[d] = v16f{};
  RowStat st{-INFINITY, 0.f};
  const int tr = 4 * h + ((lane & 15) >> 2), tc = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);

  for (int t0 = 0; t0 < end; t0 += kXTile) {
    __syncthreads();
    // a wave loads 2 KiB of the keys, 1 KiB of the rotary parts, 2 KiB of the values
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int j = 2 * wave + u, r = 4 * j + (lane >> 4), key = t0 + r;
      const char* p = A.kv + ((int64_t)(k0 + key) * A.kv_token + head * A.kv_head) * 2 + (((lane & 15) ^ row_swz(r)) << 4);
      const char* z = reinterpret_cast<const char*>(kXZero) + ((lane & 15) << 4);
      xdma16(key < Lk ? p : z, s_tile + kXKey + j * 1024);
      xdma16(key < Lk ? p + kNope * 2 : z, s_tile + kXVal + j * 1024);
    }
    {
      const int r = 8 * wave + (lane >> 3), key = t0 + r;
      const char* p = A.rope + (int64_t)(k0 + key) * A.rope_token * 2 + (((lane & 7) ^ rot_swz(r)) << 4);
      xdma16(key < Lk ? p : reinterpret_cast<const char*>(kXZero), s_tile + kXRope + wave * 1024);
    }
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();

    v16f x = {};
#pragma unroll
    for (int s = 0; s < kXSteps; ++s) {
      const int chunk = 2 * s + h;
      const char* p = s < kXNopeSteps ? s_tile + kXKey + col * (kNope * 2) + ((chunk ^ row_swz(col)) << 4)
                                      : s_tile + kXRope + col * (kRope * 2) + (((chunk - 2 * kXNopeSteps) ^ rot_swz(col)) << 4);
      x = T::mfma(lds_read<typename T::v8>(p), q[s], x);
    }
    if (t0 + kXTile > limit) {
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (t0 + key_of(r, h) >= limit) x[r] = -INFINITY;
    }
    const float mx = tile_max(x, A.c);
    if (must_move(st, mx)) {
      const float alpha = move_reference(st, mx);
#pragma unroll
      for (int d = 0; d < kXCols; ++d) o[d] *= alpha;
    }
    softmax_tile(x, st, A.c);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const typename T::v8 p = p_operand<T>(x, s);
#pragma unroll
      for (int d = 0; d < kXCols; ++d) {
        typename T::v4 v[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int r = 16 * s + 8 * u + tr;
          v[u] = lds_read_tr<T>(s_tile + kXVal + r * (kValue * 2) + (((4 * d + tc) ^ row_swz(r)) << 4) + (lane & 1) * 8);
        }
        o[d] = T::mfma(cat<T>(v[0], v[1]), p, o[d]);
      }
    }
  }

  const float l = st.l + other_half(st.l);
  if (!have) return;
  const int64_t at = (int64_t)(q0 + row) * A.H + head;
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  typename T::elem* out = reinterpret_cast<typename T::elem*>(A.out) + at * kValue;
#pragma unroll
  for (int d = 0; d < kXCols; ++d)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      typename T::v4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = (typename T::elem)(l == 0.f ? 0.f : o[d][4 * g + j] * inv);
      *reinterpret_cast<typename T::v4*>(out + 32 * d + 8 * g + 4 * h) = v;
    }
  if (A.lse && h == 0) A.lse[at] = row_lse(st.m, l);
}

// ------------------------------------------------------------------ host

static inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
static bool bad_stride(int64_t s) { return s < 0 || (s & 7) != 0; }

size_t latent_expanded_workspace_bytes(int32_t Tq, int32_t B, int32_t max_q, int32_t max_k, int32_t H) {
  if (Tq < 0 || B < 0 || max_q < 0 || max_k < 0 || H < 1 || H > kMaxHeads) return 0;
  return 256;
}

int latent_expanded(const void* q, int64_t q_token, int64_t q_head, const void* kv, int64_t kv_token,
                    int64_t kv_head, const void* k_rope, int64_t rope_token, const int32_t* cu_q,
                    const int32_t* cu_k, int32_t B, int32_t Tq, int32_t Tk, int32_t max_q, int32_t max_k, int32_t H,
                    float scale, int32_t causal, int32_t dtype, void* out, float* lse, void* workspace,
                    size_t workspace_bytes, hipStream_t stream) {
  if (B < 0 || Tq < 0 || Tk < 0 || max_q < 0 || max_k < 0 || H < 1 || !(scale > 0.f) || !(scale < INFINITY)) return IDX_EINVAL;
  if (dtype != IDX_TOPK_BF16 && dtype != IDX_TOPK_F16) return IDX_EINVAL;
  if (bad_stride(q_token) || bad_stride(q_head) || bad_stride(kv_token) || bad_stride(kv_head) || bad_stride(rope_token))
    return IDX_EINVAL;
  if (H > kMaxHeads || B > 65535) return IDX_EUNSUPPORTED;
  if (B == 0 || Tq == 0 || max_q == 0) return IDX_OK;
  if (max_q > Tq) max_q = Tq;
  const int64_t blocks = ((int64_t)max_q + kXRows - 1) / kXRows;
  if (blocks > 65535) return IDX_EUNSUPPORTED;
  if (!q || !out || !cu_q || !cu_k || (Tk > 0 && (!kv || !k_rope))) return IDX_EINVAL;
  if (!aligned16(q) || !aligned16(kv) || !aligned16(k_rope) || !aligned16(out)) return IDX_EINVAL;
  if (!workspace || workspace_bytes < latent_expanded_workspace_bytes(Tq, B, max_q, max_k, H)) return IDX_EWORKSPACE;
  if (((uintptr_t)workspace & 255u) != 0) return IDX_EINVAL;
  const ExpArgs A{static_cast<const char*>(q), q_token, q_head, static_cast<const char*>(kv), kv_token, kv_head,
                  static_cast<const char*>(k_rope), rope_token, cu_q, cu_k, Tq, Tk, H, causal, scale * kLog2e,
                  static_cast<char*>(out), lse};
  const dim3 grid((uint32_t)H, (uint32_t)blocks, (uint32_t)B);
  if (dtype == IDX_TOPK_BF16) k_expanded<TBf16><<<grid, dim3(64 * kXWaves), 0, stream>>>(A);
  else k_expanded<TF16><<<grid, dim3(64 * kXWaves), 0, stream>>>(A);
  return hipGetLastError() == hipSuccess ? IDX_OK : IDX_EHIP;
}

}  // namespace idxk
