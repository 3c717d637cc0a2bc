// Latent attention, absorbed form (gfx950): keys and values of all heads are one cache row a
// token, the 512 latent numbers (key and value) and the 64 rotary numbers (key only):
//
//   x[h,i] = scale * q[h,:] . row_i[0:576],  o[h,:] = sum_i softmax_i(x[h,:]) row_i[0:512]
//
// over the rows that a list names (latent_selected: the indexer's output) or over all of a paged
// sequence (latent_paged).  A key costs 2*(576+512) operations a head and 1152 bytes: with 64
// heads 121 operations a byte.
//
// A workgroup takes one token (or sequence) and up to 128 rows (heads, or steps x heads), 32 a
// wave; all its waves share each 32-key tile in LDS (idx_attn.hpp has the arithmetic).
#include "idx_attn.hpp"
#include "idx_latent.hpp"

namespace idxk {

constexpr int kTileKeys = 32;
constexpr int kSteps = kLatRow / 16;      // 16-deep steps of the first product
constexpr int kLatSteps = kLatent / 16;   // ... of which in the latent part
constexpr int kCols = kLatent / 32;       // 32-column blocks of the values
constexpr int kRopeOff = kTileKeys * kLatent * 2;             // rotary part of a tile, behind the latent parts
constexpr int kTileBytes = kTileKeys * kLatRow * 2;
constexpr int kMaxList = IDX_TOPK_KMAX;

struct LatArgs {
  const char* q;
  int64_t q_seq, q_token, q_head;  // in numbers
  const char* cache;
  int64_t num_slots;
  const int32_t* list;             // slots [T][K], or page ids [B][K]
  const int32_t* lens;             // paged: [B]
  int32_t K, B, S, H;
  int32_t row_blocks;
  float c;                         // scale * log2(e)
  char* out;
  float* lse;
};

// A row of zeros for keys that a tile does not have: they are masked, and
// their values must not be NaN.
__device__ const uint4 kZeroRow[kLatRow * 2 / 16] = {};

// LDS image of a tile: rows of 64 (latent) or 8 (rotary) 16-byte chunks; chunk
// c of row r stands at c ^ lat_swz(r) or c ^ rope_swz(r), so that the 16-byte
// reads of 16 rows at one chunk (first product) and the transposing 8-byte
// reads of 4 rows x 4 chunks (second product) each cover all 64 banks once.
__device__ __forceinline__ int lat_swz(int r) { return ((r & 3) << 2) | ((r >> 2) & 3); }
__device__ __forceinline__ int rope_swz(int r) { return (r >> 1) & 7; }

// 16 bytes a lane from memory to 1 KiB of LDS (lane order), without registers.
__device__ __forceinline__ void dma16(const char* src, char* dst) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                   (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}

template <class T, int HG, bool PAGED>
__global__ __launch_bounds__(64 * HG) __attribute__((amdgpu_waves_per_eu(1, 1))) void k_latent(LatArgs A) {
  __shared__ __attribute__((aligned(1024))) char s_tile[kTileBytes];
  __shared__ int32_t s_list[PAGED ? 1 : kMaxList];
  const int tid = threadIdx.x, lane = tid & 63, hg = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 5, col = lane & 31;
  const int b = blockIdx.x / A.row_blocks, rb = blockIdx.x % A.row_blocks;
  const int row = (rb * HG + hg) * 32 + col;
  const bool have = row < A.S * A.H;
  const int step = have ? row / A.H : 0, head = have ? row % A.H : 0;

  int len = A.K, limit;  // keys of the walk; this lane's row sees keys below `limit`
  if (PAGED) {
    len = A.lens[b];
    if (len < 0 || (int64_t)len > (int64_t)A.K * IDX_TOPK_PAGE) len = 0;
    limit = len - A.S + 1 + step;
  } else {
    limit = len;
    for (int i = tid; i < len; i += 64 * HG) s_list[i] = A.list[(int64_t)b * A.K + i];
  }

  typename T::v8 q[kSteps];
  {
    const typename T::elem* p = reinterpret_cast<const typename T::elem*>(A.q) + b * A.q_seq + step * A.q_token +
                                head * A.q_head + 8 * h;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      if (have) q[s] = *reinterpret_cast<const typename T::v8*>(p + 16 * s);
      else q[s] = typename T::v8{};
    }
  }
  v16f o[kCols];
#pragma unroll
  for (int d = 0; d < kCols; ++d) o[d] = v16f{};
  RowStat st{-INFINITY, 0.f};
  // this lane's LDS byte offsets: its key's row (first product; step s at
  // chunk 2s + h), and its two rows of the transposing reads (second)
  const int tr = 4 * h + ((lane & 15) >> 2), tc = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
  int kaddr = col * (kLatent * 2) + ((h ^ lat_swz(col)) << 4), raddr = col * (kRope * 2) + ((h ^ rope_swz(col)) << 4);
  int vaddr0 = tr * (kLatent * 2) + ((tc ^ lat_swz(tr)) << 4) + (lane & 1) * 8;
  int vaddr1 = (tr + 8) * (kLatent * 2) + ((tc ^ lat_swz(tr + 8)) << 4) + (lane & 1) * 8;

  // Loads the tile at k0 and computes its logits, masked.
  const auto logits = [&](int k0) {
    __syncthreads();  // the last tile is read (first: the list is there)
    // slots of the tile's keys: lane i (and i + 32) key i
    int64_t slot = -1;
    if (k0 + col < len) {
      if (PAGED) {
        const int key = k0 + col;
        const int pg = A.list[(int64_t)b * A.K + key / IDX_TOPK_PAGE];
        slot = pg < 0 ? -1 : (int64_t)pg * IDX_TOPK_PAGE + key % IDX_TOPK_PAGE;
      } else {
        slot = s_list[k0 + col];
      }
      if (slot >= A.num_slots) slot = -1;
    }
    const uint32_t live = (uint32_t)__ballot(slot >= 0);
    const char* src = slot >= 0 ? A.cache + slot * (kLatRow * 2) : reinterpret_cast<const char*>(kZeroRow);
    for (int r = hg * (kTileKeys / HG); r < (hg + 1) * (kTileKeys / HG); ++r) {
      const int64_t p = __shfl((long long)(intptr_t)src, r, 64);
      dma16(reinterpret_cast<const char*>(p) + ((lane ^ lat_swz(r)) << 4), s_tile + r * (kLatent * 2));
    }
    for (int j = hg * (4 / HG); j < (hg + 1) * (4 / HG); ++j) {
      const int r = 8 * j + (lane >> 3);
      const int64_t p = __shfl((long long)(intptr_t)src, r, 64);
      dma16(reinterpret_cast<const char*>(p) + kLatent * 2 + (((lane & 7) ^ rope_swz(r)) << 4), s_tile + kRopeOff + j * 1024);
    }
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();

    asm volatile("" : "+v"(kaddr), "+v"(raddr), "+v"(vaddr0), "+v"(vaddr1));  // the offsets below are made here, not kept in registers
    v16f x;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const char* p = s_tile + (kaddr ^ (j << 5));
#pragma unroll
      for (int u = 0; u < kLatSteps / 8; ++u) T::mfma_v(x, lds_read<typename T::v8>(p + 256 * u), q[8 * u + j], j + u == 0);
    }
#pragma unroll
    for (int j = 0; j < kRope / 16; ++j)
      T::mfma_v(x, lds_read<typename T::v8>(s_tile + kRopeOff + (raddr ^ (j << 5))), q[kLatSteps + j], false);
    mfma_v_done(x);
    if (live != ~0u || k0 + kTileKeys > limit) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int k = key_of(r, h);
        if (!(live >> k & 1) || k0 + k >= limit) x[r] = -INFINITY;
      }
    }
    return x;
  };

  // The inner loop never touches o' but by MFMA: it leaves to the outer one
  // where a reference moves.
  int k0 = 0;
  if (len > 0) {
    v16f x = logits(0);
    float mx = tile_max(x, A.c);
    for (;;) {
      const float alpha = move_reference(st, mx);
#pragma unroll
      for (int d = 0; d < kCols; ++d) o[d] *= alpha;
      for (;;) {
        softmax_tile(x, st, A.c);
        const typename T::v8 p0 = p_operand<T>(x, 0), p1 = p_operand<T>(x, 1);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const char* pa = s_tile + (vaddr0 ^ (j << 6));
          const char* pb = s_tile + (vaddr1 ^ (j << 6));
#pragma unroll
          for (int u = 0; u < kCols / 4; ++u) {
            const int d = 4 * u + j;
            o[d] = T::mfma(cat<T>(lds_read_tr<T>(pa + 256 * u), lds_read_tr<T>(pb + 256 * u)), p0, o[d]);
            o[d] = T::mfma(cat<T>(lds_read_tr<T>(pa + 256 * u + 16 * kLatent * 2), lds_read_tr<T>(pb + 256 * u + 16 * kLatent * 2)),
                           p1, o[d]);
          }
        }
        k0 += kTileKeys;
        if (k0 >= len) break;
        x = logits(k0);
        mx = tile_max(x, A.c);
        if (must_move(st, mx)) break;
      }
      if (k0 >= len) break;
    }
  }

  const float l = st.l + other_half(st.l);
  if (!have) return;
  const int64_t at = ((int64_t)b * A.S + step) * A.H + head;
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  typename T::elem* out = reinterpret_cast<typename T::elem*>(A.out) + at * kLatent;
#pragma unroll
  for (int d = 0; d < kCols; ++d)
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

template <class T, bool PAGED>
static int launch(LatArgs A, hipStream_t stream) {
  const int rows = A.S * A.H;
  const int hg = rows <= 32 ? 1 : rows <= 64 ? 2 : 4;
  A.row_blocks = (rows + 32 * hg - 1) / (32 * hg);
  const int64_t grid = (int64_t)A.B * A.row_blocks;
  if (grid > 0x7fffffffLL) return IDX_EUNSUPPORTED;
  if (hg == 1) k_latent<T, 1, PAGED><<<dim3((uint32_t)grid), dim3(64), 0, stream>>>(A);
  else if (hg == 2) k_latent<T, 2, PAGED><<<dim3((uint32_t)grid), dim3(128), 0, stream>>>(A);
  else k_latent<T, 4, PAGED><<<dim3((uint32_t)grid), dim3(256), 0, stream>>>(A);
  return hipGetLastError() == hipSuccess ? IDX_OK : IDX_EHIP;
}

static bool bad_stride(int64_t s) { return s < 0 || (s & 7) != 0; }

// What both forms check of their shared arguments.
static int check_common(const void* q, const void* cache, const int32_t* list, int32_t rows, int32_t H, float scale,
                        int32_t dtype, const void* out, const float* lse) {
  if (rows < 0 || H < 1 || !(scale > 0.f) || !(scale < INFINITY)) return IDX_EINVAL;
  if (dtype != IDX_TOPK_BF16 && dtype != IDX_TOPK_F16) return IDX_EINVAL;
  if (H > kMaxHeads) return IDX_EUNSUPPORTED;
  if (rows == 0) return IDX_OK;
  if (!q || !out || !aligned16(q) || !aligned16(out) || !aligned16(cache)) return IDX_EINVAL;
  return IDX_OK;
}

size_t latent_selected_workspace_bytes(int32_t T, int32_t H, int32_t K) {
  if (T < 0 || H < 1 || H > kMaxHeads || K < 1 || K > IDX_TOPK_KMAX) return 0;
  return 256;
}

int latent_selected(const void* q, int64_t q_token, int64_t q_head, const void* cache, int64_t num_slots,
                    const int32_t* slots, int32_t K, int32_t T, int32_t H, float scale, int32_t dtype, void* out,
                    float* lse, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (K < 1 || K > IDX_TOPK_KMAX || num_slots < 0 || bad_stride(q_token) || bad_stride(q_head)) return IDX_EINVAL;
  const int rc = check_common(q, cache, slots, T, H, scale, dtype, out, lse);
  if (rc != IDX_OK || T == 0) return rc;
  if (!slots || (!cache && num_slots > 0)) return IDX_EINVAL;
  const size_t need = latent_selected_workspace_bytes(T, H, K);
  if (!workspace || workspace_bytes < need) return IDX_EWORKSPACE;
  if (((uintptr_t)workspace & 255u) != 0) return IDX_EINVAL;
  LatArgs A{static_cast<const char*>(q), q_token, 0, q_head, static_cast<const char*>(cache), num_slots, slots,
            nullptr, K, T, 1, H, 0, scale * kLog2e, static_cast<char*>(out), lse};
  return dtype == IDX_TOPK_BF16 ? launch<TBf16, false>(A, stream) : launch<TF16, false>(A, stream);
}

size_t latent_paged_workspace_bytes(int32_t B, int32_t S, int32_t H, int32_t max_pages) {
  if (B < 0 || S < 1 || S > IDX_TOPK_MAX_STEPS || H < 1 || H > kMaxHeads || max_pages < 0) return 0;
  return 256;
}

int latent_paged(const void* q, int64_t q_seq, int64_t q_token, int64_t q_head, const void* cache,
                 int32_t num_pages, const int32_t* page_table, int32_t max_pages, const int32_t* seq_lens, int32_t B,
                 int32_t S, int32_t H, float scale, int32_t dtype, void* out, float* lse, void* workspace,
                 size_t workspace_bytes, hipStream_t stream) {
  if (S < 1 || S > IDX_TOPK_MAX_STEPS || max_pages < 0 || num_pages < 0 || bad_stride(q_seq) || bad_stride(q_token) ||
      bad_stride(q_head))
    return IDX_EINVAL;
  if (max_pages > 0x7fffffff / IDX_TOPK_PAGE) return IDX_EUNSUPPORTED;
  const int rc = check_common(q, cache, page_table, B, H, scale, dtype, out, lse);
  if (rc != IDX_OK || B == 0) return rc;
  if (!seq_lens || (!page_table && max_pages > 0) || (!cache && num_pages > 0)) return IDX_EINVAL;
  const size_t need = latent_paged_workspace_bytes(B, S, H, max_pages);
  if (!workspace || workspace_bytes < need) return IDX_EWORKSPACE;
  if (((uintptr_t)workspace & 255u) != 0) return IDX_EINVAL;
  LatArgs A{static_cast<const char*>(q), q_seq, q_token, q_head, static_cast<const char*>(cache),
            (int64_t)num_pages * IDX_TOPK_PAGE, page_table, seq_lens, max_pages, B, S, H, 0, scale * kLog2e,
            static_cast<char*>(out), lse};
  return dtype == IDX_TOPK_BF16 ? launch<TBf16, true>(A, stream) : launch<TF16, true>(A, stream);
}

}  // namespace idxk
