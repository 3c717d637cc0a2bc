// Latent attention, expanded form (gfx950): causal attention over packed prompts with per-head
// keys (128 numbers, and 64 rotary numbers that all heads share) and values (128 numbers).
// A (query, key, head) costs 2*(192+128) operations, and a 64-key tile of a head (40 KiB) serves
// every query of the prompt, so the matrix cores are the bound; a wave of 32 queries reads each
// tile from LDS once, which is as many clocks of the LDS as its products are of a matrix core.
// A workgroup takes 256 query tokens of one head of one prompt, 32 a wave, two waves a SIMD, so
// that one wave's softmax runs beside another's products; the tiles come from memory straight
// into a ring of three in LDS.  Few queries over many keys (a chunk of a long prompt) have their
// keys split over workgroups, joined by a second kernel.  idx_attn.hpp has the arithmetic.
//
// Measured: 8192 tokens x 32 heads in 632 us, 1090 TFLOP/s of useful work; the matrix cores are 55%
// busy at 1.9 GHz (their products alone, at the 1.6 GHz that power leaves them, take 430 us).  500
// tokens over 16384 keys, 16 heads: 102 us, 9 of them the join.  64 rows a wave (half the LDS reads, but
// one wave a SIMD) takes as long, and so does the softmax spread between the products within a wave:
// 12% fewer clocks, 4% less time on long prompts and 5% more on short ones.
#include "idx_attn.hpp"
#include "idx_latent.hpp"

namespace idxk {

constexpr int kXTile = 64;                 // keys of a tile
constexpr int kXWaves = 8;
constexpr int kXRows = 32 * kXWaves;       // query tokens of a workgroup
constexpr int kXRing = 3;                  // tiles in LDS: 120 of the 160 KiB
constexpr int kXWidth = kNope + kRope;
constexpr int kXSteps = kXWidth / 16, kXNopeSteps = kNope / 16;
constexpr int kXCols = kValue / 32;
constexpr int kXRope = kXTile * kNope * 2, kXVal = kXRope + kXTile * kRope * 2;  // parts of a tile, the keys first
constexpr int kXBytes = kXVal + kXTile * kValue * 2;
constexpr int kXLoads = kXBytes / 1024 / kXWaves;  // a wave's loads to LDS a tile

struct ExpArgs {
  const char* q;
  int64_t q_token, q_head;
  const char* kv;
  int64_t kv_token, kv_head;
  const char* rope;
  int64_t rope_token;
  const int32_t *cu_q, *cu_k;
  int32_t Tq, Tk, H, causal, parts;
  float c;
  char* out;
  float* lse;
  float* part_o;    // [parts][Tq][H][128]
  float2* part_ml;  // [parts][Tq][H]
};

__device__ const uint4 kXZero[16] = {};

// As in the absorbed form: chunk c of a row of 16 (8) chunks stands at c ^ swz.
__device__ __forceinline__ int row_swz(int r) { return ((r & 3) << 2) | ((r >> 2) & 3); }
__device__ __forceinline__ int rot_swz(int r) { return (r >> 1) & 7; }

template <class T>
__global__ __launch_bounds__(64 * kXWaves, 2) void k_expanded(ExpArgs A) {
  __shared__ __attribute__((aligned(1024))) char s_tile[kXRing * kXBytes];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 5, col = lane & 31, head = blockIdx.x, b = blockIdx.z;
  const int q0 = A.cu_q[b], q1 = A.cu_q[b + 1], k0 = A.cu_k[b], k1 = A.cu_k[b + 1];
  if (q0 < 0 || q1 < q0 || q1 > A.Tq || k0 < 0 || k1 < k0 || k1 > A.Tk) return;
  const int Lq = q1 - q0, Lk = k1 - k0;
  // the last queries, which see the most keys, come first
  const int yr = gridDim.y - 1 - blockIdx.y, part = yr % A.parts, first = yr / A.parts * kXRows;
  if (first >= Lq) return;
  const int row = first + wave * 32 + col;
  const bool have = row < Lq;
  const int past = A.causal ? Lk - Lq : Lk;  // row i sees the keys below i + 1 + past (causal) or past
  const int limit = A.causal ? row + 1 + past : Lk;
  const int wave_rows = first + wave * 32;
  const int see_all = A.causal ? wave_rows + 1 + past : Lk;                       // every row of the wave sees keys below
  const int see_any = A.causal ? min(wave_rows + 32, Lq) + past : Lk;             // some row does
  const int end = A.causal ? max(0, min(first + kXRows, Lq) + past) : Lk;         // some row of the workgroup does
  const int tiles = (end + kXTile - 1) / kXTile;
  const int tile0 = (int)((int64_t)tiles * part / A.parts), tile1 = (int)((int64_t)tiles * (part + 1) / A.parts);

  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)s_tile;
  const char* const kv = A.kv + ((int64_t)k0 * A.kv_token + head * A.kv_head) * 2;
  const char* const rope = A.rope + (int64_t)k0 * A.rope_token * 2;
  // A wave loads 8 rows of the keys, of the rotary parts and of the values: two, one and two
  // loads of 1 KiB.  This lane's bytes in them:
  const int kr = 8 * wave + (lane >> 4), rr = 8 * wave + (lane >> 3);
  const int koff0 = kr * (int)A.kv_token * 2 + (((lane & 15) ^ row_swz(kr)) << 4);
  const int koff1 = (kr + 4) * (int)A.kv_token * 2 + (((lane & 15) ^ row_swz(kr + 4)) << 4);
  const int roff = rr * (int)A.rope_token * 2 + (((lane & 7) ^ rot_swz(rr)) << 4);
  const auto load = [&](int t) __attribute__((always_inline)) {
    const uint32_t dst = lds0 + t % kXRing * kXBytes + wave * 2048;
    const uint32_t rdst = lds0 + t % kXRing * kXBytes + kXRope + wave * 1024;
    const char* kt = kv + (int64_t)t * kXTile * A.kv_token * 2;
    const char* rt = rope + (int64_t)t * kXTile * A.rope_token * 2;
    if ((t + 1) * kXTile <= Lk) {
      dma_row(kt, koff0, dst);
      dma_row(kt, koff1, dst + 1024);
      dma_row(kt + kNope * 2, koff0, dst + kXVal);
      dma_row(kt + kNope * 2, koff1, dst + kXVal + 1024);
      dma_row(rt, roff, rdst);
    } else {  // zeros for the keys that are not there: masked, but their values must not be NaN
      const char* const zero = reinterpret_cast<const char*>(kXZero);
      const bool in0 = t * kXTile + kr < Lk, in1 = t * kXTile + kr + 4 < Lk, inr = t * kXTile + rr < Lk;
      dma_lanes(in0 ? kt + koff0 : zero, dst);
      dma_lanes(in1 ? kt + koff1 : zero, dst + 1024);
      dma_lanes(in0 ? kt + kNope * 2 + koff0 : zero, dst + kXVal);
      dma_lanes(in1 ? kt + kNope * 2 + koff1 : zero, dst + kXVal + 1024);
      dma_lanes(inr ? rt + roff : zero, rdst);
    }
  };
#pragma unroll
  for (int i = 0; i < kXRing - 1; ++i)
    if (tile0 + i < tile1) load(tile0 + i);

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
  const int kaddr = col * (kNope * 2) + ((h ^ row_swz(col)) << 4), raddr = kXRope + col * (kRope * 2) + ((h ^ rot_swz(col)) << 4);
  const int vaddr0 = kXVal + tr * (kValue * 2) + ((tc ^ row_swz(tr)) << 4) + (lane & 1) * 8;
  const int vaddr1 = kXVal + (tr + 8) * (kValue * 2) + ((tc ^ row_swz(tr + 8)) << 4) + (lane & 1) * 8;
  __builtin_amdgcn_s_waitcnt(0x0F70);  // every register load is done: the waits below count tile loads only

  for (int t = tile0; t < tile1; ++t) {
    if (t + kXRing - 1 <= tile1) dma_wait<(kXRing - 2) * kXLoads>();
    else dma_wait<0>();
    tile_barrier();  // tile t is there, tile t - 1 is read: its buffer takes the next load
    if (t + kXRing - 1 < tile1) load(t + kXRing - 1);
    const int t0 = t * kXTile;
    if (t0 >= see_any) continue;
    const char* tile = s_tile + t % kXRing * kXBytes;
    v16f x[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      x[u] = v16f{};
#pragma unroll
      for (int s = 0; s < kXNopeSteps; ++s)
        x[u] = T::mfma(lds_read<typename T::v8>(tile + (kaddr ^ (s << 5)) + u * 32 * kNope * 2), q[s], x[u]);
#pragma unroll
      for (int s = 0; s < kRope / 16; ++s)
        x[u] = T::mfma(lds_read<typename T::v8>(tile + (raddr ^ (s << 5)) + u * 32 * kRope * 2), q[kXNopeSteps + s], x[u]);
    }
    if (t0 + kXTile > see_all) {
      const int below = limit - t0 - 4 * h;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (32 * u + key_of(r, 0) >= below) x[u][r] = -INFINITY;
    }
    const float mx = fmaxf(tile_max(x[0], A.c), tile_max(x[1], A.c));
    if (must_move<T>(st, mx)) {
      const float alpha = move_reference<T>(st, mx);
#pragma unroll
      for (int d = 0; d < kXCols; ++d) o[d] *= alpha;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      softmax_tile(x[u], st, A.c);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const typename T::v8 p = p_operand<T>(x[u], s);
        const int at = (2 * u + s) * 16 * kValue * 2;
#pragma unroll
        for (int d = 0; d < kXCols; ++d)
          o[d] = T::mfma(cat<T>(lds_read_tr<T>(tile + (vaddr0 ^ (d << 6)) + at), lds_read_tr<T>(tile + (vaddr1 ^ (d << 6)) + at)), p, o[d]);
      }
    }
  }

  const float l = st.l + other_half(st.l);
  if (!have) return;
  const int64_t at = (int64_t)(q0 + row) * A.H + head;
  if (A.parts > 1) {
    const int64_t pat = (int64_t)part * A.Tq * A.H + at;
    float* po = A.part_o + pat * kValue;
#pragma unroll
    for (int d = 0; d < kXCols; ++d)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<float4*>(po + 32 * d + 8 * g + 4 * h) =
            make_float4(o[d][4 * g], o[d][4 * g + 1], o[d][4 * g + 2], o[d][4 * g + 3]);
    if (h == 0) A.part_ml[pat] = make_float2(st.m, l);
    return;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  typename T::elem* out = reinterpret_cast<typename T::elem*>(A.out) + at * kValue;
#pragma unroll
  for (int d = 0; d < kXCols; ++d)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      typename T::v4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = T::out(o[d][4 * g + j] * inv);
      *reinterpret_cast<typename T::v4*>(out + 32 * d + 8 * g + 4 * h) = v;
    }
  if (A.lse && h == 0) A.lse[at] = row_lse(st.m, l);
}

// Joins the parts of the rows of every prompt whose range is valid: 32 threads
// a row, four columns each.
template <class T>
__global__ __launch_bounds__(256) void k_expanded_join(ExpArgs A, int max_q) {
  const int b = blockIdx.y;
  const int q0 = A.cu_q[b], q1 = A.cu_q[b + 1], k0 = A.cu_k[b], k1 = A.cu_k[b + 1];
  if (q0 < 0 || q1 < q0 || q1 > A.Tq || k0 < 0 || k1 < k0 || k1 > A.Tk) return;
  const int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  // the walk computes whole blocks of queries of the first max_q
  if (i >= (int64_t)min(q1 - q0, (max_q + kXRows - 1) / kXRows * kXRows) * A.H) return;
  const int64_t at = (int64_t)q0 * A.H + i, stride = (int64_t)A.Tq * A.H;
  const int c = (threadIdx.x & 31) * 4;
  float m = -INFINITY;
  for (int p = 0; p < A.parts; ++p) m = fmaxf(m, A.part_ml[p * stride + at].x);
  const float m0 = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int p = 0; p < A.parts; ++p) {
    const float2 ml = A.part_ml[p * stride + at];
    const float4 v = *reinterpret_cast<const float4*>(A.part_o + (p * stride + at) * kValue + c);
    const float f = __builtin_amdgcn_exp2f(ml.x - m0);
    l = fmaf(ml.y, f, l);
    o.x = fmaf(v.x, f, o.x); o.y = fmaf(v.y, f, o.y); o.z = fmaf(v.z, f, o.z); o.w = fmaf(v.w, f, o.w);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  typename T::v4 v;
  v[0] = T::out(o.x * inv); v[1] = T::out(o.y * inv); v[2] = T::out(o.z * inv); v[3] = T::out(o.w * inv);
  *reinterpret_cast<typename T::v4*>(reinterpret_cast<typename T::elem*>(A.out) + at * kValue + c) = v;
  if (A.lse && c == 0) A.lse[at] = row_lse(m, l);
}

// ------------------------------------------------------------------ host

static inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
static inline bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
static bool bad_stride(int64_t s) { return s < 0 || (s & 7) != 0; }

static inline size_t a256(size_t x) { return (x + 255) & ~(size_t)255; }

// Parts that each prompt's keys are split into: enough workgroups for the 256
// compute units, at least four tiles a part of the longest prompt.
static int expanded_parts(int32_t B, int32_t max_q, int32_t max_k, int32_t H) {
  const int64_t groups = ((int64_t)max_q + kXRows - 1) / kXRows * H * B;
  int64_t parts = groups > 0 ? 256 / groups : 1;
  const int64_t most = max_k / (4 * kXTile);
  if (parts > most) parts = most;
  return parts < 1 ? 1 : (int)parts;
}

size_t latent_expanded_workspace_bytes(int32_t Tq, int32_t B, int32_t max_q, int32_t max_k, int32_t H) {
  if (Tq < 0 || B < 0 || max_q < 0 || max_k < 0 || H < 1 || H > kMaxHeads) return 0;
  const int parts = expanded_parts(B, max_q < Tq ? max_q : Tq, max_k, H);
  const size_t rows = parts > 1 ? (size_t)parts * Tq * H : 0;
  return a256(rows * kValue * 4) + a256(rows * 8) + 256;
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
  // a tile's rows are addressed by 31-bit offsets from its first
  if (kv_token > 0x7fffffff / (2 * (kXTile + 1)) || rope_token > 0x7fffffff / (2 * (kXTile + 1))) return IDX_EUNSUPPORTED;
  if (B == 0 || Tq == 0 || max_q == 0) return IDX_OK;
  if (max_q > Tq) max_q = Tq;
  const int parts = expanded_parts(B, max_q, max_k, H);
  const int64_t blocks = ((int64_t)max_q + kXRows - 1) / kXRows * parts;
  if (blocks > 65535) return IDX_EUNSUPPORTED;
  if (!q || !out || !cu_q || !cu_k || (Tk > 0 && (!kv || !k_rope))) return IDX_EINVAL;
  if (!aligned16(q) || !aligned16(kv) || !aligned16(k_rope) || !aligned16(out) || !aligned4(cu_q) || !aligned4(cu_k) || !aligned4(lse))
    return IDX_EINVAL;
  if (!workspace || workspace_bytes < latent_expanded_workspace_bytes(Tq, B, max_q, max_k, H)) return IDX_EWORKSPACE;
  if (((uintptr_t)workspace & 255u) != 0) return IDX_EINVAL;
  char* const ws = static_cast<char*>(workspace);
  const size_t rows = parts > 1 ? (size_t)parts * Tq * H : 0;
  const ExpArgs A{static_cast<const char*>(q), q_token, q_head, static_cast<const char*>(kv), kv_token, kv_head,
                  static_cast<const char*>(k_rope), rope_token, cu_q, cu_k, Tq, Tk, H, causal, parts, scale * kLog2e,
                  static_cast<char*>(out), lse, reinterpret_cast<float*>(ws),
                  reinterpret_cast<float2*>(ws + a256(rows * kValue * 4))};
  const dim3 grid((uint32_t)H, (uint32_t)blocks, (uint32_t)B), threads(64 * kXWaves);
  if (dtype == IDX_TOPK_BF16) k_expanded<TBf16><<<grid, threads, 0, stream>>>(A);
  else k_expanded<TF16><<<grid, threads, 0, stream>>>(A);
  if (parts > 1) {
    const int64_t per = ((int64_t)max_q + kXRows) * H / 8 + 1;
    const dim3 join((uint32_t)per, (uint32_t)B);
    if (dtype == IDX_TOPK_BF16) k_expanded_join<TBf16><<<join, dim3(256), 0, stream>>>(A, max_q);
    else k_expanded_join<TF16><<<join, dim3(256), 0, stream>>>(A, max_q);
  }
  return hipGetLastError() == hipSuccess ? IDX_OK : IDX_EHIP;
}

}  // namespace idxk
