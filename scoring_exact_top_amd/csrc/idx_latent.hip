// Latent attention, absorbed form (gfx950): keys and values of all heads are one cache row a
// token, the 512 latent numbers (key and value) and the 64 rotary numbers (key only):
//
//   x[h,i] = scale * q[h,:] . row_i[0:576],  o[h,:] = sum_i softmax_i(x[h,:]) row_i[0:512]
//
// over the rows that a list names (latent_selected: the indexer's output) or over all of a paged
// sequence (latent_paged).  A key costs 2*(576+512) operations a head and 1152 bytes: with 64
// heads 121 operations a byte, so that up to 128 heads a key's bytes cost more than its products
// where they are read once (16 sequences of up to 65536 keys, 128 heads: 107 us of memory, 76 of
// products), and less where thousands of tokens list the keys of one cache.
//
// A workgroup takes one token (or sequence) and up to 128 rows (heads, or steps x heads), 16 a
// wave; its waves share each 32-key tile in LDS, read from memory straight into LDS while earlier
// tiles are worked on.  With 64 rows or fewer the waves form two key groups that take every other
// tile and are joined at the end.  Where tokens or
// sequences alone leave compute units idle, the keys are split over workgroups, whose partial
// results a second kernel joins.
//
// Measured, and what bounds it (a call in a loop; walk and join as traced alone):
//   4096 tokens x 64 heads x 2048 of 32768 rows   1297 us  901 TFLOP/s; 98% of the busy clocks are LDS
//                                                  traffic (each wave reads every tile for 16 rows)
//   16 sequences to 65536 keys, 128 heads           162 us  walk 146: the same 98%, at the 1.6 GHz that
//                                                  power leaves; 3.4 TB/s, 820 TFLOP/s; join 13
//   16 tokens x 64 heads x 2048 of 262144 rows      24 us  walk 18, join 6: latency, partial results
//   one token, 128 heads, 2048 rows                 15 us  walk 11, join 3: latency
#include <type_traits>
#include "idx_attn.hpp"
#include "idx_latent.hpp"

namespace idxk {

constexpr int kTileKeys = 32;
constexpr int kRowsWave = 16;             // attention rows of a wave
constexpr int kSteps = kLatRow / 32;      // 32-deep steps of the first product
constexpr int kLatSteps = kLatent / 32;   // ... of which in the latent part
constexpr int kCols = kLatent / 16;       // 16-column blocks of the values
constexpr int kRopeOff = kTileKeys * kLatent * 2;             // rotary part of a tile, behind the latent parts
constexpr int kTileBytes = kTileKeys * kLatRow * 2;

constexpr int kBuffers = 4;               // tiles in LDS: 144 of the 160 KiB
constexpr int kMaxList = IDX_TOPK_KMAX;
constexpr int kPlanBatch = 1024;          // larger batches take one workgroup a sequence
constexpr int kUnits = 256;               // compute units: one workgroup each

struct LatArgs {
  const char* q;
  int64_t q_seq, q_token, q_head;  // in numbers
  const char* cache;
  int64_t num_slots;
  const int32_t* list;             // slots [B][K], or page ids [B][K]
  const int32_t* lens;             // paged: [B]
  int32_t K, B, S, H;
  int32_t row_blocks;
  int32_t parts;                   // listed: workgroups a token's list is split over; paged: workgroups in all
  float c;                         // scale * log2(e)
  char* out;
  float* lse;
  float* part_o;                   // [(cell * row_blocks + block) * HG + group] 16 rows x 512 columns
  float2* part_ml;                 // ... of 16 rows
  int2* plan;                      // paged: [B] first cell and number of parts
};

// A row of zeros for keys that a tile does not have: they are masked, and
// their values must not be NaN.
__device__ const uint4 kZeroRow[kLatRow * 2 / 16] = {};

// LDS image of a tile: rows of 64 (latent) or 8 (rotary) 16-byte chunks; chunk
// c of row r stands at c ^ lat_swz(r) or c ^ rope_swz(r), so that the 16-byte
// reads of 16 rows at one chunk (first product) and the transposing 8-byte
// reads of 8 rows x 2 chunks (second product) each cover all 64 banks once.
__device__ __forceinline__ int lat_swz(int r) { return (r & 7) << 1 | (r >> 2 & 1); }
__device__ __forceinline__ int rope_swz(int r) { return (r >> 1) & 7; }

// Workgroup `wg` of a paged call: its sequence, which of the sequence's parts
// it takes and how many there are.  A sequence gets parts in proportion to its
// pages, at least one and none under kMinPages; every workgroup (its first
// wave) works the plan out from the lengths.  Only the parts of sequences that
// have several write partial results: they are numbered by themselves, `cell`
// being the first of the sequence's.
struct Part {
  int b, part, parts, cell;
};
constexpr int kMinPages = 2;

__device__ __forceinline__ int wave_incl_scan(int x, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(x, d, 64);
    if (lane >= d) x += y;
  }
  return x;
}

__device__ __forceinline__ int seq_len(const LatArgs& A, int b) {
  const int n = A.lens[b];
  return n < 0 || (int64_t)n > (int64_t)A.K * IDX_TOPK_PAGE ? 0 : n;
}

__device__ __forceinline__ Part plan_part(const LatArgs& A, int wg, int lane) {
  if (A.parts == A.B) return Part{wg, 0, 1, 0};
  int64_t total = 0;
  for (int b0 = 0; b0 < A.B; b0 += 64) {
    const int n = b0 + lane < A.B ? (seq_len(A, b0 + lane) + IDX_TOPK_PAGE - 1) / IDX_TOPK_PAGE : 0;
    total += __shfl(wave_incl_scan(n, lane), 63, 64);
  }
  // sum of max(1, ceil(n / unit)) <= total / unit + B <= parts
  int unit = (int)((total + (A.parts - A.B) - 1) / (A.parts - A.B));
  unit = unit < kMinPages ? kMinPages : unit;
  int base = 0;  // sums over the sequences before: parts, and 2^16 x parts with a cell (2^11 at most each)
  for (int b0 = 0; b0 < A.B; b0 += 64) {
    const int n = b0 + lane < A.B ? (seq_len(A, b0 + lane) + IDX_TOPK_PAGE - 1) / IDX_TOPK_PAGE : 0;
    const int parts = b0 + lane < A.B ? max(1, (n + unit - 1) / unit) : 0;
    const int both = parts > 1 ? parts << 16 | parts : parts;
    const int end = base + wave_incl_scan(both, lane);
    const int last = end & 0xFFFF;
    const uint64_t mine = __ballot(wg >= last - parts && wg < last);
    if (mine) {
      const int at = __ffsll((unsigned long long)mine) - 1;
      const int n_at = __shfl(parts, at, 64), before = __shfl(end - both, at, 64);
      return Part{b0 + at, wg - (before & 0xFFFF), n_at, before >> 16};
    }
    base = __shfl(end, 63, 64);
  }
  return Part{-1, 0, 0, 0};  // a spare workgroup
}

// HG row groups of 16 (one wave each) x KG key groups: wave (kg, hg) walks
// the tiles kg, kg + KG, ... of the workgroup's range for its 16 rows.
//
// Both products are v_mfma_f32_16x16x32, transposed as in idx_attn.hpp: logits^T
// [16 keys x 16 rows] twice a tile, o'^T [16 columns x 16 rows].  In a result lane
// 16g + c holds row c's entries 4g .. 4g + 3, so that the 8 logits a lane holds
// of a tile, keys 4g + r and 16 + 4g + r, are the second product's B operand
// with those keys in that order.  A wave of 16 rows reads every tile from LDS
// for 16 rows only, twice what 32 rows would; but o' is then 128 registers and
// q 72, two waves fit a SIMD, and one wave's softmax, LDS latency and stalls on
// loads run beside the other's products.  A tile of 128 rows takes 4650 clocks
// (4352 of LDS reads and 288 of writes, 2176 of products), with 32 rows a wave and one
// wave a SIMD 4430 at a clock that power lowers from 1.64 to 1.61 GHz: 3% of
// time, and only with the softmax spread over the products and every register
// chosen by hand.
template <class T, int HG, int KG, bool PAGED>
__global__ __launch_bounds__(64 * HG * KG, HG * KG == 8 ? 2 : 1) void k_latent(LatArgs A) {
  constexpr int kAhead = 5;      // LDS reads of operands run this many products ahead (as registers allow)
  constexpr int kRing = kBuffers / KG;           // tiles of a key group in LDS
  constexpr int kRows = kTileKeys / HG;          // rows of a tile that one wave loads
  constexpr int kFlight = kRing - 1;             // of which on their way
  constexpr int kRope4 = HG < 4 ? 4 / HG : 1;    // its loads of rotary parts (with 8 waves two load each part)
  constexpr int kLoads = kRows + kRope4;         // its loads to LDS a tile
  __shared__ __attribute__((aligned(1024))) char s_tile[kBuffers * kTileBytes];
  __shared__ int32_t s_again;
  __shared__ int32_t s_list[PAGED ? 4 : kMaxList + kTileKeys];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int hg = wave % HG, kg = wave / HG;
  const int g = lane >> 4, col = lane & 15;
  // workgroups of one chiplet (every eighth) take neighbouring work
  const int total = gridDim.x, per = total >> 3, extra = total & 7, x8 = blockIdx.x & 7, i8 = blockIdx.x >> 3;
  const int work = x8 * per + min(x8, extra) + i8;
  const int wg = work / A.row_blocks, rb = work % A.row_blocks;

  Part part;
  int len, tile0, tile1;  // keys of the sequence or list, this workgroup's tiles
  if (PAGED) {
    if (wave == 0) {
      part = plan_part(A, wg, lane);
      if (lane == 0) {
        s_list[0] = part.b; s_list[1] = part.part; s_list[2] = part.parts; s_list[3] = part.cell;
        if (A.parts > A.B && rb == 0 && part.b >= 0 && part.part == 0) A.plan[part.b] = make_int2(part.cell, part.parts);
      }
    }
    __syncthreads();
    part.b = __builtin_amdgcn_readfirstlane(s_list[0]);
    part.part = __builtin_amdgcn_readfirstlane(s_list[1]);
    part.parts = __builtin_amdgcn_readfirstlane(s_list[2]);
    if (part.b < 0) return;
    len = __builtin_amdgcn_readfirstlane(seq_len(A, part.b));
    const int pages = (len + IDX_TOPK_PAGE - 1) / IDX_TOPK_PAGE;
    tile0 = 2 * (int)((int64_t)pages * part.part / part.parts);
    tile1 = min(2 * (int)((int64_t)pages * (part.part + 1) / part.parts), (len + kTileKeys - 1) / kTileKeys);
  } else {
    part.b = wg / A.parts; part.part = wg % A.parts; part.parts = A.parts;
    len = A.K;
    const int tiles = (len + kTileKeys - 1) / kTileKeys;
    tile0 = tiles * part.part / A.parts;
    tile1 = tiles * (part.part + 1) / A.parts;
  }
  const int b = part.b;
  const int row = (rb * HG + hg) * kRowsWave + col;
  const bool have = row < A.S * A.H;
  const int step = have ? row / A.H : 0, head = have ? row % A.H : 0;
  int limit = PAGED ? len - A.S + 1 + step : len;  // this lane's row sees keys below
  const int limit_min = PAGED ? len - A.S + 1 : len;     // every row does

  // The first memory the wave waits for: this range's slots (-1 for what is not
  // to be read) go to LDS behind q's loads, which are under way meanwhile.
  const int n_list = PAGED ? 0 : (tile1 - tile0) * kTileKeys + kTileKeys;
  const auto listed = [&](int i) __attribute__((always_inline)) {
    const int at = tile0 * kTileKeys + i;
    return i < n_list && at < min(len, tile1 * kTileKeys) ? A.list[(int64_t)b * A.K + at] : -1;
  };
  int slot = PAGED ? -1 : listed(tid);
  typename T::v8 q[kSteps];  // a row past the last repeats the first: its results are dropped
  {
    const typename T::elem* p = reinterpret_cast<const typename T::elem*>(A.q) + b * A.q_seq + step * A.q_token +
                                head * A.q_head + 8 * g;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) q[s] = *reinterpret_cast<const typename T::v8*>(p + 32 * s);
  }
  if (!PAGED) {
    for (int i = tid; i < n_list; i += 64 * HG * KG) {
      s_list[i] = slot >= 0 && slot < A.num_slots ? slot : -1;
      slot = listed(i + 64 * HG * KG);
    }
    __syncthreads();
  }

  w4f o[kCols];
  RowStat st{-INFINITY, 0.f};
  // This lane's LDS byte offsets in a tile: key `col` (first product; step s at
  // chunk 4s + g; key 16 + col 16 rows on), its rotary part, and the lane's row
  // of the transposing reads (second product; the other 16 rows on).  They are
  // made where they are used: registers are short.
  const auto own_lane = [&]() __attribute__((always_inline)) {
    int l = lane;
    asm volatile("" : "+v"(l));
    return l;
  };
  const auto key_at = [&](int l) __attribute__((always_inline)) { return (l & 15) * (kLatent * 2) + ((l >> 4 ^ lat_swz(l & 15)) << 4); };
  const auto rope_at = [&](int l) __attribute__((always_inline)) { return kRopeOff + (l & 15) * (kRope * 2) + ((l >> 4 ^ rope_swz(l & 15)) << 4); };
  const auto value_at = [&](int l) __attribute__((always_inline)) {
    const int r = l >> 2;  // 4 (l / 16) + (l & 15) / 4
    return r * (kLatent * 2) + (((l & 3) >> 1 ^ lat_swz(r)) << 4) + (l & 1) * 8;
  };
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)s_tile;

  const int mine = __builtin_amdgcn_readfirstlane(tile0) + kg;  // this key group's first tile
  // the same for all key groups: barriers
  const int steps = __builtin_amdgcn_readfirstlane(tile1 > tile0 ? (tile1 - tile0 + KG - 1) / KG : 0);

  // This wave's share of a tile, in kLoads loads: lane j < kRows has the address
  // of load j's row, each lane its own of the rotary parts'.  Keys that are not
  // there (bit clear in `live`) come from the zero row; so does a whole tile
  // past the walk's end, so that every step has the same loads in flight.
  // Nothing here or in load() branches: a branch between products costs more
  // than the loads.
  struct Source {
    uint32_t dst, live;
    uint32_t lo, hi, rlo[kRope4], rhi[kRope4];
  };
  const auto source = [&](int t) __attribute__((always_inline)) {
    Source f;
    f.dst = __builtin_amdgcn_readfirstlane(lds0 + (kg * kRing + t % kRing) * kTileBytes);
    asm volatile("" : "+s"(f.dst));  // the loads' addresses are made from it, not kept in registers
    const bool in = t < steps;
    const uint64_t zero = (uint64_t)(uintptr_t)kZeroRow, cache = (uint64_t)(uintptr_t)A.cache;
    const int l = own_lane();
    const int row_l = (hg * kRows + l) & (kTileKeys - 1);
    uint64_t page = 0;
    int rows = 0;  // paged: rows of the tile that are there
    if (PAGED) {
      const int key0 = (mine + t * KG) * kTileKeys;
      // a scalar load: vector loads would queue behind the tile loads.  A tile
      // lies in one page; page 0 of the table stands in for tiles past the end
      const auto* table = reinterpret_cast<const __attribute__((address_space(4))) int32_t*>((uintptr_t)A.list) + (int64_t)b * A.K;
      const bool some = in && key0 < len;
      const int pg = table[some ? key0 / IDX_TOPK_PAGE : 0];
      rows = some && pg >= 0 && (int64_t)pg * IDX_TOPK_PAGE < A.num_slots ? min(kTileKeys, len - key0) : 0;
      page = cache + ((int64_t)pg * IDX_TOPK_PAGE + key0 % IDX_TOPK_PAGE) * (kLatRow * 2);
      f.live = rows > 0 ? ~0u : 0u;
    }
    const int tile_slot = (min(t, steps - 1) * KG + kg) * kTileKeys;
    const auto row_at = [&](int r, bool& there) __attribute__((always_inline)) {
      if (PAGED) {
        there = r < rows;
        return page + (uint32_t)r * (uint32_t)(kLatRow * 2);
      }
      const int s = s_list[tile_slot + r];
      there = in && s >= 0;
      return cache + (uint64_t)(uint32_t)s * (uint32_t)(kLatRow * 2);
    };
    bool there;
    uint64_t p = row_at(row_l, there);
    if (!PAGED) {
      const uint32_t w = (uint32_t)__ballot(there);
      f.live = __builtin_amdgcn_readfirstlane(hg * kRows == 0 ? w : w << (hg * kRows) | w >> (kTileKeys - hg * kRows));
    }
    p = there ? p : zero;
    f.lo = (uint32_t)p;
    f.hi = (uint32_t)(p >> 32);
#pragma unroll
    for (int j = 0; j < kRope4; ++j) {
      const int r = 8 * ((hg * kRope4 + j) & 3) + (l >> 3);
      uint64_t o = row_at(r, there);
      o = (there ? o : zero) + kLatent * 2 + (uint32_t)(((l & 7) ^ rope_swz(r)) << 4);
      f.rlo[j] = (uint32_t)o;
      f.rhi[j] = (uint32_t)(o >> 32);
    }
    return f;
  };
  const auto load = [&](const Source& f, int j) __attribute__((always_inline)) {
    if (j < kRows) {
      const uint64_t p = (uint32_t)__builtin_amdgcn_readlane(f.lo, j) | (uint64_t)(uint32_t)__builtin_amdgcn_readlane(f.hi, j) << 32;
      const int l16 = (own_lane() ^ (HG == 1 ? 0 : lat_swz(hg * kRows))) << 4;
      dma_row(reinterpret_cast<const char*>((uintptr_t)p), l16 ^ (lat_swz(j) << 4), f.dst + (hg * kRows + j) * (kLatent * 2));
    } else {
      const int n = (hg * kRope4 + j - kRows) & 3;
      dma_lanes(reinterpret_cast<const char*>((uintptr_t)(f.rlo[j - kRows] | (uint64_t)f.rhi[j - kRows] << 32)), f.dst + kRopeOff + n * 1024);
    }
  };
  Source next;
  uint32_t live[kFlight + 1];  // of this step's tile and the ones in flight
  const auto load_first = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < kFlight; ++t) {
      next = source(t);
      live[t + 1] = next.live;
#pragma unroll
      for (int j = 0; j < kLoads; ++j) load(next, j);
    }
    next = source(kFlight);
  };
  if (tid == 0) s_again = 0;  // before the barriers of the walk
  if (steps > 0) load_first();

  // Waits for step i's tile, computes its logits x, masked, and starts the
  // loads of a later tile on the way (kMore).
  const auto logits = [&](auto kMore, int i, w4f (&x)[2]) __attribute__((always_inline)) {
    dma_wait<(kFlight - 1) * kLoads>();
    tile_barrier();  // tile i is there and tile i - 1 is read: its buffer takes the next load
    const char* tile = s_tile + (kg * kRing + i % kRing) * kTileBytes;
    const int ka = key_at(own_lane()), ra = rope_at(own_lane());
    // each product is followed by the read of the operand kAhead products on;
    // product n: keys 16 (n & 1) on, step step_of(n)
    typename T::v8 k[kAhead];
    const auto step_of = [](int n) { return n / 2 < kLatSteps ? 4 * (n / 2 & 3) + (n / 2 >> 2) : n / 2; };
    const auto read = [&](int n) __attribute__((always_inline)) {
      const int j = n >> 1, u = n & 1;  // latent step 4 (j & 3) + j / 4: four reads from one address
      k[n % kAhead] = j < kLatSteps ? lds_read<typename T::v8>(tile + (ka ^ (j >> 2 << 6)) + 256 * (j & 3) + u * 16 * kLatent * 2)
                                    : lds_read<typename T::v8>(tile + (ra ^ ((j - kLatSteps) << 6)) + u * 16 * kRope * 2);
    };
    x[0] = w4f{};
    x[1] = w4f{};
#pragma unroll
    for (int n = 0; n < kAhead; ++n) read(n);
#pragma unroll
    for (int n = 0; n < 2 * kSteps; ++n) {
      __builtin_amdgcn_sched_barrier(0);
      x[n & 1] = T::mfma16(k[n % kAhead], q[step_of(n)], x[n & 1]);
      if (n + kAhead < 2 * kSteps) read(n + kAhead);
      // a load every few products: a burst would wait for the memory pipeline
      constexpr int kEvery = 2 * kSteps / kLoads;
      if (kMore && n % kEvery == 0 && n / kEvery < kLoads) {
        __builtin_amdgcn_sched_barrier(0);
        load(next, n / kEvery);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int t = 0; t < kFlight; ++t) live[t] = live[t + 1];
    if constexpr (kMore) {
      live[kFlight] = next.live;
      next = source(i + 1 + kFlight);
    }
    const int key0 = (mine + i * KG) * kTileKeys;
    if (live[0] != ~0u || key0 + kTileKeys > limit_min) {
      const int g4 = own_lane() >> 4 << 2;
      const uint32_t live_g = live[0] >> g4;
      const int limit_g = limit - key0 - g4;
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const int key = (r & 3) + 16 * (r >> 2);
        if (!(live_g >> key & 1) || key >= limit_g) x[r >> 2][r & 3] = -INFINITY;
      }
    }
  };
  // f(i) for every step, and whether it loads.  Two key groups have one tile each under way and a last step
  // without loads: in a short walk loads of zeros would cost as much as the others (a token's 2048 keys
  // over 32 workgroups: 2900 of 18700 clocks).
  const auto walk = [&](const auto& f) __attribute__((always_inline)) {
    if constexpr (kFlight > 1) {
      for (int i = 0; i < steps; ++i) f(std::true_type{}, i);
    } else {
      for (int i = 0; i + 1 < steps; ++i) f(std::true_type{}, i);
      if (steps > 0) f(std::false_type{}, steps - 1);
    }
  };
  // The largest logit of each row in a tile, in octaves.
  const auto largest = [&](const w4f (&x)[2]) __attribute__((always_inline)) {
    float mx = fmaxf(fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[0][2], x[0][3])), fmaxf(fmaxf(x[1][0], x[1][1]), fmaxf(x[1][2], x[1][3])));
    return max_quarters(mx) * A.c;
  };

  // o' is not rescaled where a row's maximum grows.  With 16 or 32 rows a workgroup
  // it lies in accumulation registers and would have to pass through ordinary ones;
  // with more it lies in ordinary ones (253 to 256 are taken), where multiplying it in
  // place has not been tried.  The reference stays where the row's first live tile's
  // maximum puts it: p may grow to kHeadroom octaves above 1, which costs no precision.
  // A workgroup that sees more walks its keys again, first for the rows' true maxima,
  // then with those as references: 560 us instead of 229 for 16 half sequences of 40000
  // keys, 128 heads, where every row's logits (standard deviation 7) climb by more than
  // 15 octaves; bfloat16's 64 octaves take a standard deviation of 14 to be passed.
  const float lift = T::first_lift(steps);
  __builtin_amdgcn_s_waitcnt(0x0F70);  // q is there: the waits below count tile loads only
  for (int attempt = 0;; ++attempt) {
#pragma unroll
    for (int d = 0; d < kCols; ++d) o[d] = w4f{};
    if (steps == 0) break;
    bool over = false;  // a logit passed its row's reference by too much
    walk([&](auto kMore, int i) __attribute__((always_inline)) {
      w4f x[2];
      logits(kMore, i, x);
      const float mx = largest(x);
      st.m = st.m == -INFINITY ? mx - lift : st.m;
      over |= __any(mx - st.m > T::kHeadroom);
      const float m = st.m == -INFINITY ? 0.f : st.m;  // a row without a live key yet: p = 0
      typename T::v8 p;
      float l[2] = {0.f, 0.f};
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const float e = __builtin_amdgcn_exp2f(fmaf(x[r >> 2][r & 3], A.c, -m));
        l[r & 1] += e;
        p[r] = (typename T::elem)e;
      }
      st.l += l[0] + l[1];  // this quarter's keys; the quarters are added at the end
      const char* tile = s_tile + (kg * kRing + i % kRing) * kTileBytes;
      const int va = value_at(own_lane());
      typename T::v8 v[kAhead];
      // product n: column block d = n / 4 + 8 (n & 3)
      const auto read = [&](int n) __attribute__((always_inline)) {
        const char* a = tile + (va ^ (n >> 2 << 5)) + 256 * (n & 3);
        v[n % kAhead] = cat<T>(lds_read_tr<T>(a), lds_read_tr<T>(a + 16 * kLatent * 2));
      };
#pragma unroll
      for (int n = 0; n < kAhead; ++n) read(n);
#pragma unroll
      for (int n = 0; n < kCols; ++n) {
        __builtin_amdgcn_sched_barrier(0);
        const int d = (n >> 2) + 8 * (n & 3);
        o[d] = T::mfma16(v[n % kAhead], p, o[d]);
        if (n + kAhead < kCols) read(n + kAhead);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    if (over && lane == 0) s_again = 1;
    dma_wait<0>();
    tile_barrier();  // every tile is read, every load done
    if (attempt > 0 || !__builtin_amdgcn_readfirstlane(s_again)) break;
    st = RowStat{-INFINITY, 0.f};
    load_first();
    walk([&](auto kMore, int i) __attribute__((always_inline)) {
      w4f x[2];
      logits(kMore, i, x);
      st.m = fmaxf(st.m, largest(x));
    });
    st.m -= T::kFullLift;
    dma_wait<0>();
    tile_barrier();
    load_first();
  }
  float l = sum_quarters(st.l), m = st.m;

  // Key groups are joined through LDS (nothing is in flight there any more): each hands the other m, l and
  // half of o', 16 bytes a lane at a time, and goes on with its own half of the columns.
  constexpr int kOwn = kCols / KG;
  w4f r[kOwn];
  if (KG == 2) {
    char* const give = s_tile + wave * (kOwn * 1024 + 512);
    const char* const take = s_tile + (wave + HG) % (HG * KG) * (kOwn * 1024 + 512);
    *reinterpret_cast<float2*>(give + lane * 8) = make_float2(m, l);
    const auto hand = [&](auto from) __attribute__((always_inline)) {
#pragma unroll
      for (int d = 0; d < kOwn; ++d) *reinterpret_cast<w4f*>(give + 512 + d * 1024 + lane * 16) = o[from + d];
    };
    const auto add = [&](auto own, float f0, float f1) __attribute__((always_inline)) {
#pragma unroll
      for (int d = 0; d < kOwn; ++d) r[d] = o[own + d] * f0 + *reinterpret_cast<const w4f*>(take + 512 + d * 1024 + lane * 16) * f1;
    };
    const std::integral_constant<int, 0> low;
    const std::integral_constant<int, kCols / 2> high;
    if (kg == 0) hand(high);
    else hand(low);
    __syncthreads();
    const float2 ml = *reinterpret_cast<const float2*>(take + lane * 8);
    const float top = fmaxf(m, ml.x);
    const float f0 = m == top ? 1.f : __builtin_amdgcn_exp2f(m - top), f1 = ml.x == top ? 1.f : __builtin_amdgcn_exp2f(ml.x - top);
    if (kg == 0) add(low, f0, f1);
    else add(high, f0, f1);
    l = l * f0 + ml.y * f1;
    m = top;
  } else {
#pragma unroll
    for (int d = 0; d < kOwn; ++d) r[d] = o[d];
  }
  if (part.parts > 1) {
    // in the order of the registers: whole lines, and the join adds them in that order too
    const int of = PAGED ? __builtin_amdgcn_readfirstlane(s_list[3]) + part.part : wg;
    const int64_t cell = ((int64_t)of * A.row_blocks + rb) * HG + hg;
    float* po = A.part_o + cell * (kRowsWave * kLatent) + kg * kOwn * 256 + lane * 4;
#pragma unroll
    for (int d = 0; d < kOwn; ++d) *reinterpret_cast<w4f*>(po + d * 256) = r[d];
    if (g == 0 && kg == 0) A.part_ml[cell * kRowsWave + col] = make_float2(m, l);
    return;
  }
  if (!have) return;
  const int64_t at = ((int64_t)b * A.S + step) * A.H + head;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  typename T::elem* out = reinterpret_cast<typename T::elem*>(A.out) + at * kLatent + 16 * kg * kOwn + 4 * g;
#pragma unroll
  for (int d = 0; d < kOwn; ++d) {
    typename T::v4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = T::out(r[d][j] * inv);
    *reinterpret_cast<typename T::v4*>(out + 16 * d) = v;
  }
  if (A.lse && g == 0 && kg == 0) A.lse[at] = row_lse(m, l);
}

// Joins the parts of a row: o = sum_p 2^(m_p - m) o'_p / sum_p 2^(m_p - m) l_p.
// A workgroup takes 256 of the 8192 numbers of a cell (16 rows x 512 columns in
// the order of the walk's registers), each wave every fourth part, so that few
// loads wait on one another.
template <class T>
__global__ __launch_bounds__(256) void k_latent_join(LatArgs A, int hgs, bool paged) {
  __shared__ float4 s_o[3][64];
  __shared__ float2 s_ml[3][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, piece = blockIdx.x & (kCols - 1);
  const int groups = A.row_blocks * hgs;  // 16-row groups of a token or sequence
  const int unit = blockIdx.x / kCols, b = unit / groups, group = unit % groups;
  const int row = group * kRowsWave + (lane & 15);
  int first = b * A.parts, n = A.parts;
  if (paged) {
    const int2 p = A.plan[b];
    first = p.x; n = p.y;
    if (n == 1) return;  // written by the walk
  }
  if (group * kRowsWave >= A.S * A.H) return;
  const int64_t cell0 = (int64_t)first * groups + group;
  const float2* ml = A.part_ml + cell0 * kRowsWave + (lane & 15);
  const float4* po = reinterpret_cast<const float4*>(A.part_o + cell0 * (kRowsWave * kLatent) + piece * 256) + lane;
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kBatch = 8;
  for (int p0 = wave; p0 < n; p0 += 4 * kBatch) {
    float2 s[kBatch];
    float4 v[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int p = p0 + 4 * u < n ? p0 + 4 * u : p0;
      s[u] = ml[(int64_t)p * groups * kRowsWave];
      v[u] = po[(int64_t)p * groups * (kRowsWave * kLatent / 4)];
    }
    float top = m;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) top = fmaxf(top, s[u].x);
    const float t0 = top == -INFINITY ? 0.f : top, old = __builtin_amdgcn_exp2f(m - t0);
    m = top;
    l *= old; o.x *= old; o.y *= old; o.z *= old; o.w *= old;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const float f = p0 + 4 * u < n ? __builtin_amdgcn_exp2f(s[u].x - t0) : 0.f;
      l = fmaf(s[u].y, f, l);
      o.x = fmaf(v[u].x, f, o.x); o.y = fmaf(v[u].y, f, o.y); o.z = fmaf(v[u].z, f, o.z); o.w = fmaf(v[u].w, f, o.w);
    }
  }
  if (wave > 0) {
    s_o[wave - 1][lane] = o;
    s_ml[wave - 1][lane] = make_float2(m, l);
  }
  __syncthreads();
  if (wave > 0 || row >= A.S * A.H) return;
  float top = m;
#pragma unroll
  for (int w = 0; w < 3; ++w) top = fmaxf(top, s_ml[w][lane].x);
  const float t0 = top == -INFINITY ? 0.f : top, f0 = __builtin_amdgcn_exp2f(m - t0);
  l *= f0; o.x *= f0; o.y *= f0; o.z *= f0; o.w *= f0;
#pragma unroll
  for (int w = 0; w < 3; ++w) {
    const float2 s = s_ml[w][lane];
    const float4 v = s_o[w][lane];
    const float f = __builtin_amdgcn_exp2f(s.x - t0);
    l = fmaf(s.y, f, l);
    o.x = fmaf(v.x, f, o.x); o.y = fmaf(v.y, f, o.y); o.z = fmaf(v.z, f, o.z); o.w = fmaf(v.w, f, o.w);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  typename T::v4 v;
  v[0] = T::out(o.x * inv); v[1] = T::out(o.y * inv); v[2] = T::out(o.z * inv); v[3] = T::out(o.w * inv);
  const int64_t at = (int64_t)b * A.S * A.H + row;  // rows of a sequence are its steps' heads in order
  const int column = 16 * piece + 4 * (lane >> 4);
  *reinterpret_cast<typename T::v4*>(reinterpret_cast<typename T::elem*>(A.out) + at * kLatent + column) = v;
  if (A.lse && column == 0) A.lse[at] = row_lse(top, l);
}

// ------------------------------------------------------------------ host

static inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
static inline bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
static inline size_t a256(size_t x) { return (x + 255) & ~(size_t)255; }

// How a call is cut: 16 * hg rows a workgroup, `parts` as in LatArgs.
struct LatGeom {
  int hg, row_blocks, parts;
  int64_t cells;  // partial results of 16 * hg rows each (0: none), row blocks included
  size_t o, ml, plan, total;
};

// Waves that rows need: all eight of a workgroup beyond 64 rows, else half as
// many, or fewer, beside as many of a second key group.
static int row_groups(int rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : rows <= 64 ? 4 : 8; }

static LatGeom layout(LatGeom g, int64_t B) {
  const size_t rows = (size_t)(g.cells * kRowsWave * g.hg);
  size_t at = 0;
  g.o = at; at = a256(at + rows * kLatent * 4);
  g.ml = at; at = a256(at + rows * 8);
  g.plan = at; at = a256(at + (size_t)B * 8);
  g.total = at < 256 ? 256 : at;
  return g;
}

// Few tokens or sequences are cut in two ways that both fill the compute units:
// many parts of all rows, or fewer parts of fewer rows.  The fixed costs of a
// workgroup (its rows of q read, their partial results written and joined) go
// with its rows, and a step of 32 rows costs three quarters of one of 64, so
// where parts would be short the rows are halved first: 16 tokens x 64 heads x
// 2048 keys take 24 us as 8 parts of 32 rows against 28 us as 16 parts of 64.
constexpr int kManyParts = 8;     // listed: more parts a token than these are short
constexpr int kShortKeys = 512;   // paged: keys a part at most, where the table says so

// A paged call has B parts and `extra` more, and no part has more pages than
// the total over `extra` (plan_part): as many extra parts as sequences, so that
// a sequence longer than the average is cut, but no more than make the longest
// part a quarter of a compute unit's share (half of it: 6% more time for 1024
// sequences of up to 4096 keys, 128 heads).  Sequences cut into several parts have
// less than 2 * extra of them together (n / unit + 1 < 2 n / unit each): that
// many cells, at most 8 * 256 and a rounding of row blocks of 128 rows, which is
// 521 MiB whatever the batch.
constexpr int kExtraRounds = 4;

static LatGeom listed_geom(int32_t T, int32_t H, int32_t K) {
  LatGeom g{};
  g.hg = row_groups(H);
  const int most = (K + 2 * kTileKeys - 1) / (2 * kTileKeys);  // a part keeps at least two tiles
  for (;; g.hg /= 2) {
    g.row_blocks = (H + kRowsWave * g.hg - 1) / (kRowsWave * g.hg);
    const int64_t groups = (int64_t)T * g.row_blocks;
    const int64_t parts = groups > 0 ? kUnits / groups : 1;
    g.parts = parts < 1 ? 1 : parts > most ? most : (int)parts;
    if (g.hg == 1) break;
    const bool idle = 2 * groups * g.parts <= kUnits;  // half the units without work even so
    if (!idle && (g.hg == 2 || g.parts <= kManyParts)) break;
  }
  g.cells = g.parts > 1 ? (int64_t)T * g.row_blocks * g.parts : 0;
  return layout(g, 0);
}

static LatGeom paged_geom(int32_t B, int32_t S, int32_t H, int32_t max_pages) {
  LatGeom g{};
  const int rows = S * H;
  int64_t parts = B;
  for (g.hg = row_groups(rows);; g.hg /= 2) {
    g.row_blocks = (rows + kRowsWave * g.hg - 1) / (kRowsWave * g.hg);
    if (B == 0 || B > kPlanBatch || max_pages <= kMinPages) break;
    const int64_t extra = (kExtraRounds * kUnits + g.row_blocks - 1) / g.row_blocks;
    parts = kUnits / g.row_blocks;
    if (parts < B + (extra < B ? extra : B)) parts = B + (extra < B ? extra : B);
    const int64_t most = (int64_t)B * ((max_pages + kMinPages - 1) / kMinPages) + B;
    if (parts > most) parts = most;
    if (g.hg <= 2 || (int64_t)B * max_pages * IDX_TOPK_PAGE / parts >= kShortKeys) break;
  }
  g.parts = (int)parts;
  const int64_t cut = 2 * (parts - B);
  g.cells = (cut < parts ? cut : parts) * g.row_blocks;
  return layout(g, g.cells ? B : 0);
}

template <class T, bool PAGED>
static int launch(LatArgs A, const LatGeom& g, char* ws, hipStream_t stream) {
  A.row_blocks = g.row_blocks;
  A.parts = g.parts;
  A.part_o = reinterpret_cast<float*>(ws + g.o);
  A.part_ml = reinterpret_cast<float2*>(ws + g.ml);
  A.plan = reinterpret_cast<int2*>(ws + g.plan);
  const int64_t grid = (int64_t)(PAGED ? 1 : A.B) * g.parts * g.row_blocks;
  const int64_t join = (int64_t)A.B * g.row_blocks * g.hg * kCols;
  // a launch dimension takes fewer than 2^32 threads (a larger one wraps, without an error)
  const int64_t threads = 64 * (g.hg == 8 ? 8 : 2 * g.hg);
  if (grid * threads > 0xffffffffLL || (g.cells && join * 256 > 0xffffffffLL)) return IDX_EUNSUPPORTED;
  const dim3 n((uint32_t)grid);
  if (g.hg == 1) k_latent<T, 1, 2, PAGED><<<n, dim3(128), 0, stream>>>(A);
  else if (g.hg == 2) k_latent<T, 2, 2, PAGED><<<n, dim3(256), 0, stream>>>(A);
  else if (g.hg == 4) k_latent<T, 4, 2, PAGED><<<n, dim3(512), 0, stream>>>(A);
  else k_latent<T, 8, 1, PAGED><<<n, dim3(512), 0, stream>>>(A);
  if (g.cells) k_latent_join<T><<<dim3((uint32_t)join), dim3(256), 0, stream>>>(A, g.hg, PAGED);
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
  if (!q || !out || !aligned16(q) || !aligned16(out) || !aligned16(cache) || !aligned4(list) || !aligned4(lse)) return IDX_EINVAL;
  return IDX_OK;
}

size_t latent_selected_workspace_bytes(int32_t T, int32_t H, int32_t K) {
  if (T < 0 || H < 1 || H > kMaxHeads || K < 1 || K > IDX_TOPK_KMAX) return 0;
  return listed_geom(T, H, K).total;
}

int latent_selected(const void* q, int64_t q_token, int64_t q_head, const void* cache, int64_t num_slots,
                    const int32_t* slots, int32_t K, int32_t T, int32_t H, float scale, int32_t dtype, void* out,
                    float* lse, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (K < 1 || K > IDX_TOPK_KMAX || num_slots < 0 || bad_stride(q_token) || bad_stride(q_head)) return IDX_EINVAL;
  const int rc = check_common(q, cache, slots, T, H, scale, dtype, out, lse);
  if (rc != IDX_OK || T == 0) return rc;
  if (!slots || (!cache && num_slots > 0)) return IDX_EINVAL;
  const LatGeom g = listed_geom(T, H, K);
  if (!workspace || workspace_bytes < g.total) return IDX_EWORKSPACE;
  if (((uintptr_t)workspace & 255u) != 0) return IDX_EINVAL;
  LatArgs A{static_cast<const char*>(q), q_token, 0, q_head, static_cast<const char*>(cache), num_slots, slots,
            nullptr, K, T, 1, H, 0, 0, scale * kLog2e, static_cast<char*>(out), lse, nullptr, nullptr, nullptr};
  char* const ws = static_cast<char*>(workspace);
  return dtype == IDX_TOPK_BF16 ? launch<TBf16, false>(A, g, ws, stream) : launch<TF16, false>(A, g, ws, stream);
}

size_t latent_paged_workspace_bytes(int32_t B, int32_t S, int32_t H, int32_t max_pages) {
  if (B < 0 || S < 1 || S > IDX_TOPK_MAX_STEPS || H < 1 || H > kMaxHeads || max_pages < 0) return 0;
  return paged_geom(B, S, H, max_pages).total;
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
  if (!seq_lens || !aligned4(seq_lens) || (!page_table && max_pages > 0) || (!cache && num_pages > 0)) return IDX_EINVAL;
  const LatGeom g = paged_geom(B, S, H, max_pages);
  if (!workspace || workspace_bytes < g.total) return IDX_EWORKSPACE;
  if (((uintptr_t)workspace & 255u) != 0) return IDX_EINVAL;
  LatArgs A{static_cast<const char*>(q), q_seq, q_token, q_head, static_cast<const char*>(cache),
            (int64_t)num_pages * IDX_TOPK_PAGE, page_table, seq_lens, max_pages, B, S, H, 0, 0, scale * kLog2e,
            static_cast<char*>(out), lse, nullptr, nullptr, nullptr};
  char* const ws = static_cast<char*>(workspace);
  return dtype == IDX_TOPK_BF16 ? launch<TBf16, true>(A, g, ws, stream) : launch<TF16, true>(A, g, ws, stream);
}

}  // namespace idxk
