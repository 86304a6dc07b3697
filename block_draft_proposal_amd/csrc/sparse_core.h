// What the two forms of the attention over chosen pages share: a row by itself
// (sparse_attn.hip) and the rows of a request together (sparse_tile.hip).
#pragma once

#include <algorithm>

#include "kv_mfma.h"
#include "kv_sparse.h"

namespace dflash {

typedef float f32x4_t __attribute__((ext_vector_type(4)));

template <int DT, int D>
struct SparseShape {
  static constexpr int kRB = D * (DT == DFLASH_BF16 ? 2 : 1);
  static constexpr int kChunks = kRB / 16;
  static constexpr int kWaves = kRB == 512 ? 2 : 4, kThreads = 64 * kWaves;   // of a workgroup, at most
  static constexpr int kTile = 32 * kRB;                              // K (or V) of a step
  static constexpr int kLoads = kTile / 1024;                         // direct loads of K (or V) a lane
  static constexpr int kWaveStages = 2 * 2 * kTile;
  // LDS: the waves' stages, then a ring of each
  static constexpr int kRowsAt = 0;                                   // [4 steps][32] byte offsets, int64
  static constexpr int kScalesAt = 4 * 32 * 8;                        // [4 steps][K 32, V 32] fp32
  static constexpr int kMasksAt = kScalesAt + (DT == DFLASH_BF16 ? 0 : 4 * 64 * 4);   // [4 steps][32], of tiles
  static constexpr int kRing = kMasksAt + 4 * 32 * 4;
  static constexpr int kJoin = 16 * (D + 2) * 4;                      // after the loop: O, m and l of 16 rows
  static constexpr int kWaveLds = kWaveStages + kRing > kJoin ? kWaveStages + kRing : kJoin;
  static_assert(kWaves * kWaveLds <= 160 * 1024 && 2 * kLoads < 63, "LDS of a CU, loads in flight");
  // Waves that a CU holds of a kernel with row_tiles * D sums to a lane group: by
  // its LDS, and with more than 256 registers one to a SIMD.
  static constexpr int cu_waves(int row_tiles) {
    return kWaves * kWaveLds <= 80 * 1024 && row_tiles * D <= 128 ? 2 * kWaves : kWaves;
  }

  // Chunk c of stage row r lies in slot c ^ swizzle(r), so that reads of one
  // instruction fall on different banks: for K, 16 consecutive rows of one
  // chunk; for V's transposed reads, 8 consecutive rows of two chunks (16-bit
  // elements) or 8 and the 8 that are 16 further of one (8-bit).
  static constexpr int kRowsPerBanks = kRB >= 256 ? 1 : 256 / kRB;
  __device__ static __forceinline__ int k_swizzle(int r) { return (r / kRowsPerBanks) & (16 / kRowsPerBanks - 1); }
  __device__ static __forceinline__ int v_swizzle(int r) {
    constexpr int n = 8 / kRowsPerBanks;
    if constexpr (DT == DFLASH_BF16) return ((r / kRowsPerBanks) & (n - 1)) << 1;
    else return ((r / kRowsPerBanks) & (n - 1)) | (((r >> 4) & 1) * n);
  }
};

// How items are spread over the chip: waves of a workgroup, workgroups to an item.
struct Spread {
  int waves, splits;
};
// As many waves as run at once.  Few items are split over workgroups, while each
// wave has two steps of its own; of many, a workgroup has fewer waves and an item
// takes longer, rather than that the last ones wait for a place: one item's
// look-ups then run beside the products of others.  (bf16, 8 kv heads of 128, always
// 4 waves and this way: 128 rows over 16 pages of 16 50 and 30 us, 50 rows over 64
// 63 and 40, 200 rows 189 and 174; 48 x 16 drafted rows 451 and 391.)
template <class S>
Spread spread(int64_t items, int row_tiles, int64_t keys, int64_t max_parts) {
  const int64_t places = 256 * S::cu_waves(row_tiles);
  Spread x{S::kWaves, 1};
  while (x.waves > 1 && items * x.waves > places) x.waves /= 2;
  if (x.waves == S::kWaves)
    x.splits = (int)std::max<int64_t>(1, std::min({keys / (32 * S::kWaves * 2), max_parts / items, places / S::kWaves / items}));
  return x;
}

// x of the lanes 16, 32 and 48 away, combined.
__device__ __forceinline__ float quarter_max(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return half_max(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float quarter_sum(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return half_sum(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// Orders a wave's LDS accesses as they are written (the hardware keeps a
// wave's in order).
__device__ __forceinline__ void wave_order() { asm volatile("" ::: "memory"); }

// With more than 256 registers the sums lie in AGPRs, which only the matrix
// cores compute with.  Without this, at either end of the rare rescaling, the
// compiler moves them to VGPRs and back in every step.
template <bool MANY>
__device__ __forceinline__ void in_accumulators(f32x4_t& x) {
  if constexpr (MANY) asm volatile("" : "+a"(x));
}

// Whether a row sees anything: a block that its list names, the tail or a node.
// The kernels find that as they walk the row's keys; this is for requests whose
// length is beyond the table, which have none.  All lanes of a wave ask together.
__device__ __forceinline__ bool sees_any(const SparseArgs& a, int64_t row, int head, int32_t full, int32_t tail, int n) {
  if (tail > 0 || !a.mask) return true;            // a chain: every node sees itself
  const int lane = threadIdx.x & 63;
  const int32_t* chosen = a.blocks + (row * a.c.n_kv_heads + head) * a.n_take;
  const uint64_t* mask = a.mask + row * a.mask_words;
  bool any = false;
  for (int i = lane; i < a.n_take; i += 64) any = any || (chosen[i] >= 0 && chosen[i] < full && (i == 0 || chosen[i] > chosen[i - 1]));
  for (int w = lane; 64 * w < n; w += 64) any = any || (mask[w] & (n - 64 * w >= 64 ? ~0ull : (1ull << (n - 64 * w)) - 1));
  return __any(any);
}

// Whether rows of a request attend together, and how.
struct TilePlan {
  bool use;
  int nodes;                  // of a tile
  int per_req;                // tiles of a request
  int row_tiles;              // 16 (node, head) rows each
};
TilePlan sparse_tile_plan(const KvView& c, int64_t n_rows, int32_t n_take, int32_t max_nodes, int32_t n_q_heads);
size_t sparse_tile_bytes(const KvView& c, int64_t n_rows, int32_t n_take, int32_t n_q_heads);
hipError_t launch_sparse_tiles(const SparseArgs& a, const TilePlan& plan, hipStream_t stream);

}  // namespace dflash
