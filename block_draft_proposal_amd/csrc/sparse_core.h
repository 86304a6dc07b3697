// What the two forms of the attention over chosen pages share: a row by itself
// (sparse_attn.hip) and the rows of a request together (sparse_tile.hip).
#pragma once

#include "kv_mfma.h"
#include "kv_sparse.h"

namespace dflash {

typedef float f32x4_t __attribute__((ext_vector_type(4)));

template <int DT, int D>
struct SparseShape {
  static constexpr int kRB = D * (DT == DFLASH_BF16 ? 2 : 1);
  static constexpr int kChunks = kRB / 16;
  static constexpr int kWaves = kRB == 512 ? 2 : 4, kThreads = 64 * kWaves;
  static constexpr int kTile = 32 * kRB;                              // K (or V) of a step
  static constexpr int kLoads = kTile / 1024;                         // direct loads of K (or V) a lane
  static constexpr int kWaveStages = 2 * 2 * kTile;
  static constexpr int kRowsAt = kWaves * kWaveStages;                // [wave][4 steps][32] byte offsets, int64
  static constexpr int kScalesAt = kRowsAt + kWaves * 4 * 32 * 8;     // [wave][4 steps][K 32, V 32] fp32
  static constexpr int kMasksAt = kScalesAt + (DT == DFLASH_BF16 ? 0 : kWaves * 4 * 64 * 4);   // [wave][4 steps][32], of tiles
  static constexpr int kLoop = kMasksAt + kWaves * 4 * 32 * 4;
  static constexpr int kJoin = kWaves * 16 * (D + 2) * 4;             // after the loop: [wave] O, m and l of 16 rows
  static constexpr int kLds = kLoop > kJoin ? kLoop : kJoin;
  static constexpr int kPerCu = kLds <= 80 * 1024 ? 2 : 1;            // workgroups that a CU holds
  static_assert(kLds <= 160 * 1024 && 2 * kLoads < 63, "LDS of a CU, loads in flight");

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
