// The pages that a query row may need most, by the bounds of their keys.
//
// The score is a small matrix product in integers: for a tile of up to 16 rows
// of the batch and one kv head, Q' [heads x rows, 2 D] times the bounds
// [2 D, blocks] by v_mfma_i32_16x16x64_i8, Q' holding the negative part of a
// row's codes against the least keys and the positive part against the greatest.
// The largest of the group's heads becomes an order-preserving key.  Then each
// (row, kv head) finds the smallest of its n_take largest keys, and writes the
// blocks from there on in order.
//
// What it cannot do without is one pass over the bounds, 256 bytes for a block
// and kv head of 128 channels.  Blocks of 16 drafted rows do both in one
// workgroup, their keys in LDS (32 requests x 16 rows, 8 kv heads, up to 2048
// blocks, 100 MB of bounds: 46 us, the score 27 of them, 3.7 TB/s of bounds
// while it lasts).  Single rows, and few of them, are split over the chip with their
// keys in the workspace, and a second launch chooses (one row of 8192 blocks, 8
// heads: 12 + 10 us; a chain of small steps, and latency).
#include <algorithm>

#include "kv_sparse.h"

namespace dflash {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr uint32_t kForced = 0xffffffffu, kBroken = 0xfffffffeu;

// NT rows of the batch and 16 / NT heads make the 16 rows of a product; row
// h * NT + node of step s is head s * (16 / NT) + h of that node.
template <int D, int NT>
size_t query_bytes(int steps) { return (size_t)steps * (2 * D / 64) * 1024; }

// The operands of T threads' tile, as they lie: [steps][2 D / 64][64 lanes] x 16
// bytes.  Returns the request of the tile's first row, searched for while the
// queries are on their way.
template <int D, int NT, int T>
__device__ __forceinline__ int32_t read_queries(const SelectArgs& a, int group, int steps, int head, int64_t row0, int8_t* queries) {
  const KvView& c = a.c;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // Queries in 8 bits: a wave takes some of the rows.  The first 128 of a row's
  // 16-byte pieces are read once, those of all rows before the first is used.
  constexpr int kHeads = 16 / NT, kOps = 2 * D / 64, kVecs = D / 8;
  constexpr int kWaves = T / 64, kMine = NT < kWaves ? 1 : NT / kWaves;   // rows of a wave
  const int pieces = group * kVecs;
  u32x4 held[kMine][2];
  const auto tile_row = [&](int i) { return min(wave + i * kWaves, NT - 1); };
  const auto query_of = [&](int i) { return a.q + min(row0 + tile_row(i), c.n_rows - 1) * a.q_row + (int64_t)head * group * a.q_head; };
#pragma unroll
  for (int i = 0; i < kMine; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int x = min(lane + 64 * j, pieces - 1);
      held[i][j] = ld16(query_of(i) + (int64_t)(x / kVecs) * a.q_head + (x % kVecs) * 8);
    }
  RowOf at;
  row_of(c, row0, a.max_nodes, at);
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    if (wave + i * kWaves >= NT) break;
    const int n = tile_row(i);
    const uint16_t* qp = query_of(i);
    uint32_t top = 0;
    auto widen = [&](u32x4 w) {
#pragma unroll
      for (int j = 0; j < 4; ++j) top = max(top, max(w[j] & 0x7fffu, (w[j] >> 16) & 0x7fffu));
    };
    widen(held[i][0]);
    widen(held[i][1]);
    for (int x = lane + 128; x < pieces; x += 64) widen(ld16(qp + (int64_t)(x / kVecs) * a.q_head + (x % kVecs) * 8));
    top = wave_max_u32(top) << 16;
    const bool finite = top < 0x7f800000u;
    const int byte = finite ? max((int)((top + 0x1ffffu) >> 23) - 6, 27) : 127;
    const float inv = finite ? __uint_as_float((uint32_t)(254 - byte) << 23) : 0.f;
    auto store = [&](u32x4 w, int x) {
      const int d = (x % kVecs) * 8;
      float f[8];
      unpack16(w, f);
      uint32_t neg[2] = {0, 0}, pos[2] = {0, 0};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // adding 1.5 * 2^23 rounds to an integer, ties to even, whose two's
        // complement is then in the sum's low bits
        const int code = finite ? (int)(__float_as_uint(f[j] * inv + 12582912.f) << 16) >> 16 : 0;
        neg[j >> 2] |= ((uint32_t)min(code, 0) & 255u) << (8 * (j & 3));
        pos[j >> 2] |= ((uint32_t)max(code, 0) & 255u) << (8 * (j & 3));
      }
      const int slot = x / kVecs, step = slot / kHeads, m = (slot % kHeads) * NT + n;
      // byte k of the contraction: operand k / 64, lane group k % 64 / 16
      int8_t* at = queries + ((step * kOps + d / 64) * 64 + (d % 64 / 16) * 16 + m) * 16 + d % 16;
      *reinterpret_cast<uint2*>(at) = make_uint2(neg[0], neg[1]);
      *reinterpret_cast<uint2*>(at + (D / 64) * 64 * 16) = make_uint2(pos[0], pos[1]);
    };
    if (lane < pieces) store(held[i][0], lane);
    if (lane + 64 < pieces) store(held[i][1], lane + 64);
    // the rest, and heads past the group, which repeat its last
    for (int x = lane + 128; x < pieces; x += 64) store(ld16(qp + (int64_t)(x / kVecs) * a.q_head + (x % kVecs) * 8), x);
    for (int x = pieces + lane; x < steps * kHeads * kVecs; x += 64) store(ld16(qp + (int64_t)(group - 1) * a.q_head + (x % kVecs) * 8), x);
  }
  __syncthreads();
  return at.req;
}

// The keys of blocks first_block .. end_block - 1 of the tile's rows, 16 TT
// blocks a wave's step: put(row of the tile, block, key).  rows(lo, hi, blocks)
// says how many blocks rows lo .. hi - 1 have.
template <int D, int NT, int T, int TT, class Rows, class Put>
__device__ __forceinline__ void score_blocks(const SelectArgs& a, const int8_t* queries, int steps, int head, int64_t row0, int32_t req,
                                             int64_t first_block, int64_t end_block, const Rows& rows, const Put& put) {
  constexpr int kOps = 2 * D / 64, kWaveBlocks = 16 * TT, kStep = kWaveBlocks * T / 64;
  const KvView& c = a.c;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // the requests whose rows the tile holds
  int64_t row = row0;
  for (; row < min(row0 + NT, c.n_rows) && req < c.n_req; ++req) {
    const int64_t first = c.offsets[req], end = min((int64_t)c.offsets[req + 1], min(first + a.max_nodes, c.n_rows));
    const int64_t next = max(row, (int64_t)c.offsets[req + 1]);
    if (max(first, row) >= end) {
      row = next;
      continue;
    }
    const int lo = (int)(max(first, row) - row0), hi = (int)(min(end, row0 + NT) - row0);   // its rows of the tile
    row = next;
    const int32_t blocks = kv_blocks(c, c.start[req]);
    rows(lo, hi, blocks);
    const int32_t* table = c.table + req * c.table_stride;
    const int32_t to = (int32_t)min((int64_t)blocks, end_block);
    int32_t ids[TT];                               // pages of the step, looked up a step ahead
    auto look_up = [&](int64_t b0) {
#pragma unroll
      for (int t = 0; t < TT; ++t) ids[t] = table[(int32_t)min(b0 + 16 * t + (lane & 15), (int64_t)blocks - 1)];
    };
    int64_t b0 = first_block + wave * kWaveBlocks;
    if (b0 < to) look_up(b0);
    for (; b0 < to; b0 += kStep) {
      i32x4_t edge[TT][kOps];
      uint32_t byte[TT];
      bool broken[TT];
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        int32_t id = ids[t];
        broken[t] = id < 0 || id >= c.n_pages;
        if (broken[t]) id = 0;
        const int64_t at = (int64_t)id * c.n_kv_heads + head;
        const int8_t* p = a.codes + at * (2 * D) + (lane >> 4) * 16;
#pragma unroll
        for (int o = 0; o < kOps; ++o) edge[t][o] = *reinterpret_cast<const i32x4_t*>(p + 64 * o);
        byte[t] = a.scale[at];
      }
      if (b0 + kStep < to) look_up(b0 + kStep);
      int best[TT][4];
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) best[t][i] = -0x7fffffff - 1;
      for (int s = 0; s < steps; ++s) {
        i32x4_t q[kOps];
#pragma unroll
        for (int o = 0; o < kOps; ++o) q[o] = *reinterpret_cast<const i32x4_t*>(queries + ((s * kOps + o) * 64 + lane) * 16);
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          i32x4_t sum = {0, 0, 0, 0};
#pragma unroll
          for (int o = 0; o < kOps; ++o) sum = __builtin_amdgcn_mfma_i32_16x16x64_i8(q[o], edge[t][o], sum, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) best[t][i] = max(best[t][i], sum[i]);
        }
      }
      // sum[i] of lane l is row 4 (l / 16) + i of the product and block l % 16
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        if constexpr (NT <= 8) {
#pragma unroll
          for (int i = 0; i < 4; ++i) best[t][i] = max(best[t][i], __shfl_xor(best[t][i], 32, 64));
        }
        if constexpr (NT <= 4) {
#pragma unroll
          for (int i = 0; i < 4; ++i) best[t][i] = max(best[t][i], __shfl_xor(best[t][i], 16, 64));
        }
        if constexpr (NT <= 2) {
          best[t][0] = max(best[t][0], best[t][2]);
          best[t][1] = max(best[t][1], best[t][3]);
        }
        if constexpr (NT == 1) best[t][0] = max(best[t][0], best[t][1]);
        const int64_t b = b0 + 16 * t + (lane & 15);
        // whole numbers up to 2^22 times a power of two: exact.  With 2^-24
        // taken off, for any scale byte from 25 on, they are 0 or normal numbers
        // and so is a difference of two of them.
        const float unit = kv_scale_value(byte[t] == 255u ? 127u : (uint32_t)max((int)byte[t] - 24, 1));
        constexpr int kRegs = NT < 4 ? NT : 4;
        const int groups = NT < 4 ? 1 : NT / 4;   // lane groups that hold rows of their own
#pragma unroll
        for (int i = 0; i < kRegs; ++i) {
          const int n = 4 * (lane >> 4) + i;
          if ((lane >> 4) >= groups || n < lo || n >= hi || b >= to) continue;
          const uint32_t bits = __float_as_uint((float)best[t][i] * unit);
          uint32_t key = (bits & 0x80000000u) ? ~bits : bits | 0x80000000u;
          if (broken[t] || byte[t] == 255u) key = kBroken;
          if (b < a.n_first || b >= blocks - a.n_last) key = kForced;
          put(n, (int32_t)b, key);
        }
      }
    }
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads) select_score_kernel(SelectArgs a, int group, int steps, int chunk_blocks, int chunks) {
  extern __shared__ __align__(16) int8_t queries[];
  const KvView& c = a.c;
  // Consecutive workgroups, on as many XCDs, take the kv heads of the same
  // blocks.  (The heads on one XCD, so that a line of scale bytes is fetched
  // once: one row of 8192 blocks 18 us, this way 9; 512 rows of 2048 38 and 41.)
  const int head = blockIdx.x % c.n_kv_heads;
  const int rest = blockIdx.x / c.n_kv_heads, chunk = rest % chunks;
  const int64_t row0 = (int64_t)(rest / chunks) * NT;
  const int32_t req = read_queries<D, NT, kThreads>(a, group, steps, head, row0, queries);
  score_blocks<D, NT, kThreads, 4>(a, queries, steps, head, row0, req, (int64_t)chunk * chunk_blocks, ((int64_t)chunk + 1) * chunk_blocks,
                                [](int, int, int32_t) {},
                                [&](int n, int32_t b, uint32_t key) { a.keys[((row0 + n) * c.n_kv_heads + head) * c.table_width + b] = key; });
}

// --- the choice ---

// The thread's keys of the segment at s0; 0 past the last, which no key is.
template <int T, int kOwn>
__device__ __forceinline__ void load_keys(const uint32_t* keys, int tid, int64_t s0, int32_t blocks, uint32_t (&k)[kOwn]) {
  const int64_t at = s0 + (int64_t)tid * kOwn;
  typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
  if (at + kOwn <= blocks) {
#pragma unroll
    for (int i = 0; i < kOwn / 4; ++i) {
      const u32x4_a4 x = *reinterpret_cast<const u32x4_a4*>(keys + at + 4 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) k[4 * i + j] = x[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kOwn; ++i) k[i] = at + i < blocks ? keys[at + i] : 0u;
  }
}

// x of all waves, summed; `at` alternates between calls, so that one barrier is
// enough.
template <int T>
__device__ __forceinline__ uint32_t all_waves(uint32_t x, uint32_t (*sums)[T / 64], int& at) {
  at ^= 1;
  if ((threadIdx.x & 63) == 0) sums[at][threadIdx.x >> 6] = x;
  __syncthreads();
  uint32_t all = 0;
#pragma unroll
  for (int i = 0; i < T / 64; ++i) all += sums[at][i];
  return all;
}

// The score that a key stands for.
__device__ __forceinline__ float key_score(uint32_t key) { return __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key); }

// T threads for a (row, kv head), kOwn neighbouring keys each.
//
// The threshold is the smallest key that is taken.  A histogram of the scores
// between the least and the greatest leaves one bin that it lies in, and where
// few keys share it they are ranked one by one; else the bin is the next range.
// Bins are even in the score, not in the key's bits: scores of one magnitude
// share their upper bits, and all threads adding to one bin would wait in line
// (one row of 8192 blocks, 8 heads: 11 bits of the key at a time 29 us, so 10).
template <int T, int kOwn>
__global__ void __launch_bounds__(T) select_take_kernel(SelectArgs a) {
  constexpr int kSegment = kOwn * T, kBins = 2048, kEach = kBins / T, kFew = 64;
  __shared__ uint32_t bins[kBins];
  __shared__ uint32_t sums[2][T / 64], lows[T / 64], highs[T / 64];
  __shared__ uint32_t few[kFew];
  __shared__ uint32_t found[3], n_few, range[2];
  const KvView& c = a.c;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // what the table's row may have, before the row's request is known
  const uint32_t* keys = a.keys + (int64_t)blockIdx.x * c.table_width;
  uint32_t k[kOwn];
  load_keys<T, kOwn>(keys, tid, 0, c.table_width, k);
  const int64_t row = blockIdx.x / (unsigned)c.n_kv_heads;
  RowOf at;
  if (!row_of(c, row, a.max_nodes, at) || row - at.first >= a.max_nodes) return;   // the same in every thread
  const int32_t blocks = kv_blocks(c, at.start), take = a.n_take;
  int32_t* out = a.out + (int64_t)blockIdx.x * take;
  if (blocks <= take) {
    for (int i = tid; i < take; i += T) out[i] = i < blocks ? i : -1;
    return;
  }
  const bool held = blocks <= kSegment;           // the keys stay in registers
#pragma unroll
  for (int i = 0; i < kOwn; ++i) k[i] = tid * kOwn + i < blocks ? k[i] : 0u;   // no key is 0
  int at_sum = 0;
  // calls f for every key (and for the zeros past the last)
  auto for_keys = [&](auto f) {
    for (int64_t s0 = 0; s0 < blocks; s0 += kSegment) {
      if (!held) load_keys<T, kOwn>(keys, tid, s0, blocks, k);
#pragma unroll
      for (int i = 0; i < kOwn; ++i) f(k[i]);
    }
  };

  for (int i = tid; i < kBins; i += T) bins[i] = 0;
  if (tid == 0) n_few = 0;
  uint32_t low = 0xffffffffu, high = 0, forced = 0, broken = 0;
  for_keys([&](uint32_t key) {
    const bool plain = key - 1u < kBroken - 1u;
    low = min(low, plain ? key : 0xffffffffu);
    high = max(high, plain ? key : 0u);
    forced += key == kForced;
    broken += key == kBroken;
  });
  low = ~wave_max_u32(~low);
  high = wave_max_u32(high);
  if (lane == 0) {
    lows[wave] = low;
    highs[wave] = high;
  }
  forced = all_waves<T>(wave_sum_u32(forced), sums, at_sum);
  broken = all_waves<T>(wave_sum_u32(broken), sums, at_sum);
#pragma unroll
  for (int i = 0; i < T / 64; ++i) {
    low = min(low, lows[i]);
    high = max(high, highs[i]);
  }
  uint32_t threshold = low, left = (uint32_t)take;  // left: keys at the threshold that are taken, the first ones
  if (forced >= left) {
    threshold = kForced;
  } else if (forced + broken >= left) {
    threshold = kBroken;
    left -= forced;
  } else {
    left -= forced + broken;                      // of more keys in [low, high]
#pragma unroll 1
    while (low < high) {
      // the least key is in the first bin and the greatest in the last, and a
      // greater score never in a lower bin; so every round leaves a smaller range
      const float least = key_score(low), span = key_score(high) - least;
      auto bin_of = [&](uint32_t key) {
        return key == high ? kBins - 1 : min((int)((key_score(key) - least) / span * (float)(kBins - 1)), kBins - 1);
      };
      for_keys([&](uint32_t key) {
        if (key >= low && key <= high) atomicAdd(&bins[bin_of(key)], 1u);
      });
      __syncthreads();
      uint32_t own[kEach], sum = 0;               // thread t holds the bins from the top down
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        own[i] = bins[kBins - 1 - tid * kEach - i];
        sum += own[i];
      }
      uint32_t scan = sum;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const uint32_t y = (uint32_t)__shfl_up((int)scan, o, 64);
        if (lane >= o) scan += y;
      }
      at_sum ^= 1;
      if (lane == 63) sums[at_sum][wave] = scan;
      __syncthreads();
      uint32_t above = scan - sum;
#pragma unroll
      for (int i = 0; i < T / 64; ++i)
        if (i < wave) above += sums[at_sum][i];
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        if (above < left && above + own[i] >= left) {
          found[0] = kBins - 1 - tid * kEach - i;
          found[1] = left - above;
          found[2] = own[i];
        }
        above += own[i];
        bins[kBins - 1 - tid * kEach - i] = 0;    // for the next round
      }
      if (tid == 0) {
        range[0] = 0xffffffffu;
        range[1] = 0;
      }
      __syncthreads();
      const int bin = (int)found[0];
      const uint32_t in_bin = found[2], from = low, to = high;
      left = found[1];
      if (in_bin <= kFew) {
        for_keys([&](uint32_t key) {
          if (key >= from && key <= to && bin_of(key) == bin) few[atomicAdd(&n_few, 1u)] = key;
        });
        __syncthreads();
        const uint32_t mine = few[min((uint32_t)lane, in_bin - 1)];
        uint32_t greater = 0, as_great = 0;
        for (uint32_t i = 0; i < in_bin; ++i) {
          const uint32_t other = few[i];
          greater += other > mine;
          as_great += other >= mine;
        }
        const uint64_t hit = __ballot(greater < left && as_great >= left);
        const int first = __builtin_ctzll(hit);
        threshold = (uint32_t)__builtin_amdgcn_readlane((int)mine, first);
        left -= (uint32_t)__builtin_amdgcn_readlane((int)greater, first);
        break;
      }
      low = 0xffffffffu;
      high = 0;
      for_keys([&](uint32_t key) {
        if (key < from || key > to || bin_of(key) != bin) return;
        low = min(low, key);
        high = max(high, key);
      });
      atomicMin(&range[0], low);
      atomicMax(&range[1], high);
      __syncthreads();
      threshold = low = range[0];
      high = range[1];
    }
  }

  // blocks above the threshold, and the first `left` at it, in order
  uint32_t base_above = 0, base_at = 0;
  for (int64_t s0 = 0; s0 < blocks; s0 += kSegment) {
    if (!held) load_keys<T, kOwn>(keys, tid, s0, blocks, k);
    uint32_t x = 0;                               // above in the lower half, at it in the upper
#pragma unroll
    for (int i = 0; i < kOwn; ++i) x += k[i] > threshold ? 1u : k[i] == threshold ? 0x10000u : 0u;
    uint32_t scan = x;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const uint32_t y = (uint32_t)__shfl_up((int)scan, o, 64);
      if (lane >= o) scan += y;
    }
    at_sum ^= 1;
    if (lane == 63) sums[at_sum][wave] = scan;
    __syncthreads();
    uint32_t before = scan - x, total = 0;
#pragma unroll
    for (int i = 0; i < T / 64; ++i) {
      if (i < wave) before += sums[at_sum][i];
      total += sums[at_sum][i];
    }
    uint32_t above = base_above + (before & 0xffffu), at = base_at + (before >> 16);
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const bool is_above = k[i] > threshold, is_at = k[i] == threshold;
      if (is_above || (is_at && at < left)) out[above + min(at, left)] = (int32_t)(s0 + tid * kOwn + i);
      above += is_above;
      at += is_at;
    }
    base_above += total & 0xffffu;
    base_at += total >> 16;
  }
}

// One wave for a (row, kv head) of up to 64 KPL blocks; lane l holds keys l,
// l + 64, ..., so that a load is one run.
//
// The threshold is found by halving the range of the scores, and now and then
// that of the keys, which bounds the rounds whatever the scores.  Once no more
// than 64 keys are left in the range, they are put one to a lane and a round
// costs a comparison and not one for each register; equal scores need all the
// rounds, and get them there.  (4096 choices among up to 2048: 14 us of the
// fused kernel, all rounds over all registers 20; a histogram in LDS by a
// workgroup each, from the workspace, 38 against 28.)
__device__ __forceinline__ uint32_t score_key(float x) {
  const uint32_t bits = __float_as_uint(x);
  return (bits & 0x80000000u) ? ~bits : bits | 0x80000000u;
}
// A wave's sum, in all lanes.
__device__ __forceinline__ int wave_total(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);   // row_shr 1, 2, 4, 8
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);   // row_bcast 15, then 31
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);
  return __builtin_amdgcn_readlane(x, 63);
}
// The blocks of one row; k: the lane's keys, 0 past the last; few: 64 words of the wave's own.
template <int KPL>
__device__ __forceinline__ void take_of_wave(const uint32_t (&k)[KPL], int32_t blocks, int32_t take, int32_t* out, uint32_t* few) {
  const int lane = threadIdx.x & 63;
  // f(i) for the registers that hold keys, a few more among them
  auto each = [&](auto f) {
    constexpr int kPart = 6;
#pragma unroll
    for (int p = 0; p < KPL; p += kPart) {
      if (p * 64 >= blocks) break;
#pragma unroll
      for (int i = p; i < (p + kPart < KPL ? p + kPart : KPL); ++i) f(i);
    }
  };
  // how many keys are at least x > 0
  auto reach = [&](uint32_t x) -> int {
    int n = 0;
    each([&](int i) { n += k[i] >= x; });
    return wave_total(n);
  };
  uint32_t low = 0xffffffffu, high = 0;           // of the keys that are neither forced nor broken
  each([&](int i) {
    const bool plain = k[i] - 1u < kBroken - 1u;
    low = min(low, plain ? k[i] : 0xffffffffu);
    high = max(high, plain ? k[i] : 0u);
  });
  low = (uint32_t)__builtin_amdgcn_readfirstlane((int)~wave_max_u32(~low));
  high = (uint32_t)__builtin_amdgcn_readfirstlane((int)wave_max_u32(high));
  // n_low >= take keys reach `low`, and n_high < take reach beyond `high`
  int n_low = 64 * KPL, n_high = reach(kBroken);
  if (n_high >= take) {
    n_low = reach(kForced);
    low = high = n_low >= take ? kForced : kBroken;
    if (low == kForced) n_high = 0;
    else n_high = n_low;
  }
  auto next_mid = [&](int round) -> uint32_t {
    uint32_t mid = low + (high - low + 1) / 2;
    if (round % 8) mid = min(max(score_key(0.5f * key_score(low) + 0.5f * key_score(high)), low + 1), high);
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)mid);
  };
  bool exact = false;                             // n_low == take
  int round = 1;
  for (; low < high && n_low - n_high > 64; ++round) {
    const uint32_t mid = next_mid(round);
    const int n = reach(mid);
    if (n < take) {
      high = mid - 1;
      n_high = n;
    } else {
      low = mid;
      n_low = n;
      if (n == take) {
        exact = true;
        break;
      }
    }
  }
  if (low < high && !exact) {
    // the keys that are left, one to a lane
    int n_few = 0;
    const uint32_t span = high - low;
    each([&](int i) {
      const bool in = k[i] - low <= span;
      const uint64_t who = __ballot(in);
      const int at = (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)who, n_few));
      if (in) few[at] = k[i];
      n_few += __builtin_popcountll(who);
    });
    asm volatile("" ::: "memory");                // the wave's accesses are in order
    const uint32_t mine = lane < n_few ? few[lane] : 0u;
    const int beyond = n_high;
    for (; low < high; ++round) {
      const uint32_t mid = next_mid(round);
      const int n = beyond + __builtin_popcountll(__ballot(mine >= mid));
      if (n < take) {
        high = mid - 1;
        n_high = n;
      } else {
        low = mid;
        n_low = n;
        if (n == take) break;
      }
    }
  }
  const uint32_t threshold = low;
  int above = 0;                                  // so many keys before
  if (n_low == take) {                            // all at the threshold
    each([&](int i) {
      const uint64_t who = __ballot(k[i] >= threshold);
      const int at = (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)who, above));
      if (k[i] >= threshold) out[at] = i * 64 + lane;
      above += __builtin_popcountll(who);
    });
    return;
  }
  const int left = take - n_high;                 // keys at the threshold that are taken, the first ones
  int at = 0;
  each([&](int i) {
    const uint64_t is_above = __ballot(k[i] > threshold), is_at = __ballot(k[i] == threshold);
    const int my_above = (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(is_above >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)is_above, above));
    const int my_at = (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(is_at >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)is_at, at));
    if (k[i] > threshold || (k[i] == threshold && my_at < left)) out[my_above + min(my_at, left)] = i * 64 + lane;
    above += __builtin_popcountll(is_above);
    at += __builtin_popcountll(is_at);
  });
}
template <int KPL>
__global__ void __launch_bounds__(kThreads) select_take_wave_kernel(SelectArgs a, int64_t n_items) {
  const KvView& c = a.c;
  const int lane = threadIdx.x & 63;
  const int64_t item = (int64_t)blockIdx.x * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (item >= n_items) return;                    // waves do not wait for each other
  // all that the table's row may have, before the row's request is known
  const uint32_t* keys = a.keys + item * c.table_width;
  uint32_t k[KPL];
#pragma unroll
  for (int i = 0; i < KPL; ++i) k[i] = keys[min(i * 64 + lane, c.table_width - 1)];
  const int64_t row = item / c.n_kv_heads;
  RowOf at;
  if (!row_of(c, row, a.max_nodes, at) || row - at.first >= a.max_nodes) return;   // the same in every lane
  const int32_t blocks = __builtin_amdgcn_readfirstlane(kv_blocks(c, at.start)), take = a.n_take;
  int32_t* out = a.out + item * take;
  if (blocks <= take) {
    for (int i = lane; i < take; i += 64) out[i] = i < blocks ? i : -1;
    return;
  }
#pragma unroll
  for (int i = 0; i < KPL; ++i) k[i] = i * 64 + lane < blocks ? k[i] : 0u;   // no key is 0
  __shared__ uint32_t few[kThreads / 64][64];
  take_of_wave<KPL>(k, blocks, take, out, few[threadIdx.x >> 6]);
}

// Score and choice of NT rows and a kv head in one workgroup, a wave for each
// row's choice: the keys stay in LDS, [NT][key_row].  Two tiles of 16 blocks a
// step, so that 16 waves fit a CU: with four, and 8 waves, 54 us, now 41.
constexpr int kFusedKeys = 36;
template <int D, int NT>
__global__ void __launch_bounds__(64 * NT, (D == 256 ? NT / 4 : 4)) select_fused_kernel(SelectArgs a, int group, int steps, int key_row) {
  constexpr int T = 64 * NT;
  extern __shared__ __align__(16) int8_t queries[];
  __shared__ int32_t row_blocks[NT];              // -1: none of a request
  uint32_t* keys = reinterpret_cast<uint32_t*>(queries + steps * (2 * D / 64) * 1024);
  const KvView& c = a.c;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int head = blockIdx.x % c.n_kv_heads;
  const int64_t row0 = (int64_t)(blockIdx.x / c.n_kv_heads) * NT;
  if (tid < NT) row_blocks[tid] = -1;
  const int32_t req = read_queries<D, NT, T>(a, group, steps, head, row0, queries);
  score_blocks<D, NT, T, 2>(a, queries, steps, head, row0, req, 0, c.table_width,
                            [&](int lo, int hi, int32_t blocks) {
                              if (tid >= lo && tid < hi) row_blocks[tid] = blocks;
                            },
                            [&](int n, int32_t b, uint32_t key) { keys[n * key_row + b] = key; });
  __syncthreads();
  const int32_t blocks = __builtin_amdgcn_readfirstlane(row_blocks[wave]), take = a.n_take;
  if (blocks < 0) return;
  int32_t* out = a.out + ((row0 + wave) * c.n_kv_heads + head) * take;
  if (blocks <= take) {
    for (int i = lane; i < take; i += 64) out[i] = i < blocks ? i : -1;
    return;
  }
  uint32_t k[kFusedKeys];
  uint32_t* mine = keys + wave * key_row;
#pragma unroll
  for (int i = 0; i < kFusedKeys; ++i) k[i] = i * 64 + lane < blocks ? mine[i * 64 + lane] : 0u;   // no key is 0
  take_of_wave<kFusedKeys>(k, blocks, take, out, mine);   // whose keys are in registers now
}

template <int D, int NT>
hipError_t run(const SelectArgs& a, hipStream_t s) {
  const int group = a.n_q_heads / a.c.n_kv_heads, steps = (group + 16 / NT - 1) / (16 / NT);
  const int64_t tiles = (a.c.n_rows + NT - 1) / NT * a.c.n_kv_heads;
  if constexpr (NT >= 8) {
    // One launch where the keys fit LDS and the tiles half the chip.  (8 kv heads
    // of 128, 16 rows to a request, 2048 blocks: 16 requests 35 us and the two
    // launches 37, 32: 42 and 52, 64: 78 and 99; 8 rows, 64 requests: 57 and 75;
    // 1024 blocks, 8 requests: 22 both ways.  Only very many short tables lose: 100
    // blocks of 512 requests of 8 rows 78 and 68.)
    const int key_row = (a.c.table_width + 15) / 16 * 16 + 4;   // rows 4 apart on other banks
    const size_t lds = query_bytes<D, NT>(steps) + (size_t)NT * key_row * 4;
    if (a.c.table_width <= 64 * kFusedKeys && lds + NT * 4 <= 160 * 1024 && tiles >= 128) {
      select_fused_kernel<D, NT><<<(unsigned)tiles, 64 * NT, lds, s>>>(a, group, steps, key_row);
      return hipGetLastError();
    }
  }
  // Blocks of a workgroup: a share that makes as many workgroups as run at once.
  constexpr int kStep = 16 * 4 * (kThreads / 64);   // of its step
  const int64_t wanted = std::max<int64_t>(1, 768 / tiles);
  const int64_t share = (a.c.table_width + wanted - 1) / wanted;
  const int64_t chunk = (share + kStep - 1) / kStep * kStep;
  const int chunks = (int)((a.c.table_width + chunk - 1) / chunk);
  select_score_kernel<D, NT><<<(unsigned)(tiles * chunks), kThreads, query_bytes<D, NT>(steps), s>>>(a, group, steps, (int)chunk, chunks);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // A wave for a (row, kv head) where it holds the longest prefix's keys; else a
  // workgroup.
  const int64_t items = a.c.n_rows * a.c.n_kv_heads;
  const unsigned waves = (unsigned)((items + kThreads / 64 - 1) / (kThreads / 64));
  // (A table has a few pages more than a power of two: for the nodes.)
  if (a.c.table_width <= 18 * 64) select_take_wave_kernel<18><<<waves, kThreads, 0, s>>>(a, items);
  else if (a.c.table_width <= 36 * 64) select_take_wave_kernel<36><<<waves, kThreads, 0, s>>>(a, items);
  else if (a.c.table_width <= 68 * 64) select_take_wave_kernel<68><<<waves, kThreads, 0, s>>>(a, items);
  else select_take_kernel<1024, 8><<<(unsigned)items, 1024, 0, s>>>(a);
  return hipGetLastError();
}
template <int D>
hipError_t run_dim(const SelectArgs& a, hipStream_t s) {
  // rows of a tile: as few as hold a request, for the rest of the product is
  // filled with heads; and no more than 64 KB of operands hold
  const int group = a.n_q_heads / a.c.n_kv_heads;
  int rows = 16;
  while (rows > 1 && (rows / 2 >= a.max_nodes || (int64_t)group * rows * D > 32768)) rows /= 2;
  if (rows == 1) return run<D, 1>(a, s);
  if (rows == 2) return run<D, 2>(a, s);
  if (rows == 4) return run<D, 4>(a, s);
  if (rows == 8) return run<D, 8>(a, s);
  return run<D, 16>(a, s);
}

}  // namespace

size_t kv_select_bytes(int64_t n_rows, int32_t n_kv_heads, int32_t table_width) {
  return ((size_t)n_rows * n_kv_heads * table_width * 4 + 255) / 256 * 256;
}

hipError_t launch_kv_select(const SelectArgs& a, hipStream_t stream) {
  if (a.c.head_dim == 64) return run_dim<64>(a, stream);
  if (a.c.head_dim == 128) return run_dim<128>(a, stream);
  return run_dim<256>(a, stream);
}

}  // namespace dflash
