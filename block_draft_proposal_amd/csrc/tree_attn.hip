// Attention of drafted nodes over a paged cache.
//
// One request and kv head form n * group query rows over the same keys.  A
// workgroup takes kRows = 32 RW of them (an item) and walks kKeys keys a step:
//
//   S^T = K Q^T        v_mfma_f32_32x32x16_bf16, a lane holds 16 scores of one row
//   running maximum, p = 2^(s - m), running sum          in registers
//   O^T += V^T P^T     the same lane's p, packed to bf16, are the operand as they lie
//
// Transposed products keep a row's softmax inside a lane and its partner 32
// lanes away, and need no movement of P: the contraction over keys may take
// them in any order, and V's transposed reads (ds_read_b64_tr) use the order
// that the scores already have.  K and V come by 16-byte direct global -> LDS
// loads into two stages; the 16-byte chunks of a row are swizzled so that
// neither product's reads collide on banks.  8-bit codes stay 8 bits in LDS
// and become bf16 (exactly) on the way into the product; their scales, powers
// of two, multiply the scores and the weights.
//
// A workgroup's waves are RW (rows) x KW (keys of a step): few rows leave
// waves to spare, which split the keys and join their sums at the end.
//
// Work is split evenly whatever the lengths: the steps of all items, with a
// constant for what an item costs besides, form one line that is cut into
// equal pieces, one for each workgroup.  A piece that covers an item writes
// its result; pieces of a cut item leave (m, l, O) in the workspace, at most
// two to a workgroup, and a second kernel joins them in a fixed order (32
// requests x 16 nodes, bf16: 73 us and 10).
//
// Loads run two steps ahead of the products and do not stop at an item's end:
// each step's rows are looked up (page table, then addresses into LDS) by one
// thread a row, two steps before its direct loads are issued.
//
// Measured (pages of 16, 8 kv heads of 128, all requests alike; us, both
// kernels, passes in one graph; boxes differ by 2 %): 64 requests x 4 nodes x
// 32 heads over 8160 positions, bf16 382 (5.6 TB/s; a plain read of 2 GiB runs
// at 6.7), e4m3 208 (5.2), int8 214 (5.1): bound by HBM, each byte read once.
// 16 nodes: 396, 262, 302; in int8 the vector units issue for half of the
// time, mostly conversions.  8 requests x 64 nodes x 64 heads over 16384: 335
// to 344, 343, 426 (800 to 820, 803, 646 TFLOP/s; a library product of 8192^3
// reaches 1430): the matrix cores are busy for 31 % of the time, vector units
// issue for 23, LDS is read for 17: a wave waits in turn for each, two waves to
// a SIMD.  One token over 200 positions: 14.0, main kernel 27 000 cycles in a
// row (plan 2400, query and cursor 2700, two iterations that look rows up and
// issue their loads 3000, their arrival 2700, first step 2100, second step and
// the join of the key waves 11 100, output 1900, the loop's end 1500).
// Tried without gain (each beside the kernel of its day, wide: the bf16 shape
// of 64 nodes above): a ring of four stages with one barrier a step (wide 330
// for 337, but 16 nodes e4m3 276 for 263), two row tiles to a wave (wide 356
// for 337), sums of the rounded weights (wide 346 for 337, error 2.0e-3 for
// 2.1e-3), steps priced by their rows (256 requests 502 for 484).
#include <algorithm>
#include <type_traits>

#include "kv_cache.h"

namespace dflash {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef int i32x2_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void lds_void_t;

template <int DT, int D, int RW>
struct Shape {
  static constexpr int kRowBytes = D * (DT == DFLASH_BF16 ? 2 : 1);
  static constexpr int kKeyWaves = kRowBytes == 512 ? (RW == 1 ? 2 : 1) : RW == 8 ? 1 : 4 / RW;
  static constexpr int kKeys = kRowBytes == 512 ? (RW == 1 ? 64 : 32)      // keys of a step
                               : RW == 1 || RW == 8 ? 128
                               : RW == 2        ? (DT == DFLASH_BF16 && D == 128 ? 64 : 128)
                                                : 64;
  static constexpr int kRows = 32 * RW;
  static constexpr int kWaves = RW * kKeyWaves, kThreads = 64 * kWaves;
  static constexpr int kSubs = kKeys / kKeyWaves / 32;                     // 32-key blocks of a wave in a step
  static constexpr int kChunks = kRowBytes / 16;
  static constexpr int kTile = kKeys * kRowBytes;                          // bytes of K (or V) in a step
  static constexpr int kLoads = kTile / 1024 / kWaves;                     // direct loads of K (or V) per thread
  static constexpr int kRowsAt = 4 * kTile;                                // [2 stages][kKeys] byte offsets, int64
  static constexpr int kScalesAt = kRowsAt + 16 * kKeys;                   // [2 stages][K, V][kKeys] fp32
  static constexpr int kBadAt = kScalesAt + (DT == DFLASH_BF16 ? 0 : 16 * kKeys);   // [4 steps][2] a row without a page
  static constexpr int kStatsAt = kBadAt + 32;                             // [kKeyWaves][kRows] m, l
  static constexpr int kLds = kStatsAt + 8 * kKeyWaves * kRows;
  // Workgroups of a CU, by their LDS and by registers: two waves to a SIMD,
  // one with heads of 256 (8 x 64 nodes x 64 heads of 256 over 8192, bf16: 445
  // us, with pieces for twice as many 479).
  static constexpr int kPerCu = kLds <= 80 * 1024 && kWaves * (D == 256 ? 2 : 1) <= 4 ? 2 : 1;
  static constexpr int kPartOdd = kRows * (D + 2);                         // a partial: O [kRows][D], m and l of each
  static constexpr int kPartFloats = kPartOdd + 4;                         // row, whether odd values were left out
  static_assert(kSubs >= 1 && kSubs <= 4 && kLoads >= 1 && kTile % (1024 * kWaves) == 0, "a step splits over the waves");
  static_assert(kKeyWaves / 2 * kRows * D * 4 <= 2 * kTile, "the join fits where one stage was");
  static_assert(kKeys <= kThreads && kKeys <= 128, "one thread looks up a row");
  static_assert(kLds <= 160 * 1024, "LDS of a CU");

  // Chunk c of stage row r lies in slot c ^ swizzle(r), so that reads of one
  // instruction fall on different banks: for K, 16 consecutive rows of one
  // chunk; for V's transposed reads, rows r .. r+3 of four chunks (16-bit
  // elements) or rows r .. r+3, r+8 .. r+11 of two (8-bit).
  static constexpr int kRowsPerBanks = kRowBytes >= 256 ? 1 : 256 / kRowBytes;
  __device__ static __forceinline__ int k_swizzle(int r) { return (r / kRowsPerBanks) & (16 / kRowsPerBanks - 1); }
  __device__ static __forceinline__ int v_swizzle(int r) {
    if constexpr (DT == DFLASH_BF16) return kRowBytes == 128 ? ((r >> 1) & 1) << 2 : (r & 3) << 2;
    else if constexpr (kRowBytes == 256) return ((r & 3) | ((r >> 1) & 4)) << 1;
    else if constexpr (kRowBytes == 128) return (((r >> 1) & 1) | ((r >> 2) & 2)) << 1;
    else return ((r >> 3) & 1) << 1;
  }
};

// What an item costs besides its steps, in steps: the first step's latency,
// the join of the key waves and the output.  (bf16, 32 ragged requests of 16
// nodes, up to 4096 positions: 85 us, priced at 0 steps 99, at 4 the same.)
constexpr int kItemCost = 2;
// A piece is at least this long.  One token over 2000 positions: 16.6 us, with
// pieces of 4 19.3, of 1 15.7, but 16 over 4000 22.2, 28.3 and 25.6.
constexpr int kMinPiece = 2;
// Lengths beyond this, or beyond the page table, have no positions: such a
// request takes one step, whatever its length claims to be, and is NaN.
constexpr int kMaxLen = 0x7fffffff - (1 << 17);

template <int N>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
// A barrier that leaves direct loads in flight (each thread has waited for
// those it needs): only this thread's LDS accesses are waited for.
__device__ __forceinline__ void step_barrier() {
  __builtin_amdgcn_s_waitcnt((0 << 8) | (7 << 4) | 15 | (3 << 14));
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// x of the lane 32 away, combined.
__device__ __forceinline__ float half_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// 8 codes (two words) as 8 bf16, exactly.
template <int DT>
__device__ __forceinline__ bf16x8_t codes_to_bf16(uint32_t a, uint32_t b) {
  u32x4 o;
  if constexpr (DT == DFLASH_E4M3) {
    o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, false));
    o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, true));
    o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, false));
    o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, true));
  } else {
    float x[4], y[4];
    unpack_codes<DT>(a, x);
    unpack_codes<DT>(b, y);
    // an integer below 256 has no bits under bf16's: the upper halves are exact
    o[0] = __builtin_amdgcn_perm(__float_as_uint(x[1]), __float_as_uint(x[0]), 0x07060302u);
    o[1] = __builtin_amdgcn_perm(__float_as_uint(x[3]), __float_as_uint(x[2]), 0x07060302u);
    o[2] = __builtin_amdgcn_perm(__float_as_uint(y[1]), __float_as_uint(y[0]), 0x07060302u);
    o[3] = __builtin_amdgcn_perm(__float_as_uint(y[3]), __float_as_uint(y[2]), 0x07060302u);
  }
  return __builtin_bit_cast(bf16x8_t, o);
}

__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u; }

// A transposed read of V: among 16 lanes, lane i gets column i of the 16 x
// 16-bit by 4-row (8-bit: 8-row) block whose pieces of 8 bytes the lanes
// address.  The parameter is restrict so that the compiler tells the read from
// the direct loads in flight (into the other stage), and does not wait for them.
typedef short i16x4_t __attribute__((ext_vector_type(4)));
template <int DT>
__device__ __forceinline__ i32x2_t read_transposed(const __attribute__((address_space(3))) unsigned char* __restrict__ p) {
  if constexpr (DT == DFLASH_BF16)
    return __builtin_bit_cast(i32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4_t*)p));
  else
    return __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2_t*)p);
}

// Sets the elements of w that are not finite to zero; whether there were any.
template <int DT>
__device__ __forceinline__ bool odd_values(u32x4& w) {
  bool any = false;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    // the top bit of each element whose magnitude bits are all those of an infinity or NaN
    const uint32_t hit = DT == DFLASH_BF16 ? ((w[j] & 0x7f807f80u) + 0x00800080u) & 0x80008000u
                                           : ((w[j] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
    if (hit) {
      any = true;
      const uint32_t one = DT == DFLASH_BF16 ? 0x00010001u : 0x01010101u, top = DT == DFLASH_BF16 ? 15 : 7;
      w[j] &= ~(((hit >> top) & one) * (DT == DFLASH_BF16 ? 0xffffu : 0xffu));
    }
  }
  return any;
}

// Uniform loads of a batch's arrays, which no kernel here writes: through the
// constant address space they are scalar loads, which do not wait for (or
// make anything wait for) the vector loads in flight.
__device__ __forceinline__ int32_t uniform_load(const int32_t* p, int64_t i) {
  return ((const __attribute__((address_space(4))) int32_t*)(uintptr_t)p)[i];
}

// A request's share of the line.
struct Req {
  int32_t first;             // its first row
  int32_t n;                 // nodes
  int32_t start;             // prefix positions
  int32_t len;               // start + n; 1 where over
  int32_t steps;             // ceil(len / keys); 0 without nodes
  int32_t tiles;             // row tiles
  bool over;                 // start + n is beyond kMaxLen or the table
  __device__ __forceinline__ int64_t cost(int heads) const {
    return steps ? (int64_t)(steps + kItemCost) * (tiles * heads) : 0;
  }
};
template <int KEYS, int ROWS>
__device__ __forceinline__ Req make_request(const TreeArgs& a, int32_t first, int32_t end, int32_t start, int group) {
  Req q;
  const int64_t n = first < 0 ? 0 : max((int64_t)0, min(min((int64_t)end, a.c.n_rows) - first, (int64_t)a.max_nodes));
  q.first = first;
  q.n = (int32_t)n;
  q.start = max(start, 0);
  q.over = q.start + n > min((int64_t)kMaxLen, (int64_t)a.c.table_width * a.c.page_size);
  q.len = q.over ? 1 : (int32_t)(q.start + n);
  q.steps = n > 0 ? (q.len + KEYS - 1) / KEYS : 0;
  q.tiles = (q.n * group + ROWS - 1) / ROWS;
  return q;
}

// The line and this workgroup's piece [u0, u1) of it; req and before: the
// request that u0 lies in and the line before it.
struct Piece {
  int64_t total, u0, u1, before;
  int32_t pieces, w, req;
  __device__ __forceinline__ int64_t begin(int64_t i) const { return total * i / pieces; }
  // the piece that point u lies in
  __device__ __forceinline__ int32_t of(int64_t u) const { return (int32_t)(((u + 1) * pieces - 1) / total); }
};

// x of the lanes that a DPP control names, 0 where there is none.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ int64_t dpp_i64(int64_t x) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)x, CTRL, ROW_MASK, 0xf, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(x >> 32), CTRL, ROW_MASK, 0xf, false);
  return (int64_t)(((uint64_t)hi << 32) | lo);
}
// Inclusive sums along a wave.
__device__ __forceinline__ int64_t wave_scan(int64_t x) {
  x += dpp_i64<0x111, 0xf>(x);                    // row_shr 1, 2, 4, 8
  x += dpp_i64<0x112, 0xf>(x);
  x += dpp_i64<0x114, 0xf>(x);
  x += dpp_i64<0x118, 0xf>(x);
  x += dpp_i64<0x142, 0xa>(x);                    // row_bcast 15, then 31
  x += dpp_i64<0x143, 0xc>(x);
  return x;
}

// x of the first lane, known to be the same in all: kept in scalar registers.
__device__ __forceinline__ int64_t uniform_i64(int64_t x) {
  return ((int64_t)__builtin_amdgcn_readfirstlane((int32_t)(x >> 32)) << 32) |
         (uint32_t)__builtin_amdgcn_readfirstlane((int32_t)x);
}

template <class S>
__device__ __forceinline__ Piece find_piece(const TreeArgs& a, int group) {
  __shared__ int64_t sums[S::kWaves];
  __shared__ int64_t found[2];
  const int tid = threadIdx.x, wave = tid >> 6, n_req = a.c.n_req;
  auto cost_of = [&](int r) -> int64_t {
    if (r >= n_req) return 0;
    return make_request<S::kKeys, S::kRows>(a, a.c.offsets[r], a.c.offsets[r + 1], a.c.start[r], group).cost(a.c.n_kv_heads);
  };
  // the first kThreads requests' sums stay in registers; more come in rounds
  const int64_t own0 = cost_of(tid), scan0 = wave_scan(own0);
  Piece p;
  p.total = 0;
  for (int r0 = 0; r0 < n_req; r0 += S::kThreads) {
    const int64_t scan = r0 == 0 ? scan0 : wave_scan(cost_of(r0 + tid));
    if (r0) __syncthreads();
    if ((tid & 63) == 63) sums[wave] = scan;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < S::kWaves; ++i) p.total += sums[i];
  }
  p.total = uniform_i64(p.total);
  p.pieces = (int32_t)min((int64_t)gridDim.x, (p.total + kMinPiece - 1) / kMinPiece);
  p.w = (int)blockIdx.x < p.pieces ? (int)xcd_contiguous(blockIdx.x, p.pieces) : (int)blockIdx.x;
  p.u0 = p.u1 = p.before = 0;
  p.req = n_req;
  if (p.w >= p.pieces) return p;                  // the whole workgroup: nothing to do
  p.u0 = p.begin(p.w);
  p.u1 = p.begin(p.w + 1);
  int64_t run = 0;
  for (int r0 = 0; r0 < n_req && uniform_i64(run) <= p.u0; r0 += S::kThreads) {
    int64_t own = own0, scan = scan0;
    if (n_req > S::kThreads) {                    // sums holds the last round's
      if (r0) {
        own = cost_of(r0 + tid);
        scan = wave_scan(own);
      }
      __syncthreads();
      if ((tid & 63) == 63) sums[wave] = scan;
      __syncthreads();
    }
    int64_t all = 0;
    scan += run;
#pragma unroll
    for (int i = 0; i < S::kWaves; ++i) {
      if (i < wave) scan += sums[i];
      all += sums[i];
    }
    if (scan - own <= p.u0 && p.u0 < scan) {
      found[0] = r0 + tid;
      found[1] = scan - own;
    }
    run += all;
  }
  __syncthreads();
  p.req = __builtin_amdgcn_readfirstlane((int32_t)found[0]);
  p.before = uniform_i64(found[1]);
  return p;
}

// Walks the steps of a piece.
template <class S>
struct Cursor {
  Req q;
  int64_t at;                // where the item begins on the line
  int64_t u0, u1;
  int32_t req, item, head, tile, t, t1;
  bool valid;

  // The item's steps that lie in the piece; on to the next item where there are none.
  __device__ __forceinline__ void settle(const TreeArgs& a, int group) {
    for (;;) {
      if (at >= u1) {
        valid = false;
        return;
      }
      if (item >= q.tiles * a.c.n_kv_heads || q.steps == 0) {
        if (++req >= a.c.n_req) {
          valid = false;
          return;
        }
        load(a, group);
        item = 0;
        continue;
      }
      const int64_t lo = u0 - at - kItemCost, hi = u1 - at - kItemCost;
      t = (int32_t)max(lo, (int64_t)0);
      t1 = (int32_t)min(hi, (int64_t)q.steps);
      if (t < t1) {
        head = item / q.tiles;
        tile = item - head * q.tiles;
        return;
      }
      at += q.steps + kItemCost;
      ++item;
    }
  }
  __device__ __forceinline__ void load(const TreeArgs& a, int group) {
    q = make_request<S::kKeys, S::kRows>(a, uniform_load(a.c.offsets, req), uniform_load(a.c.offsets, req + 1),
                                         uniform_load(a.c.start, req), group);
  }
  __device__ __forceinline__ void begin(const TreeArgs& a, const Piece& p, int group) {
    u0 = p.u0;
    u1 = p.u1;
    req = p.req;
    load(a, group);
    const int32_t per_item = q.steps + kItemCost;
    item = (int32_t)((p.u0 - p.before) / per_item);
    at = p.before + (int64_t)item * per_item;
    valid = true;
    settle(a, group);
  }
  __device__ __forceinline__ void next_item(const TreeArgs& a, int group) {
    at += q.steps + kItemCost;
    ++item;
    settle(a, group);
  }
};

// What the join needs of a cut item (n: its pieces; 0: none).
struct JoinItem {
  int32_t piece, n, rows;           // first piece (the item in its slot 1, in later ones' slot 0)
  int32_t first, nodes, start, req, head, tile;
  int32_t pad[3];
};

// Whether a node sees anything: a prefix, or a bit of its mask.
__device__ __forceinline__ bool sees_any(const TreeArgs& a, int32_t first, int32_t n, int32_t start, int node) {
  if (start > 0 || !a.mask) return true;
  const uint64_t* m = a.mask + (int64_t)(first + node) * a.mask_words;
  uint64_t any = 0;
  for (int w = 0; w * 64 < n; ++w) {
    const int left = n - w * 64;
    any |= m[w] & (left >= 64 ? ~0ull : (1ull << left) - 1);
  }
  return any != 0;
}

// Adds to 4 elements of a row's result, at d, the values at the nodes it sees
// that are not finite (a sum with such a value is that value, and of both
// infinities NaN, whatever the weights).
template <int DT, int D>
__device__ __forceinline__ void add_odd(const TreeArgs& a, int32_t first, int32_t n, int32_t start, int req, int head,
                                        int node, int d, float (&f)[4]) {
  constexpr int kSize = DT == DFLASH_BF16 ? 2 : 1;
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    if (a.mask ? !((a.mask[(int64_t)(first + node) * a.mask_words + (j >> 6)] >> (j & 63)) & 1) : j > node) continue;
    int64_t page;
    int32_t slot;
    if (!kv_locate(a.c, a.c.table + req * a.c.table_stride, (int64_t)start + j, page, slot)) continue;
    const unsigned char* v = a.c.v + page * a.c.page_bytes + ((int64_t)(head * a.c.page_size + slot) * D + d) * kSize;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x;
      if constexpr (DT == DFLASH_BF16) x = bf16_to_f32(reinterpret_cast<const uint16_t*>(v)[i]);
      else x = __builtin_amdgcn_cvt_f32_fp8((int)v[i], 0);
      if (!isfinite(x)) f[i] += x;
    }
  }
}

template <int DT, int D, int RW>
__global__ void __launch_bounds__((Shape<DT, D, RW>::kThreads), (D == 256 ? 1 : 2))
    tree_attention_kernel(TreeArgs a, FastDiv per_group) {
  using S = Shape<DT, D, RW>;
  constexpr int kRB = S::kRowBytes, kKeys = S::kKeys, kBlocks = D / 32, kSteps16 = D / 16;
  constexpr int kPerBlock = DT == DFLASH_BF16 ? 4 : 2;   // chunks of a 32-column block
  extern __shared__ __align__(16) unsigned char ta_smem[];
  int64_t* row_at = reinterpret_cast<int64_t*>(ta_smem + S::kRowsAt);
  float* scales = reinterpret_cast<float*>(ta_smem + S::kScalesAt);
  int32_t* bad_pages = reinterpret_cast<int32_t*>(ta_smem + S::kBadAt);
  float2* stats = reinterpret_cast<float2*>(ta_smem + S::kStatsAt);
  const KvView& c = a.c;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rw = wave % RW, kw = wave / RW, half = lane >> 5, l32 = lane & 31;
  const int group = per_group.d;
  const Piece piece = find_piece<S>(a, group);
  JoinItem* joins = static_cast<JoinItem*>(a.workspace);
  if (tid == 0) joins[piece.w * 2].n = joins[piece.w * 2 + 1].n = 0;
  if (piece.w >= piece.pieces) return;
  float* parts = reinterpret_cast<float*>(joins + 2 * gridDim.x) + (int64_t)piece.w * 2 * S::kPartFloats;
  // log2(e) and the softmax scale; an int8 cache carries it in K's scales
  const float c2 = a.scale * 1.44269504088896340736f, cs = DT == DFLASH_I8 ? 1.f : c2;

  // K reads: row l32 of a 32-key block, chunk 2t + half in slot (2t) ^ kx
  const int kx = half ^ S::k_swizzle(l32);
  // V reads: lane i of a 16-lane group addresses row vr of a 16-key block
  // (plus 8 for the second half of 16-bit ones) and 8 bytes of a 16-column block
  const int g16 = lane >> 4, i16 = lane & 15;
  const int vj = DT == DFLASH_BF16 ? i16 >> 2 : i16 >> 1;
  const int vr = DT == DFLASH_BF16 ? 4 * half + vj : 8 * (vj >> 2) + 4 * half + (vj & 3);
  const int vx = (DT == DFLASH_BF16 ? 2 * (g16 & 1) + ((i16 >> 1) & 1) : g16 & 1) ^ S::v_swizzle(vr);
  const int vbase = vr * kRB + (i16 & 1) * 8;
  // direct loads: this lane's row in the first of its wave's blocks of 1 KB, and its chunk's place in the row
  const int lane_row = wave * (1024 / kRB) + lane / S::kChunks, lslot = lane % S::kChunks;
  const int64_t* lane_rows = row_at + lane_row;

  // The step being looked up, two or three ahead of the products.
  Cursor<S> feed;
  feed.begin(a, piece, group);
  Cursor<S> w = feed;                              // the step of the products
  const bool feeder = tid < kKeys;                 // this thread looks up row tid of each step
  int32_t page_id = 0, row_in_page = 0;            // of the next step to get addresses
  uint32_t k_byte = 0, v_byte = 0;                 // scale bytes of the step after

  bf16x8_t qf[kSteps16];                           // this row's query, in the order K's chunks have in the product
  int row = rw * 32 + l32, rows = 0, node = 0, gh = 0;   // this lane's row of the item, its node and head of the group
  auto load_query = [&]() {
    rows = min(S::kRows, w.q.n * group - w.tile * S::kRows);
    const int flat = w.tile * S::kRows + min(row, rows - 1);
    node = per_group.div(flat);
    gh = flat - node * group;
    const uint16_t* qp = a.q + (int64_t)(w.q.first + node) * a.q_row + (int64_t)(w.head * group + gh) * a.q_head;
#pragma unroll
    for (int t = 0; t < kSteps16; ++t) {
      const int d = DT == DFLASH_BF16 ? 16 * t + 8 * half : 32 * (t / 2) + 16 * half + 8 * (t & 1);
      qf[t] = __builtin_bit_cast(bf16x8_t, ld16(qp + d));
    }
  };

  // Starts the look-up of the next step's pages; false after the last.
  auto look_up = [&]() -> bool {
    if (!feed.valid) return false;
    if (feeder) {
      // rows past the end repeat the last position; they are masked
      const int pos = min(feed.t * kKeys + tid, feed.q.len - 1), idx = c.per_page.div(pos);
      row_in_page = feed.head * c.page_size + (pos - idx * c.page_size);
      page_id = -1;
      if (idx < c.table_width) page_id = c.table[feed.req * c.table_stride + idx];
    }
    if (++feed.t == feed.t1) feed.next_item(a, group);
    return true;
  };

  // With more than 256 registers the accumulators lie in AGPRs, which only the
  // matrix cores compute with.  Without this, at either end of the rare
  // rescaling, the compiler moves them to VGPRs and back in every step (8 x 64
  // nodes x 64 heads of 256 over 8192, bf16: 542 us, with it 445).
  auto in_accumulators = [](f32x16_t& x) {
    if constexpr (D == 256) asm volatile("" : "+a"(x));
  };
  f32x16_t o[kBlocks];
  float m, l;                                      // of this lane's row; l over this lane's keys only
  bool bad, odd;                                   // a position without a page; a node's value that is not finite
  int t_first;                                     // the item's first step here
  auto clear = [&]() {
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[b][i] = 0.f;
    m = -INFINITY;
    l = 0.f;
    bad = w.q.over;
    odd = false;
    t_first = w.t;
  };
  if (!w.valid) return;                            // the whole workgroup: its piece has no steps
  load_query();
  clear();

  // The products of a step with this wave's rows and keys, 32 keys at a time.
  // masked: some of the keys are nodes, or past the end.  The scores of the
  // next 32 keys (matrix cores) run under the exponentials of these.
  auto products = [&](const unsigned char* stage, int g, int p0, bool masked) {
    const int kb0 = kw * S::kSubs * 32;             // first key of this wave
    const unsigned char* krow = stage + (kb0 + l32) * kRB;
    const auto* v0 = (const __attribute__((address_space(3))) unsigned char*)(stage + S::kTile + kb0 * kRB) + vbase;
    u32x4 kf[kRB / 32];
    auto read_keys = [&](int sub) {
#pragma unroll
      for (int i = 0; i < kRB / 32; ++i) kf[i] = ld16(krow + sub * 32 * kRB + (((2 * i) ^ kx) << 4));
    };
    auto scores = [&](f32x16_t& s) {
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = 0.f;
      if constexpr (DT == DFLASH_BF16) {
#pragma unroll
        for (int t16 = 0; t16 < kSteps16; ++t16)
          s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, kf[t16]), qf[t16], s, 0, 0, 0);
      } else {
#pragma unroll
        for (int t32 = 0; t32 < kSteps16 / 2; ++t32) {
          const u32x4 x = kf[t32];
          s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(codes_to_bf16<DT>(x[0], x[1]), qf[2 * t32], s, 0, 0, 0);
          s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(codes_to_bf16<DT>(x[2], x[3]), qf[2 * t32 + 1], s, 0, 0, 0);
        }
      }
    };
    read_keys(0);
    f32x16_t s;
    scores(s);
#pragma unroll
    for (int sub = 0; sub < S::kSubs; ++sub) {
      // s[i]: key 8 (i / 4) + 4 half + i % 4 of the block of 32
      if constexpr (DT != DFLASH_BF16) {
        const float* kscale = scales + g * 2 * kKeys + kb0 + sub * 32 + 4 * half;
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] *= kscale[8 * (i >> 2) + (i & 3)];
      }
      uint32_t vis = ~0u;
      if (masked) {
        const int k0 = p0 + kb0 + sub * 32, rel = k0 - w.q.start;   // rel: the node of key 0 of the block
        const int pre = min(max(-rel, 0), 32);
        uint32_t bits = 0;
        int seen = w.q.n;
        if (!a.mask) {
          seen = min(seen, node + 1);
          bits = ~0u;
        } else if (rel < w.q.n && pre < 32) {
          const uint64_t* mw = a.mask + (int64_t)(w.q.first + node) * a.mask_words;
          if (rel < 0) {
            bits = (uint32_t)(mw[0] << -rel);
          } else {
            const int word = rel >> 6, sh = rel & 63;
            uint64_t x = mw[word] >> sh;
            if (sh > 32 && word + 1 < a.mask_words) x |= mw[word + 1] << (64 - sh);
            bits = (uint32_t)x;
          }
        }
        bits &= low_bits(seen - rel);
        vis = (low_bits(pre) | (bits & ~low_bits(pre))) >> (4 * half);   // bit 8 (i / 4) + i % 4 for s[i]
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = (vis >> (8 * (i >> 2) + (i & 3))) & 1 ? s[i] : -INFINITY;
      }
      float top = s[0];
#pragma unroll
      for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i]);
      top = half_max(top);
      // The sums keep the maximum they were built with until a row's passes it
      // by 2^8: weights up to 256 are as exact as those up to 1, and most
      // blocks then leave O alone (8 x 64 nodes x 64 heads over 16384, bf16:
      // 338 us, rescaled at every new maximum 349).
      if (__any((top - m) * cs > 8.f)) {
        const float next = fmaxf(m, top), keep = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((m - next) * cs);
        m = next;
        l *= keep;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          in_accumulators(o[b]);
#pragma unroll
          for (int i = 0; i < 16; ++i) o[b][i] *= keep;
          in_accumulators(o[b]);
          if (D == 256) __builtin_amdgcn_sched_barrier(0);   // a block at a time: few registers
        }
      }
      const float base = m == -INFINITY ? 0.f : m * cs;
      if (sub + 1 < S::kSubs) read_keys(sub + 1);
      // V of up to four blocks of 32 columns: [column block][16-key operand]
      constexpr int kGroup = kBlocks < 4 ? kBlocks : 4, kPieces = DT == DFLASH_BF16 ? 4 : 2;
      i32x2_t r[kGroup][kPieces];
      auto read_group = [&](int b) {
#pragma unroll
        for (int i = 0; i < kGroup; ++i)
#pragma unroll
          for (int x = 0; x < kPieces; ++x)
            r[i][x] = read_transposed<DT>(v0 + (((kPerBlock * (b + i)) ^ vx) << 4) +
                                          (sub * 32 + x * (DT == DFLASH_BF16 ? 8 : 16)) * kRB);
      };
      read_group(0);
      __builtin_amdgcn_sched_barrier(0);
      f32x16_t next_s;
      if (sub + 1 < S::kSubs) scores(next_s);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[i] = __builtin_amdgcn_exp2f(DT != DFLASH_I8 ? fmaf(s[i], cs, -base) : s[i] - base);
        sum += s[i];
      }
      l += sum;
      if constexpr (DT != DFLASH_BF16) {
        const float* vscale = scales + g * 2 * kKeys + kKeys + kb0 + sub * 32 + 4 * half;
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] *= vscale[8 * (i >> 2) + (i & 3)];
        if (masked) {                               // 0 * NaN: an unseen key's scale
#pragma unroll
          for (int i = 0; i < 16; ++i) s[i] = (vis >> (8 * (i >> 2) + (i & 3))) & 1 ? s[i] : 0.f;
        }
      }
      // weights rounded to bf16 (half a step, 2^-8 of each): the product with
      // V is bf16 x bf16 on the matrix cores; l sums them unrounded
      bf16x8_t pf[2];
#pragma unroll
      for (int u16 = 0; u16 < 2; ++u16) {
        const u32x4 pw = {pack_bf16(s[8 * u16], s[8 * u16 + 1]), pack_bf16(s[8 * u16 + 2], s[8 * u16 + 3]),
                          pack_bf16(s[8 * u16 + 4], s[8 * u16 + 5]), pack_bf16(s[8 * u16 + 6], s[8 * u16 + 7])};
        pf[u16] = __builtin_bit_cast(bf16x8_t, pw);
      }
      if (sub + 1 < S::kSubs) {
#pragma unroll
        for (int i = 0; i < kSteps16; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x002, (DT == DFLASH_BF16 ? 56 : DT == DFLASH_E4M3 ? 104 : 168) / kSteps16, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int b = 0; b < kBlocks; b += kGroup) {
        if (b) read_group(b);
#pragma unroll
        for (int x = 0; x < 2 * kGroup; ++x) {
          const int i = x % kGroup, u16 = x / kGroup;
          bf16x8_t vf;
          if constexpr (DT == DFLASH_BF16)
            vf = __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(r[i][2 * u16], r[i][2 * u16 + 1], 0, 1, 2, 3));
          else
            vf = codes_to_bf16<DT>((uint32_t)r[i][u16][0], (uint32_t)r[i][u16][1]);
          o[b + i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, pf[u16], o[b + i], 0, 0, 0);
        }
      }
      if (sub + 1 < S::kSubs) s = next_s;
    }
  };

  // e0, e1, e2: whether steps g, g+1, g+2 exist.  Iteration g multiplies step
  // g, writes step g+1's scales, gives step g+2 its addresses and its direct
  // loads, and looks up step g+3's pages; the first two only fill.
  bool e0 = false, e1 = false, e2 = look_up();
  wait_vm<0>();
  for (int s4 = 2;; s4 = (s4 + 1) & 3) {           // the iteration's step, modulo 4
    const int g = s4 & 1;                          // its stage
    wait_vm<2 * S::kLoads>();                      // all but step g+1's direct loads have arrived
    step_barrier();
    unsigned char* stage = ta_smem + g * 2 * S::kTile;
    if (feeder) {
      if constexpr (DT != DFLASH_BF16) {
        float* sc = scales + (g ^ 1) * 2 * kKeys + tid;
        sc[0] = DT == DFLASH_I8 ? kv_scale_value(k_byte) * c2 : kv_scale_value(k_byte);
        sc[kKeys] = kv_scale_value(v_byte);
      }
      const bool no_page = page_id < 0 || page_id >= c.n_pages, use = e2 && !no_page;
      const int64_t id = use ? page_id : 0;
      const int32_t at = use ? row_in_page : 0;
      row_at[g * kKeys + tid] = id * c.page_bytes + (int64_t)at * kRB;
      const uint64_t any = __ballot(no_page);
      if (lane == 0) bad_pages[((s4 + 2) & 3) * 2 + wave] = any != 0;
      if constexpr (DT != DFLASH_BF16) {
        k_byte = c.k_scale[id * c.scale_page_bytes + at];
        v_byte = c.v_scale[id * c.scale_page_bytes + at];
      }
    }
    const bool e3 = look_up();
    bool ends = false;
    if (e0) {
#pragma unroll
      for (int i = 0; i < (kKeys + 63) / 64; ++i) bad = bad || bad_pages[s4 * 2 + i];
      const int p0 = w.t * kKeys;
      const bool masked = p0 + kKeys > w.q.start;   // the step reaches the tree (or the end)
      if constexpr (DT != DFLASH_I8) {
        if (masked) {
          // A weight of zero times an infinity is no zero: a node's value that
          // is not finite must not reach the rows that do not see it.  Such
          // elements become zeros here and are added at the end, where seen.
          unsigned char* vw = stage + S::kTile;
          for (int x = tid; x < S::kTile / 16; x += S::kThreads) {
            if (p0 + x / S::kChunks < w.q.start) continue;
            u32x4 v = ld16(vw + x * 16);
            if (odd_values<DT>(v)) {
              odd = true;
              st16(vw + x * 16, v);
            }
          }
          step_barrier();
        }
      }
      if (rw * 32 < rows) products(stage, g, p0, masked);
      ends = ++w.t == w.t1;
    }
    step_barrier();                                 // every wave is done with this stage; the addresses are there
    if (ends) {
      const JoinItem it = {0, 0, rows, w.q.first, w.q.n, w.q.start, w.req, w.head, w.tile, {0, 0, 0}};
      const int t_last = w.t, steps = w.q.steps, out_node = node, out_gh = gh;
      const int64_t item_at = w.at + kItemCost;
      const bool item_bad = bad, item_odd = odd, whole = t_first == 0 && t_last == steps;
      const int slot = item_at < piece.u0 ? 0 : 1;  // a cut item that began before the piece, or in it
      float mc = m == -INFINITY ? -INFINITY : m * cs;
      l = half_sum(l);
      w.next_item(a, group);
      if (w.valid) load_query();                    // arrives while this item is finished
      // join the key waves, two halves at a time, through the free stage
      if constexpr (S::kKeyWaves > 1) {
        if (half == 0) stats[kw * S::kRows + row] = make_float2(mc, l);
        step_barrier();
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < S::kKeyWaves; ++i) top = fmaxf(top, stats[i * S::kRows + row].x);
        const float keep = mc == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mc - top);
        l = 0.f;
#pragma unroll
        for (int i = 0; i < S::kKeyWaves; ++i) {
          const float2 x = stats[i * S::kRows + row];
          l += x.x == -INFINITY ? x.y : x.y * __builtin_amdgcn_exp2f(x.x - top);
        }
        mc = top;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[b][i] *= keep;
#pragma unroll
        for (int from = S::kKeyWaves / 2; from > 0; from /= 2) {
          float4* pool = reinterpret_cast<float4*>(stage) + ((kw % from) * RW + rw) * (D / 8) * 64 + lane;
          if (kw >= from && kw < 2 * from) {
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                pool[(4 * b + i) * 64] = make_float4(o[b][4 * i], o[b][4 * i + 1], o[b][4 * i + 2], o[b][4 * i + 3]);
          }
          step_barrier();
          if (kw < from) {
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float4 f = pool[(4 * b + i) * 64];
                o[b][4 * i] += f.x;
                o[b][4 * i + 1] += f.y;
                o[b][4 * i + 2] += f.z;
                o[b][4 * i + 3] += f.w;
              }
          }
          step_barrier();
        }
      }
      if (item_bad) l = __builtin_nanf("");         // every thread has seen every step's pages
      const bool any_odd = DT != DFLASH_I8 && __syncthreads_or(item_odd);
      if (kw == 0 && row < it.rows) {
        if (whole) {
          const float inv = sees_any(a, it.first, it.nodes, it.start, out_node) ? 1.f / l : 0.f;
          uint16_t* op = a.out + ((int64_t)(it.first + out_node) * a.n_q_heads + it.head * group + out_gh) * D;
#pragma unroll
          for (int b = 0; b < kBlocks; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint2*>(op + 32 * b + 8 * i + 4 * half) =
                  make_uint2(pack_bf16(o[b][4 * i] * inv, o[b][4 * i + 1] * inv),
                             pack_bf16(o[b][4 * i + 2] * inv, o[b][4 * i + 3] * inv));
          if (any_odd) {
#pragma unroll 1
            for (int x = 0; x < D / 8; ++x) {       // this lane's own 4 elements of each 8
              uint2* at = reinterpret_cast<uint2*>(op + 8 * x + 4 * half);
              const uint2 v = *at;
              float f[4] = {bf16_to_f32(v.x & 0xffffu), bf16_to_f32(v.x >> 16), bf16_to_f32(v.y & 0xffffu),
                            bf16_to_f32(v.y >> 16)};
              add_odd<DT, D>(a, it.first, it.nodes, it.start, it.req, it.head, out_node, 8 * x + 4 * half, f);
              *at = make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
            }
          }
        } else {
          float* part = parts + slot * S::kPartFloats;
#pragma unroll
          for (int b = 0; b < kBlocks; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<float4*>(part + row * D + 32 * b + 8 * i + 4 * half) =
                  make_float4(o[b][4 * i], o[b][4 * i + 1], o[b][4 * i + 2], o[b][4 * i + 3]);
          if (half == 0) *reinterpret_cast<float2*>(part + S::kRows * D + 2 * row) = make_float2(mc, l);
          if (tid == 0) {
            part[S::kPartOdd] = any_odd ? 1.f : 0.f;
            JoinItem j = it;
            j.piece = piece.of(item_at);
            j.n = piece.of(item_at + steps - 1) - j.piece + 1;
            joins[piece.w * 2 + slot] = j;
          }
        }
      }
      clear();
      step_barrier();                               // the stage and the statistics are free
    }
    // Past the last step the same number of loads takes row 0 of the pool (into
    // a stage that nothing reads any more): at the loop's top, on every path,
    // all but these are older than the count waited for, and the compiler adds
    // no waits of its own at the other loads' uses.
    constexpr int kStride = S::kWaves * (1024 / kRB);     // rows between a lane's; swizzles repeat after 16
    int64_t rows_at[S::kLoads];
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) rows_at[i] = lane_rows[g * kKeys + i * kStride];
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) {
      const int64_t at = rows_at[i];
      const int r = lane_row + i * kStride % 16;
      unsigned char* to = stage + wave * 1024 + i * S::kWaves * 1024;
      __builtin_amdgcn_global_load_lds((const void*)(c.k + at + ((lslot ^ S::k_swizzle(r)) << 4)), (lds_void_t*)to, 16, 0, 0);
      __builtin_amdgcn_global_load_lds((const void*)(c.v + at + ((lslot ^ S::v_swizzle(r)) << 4)),
                                       (lds_void_t*)(to + S::kTile), 16, 0, 0);
    }
    e0 = e1;
    e1 = e2;
    e2 = e3;
    if (!(e0 || e1 || e2)) break;
  }
  wait_vm<0>();
}

// Joins the pieces of cut items, in the order of the line: nothing depends on
// which piece finished first.  kJoinWgs workgroups for each piece share the
// rows of its items.  Up to 8 pieces, a thread adds the parts of its 4
// elements; with more, 16 threads do, and their sums are added in their order.
// (One workgroup for each: 16 nodes over 4000 positions 27.7 us, with 4 22.2.)
constexpr int kJoinWgs = 4;

struct JoinSum {
  float top = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  __device__ __forceinline__ void add(float m2, float l2, const float (&p)[4]) {
    const float next = fmaxf(top, m2);
    // a part that saw nothing has l = 0, or NaN for a bad page, and O = 0
    const float w1 = top == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(top - next);
    const float w2 = m2 == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m2 - next);
    top = next;
    l = l * w1 + l2 * w2;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = o[i] * w1 + p[i] * w2;
  }
};

template <int DT, int D, int RW>
__global__ void __launch_bounds__(256) tree_join_kernel(TreeArgs a, FastDiv per_group) {
  using S = Shape<DT, D, RW>;
  __shared__ float sh[256][7];
  const JoinItem* joins = static_cast<const JoinItem*>(a.workspace);
  const float* parts = reinterpret_cast<const float*>(joins + 2 * gridDim.x);
  const int tid = threadIdx.x, group = per_group.d;
  for (int slot = 0; slot < 2; ++slot) {
    const JoinItem it = joins[blockIdx.x * 2 + slot];
    if (it.n == 0) continue;
    const int total = it.rows * (D / 4), wg = ((int)blockIdx.x - it.piece) * kJoinWgs + (int)blockIdx.y;
    const bool few = it.n <= 8;
    const int groups = few ? 1 : 16, vecs = 256 / groups, mine = tid / vecs;
    for (int v0 = wg * vecs; v0 < total; v0 += it.n * kJoinWgs * vecs) {
      const int e = min(v0 + tid % vecs, total - 1), row = e / (D / 4), d = (e % (D / 4)) * 4;
      JoinSum s;
      float odd = 0.f;
#pragma unroll 4
      for (int x = mine; x < it.n; x += groups) {
        const float* p = parts + ((int64_t)(it.piece + x) * 2 + (x == 0 ? 1 : 0)) * S::kPartFloats;
        const float2 ml = *reinterpret_cast<const float2*>(p + S::kRows * D + 2 * row);
        const float4 f = *reinterpret_cast<const float4*>(p + row * D + d);
        odd += p[S::kPartOdd];
        s.add(ml.x, ml.y, {f.x, f.y, f.z, f.w});
      }
      if (!few) {
        __syncthreads();
        sh[tid][0] = s.top;
        sh[tid][1] = s.l;
#pragma unroll
        for (int i = 0; i < 4; ++i) sh[tid][2 + i] = s.o[i];
        sh[tid][6] = odd;
        __syncthreads();
        if (mine == 0) {
#pragma unroll
          for (int x = 1; x < 16; ++x) {
            const float(&f)[7] = sh[x * vecs + tid];
            odd += f[6];
            s.add(f[0], f[1], {f[2], f[3], f[4], f[5]});
          }
        }
      }
      if (mine != 0 || v0 + tid >= total) continue;
      const int flat = it.tile * S::kRows + row, node = per_group.div(flat), gh = flat - node * group;
      const float inv = sees_any(a, it.first, it.nodes, it.start, node) ? 1.f / s.l : 0.f;
      float f[4] = {s.o[0] * inv, s.o[1] * inv, s.o[2] * inv, s.o[3] * inv};
      if constexpr (DT != DFLASH_I8) {
        if (odd != 0.f) add_odd<DT, D>(a, it.first, it.nodes, it.start, it.req, it.head, node, d, f);
      }
      *reinterpret_cast<uint2*>(a.out + ((int64_t)(it.first + node) * a.n_q_heads + it.head * group + gh) * D + d) =
          make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
    }
  }
}

// Row waves, 32 rows each, by the most rows that a request may have for a kv
// head; the waves left of 4 split the keys.  With 32 rows (e4m3, 16 requests x
// 8 kv heads over 8192) 1, 2, 4 and 8 row waves take 74, 79, 93 and 133 us,
// with 64 rows 2, 4 and 8 take 84, 111 and 138, with 128 rows 4 and 8 127 and
// 143.  8 row waves read K and V once for 256 rows, but leave more of them
// empty: where the tiles of 128 come in pairs they win (512 rows, 8 x 16384,
// bf16 337 us against 358), where the last is odd they lose (320 rows, e4m3
// 325 against 299).  Heads of 256 have no registers for 8.  The rows are
// known to the host as max_nodes alone: a caller that allows many more nodes
// than it sends pays the difference above.
int row_waves(const KvView& c, int32_t max_nodes, int32_t group) {
  const int64_t rows = (int64_t)max_nodes * group;
  if (rows <= 64) return rows <= 32 ? 1 : 2;
  return c.head_dim < 256 && (rows + 127) / 128 % 2 == 0 ? 8 : 4;
}

template <int DT, int D, int RW>
struct Launch {
  using S = Shape<DT, D, RW>;
  static int grid() { return 256 * S::kPerCu; }
  static size_t bytes() { return (size_t)grid() * 2 * (sizeof(JoinItem) + S::kPartFloats * sizeof(float)); }
  static hipError_t run(const TreeArgs& a, hipStream_t s) {
    const FastDiv per_group = FastDiv::make(a.n_q_heads / a.c.n_kv_heads);
    tree_attention_kernel<DT, D, RW><<<grid(), S::kThreads, S::kLds, s>>>(a, per_group);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    tree_join_kernel<DT, D, RW><<<dim3(grid(), kJoinWgs), 256, 0, s>>>(a, per_group);
    return hipGetLastError();
  }
};

// Calls f with the Launch type for this cache and number of row waves.
template <int DT, int D, class F>
auto with_rows(int rw, const F& f) {
  if (rw == 1) return f(Launch<DT, D, 1>{});
  if (rw == 2) return f(Launch<DT, D, 2>{});
  if constexpr (D < 256) {
    if (rw == 8) return f(Launch<DT, D, 8>{});
  }
  return f(Launch<DT, D, 4>{});
}
template <int DT, class F>
auto with_dim(int dim, int rw, const F& f) {
  if (dim == 64) return with_rows<DT, 64>(rw, f);
  if (dim == 128) return with_rows<DT, 128>(rw, f);
  return with_rows<DT, 256>(rw, f);
}
template <class F>
auto with_shape(const KvView& c, int rw, const F& f) {
  if (c.dtype == DFLASH_BF16) return with_dim<DFLASH_BF16>(c.head_dim, rw, f);
  if (c.dtype == DFLASH_E4M3) return with_dim<DFLASH_E4M3>(c.head_dim, rw, f);
  return with_dim<DFLASH_I8>(c.head_dim, rw, f);
}

}  // namespace

// The most that any call with up to max_nodes nodes takes, so that a workspace
// for many nodes serves fewer.  (The forms alone do not grow with their rows:
// 64 and 128 are 33 KB apart, the smaller the larger.)  A form of rw row waves
// is for more than 16 rw rows.
size_t tree_attention_bytes(const KvView& c, int32_t n_req, int32_t max_nodes, int32_t n_q_heads) {
  const int64_t rows = (int64_t)max_nodes * (n_q_heads / c.n_kv_heads);
  size_t most = 0;
  for (int rw = 1; rw <= 8 && (rw == 1 || rows > 16 * rw); rw *= 2)
    most = std::max(most, with_shape(c, rw, [](auto l) { return decltype(l)::bytes(); }));
  return most;
}

hipError_t launch_tree_attention(const TreeArgs& a, hipStream_t stream) {
  return with_shape(a.c, row_waves(a.c, a.max_nodes, a.n_q_heads / a.c.n_kv_heads),
                    [&](auto l) { return decltype(l)::run(a, stream); });
}

}  // namespace dflash
