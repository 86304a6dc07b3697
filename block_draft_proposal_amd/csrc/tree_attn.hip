// Attention of drafted nodes over a paged cache.
//
// One request and kv head form M = nodes * group query rows over the same
// keys.  A workgroup takes MT = 32 RW of them and walks KT keys a step:
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
// W = RW KW waves: RW share the rows, KW the keys of a step (few rows leave
// waves to spare; they join their sums at the end).
//
// Work is split evenly whatever the lengths: the steps of all (request, kv
// head, row tile) items form one line that is cut into equal pieces, one for
// each workgroup.  A piece that covers an item writes its result; pieces of a
// cut item leave (m, l, O) in the workspace, at most two to a workgroup, and a
// second kernel joins them in a fixed order.
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
  static constexpr int kKeyWaves = kRowBytes == 512 ? (RW == 1 ? 2 : 1) : 4 / RW;
  static constexpr int kKeys = kRowBytes == 512 ? (RW == 1 ? 64 : 32)      // keys of a step
                               : RW == 1        ? 128
                               : RW == 2        ? (kRowBytes == 256 ? 64 : 128)
                                                : 64;
  static constexpr int kRows = 32 * RW;
  static constexpr int kWaves = RW * kKeyWaves, kThreads = 64 * kWaves;
  static constexpr int kSubs = kKeys / kKeyWaves / 32;                     // 32-key blocks of a wave in a step
  static constexpr int kChunks = kRowBytes / 16;
  static constexpr int kTile = kKeys * kRowBytes;                          // bytes of K (or V) in a step
  static constexpr int kLoads = kTile / 1024 / kWaves;                     // direct loads of K (or V) per thread
  static constexpr int kPages = 1024;                                      // page ids held in LDS
  static constexpr int kIdsAt = 4 * kTile;
  static constexpr int kScalesAt = kIdsAt + 4 * kPages;                    // [2 stages][K, V][kKeys] fp32
  static constexpr int kStatsAt = kScalesAt + (DT == DFLASH_BF16 ? 0 : 16 * kKeys);   // [kKeyWaves][kRows] m, l
  static constexpr int kLds = kStatsAt + 8 * kKeyWaves * kRows;
  static constexpr int kPerCu = kLds <= 80 * 1024 ? 2 : 1;                 // workgroups of a CU
  static constexpr int kPartOdd = kRows * (D + 2);                         // a partial: O [kRows][D], m and l of each
  static constexpr int kPartFloats = kPartOdd + 4;                         // row, whether odd values were left out
  static_assert(kSubs >= 1 && kLoads >= 1 && kTile % (1024 * kWaves) == 0, "a step splits over the waves");
  static_assert((kKeyWaves - 1) * kRows * D * 4 <= 4 * kTile, "the join fits where the stages were");
  static_assert(DT == DFLASH_BF16 || 2 * kKeys <= kThreads, "one scale per thread");
  static_assert(kLds <= 160 * 1024, "LDS of a CU");

  // Chunk c of stage row r lies in slot c ^ swizzle(r).  8 lanes of a 16-byte
  // read (8 consecutive rows, one chunk) and 16 lanes of a transposed read
  // (rows r .. r+3 and two chunks of 16-bit elements; r .. r+3, r+8 .. r+11
  // and one chunk of 8-bit ones) fall on different banks.
  __device__ static __forceinline__ int swizzle(int r) {
    if constexpr (DT == DFLASH_BF16) return kRowBytes == 128 ? ((r >> 1) & 3) << 1 : (r & 7) << 1;
    else return kRowBytes == 256 ? r & 15 : kRowBytes == 128 ? (r >> 1) & 7 : (r >> 2) & 3;
  }
};

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

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const unsigned char*)p;
}

// Transposed reads of V at LDS addresses a[i] + O0 and a[i] + O1: among 16
// lanes, lane i gets column i of the 16 x 16-bit by 4-row (8-bit: 8-row) block
// whose pieces of 8 bytes the lanes address.  One block of assembly with its
// own wait: the compiler takes the builtins to depend on every direct load in
// flight and would wait for the next step's.
template <bool WIDE, int O0, int O1>
__device__ __forceinline__ void read_transposed(const uint32_t (&a)[4], i32x2_t (&r)[4][2]) {
  if constexpr (WIDE)
    asm volatile(
        "ds_read_b64_tr_b16 %0, %8 offset:%12\n\tds_read_b64_tr_b16 %1, %8 offset:%13\n\t"
        "ds_read_b64_tr_b16 %2, %9 offset:%12\n\tds_read_b64_tr_b16 %3, %9 offset:%13\n\t"
        "ds_read_b64_tr_b16 %4, %10 offset:%12\n\tds_read_b64_tr_b16 %5, %10 offset:%13\n\t"
        "ds_read_b64_tr_b16 %6, %11 offset:%12\n\tds_read_b64_tr_b16 %7, %11 offset:%13\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(r[0][0]), "=&v"(r[0][1]), "=&v"(r[1][0]), "=&v"(r[1][1]), "=&v"(r[2][0]), "=&v"(r[2][1]),
          "=&v"(r[3][0]), "=&v"(r[3][1])
        : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "n"(O0), "n"(O1));
  else
    asm volatile(
        "ds_read_b64_tr_b8 %0, %8 offset:%12\n\tds_read_b64_tr_b8 %1, %8 offset:%13\n\t"
        "ds_read_b64_tr_b8 %2, %9 offset:%12\n\tds_read_b64_tr_b8 %3, %9 offset:%13\n\t"
        "ds_read_b64_tr_b8 %4, %10 offset:%12\n\tds_read_b64_tr_b8 %5, %10 offset:%13\n\t"
        "ds_read_b64_tr_b8 %6, %11 offset:%12\n\tds_read_b64_tr_b8 %7, %11 offset:%13\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(r[0][0]), "=&v"(r[0][1]), "=&v"(r[1][0]), "=&v"(r[1][1]), "=&v"(r[2][0]), "=&v"(r[2][1]),
          "=&v"(r[3][0]), "=&v"(r[3][1])
        : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "n"(O0), "n"(O1));
}
template <int O0, int O1>
__device__ __forceinline__ void read_transposed_8bit(const uint32_t (&a)[2], i32x2_t (&r)[2][2]) {
  asm volatile(
      "ds_read_b64_tr_b8 %0, %4 offset:%6\n\tds_read_b64_tr_b8 %1, %4 offset:%7\n\t"
      "ds_read_b64_tr_b8 %2, %5 offset:%6\n\tds_read_b64_tr_b8 %3, %5 offset:%7\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(r[0][0]), "=&v"(r[0][1]), "=&v"(r[1][0]), "=&v"(r[1][1])
      : "v"(a[0]), "v"(a[1]), "n"(O0), "n"(O1));
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

// A request's share of the line of steps.
struct Req {
  int32_t first;             // its first row
  int32_t n;                 // nodes
  int64_t start;             // prefix positions
  int64_t len;               // start + n
  int32_t steps;             // ceil(len / keys)
  int32_t tiles;             // row tiles
};
__device__ __forceinline__ Req request(const TreeArgs& a, int r, int keys, int rows, int group) {
  Req q;
  const int64_t first = a.c.offsets[r], end = min((int64_t)a.c.offsets[r + 1], a.c.n_rows);
  const int64_t n = first < 0 ? 0 : max((int64_t)0, min(end - first, (int64_t)a.max_nodes));
  q.first = (int32_t)first;
  q.n = (int32_t)n;
  q.start = max(a.c.start[r], 0);
  q.len = q.start + n;
  q.steps = n > 0 ? (int32_t)((q.len + keys - 1) / keys) : 0;
  q.tiles = (int32_t)((n * group + rows - 1) / rows);
  return q;
}

// The line of steps: its length, this workgroup's piece [u0, u1), and the
// request that holds u0 with the steps before it.
struct Piece {
  int64_t total, u0, u1, before;
  int32_t pieces, w, req;
  __device__ __forceinline__ int64_t begin(int64_t i) const { return total * i / pieces; }
  // the piece that step u lies in
  __device__ __forceinline__ int32_t of(int64_t u) const { return (int32_t)(((u + 1) * pieces - 1) / total); }
};

template <int THREADS>
__device__ __forceinline__ Piece find_piece(const TreeArgs& a, int keys, int rows, int group) {
  constexpr int kWaves = THREADS / 64;
  __shared__ int64_t sums[kWaves];
  __shared__ int64_t found[2];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n_req = a.c.n_req;
  auto steps_of = [&](int r) -> int64_t {
    if (r >= n_req) return 0;
    const Req q = request(a, r, keys, rows, group);
    return (int64_t)q.steps * q.tiles * a.c.n_kv_heads;
  };
  const int64_t mine = steps_of(tid);
  int64_t sum = mine;
  for (int r = tid + THREADS; r < n_req; r += THREADS) sum += steps_of(r);
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
  if (lane == 0) sums[wave] = sum;
  __syncthreads();
  Piece p;
  p.total = 0;
  for (int i = 0; i < kWaves; ++i) p.total += sums[i];
  __syncthreads();
  p.pieces = (int32_t)min((int64_t)gridDim.x, p.total);
  p.w = (int)blockIdx.x < p.pieces ? (int)xcd_contiguous(blockIdx.x, p.pieces) : p.pieces;
  p.u0 = p.u1 = 0;
  p.req = n_req;
  p.before = 0;
  if (p.w >= p.pieces) return p;                  // the whole workgroup: nothing to do
  p.u0 = p.begin(p.w);
  p.u1 = p.begin(p.w + 1);
  int64_t run = 0;
  for (int r0 = 0; r0 < n_req; r0 += THREADS) {
    int64_t x = r0 == 0 ? mine : steps_of(r0 + tid);
    const int64_t own = x;
    for (int o = 1; o < 64; o <<= 1) {
      const int64_t y = __shfl_up(x, o, 64);
      if (lane >= o) x += y;
    }
    if (lane == 63) sums[wave] = x;
    __syncthreads();
    int64_t ahead = run, all = 0;
    for (int i = 0; i < kWaves; ++i) {
      if (i < wave) ahead += sums[i];
      all += sums[i];
    }
    x += ahead;                                   // steps up to and with request r0 + tid
    if (x - own <= p.u0 && p.u0 < x) {
      found[0] = r0 + tid;
      found[1] = x - own;
    }
    run += all;
    __syncthreads();
    if (run > p.u0) break;
  }
  p.req = (int32_t)found[0];
  p.before = found[1];
  __syncthreads();
  return p;
}

// Whether a node sees anything: a prefix, or a bit of its mask.
__device__ __forceinline__ bool sees_any(const TreeArgs& a, const Req& q, int node) {
  if (q.start > 0 || !a.mask) return true;
  const uint64_t* m = a.mask + (int64_t)(q.first + node) * a.mask_words;
  uint64_t any = 0;
  for (int w = 0; w * 64 < q.n; ++w) {
    const int left = q.n - w * 64;
    any |= m[w] & (left >= 64 ? ~0ull : (1ull << left) - 1);
  }
  return any != 0;
}

// Adds to 4 elements of a row's result, at d, the values at the nodes it sees
// that are not finite (a sum with such a value is that value, and of both
// infinities NaN, whatever the weights).
template <int DT, int D>
__device__ __forceinline__ void add_odd(const TreeArgs& a, const Req& q, int req, int head, int node, int d,
                                                  float (&f)[4]) {
  constexpr int kSize = DT == DFLASH_BF16 ? 2 : 1;
#pragma unroll 1
  for (int j = 0; j < q.n; ++j) {
    if (a.mask ? !((a.mask[(int64_t)(q.first + node) * a.mask_words + (j >> 6)] >> (j & 63)) & 1) : j > node) continue;
    int64_t page;
    int32_t slot;
    if (!kv_locate(a.c, a.c.table + req * a.c.table_stride, q.start + j, page, slot)) continue;
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
  int32_t* ids = reinterpret_cast<int32_t*>(ta_smem + S::kIdsAt);
  float* scales = reinterpret_cast<float*>(ta_smem + S::kScalesAt);
  float* stats = reinterpret_cast<float*>(ta_smem + S::kStatsAt);
  const KvView& c = a.c;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rw = wave % RW, kw = wave / RW, half = lane >> 5, l32 = lane & 31;
  const int group = per_group.d;
  const Piece piece = find_piece<S::kThreads>(a, kKeys, S::kRows, group);
  if (piece.w >= piece.pieces) return;
  // log2(e) and the softmax scale; 8-bit caches carry it in K's scales
  const float c2 = a.scale * 1.44269504088896340736f, cs = DT == DFLASH_BF16 ? c2 : 1.f;

  // K reads: row l32 of a 32-key block, chunk 2t + half in slot (2t) ^ kx
  const int kx = half ^ S::swizzle(l32);
  // V reads: lane i of a 16-lane group addresses row vr of a 16-key block
  // (plus 8 for the second half of 16-bit ones) and 8 bytes of a 16-column block
  const int g16 = lane >> 4, i16 = lane & 15;
  const int vj = DT == DFLASH_BF16 ? i16 >> 2 : i16 >> 1;
  const int vr = DT == DFLASH_BF16 ? 4 * half + vj : 8 * (vj >> 2) + 4 * half + (vj & 3);
  const int vx = (DT == DFLASH_BF16 ? 2 * (g16 & 1) + ((i16 >> 1) & 1) : g16 & 1) ^ S::swizzle(vr);
  const int vbase = vr * kRB + (i16 & 1) * 8;

  int req = piece.req;
  int64_t req_begin = piece.before, u = piece.u0;
  while (u < piece.u1) {
    const Req q = request(a, req, kKeys, S::kRows, group);
    const int64_t req_units = (int64_t)q.steps * q.tiles * c.n_kv_heads;
    if (u >= req_begin + req_units) {              // also requests without nodes
      req_begin += req_units;
      ++req;
      continue;
    }
    const int32_t item = (int32_t)((u - req_begin) / q.steps), t0 = (int32_t)((u - req_begin) - (int64_t)item * q.steps);
    const int32_t t1 = (int32_t)min((int64_t)q.steps, t0 + (piece.u1 - u));
    const int head = item / q.tiles, tile = item - head * q.tiles;
    const int rows = min(S::kRows, q.n * group - tile * S::kRows);   // rows of this tile
    const bool whole = t0 == 0 && t1 == q.steps, first_item = u == piece.u0;
    const int row = rw * 32 + l32;                 // this lane's row of the tile, and its node and head
    const int flat = tile * S::kRows + min(row, rows - 1), node = per_group.div(flat), gh = flat - node * group;
    const int32_t* table = c.table + req * c.table_stride;

    // this row's query, in the order K's chunks have in the product
    bf16x8_t qf[kSteps16];
    {
      const uint16_t* qp = a.q + (int64_t)(q.first + node) * a.q_row + (int64_t)(head * group + gh) * a.q_head;
#pragma unroll
      for (int t = 0; t < kSteps16; ++t) {
        const int d = DT == DFLASH_BF16 ? 16 * t + 8 * half : 32 * (t / 2) + 16 * half + 8 * (t & 1);
        qf[t] = __builtin_bit_cast(bf16x8_t, ld16(qp + d));
      }
    }

    // page ids in LDS, a window of them at a time
    const int last_page = c.per_page.div((int)min(q.len - 1, (int64_t)0x7fffffff));
    int page0 = 0, page_end = 0;
    bool bad = q.len > 0x7fffffff;
    auto load_pages = [&](int from) {
      step_barrier();
      page0 = from;
      page_end = min(from + S::kPages, last_page + 1);
      for (int i = from + tid; i < page_end; i += S::kThreads) {
        int id = i < c.table_width ? table[i] : -1;
        if (id < 0 || id >= c.n_pages) {
          bad = true;
          id = 0;
        }
        ids[i - from] = id;
      }
      step_barrier();
    };
    // page id and row within its head's rows of position pos (at most the
    // last held one: later rows of a step repeat it and are masked)
    auto locate = [&](int64_t pos, int32_t& id, int32_t& r) {
      const int p = (int)min(pos, min(q.len - 1, (int64_t)0x7fffffff)), idx = c.per_page.div(p);
      id = ids[idx - page0];
      r = head * c.page_size + (p - idx * c.page_size);
    };
    uint32_t scale_next = 0;                       // this thread's scale byte of the step issued last
    auto issue = [&](int t) {
      const int64_t p0 = (int64_t)t * kKeys;
      const int need = c.per_page.div((int)min(min(p0 + kKeys, q.len) - 1, (int64_t)0x7fffffff));
      if (need >= page_end) load_pages(c.per_page.div((int)min(p0, (int64_t)0x7fffffff)));
      unsigned char* stage = ta_smem + (t & 1) * 2 * S::kTile;
      if constexpr (DT != DFLASH_BF16) {
        if (tid < 2 * kKeys) {
          int32_t id, r;
          locate(p0 + tid % kKeys, id, r);
          scale_next = (tid < kKeys ? c.k_scale : c.v_scale)[id * c.scale_page_bytes + r];
        }
      }
#pragma unroll
      for (int i = 0; i < S::kLoads; ++i) {
        const int blk = i * S::kWaves + wave, r = blk * (1024 / kRB) + lane / S::kChunks;
        int32_t id, at;
        locate(p0 + r, id, at);
        const int64_t off = id * c.page_bytes + (int64_t)at * kRB + (((lane % S::kChunks) ^ S::swizzle(r)) << 4);
        __builtin_amdgcn_global_load_lds((const void*)(c.k + off), (lds_void_t*)(stage + blk * 1024), 16, 0, 0);
        __builtin_amdgcn_global_load_lds((const void*)(c.v + off), (lds_void_t*)(stage + S::kTile + blk * 1024), 16, 0, 0);
      }
    };

    bool odd = false;                              // a node's value was not finite
    f32x16_t o[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[b][i] = 0.f;
    float m = -INFINITY, l = 0.f;                  // of this lane's row; l over this lane's keys only

    step_barrier();                                // the LDS is free of the previous item
    issue(t0);
    // the queries have arrived before the loop: no wait in it may be for them
#pragma unroll
    for (int i = 0; i < kSteps16; ++i) {
      u32x4 w = __builtin_bit_cast(u32x4, qf[i]);
      asm volatile("" : "+v"(w));
      qf[i] = __builtin_bit_cast(bf16x8_t, w);
    }
    uint32_t scale_now = scale_next;
    if (t0 + 1 < t1) issue(t0 + 1);
    for (int t = t0; t < t1; ++t) {
      if (t + 1 < t1) wait_vm<2 * S::kLoads>();
      else wait_vm<0>();
      if constexpr (DT != DFLASH_BF16) {
        if (tid < 2 * kKeys)
          scales[(t & 1) * 2 * kKeys + tid] = tid < kKeys ? kv_scale_value(scale_now) * c2 : kv_scale_value(scale_now);
      }
      step_barrier();
      const unsigned char* ks = ta_smem + (t & 1) * 2 * S::kTile;
      const unsigned char* vs = ks + S::kTile;
      const int64_t p0 = (int64_t)t * kKeys;
      const bool masked = p0 + kKeys > q.start;     // the step reaches the tree (or the end)
      if constexpr (DT != DFLASH_I8) {
        if (masked) {
          // A weight of zero times an infinity is no zero: a node's value that
          // is not finite must not reach the rows that do not see it.  Such
          // elements become zeros here and are added at the end, where seen.
          unsigned char* vw = ta_smem + (t & 1) * 2 * S::kTile + S::kTile;
          for (int x = tid; x < S::kTile / 16; x += S::kThreads) {
            if (p0 + x / S::kChunks < q.start) continue;
            u32x4 w = ld16(vw + x * 16);
            if (odd_values<DT>(w)) {
              odd = true;
              st16(vw + x * 16, w);
            }
          }
          step_barrier();
        }
      }
#pragma unroll
      for (int sub = 0; sub < S::kSubs; ++sub) {
        const int kb = (kw * S::kSubs + sub) * 32;  // first key of the block within the step
        f32x16_t s;
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = 0.f;
        const unsigned char* krow = ks + (kb + l32) * kRB;
        if constexpr (DT == DFLASH_BF16) {
#pragma unroll
          for (int t16 = 0; t16 < kSteps16; ++t16) {
            const bf16x8_t kf = __builtin_bit_cast(bf16x8_t, ld16(krow + (((2 * t16) ^ kx) << 4)));
            s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[t16], s, 0, 0, 0);
          }
        } else {
#pragma unroll
          for (int t32 = 0; t32 < kSteps16 / 2; ++t32) {
            const u32x4 w = ld16(krow + (((2 * t32) ^ kx) << 4));
            s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(codes_to_bf16<DT>(w[0], w[1]), qf[2 * t32], s, 0, 0, 0);
            s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(codes_to_bf16<DT>(w[2], w[3]), qf[2 * t32 + 1], s, 0, 0, 0);
          }
          const float* kscale = scales + (t & 1) * 2 * kKeys + kb + 4 * half;
#pragma unroll
          for (int i = 0; i < 16; ++i) s[i] *= kscale[8 * (i >> 2) + (i & 3)];
        }
        // s[i]: key 8 (i / 4) + 4 half + i % 4 of the block
        uint32_t vis = ~0u;
        if (masked) {
          const int64_t k0 = p0 + kb;
          const int pre = (int)min(max(q.start - k0, (int64_t)0), (int64_t)32);
          const int64_t rel = k0 - q.start;         // the node of key 0 of the block
          uint32_t bits = 0;
          int64_t seen = q.n;
          if (!a.mask) {
            seen = min(seen, (int64_t)node + 1);
            bits = ~0u;
          } else if (rel < q.n && pre < 32) {
            const uint64_t* mw = a.mask + (int64_t)(q.first + node) * a.mask_words;
            if (rel < 0) {
              bits = (uint32_t)(mw[0] << -rel);
            } else {
              const int w = (int)(rel >> 6), sh = (int)(rel & 63);
              uint64_t x = mw[w] >> sh;
              if (sh > 32 && w + 1 < a.mask_words) x |= mw[w + 1] << (64 - sh);
              bits = (uint32_t)x;
            }
          }
          bits &= low_bits((int)min(max(seen - rel, (int64_t)0), (int64_t)32));
          vis = low_bits(pre) | (bits & ~low_bits(pre));
          vis >>= 4 * half;                         // now bit 8 (i / 4) + i % 4 for s[i]
#pragma unroll
          for (int i = 0; i < 16; ++i) s[i] = (vis >> (8 * (i >> 2) + (i & 3))) & 1 ? s[i] : -INFINITY;
        }
        float top = s[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i]);
        top = half_max(top);
        // The sums keep the maximum they were built with until a row's passes
        // it by 2^8: weights up to 256 are as exact as those up to 1, and most
        // blocks then leave O alone.
        if (__any((top - m) * cs > 8.f)) {
          const float next = fmaxf(m, top), keep = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((m - next) * cs);
          m = next;
          l *= keep;
#pragma unroll
          for (int b = 0; b < kBlocks; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[b][i] *= keep;
        }
        const float base = m == -INFINITY ? 0.f : m * cs;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[i] = __builtin_amdgcn_exp2f(DT == DFLASH_BF16 ? fmaf(s[i], cs, -base) : s[i] - base);
          sum += s[i];
        }
        l += sum;
        if constexpr (DT != DFLASH_BF16) {
          const float* vscale = scales + (t & 1) * 2 * kKeys + kKeys + kb + 4 * half;
#pragma unroll
          for (int i = 0; i < 16; ++i) s[i] *= vscale[8 * (i >> 2) + (i & 3)];
          if (masked) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = (vis >> (8 * (i >> 2) + (i & 3))) & 1 ? s[i] : 0.f;
          }
        }
        const unsigned char* vblk = vs + kb * kRB;
        // weights rounded to bf16 (half a step, 2^-8 of each): the product with
        // V is bf16 x bf16 on the matrix cores; l sums them unrounded
        bf16x8_t pf[2];
#pragma unroll
        for (int u16 = 0; u16 < 2; ++u16) {
          const u32x4 pw = {pack_bf16(s[8 * u16], s[8 * u16 + 1]), pack_bf16(s[8 * u16 + 2], s[8 * u16 + 3]),
                            pack_bf16(s[8 * u16 + 4], s[8 * u16 + 5]), pack_bf16(s[8 * u16 + 6], s[8 * u16 + 7])};
          pf[u16] = __builtin_bit_cast(bf16x8_t, pw);
        }
        const uint32_t v0 = lds_address(vblk) + vbase;
        auto v_at = [&](int b) { return v0 + (uint32_t)(((kPerBlock * b) ^ vx) << 4); };   // column block b, first keys
        auto add = [&](int b, int u16, bf16x8_t vf) {
          o[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, pf[u16], o[b], 0, 0, 0);
        };
        auto join16 = [](const i32x2_t (&r)[2]) {
          return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(r[0], r[1], 0, 1, 2, 3));
        };
        auto codes = [](i32x2_t r) { return codes_to_bf16<DT>((uint32_t)r[0], (uint32_t)r[1]); };
        i32x2_t r[4][2];
        if constexpr (DT == DFLASH_BF16 && D == 64) {
          const uint32_t at[4] = {v_at(0), v_at(1), v_at(0) + 16 * kRB, v_at(1) + 16 * kRB};
          read_transposed<true, 0, 8 * kRB>(at, r);
#pragma unroll
          for (int i = 0; i < 4; ++i) add(i & 1, i >> 1, join16(r[i]));
        } else if constexpr (DT == DFLASH_BF16) {
#pragma unroll
          for (int b = 0; b < kBlocks; b += 4) {
            const uint32_t at[4] = {v_at(b), v_at(b + 1), v_at(b + 2), v_at(b + 3)};
            read_transposed<true, 0, 8 * kRB>(at, r);
#pragma unroll
            for (int i = 0; i < 4; ++i) add(b + i, 0, join16(r[i]));
            read_transposed<true, 16 * kRB, 24 * kRB>(at, r);
#pragma unroll
            for (int i = 0; i < 4; ++i) add(b + i, 1, join16(r[i]));
          }
        } else if constexpr (D == 64) {
          const uint32_t at[2] = {v_at(0), v_at(1)};
          i32x2_t r2[2][2];
          read_transposed_8bit<0, 16 * kRB>(at, r2);
#pragma unroll
          for (int i = 0; i < 4; ++i) add(i >> 1, i & 1, codes(r2[i >> 1][i & 1]));
        } else {
#pragma unroll
          for (int b = 0; b < kBlocks; b += 4) {
            const uint32_t at[4] = {v_at(b), v_at(b + 1), v_at(b + 2), v_at(b + 3)};
            read_transposed<false, 0, 16 * kRB>(at, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) add(b + (i >> 1), i & 1, codes(r[i >> 1][i & 1]));
          }
        }
      }
      step_barrier();                              // every wave is done with this stage
      scale_now = scale_next;
      if (t + 2 < t1) issue(t + 2);
    }

    // join the key waves: O of all but the first through LDS
    l = half_sum(l);
    float mc = m == -INFINITY ? -INFINITY : m * cs;
    if constexpr (S::kKeyWaves > 1) {
      float2* st = reinterpret_cast<float2*>(stats);
      if (half == 0) st[kw * S::kRows + row] = make_float2(mc, l);
      step_barrier();
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < S::kKeyWaves; ++i) top = fmaxf(top, st[i * S::kRows + row].x);
      const float keep = mc == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mc - top);
      l = 0.f;
#pragma unroll
      for (int i = 0; i < S::kKeyWaves; ++i) {
        const float2 x = st[i * S::kRows + row];
        l += x.x == -INFINITY ? x.y : x.y * __builtin_amdgcn_exp2f(x.x - top);
      }
      mc = top;
      float4* pool = reinterpret_cast<float4*>(ta_smem) + rw * (D / 8) * 64 + lane;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[b][i] *= keep;
      if (kw > 0) {
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            pool[((kw - 1) * RW * (D / 8) + 4 * b + i) * 64] =
                make_float4(o[b][4 * i], o[b][4 * i + 1], o[b][4 * i + 2], o[b][4 * i + 3]);
      }
      step_barrier();
      if (kw == 0) {
#pragma unroll
        for (int x = 0; x < S::kKeyWaves - 1; ++x)
#pragma unroll
          for (int b = 0; b < kBlocks; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 f = pool[(x * RW * (D / 8) + 4 * b + i) * 64];
              o[b][4 * i] += f.x;
              o[b][4 * i + 1] += f.y;
              o[b][4 * i + 2] += f.z;
              o[b][4 * i + 3] += f.w;
            }
      }
    }
    if (__syncthreads_or(bad)) l = __builtin_nanf("");
    const bool any_odd = DT != DFLASH_I8 && __syncthreads_or(odd);
    if (kw == 0 && row < rows) {
      if (whole) {
        const float inv = sees_any(a, q, node) ? 1.f / l : 0.f;
        uint16_t* op = a.out + ((int64_t)(q.first + node) * a.n_q_heads + head * group + gh) * D;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint2*>(op + 32 * b + 8 * i + 4 * half) =
                make_uint2(pack_bf16(o[b][4 * i] * inv, o[b][4 * i + 1] * inv),
                           pack_bf16(o[b][4 * i + 2] * inv, o[b][4 * i + 3] * inv));
        if (any_odd) {
#pragma unroll 1
          for (int x = 0; x < D / 8; ++x) {         // this lane's own 4 elements of each 8
            uint2* at = reinterpret_cast<uint2*>(op + 8 * x + 4 * half);
            const uint2 w = *at;
            float f[4] = {bf16_to_f32(w.x & 0xffffu), bf16_to_f32(w.x >> 16), bf16_to_f32(w.y & 0xffffu), bf16_to_f32(w.y >> 16)};
            add_odd<DT, D>(a, q, req, head, node, 8 * x + 4 * half, f);
            *at = make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
          }
        }
      } else {
        float* part = static_cast<float*>(a.workspace) + ((int64_t)piece.w * 2 + (first_item ? 0 : 1)) * S::kPartFloats;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float4*>(part + row * D + 32 * b + 8 * i + 4 * half) =
                make_float4(o[b][4 * i], o[b][4 * i + 1], o[b][4 * i + 2], o[b][4 * i + 3]);
        if (half == 0) *reinterpret_cast<float2*>(part + S::kRows * D + 2 * row) = make_float2(mc, l);
        if (tid == 0) part[S::kPartOdd] = any_odd ? 1.f : 0.f;
      }
    }
    u += t1 - t0;
  }
}

// Joins the pieces of cut items.  The workgroups of an item's pieces share its
// rows; the pieces are summed in the order of the line, so the result does not
// depend on which finished first.
template <int DT, int D, int RW>
__global__ void __launch_bounds__(256) tree_join_kernel(TreeArgs a, FastDiv per_group) {
  using S = Shape<DT, D, RW>;
  const Piece piece = find_piece<256>(a, S::kKeys, S::kRows, per_group.d);
  if (piece.w >= piece.pieces) return;
  const KvView& c = a.c;
  const int group = per_group.d;
  int req = piece.req;
  int64_t req_begin = piece.before, u = piece.u0;
  while (u < piece.u1) {
    const Req q = request(a, req, S::kKeys, S::kRows, group);
    const int64_t req_units = (int64_t)q.steps * q.tiles * c.n_kv_heads;
    if (u >= req_begin + req_units) {
      req_begin += req_units;
      ++req;
      continue;
    }
    const int32_t item = (int32_t)((u - req_begin) / q.steps);
    const int64_t i0 = req_begin + (int64_t)item * q.steps, i1 = i0 + q.steps;
    u = i1;
    if (i0 >= piece.u0 && i1 <= piece.u1) {        // whole: on to the piece's last item
      const int64_t skip = (min(piece.u1, req_begin + req_units) - i1) / q.steps;
      u += skip * q.steps;
      continue;
    }
    const int first = piece.of(i0), last = piece.of(i1 - 1), n = last - first + 1;
    const int head = item / q.tiles, tile = item - head * q.tiles;
    const int rows = min(S::kRows, q.n * group - tile * S::kRows);
    const float* parts = static_cast<const float*>(a.workspace);
    const bool first_starts = piece.begin(first) == i0;
    auto part = [&](int x) {
      const int slot = x == 0 && !first_starts ? 1 : 0;
      return parts + ((int64_t)(first + x) * 2 + slot) * S::kPartFloats;
    };
    for (int e = (piece.w - first) * 256 + (int)threadIdx.x; e < rows * (D / 4); e += n * 256) {
      const int row = e / (D / 4), d = (e % (D / 4)) * 4;
      float top = -INFINITY;
      for (int x = 0; x < n; ++x) top = fmaxf(top, part(x)[S::kRows * D + 2 * row]);
      float l = 0.f, o0 = 0.f, o1 = 0.f, o2 = 0.f, o3 = 0.f;
      for (int x = 0; x < n; ++x) {
        const float* p = part(x);
        const float2 ml = *reinterpret_cast<const float2*>(p + S::kRows * D + 2 * row);
        const float4 f = *reinterpret_cast<const float4*>(p + row * D + d);
        const float w = ml.x == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ml.x - top);
        l += ml.x == -INFINITY ? ml.y : ml.y * w;   // a part that saw nothing has l = 0, or NaN for a bad page
        o0 = fmaf(f.x, w, o0);
        o1 = fmaf(f.y, w, o1);
        o2 = fmaf(f.z, w, o2);
        o3 = fmaf(f.w, w, o3);
      }
      const int flat = tile * S::kRows + row, node = per_group.div(flat), gh = flat - node * group;
      const float inv = sees_any(a, q, node) ? 1.f / l : 0.f;
      float f[4] = {o0 * inv, o1 * inv, o2 * inv, o3 * inv};
      if constexpr (DT != DFLASH_I8) {
        bool odd = false;
        for (int x = 0; x < n; ++x) odd = odd || part(x)[S::kPartOdd] != 0.f;
        if (odd) add_odd<DT, D>(a, q, req, head, node, d, f);
      }
      *reinterpret_cast<uint2*>(a.out + ((int64_t)(q.first + node) * a.n_q_heads + head * group + gh) * D + d) =
          make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
    }
  }
}

// Row waves: 32 rows a wave up to 128 rows a workgroup.
int row_waves(int32_t max_nodes, int32_t group) {
  const int64_t rows = (int64_t)max_nodes * group;
  return rows <= 32 ? 1 : rows <= 64 ? 2 : 4;
}

template <int DT, int D, int RW>
struct Launch {
  using S = Shape<DT, D, RW>;
  static int grid() { return 256 * S::kPerCu; }
  static size_t bytes() { return (size_t)grid() * 2 * S::kPartFloats * sizeof(float); }
  static hipError_t run(const TreeArgs& a, hipStream_t s) {
    const FastDiv per_group = FastDiv::make(a.n_q_heads / a.c.n_kv_heads);
    tree_attention_kernel<DT, D, RW><<<grid(), S::kThreads, S::kLds, s>>>(a, per_group);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    tree_join_kernel<DT, D, RW><<<grid(), 256, 0, s>>>(a, per_group);
    return hipGetLastError();
  }
};

// Calls f with the Launch type for this cache and number of row waves.
template <int DT, int D, class F>
auto with_rows(int rw, const F& f) {
  if (rw == 1) return f(Launch<DT, D, 1>{});
  if (rw == 2) return f(Launch<DT, D, 2>{});
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

size_t tree_attention_bytes(const KvView& c, int32_t n_req, int32_t max_nodes, int32_t n_q_heads) {
  return with_shape(c, row_waves(max_nodes, n_q_heads / c.n_kv_heads), [](auto l) { return decltype(l)::bytes(); });
}

hipError_t launch_tree_attention(const TreeArgs& a, hipStream_t stream) {
  return with_shape(a.c, row_waves(a.max_nodes, a.n_q_heads / a.c.n_kv_heads),
                    [&](auto l) { return decltype(l)::run(a, stream); });
}

}  // namespace dflash
