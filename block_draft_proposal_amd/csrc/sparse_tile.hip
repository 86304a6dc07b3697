// Attention over chosen pages for the rows of a request together.
//
// Drafted nodes of one request choose much the same pages: read row by row, the
// same keys come through the caches again and again.  Here up to 64 (node, query
// head) rows of a request and kv head are one tile, which walks the union of its
// nodes' pages once, each page with a bit for every node that chose it.
//
// A first kernel makes the union: for each tile and kv head a word of bits per
// block in LDS, then the blocks with a bit in order, as (page, bits), into the
// workspace.  The main kernel is that of single rows (see there for the layout of
// products, stages and waits) with up to four tiles of 16 rows to a step, and a
// word of bits beside each key: a lane's column is one (node, head), and keys
// without its node's bit have score -inf there.
//
// The rows of a tile share V's operand, and 0 times an infinity or a NaN that
// another row sees would be no zero.  Such values are rare enough that nothing
// looks for them: a row whose result is not finite is computed again by itself,
// over its own keys alone.
//
// Measured: 32 requests of 16 drafted rows, 128 pages of 16 a row, 8 kv heads of
// 128, 4 query heads each, bf16: 113 us and 7 for the unions, which name 490 MB of
// keys and values (463 fetched, 4.1 TB/s); row by row 460 us.
#include "sparse_core.h"

namespace dflash {
namespace {

constexpr int kThreads = 256, kUnionThreads = 512;
constexpr int kMaxBlocks = 16384;                 // of a table's row: a word each in LDS
constexpr int kMaxTileNodes = 32;                 // bits of a word
constexpr int kMaxTileParts = 512;
constexpr size_t kMaxLists = (size_t)1 << 30;     // bytes

// (node, head) rows that a tile may have: heads of 256 have no registers for more.
int max_rows(int head_dim) { return head_dim == 256 ? 32 : 64; }

constexpr size_t up256(size_t n) { return (n + 255) / 256 * 256; }
// A split tile's sums: O [16 GT][D], (m, l) of each row, the nodes that saw
// anything, those that saw a position without a page.
__host__ __device__ inline int64_t part_floats(int row_tiles, int d) { return (int64_t)16 * row_tiles * (d + 2) + 4; }

struct Lists {
  uint2* entries;                                 // tile of nt rows from row0 on, head h: nt * n_take at (row0 * heads + h * nt) * n_take
  int32_t* counts;                                // [row0 * heads + h]
  float* parts;
  size_t bytes;
  Lists(void* base, int64_t n_rows, int32_t heads, int32_t n_take, int32_t head_dim) {
    unsigned char* p = static_cast<unsigned char*>(base);
    const size_t items = (size_t)n_rows * heads;
    const size_t entry_bytes = up256(std::min(items * n_take * sizeof(uint2), kMaxLists)), count_bytes = up256(items * 4);
    entries = reinterpret_cast<uint2*>(p);
    counts = reinterpret_cast<int32_t*>(p + entry_bytes);
    parts = reinterpret_cast<float*>(p + entry_bytes + count_bytes);
    bytes = entry_bytes + count_bytes + up256((size_t)kMaxTileParts * part_floats(max_rows(head_dim) / 16, head_dim) * sizeof(float));
  }
};

// Rows row0 .. row0 + nt - 1: nodes n0 .. of request req, which has n.
struct Tile {
  int64_t row0;
  int req, n0, nt, n;
  int32_t start, full;                            // positions of the prefix, full pages
  bool over;                                      // start + n is beyond the table
};
// false for a tile without rows
__device__ __forceinline__ bool tile_at(const SparseArgs& a, int tile, int nodes, int per_req, Tile& t) {
  const KvView& c = a.c;
  t.req = tile / per_req;
  t.n0 = (tile - t.req * per_req) * nodes;
  const int64_t first = c.offsets[t.req], end = c.offsets[t.req + 1];
  t.start = max(c.start[t.req], 0);               // with the offsets, not behind them
  t.n = (int)max((int64_t)0, min(min(end, c.n_rows) - first, (int64_t)a.max_nodes));
  t.nt = min(nodes, t.n - t.n0);
  if (first < 0 || t.nt <= 0) return false;
  t.row0 = first + t.n0;
  t.full = kv_blocks(c, t.start);
  t.over = (int64_t)t.start + t.n > min((int64_t)kMaxLen, (int64_t)c.table_width * c.page_size);
  return true;
}

__global__ void __launch_bounds__(kUnionThreads) sparse_union_kernel(SparseArgs a, Lists lists, int nodes, int per_req) {
  extern __shared__ uint32_t bits[];              // [full]
  __shared__ uint32_t sums[kUnionThreads / 64];
  const KvView& c = a.c;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int head = blockIdx.x % c.n_kv_heads;
  Tile t;
  if (!tile_at(a, blockIdx.x / c.n_kv_heads, nodes, per_req, t)) return;
  for (int b = tid; b < t.full; b += kUnionThreads) bits[b] = 0;
  __syncthreads();
  if (!t.over) {
    for (int node = wave; node < t.nt; node += kUnionThreads / 64) {
      const int32_t* chosen = a.blocks + ((t.row0 + node) * c.n_kv_heads + head) * a.n_take;
#pragma unroll 4
      for (int e = lane; e < a.n_take; e += 64) {
        const int32_t b = chosen[e], before = e > 0 ? chosen[e - 1] : -1;
        if (b >= 0 && b < t.full && b > before) atomicOr(&bits[b], 1u << node);
      }
    }
  }
  __syncthreads();
  // the blocks with a bit, in order: a thread takes neighbours
  const int each = (t.full + kUnionThreads - 1) / kUnionThreads, lo = min(tid * each, t.full), hi = min(lo + each, t.full);
  uint32_t n = 0;
  for (int b = lo; b < hi; ++b) n += bits[b] != 0;
  uint32_t scan = n;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t y = (uint32_t)__shfl_up((int)scan, o, 64);
    if (lane >= o) scan += y;
  }
  if (lane == 63) sums[wave] = scan;
  __syncthreads();
  uint32_t at = scan - n, total = 0;
#pragma unroll
  for (int i = 0; i < kUnionThreads / 64; ++i) {
    if (i < wave) at += sums[i];
    total += sums[i];
  }
  uint2* out = lists.entries + (t.row0 * c.n_kv_heads + (int64_t)head * t.nt) * a.n_take;
  const int32_t* table = c.table + t.req * c.table_stride;
  for (int b = lo; b < hi; ++b)
    if (bits[b]) out[at++] = make_uint2((uint32_t)table[b], bits[b]);
  if (tid == 0) lists.counts[t.row0 * c.n_kv_heads + head] = (int32_t)total;
}

// One row and query head by itself, over the keys that it sees: a wave, a key a
// lane for the scores and a few channels a lane for the values.
template <int DT, int D>
__device__ __forceinline__ void alone(const SparseArgs& a, const Tile& t, int node, int head, int q_head) {
  constexpr int kSize = DT == DFLASH_BF16 ? 2 : 1, kOwn = D / 64;
  const KvView& c = a.c;
  const int lane = threadIdx.x & 63;
  const int64_t row = t.row0 + node;
  const int32_t* table = c.table + t.req * c.table_stride;
  const int32_t* chosen = a.blocks + (row * c.n_kv_heads + head) * a.n_take;
  const uint64_t* mask = a.mask ? a.mask + row * a.mask_words : nullptr;
  const uint16_t* q = a.q + row * a.q_row + (int64_t)q_head * a.q_head;
  const int32_t chosen_keys = a.n_take * c.page_size, tail = t.start - t.full * c.page_size;
  const int64_t keys = (int64_t)chosen_keys + tail + t.n;
  float m = -INFINITY, l = 0.f, o[kOwn];
#pragma unroll
  for (int i = 0; i < kOwn; ++i) o[i] = 0.f;
  auto value = [&](const unsigned char* p, int d, float scale) -> float {
    if constexpr (DT == DFLASH_BF16) return bf16_to_f32(reinterpret_cast<const uint16_t*>(p)[d]);
    else if constexpr (DT == DFLASH_E4M3) return __builtin_amdgcn_cvt_f32_fp8((int)p[d], 0) * scale;
    else return (float)reinterpret_cast<const int8_t*>(p)[d] * scale;
  };
  for (int64_t x0 = 0; x0 < keys; x0 += 64) {
    const int64_t x = x0 + lane;
    bool see = x < keys;
    int32_t pos = 0;
    if (see && x < chosen_keys) {
      const int e = c.per_page.div((int32_t)x);
      const int32_t b = chosen[e], before = e > 0 ? chosen[e - 1] : -1;
      see = b >= 0 && b < t.full && b > before;
      if (see) pos = b * c.page_size + ((int32_t)x - e * c.page_size);
    } else if (see) {
      const int32_t y = (int32_t)(x - chosen_keys), j = y - tail;
      pos = t.full * c.page_size + y;
      if (j >= 0) see = mask ? (mask[j >> 6] >> (j & 63)) & 1 : j <= t.n0 + node;
    }
    if (!__any(see)) continue;
    int64_t page = 0;
    int32_t slot = 0;
    see = see && kv_locate(c, table, pos, page, slot);   // a row that sees a position without a page is NaN before it comes here
    const int64_t at = page * c.page_bytes + ((int64_t)head * c.page_size + slot) * D * kSize;
    const int64_t scale_at = page * c.scale_page_bytes + (int64_t)head * c.page_size + slot;
    float s = -INFINITY, v_scale = 1.f;
    if (see) {
      const float k_scale = DT == DFLASH_BF16 ? 1.f : kv_scale_value(c.k_scale[scale_at]);
      if (DT != DFLASH_BF16) v_scale = kv_scale_value(c.v_scale[scale_at]);
      s = 0.f;
      for (int d = 0; d < D; ++d) s += bf16_to_f32(q[d]) * value(c.k + at, d, k_scale);
      s *= a.scale * 1.44269504088896340736f;
    }
    const float next = fmaxf(m, wave_max_f32(s));
    const float keep = m == -INFINITY ? 0.f : exp2f(m - next);
    float p = see ? exp2f(s - (next == -INFINITY ? 0.f : next)) : 0.f;
    m = next;
    float sum = p;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
    l = l * keep + sum;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) o[i] *= keep;
    for (uint64_t left = __ballot(see); left; left &= left - 1) {
      const int j = __builtin_ctzll(left);
      const float w = __shfl(p, j, 64), scale = __shfl(v_scale, j, 64);
      const unsigned char* v = c.v + __shfl(at, j, 64);
#pragma unroll
      for (int i = 0; i < kOwn; ++i) o[i] += w * value(v, lane * kOwn + i, scale);
    }
  }
  uint16_t* out = a.out + (row * a.n_q_heads + q_head) * D + lane * kOwn;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) out[i] = (uint16_t)f32_to_bf16_rne(o[i] / l);
}

template <int DT, int D, int GT>
__global__ void __launch_bounds__((SparseShape<DT, D>::kThreads), (GT * D <= 128 ? 2 : 1))
    sparse_tile_kernel(SparseArgs a, Lists lists, FastDiv per_group, int nodes, int per_req, int splits) {
  using S = SparseShape<DT, D>;
  constexpr int kRB = S::kRB, kOps = D / 32, kBlocks = D / 16;
  extern __shared__ __align__(16) unsigned char st_smem[];
  __shared__ uint32_t node_sets[2];                // nodes that see anything; that see a position without a page
  __shared__ uint64_t odd_rows;
  const KvView& c = a.c;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = blockDim.x >> 6;
  const int l16 = lane & 15, g16 = lane >> 4, l32 = lane & 31, group = per_group.d;
  // tiles of one kv head are neighbours on one XCD
  const uint32_t w = xcd_contiguous(blockIdx.x, gridDim.x);
  const uint32_t tiles = (uint32_t)c.n_req * (uint32_t)per_req;
  const int split = (int)(w % (uint32_t)splits), head = (int)(w / (uint32_t)splits / tiles);
  Tile t;
  if (!tile_at(a, (int)(w / (uint32_t)splits % tiles), nodes, per_req, t)) return;   // the whole workgroup
  const int rows = t.nt * group;                   // of this tile: node 0's heads, node 1's ...
  const int32_t* table = c.table + t.req * c.table_stride;
  const uint2* entries = lists.entries + (t.row0 * c.n_kv_heads + (int64_t)head * t.nt) * a.n_take;
  const uint32_t* mask = a.mask ? reinterpret_cast<const uint32_t*>(a.mask + t.row0 * a.mask_words) : nullptr;
  const uint32_t all_nodes = t.nt == 32 ? ~0u : (1u << t.nt) - 1u;

  // the line: the union's pages, the tail, the nodes
  const int32_t chosen_keys = t.over ? 0 : lists.counts[t.row0 * c.n_kv_heads + head] * c.page_size;
  const int32_t tail = t.start - t.full * c.page_size, rest = t.over ? 0 : tail + (mask ? t.n : t.n0 + t.nt);
  const int64_t steps = ((int64_t)chosen_keys + rest + 31) / 32, slots = (int64_t)splits * waves, me = split * waves + wave;
  const int t0 = __builtin_amdgcn_readfirstlane((int)(steps * me / slots)), t1 = __builtin_amdgcn_readfirstlane((int)(steps * (me + 1) / slots));

  unsigned char* stages = st_smem + wave * S::kWaveStages;
  unsigned char* ring = st_smem + waves * S::kWaveStages + wave * S::kRing;
  int64_t* row_at = reinterpret_cast<int64_t*>(ring + S::kRowsAt);
  float* scales = reinterpret_cast<float*>(ring + S::kScalesAt);
  uint32_t* masks = reinterpret_cast<uint32_t*>(ring + S::kMasksAt);
  const float c2 = a.scale * 1.44269504088896340736f, cs = DT == DFLASH_BF16 ? c2 : 1.f;
  if (tid == 0) {
    node_sets[0] = node_sets[1] = 0;
    odd_rows = 0;
  }

  // queries; rows past the tile's repeat its last
  bf16x8_t qf[GT][kOps];
  int node[GT];                                    // of this lane's column
#pragma unroll
  for (int u = 0; u < GT; ++u) {
    const int f = min(16 * u + l16, rows - 1);
    node[u] = per_group.div(f);
    const uint16_t* qp = a.q + (t.row0 + node[u]) * a.q_row + ((int64_t)head * group + (f - node[u] * group)) * a.q_head;
#pragma unroll
    for (int o = 0; o < kOps; ++o) {
      const int d = DT == DFLASH_BF16 ? 32 * o + 8 * g16 : 64 * (o / 2) + 16 * g16 + 8 * (o & 1);
      qf[u][o] = __builtin_bit_cast(bf16x8_t, ld16(qp + d));
    }
  }

  f32x4_t o[GT][kBlocks];
  float m[GT], l[GT];                              // l over this lane's keys only
#pragma unroll
  for (int u = 0; u < GT; ++u) {
    m[u] = -INFINITY;
    l[u] = 0.f;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) o[u][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
  uint32_t seen = 0, bad = 0;                      // over this lane's keys
  if (t.over) {
    for (int i = 0; i < t.nt; ++i) seen |= (uint32_t)sees_any(a, t.row0 + i, head, t.full, tail, t.n) << i;
    bad = seen;
  }

  // Two values to choose from, not two places of the arguments to load one from.
  uint64_t k_scales = reinterpret_cast<uint64_t>(c.k_scale), v_scales = reinterpret_cast<uint64_t>(c.v_scale);
  asm volatile("" : "+s"(k_scales), "+s"(v_scales));
  const unsigned char* row_scales = reinterpret_cast<const unsigned char*>(lane < 32 ? k_scales : v_scales);

  // --- looking up: lanes 0 .. 31 and 32 .. 63 both hold the step's 32 keys ---
  // Every look-up is the same loads on every path, whose values stay in the
  // registers that they came to until the next iteration uses them: so nothing
  // waits for the direct loads in flight.  Keys that are none load what is there.
  int32_t a_page = -1, a_off = 0;
  uint32_t a_bits = 0, a_mask = 0;                 // a_bits: of a chosen page; a_mask: which of them count, or the nodes of the rest
  uint32_t vis0 = 0, vis1 = 0, vis2 = 0, vis3 = 0; // keys of a step that some node sees
  bool a_chosen = false, c_ok = false;
  bool all0 = false, all1 = false, all2 = false, all3 = false;   // whether all nodes see all of a step's keys

  auto find_page = [&](int step) {
    const int64_t x = (int64_t)step * 32 + l32;
    const bool ok = step < t1 && x < (int64_t)chosen_keys + rest;
    a_chosen = ok && x < chosen_keys;
    const int32_t y = ok && !a_chosen ? (int32_t)(x - chosen_keys) : 0;   // among the rest
    const int32_t p = a_chosen ? (int32_t)x : t.full * c.page_size + y, d = c.per_page.div(p), j = y - tail;
    a_off = p - d * c.page_size;
    a_mask = ok ? all_nodes : 0u;
    if (ok && !a_chosen && j >= 0) {
      if (mask) {
        a_mask = 0;
        for (int i = 0; i < t.nt; ++i) a_mask |= ((mask[(int64_t)i * 2 * a.mask_words + (j >> 5)] >> (j & 31)) & 1u) << i;
      } else if (j > t.n0) {
        a_mask = j - t.n0 >= 32 ? 0u : all_nodes & (~0u << (j - t.n0));
      }
    }
    const int32_t* from = a_chosen ? reinterpret_cast<const int32_t*>(entries + d) : table + (ok ? d : 0);   // within the table: start + n is
    a_page = from[0];
    a_bits = (uint32_t)(a_chosen ? from + 1 : from)[0];
  };
  auto find_row = [&](int step) {
    const uint32_t who = a_chosen ? a_bits : a_mask;
    const bool held = a_page >= 0 && a_page < c.n_pages;
    seen |= who;
    if (!held) bad |= who;
    c_ok = who != 0 && held;
    const int64_t id = c_ok ? a_page : 0;
    const int32_t at = c_ok ? head * c.page_size + a_off : 0;
    vis3 = (uint32_t)__ballot(c_ok);
    all3 = __all(c_ok && who == all_nodes);
    if (lane < 32) {
      row_at[(step & 3) * 32 + lane] = id * c.page_bytes + (int64_t)at * kRB;
      masks[(step & 3) * 32 + lane] = c_ok ? who : 0u;
    }
    // the scale's byte, as a word of the lane, into the ring's place
    if constexpr (DT != DFLASH_BF16)
      __builtin_amdgcn_global_load_lds((const void*)(row_scales + id * c.scale_page_bytes + at), (lds_void_t*)(scales + (step & 3) * 64), 1, 0, 0);
  };
  auto put_scale = [&](int step) {
    if constexpr (DT != DFLASH_BF16) {
      float* at = scales + (step & 3) * 64 + lane;
      *at = c_ok ? kv_scale_value(__float_as_uint(*at)) * (lane < 32 ? c2 : 1.f) : 0.f;
    }
  };

  // --- the products of a step ---
  const int kx = S::k_swizzle(l16);
  const int vr = DT == DFLASH_BF16 ? 4 * g16 + (l16 >> 2) : 16 * (l16 >> 3) + 4 * g16 + ((l16 >> 1) & 3);
  const int vx = (DT == DFLASH_BF16 ? (l16 >> 1) & 1 : 0) ^ S::v_swizzle(vr);
  const int vbase = vr * kRB + (l16 & 1) * 8;

  auto products = [&](int step, uint32_t vis, bool all) {
    unsigned char* stage = stages + (step & 1) * 2 * S::kTile;
    if (DT != DFLASH_I8 && vis != ~0u) {
      for (int x = lane; x < S::kTile / 16; x += 64)
        if (!((vis >> (x / S::kChunks)) & 1u)) st16(stage + S::kTile + x * 16, u32x4{0, 0, 0, 0});
      asm volatile("" ::: "memory");
    }
    // All of K's operands, scales and masks are read before the first product,
    // and V's while the scores become weights: one wave to a SIMD has nobody to
    // fill its waits.
    u32x4 kf[2][kRB / 64];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int i = 0; i < kRB / 64; ++i) kf[kb][i] = ld16(stage + (16 * kb + l16) * kRB + (((4 * i + g16) ^ kx) << 4));
    float ks[2][4], vs[2][4];                      // s[u][kb][i]: key 16 kb + 4 g16 + i, row 16 u + l16
    uint32_t who[2][4];
    if constexpr (DT != DFLASH_BF16) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ks[kb][i] = scales[(step & 3) * 64 + 16 * kb + 4 * g16 + i];
          vs[kb][i] = scales[(step & 3) * 64 + 32 + 16 * kb + 4 * g16 + i];
        }
    }
    if (!all) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 4; ++i) who[kb][i] = masks[(step & 3) * 32 + 16 * kb + 4 * g16 + i];
    }
    __builtin_amdgcn_sched_barrier(0);
    f32x4_t s[GT][2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
      for (int u = 0; u < GT; ++u) s[u][kb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < kRB / 64; ++i) {
        const u32x4 x = kf[kb][i];
        if constexpr (DT == DFLASH_BF16) {
#pragma unroll
          for (int u = 0; u < GT; ++u)
            s[u][kb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, x), qf[u][i], s[u][kb], 0, 0, 0);
        } else {
          const bf16x8_t lo = codes_to_bf16<DT>(x[0], x[1]), hi = codes_to_bf16<DT>(x[2], x[3]);
#pragma unroll
          for (int u = 0; u < GT; ++u) {
            s[u][kb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, qf[u][2 * i], s[u][kb], 0, 0, 0);
            s[u][kb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, qf[u][2 * i + 1], s[u][kb], 0, 0, 0);
          }
        }
      }
    }
    // V of up to eight blocks of 16 columns
    const auto* v0 = (const __attribute__((address_space(3))) unsigned char*)(stage + S::kTile) + vbase;
    constexpr int kGroup = kBlocks < 8 ? kBlocks : 8, kPieces = DT == DFLASH_BF16 ? 2 : 1;
    i32x2_t vr2[kGroup][kPieces];
    auto read_group = [&](int b0) {
#pragma unroll
      for (int b = 0; b < kGroup; ++b)
#pragma unroll
        for (int x = 0; x < kPieces; ++x)
          vr2[b][x] = read_transposed<DT>(v0 + ((((DT == DFLASH_BF16 ? 2 : 1) * (b0 + b)) ^ vx) << 4) + x * 16 * kRB);
    };
    read_group(0);
    __builtin_amdgcn_sched_barrier(0);
    // The row tiles' maxima first, one decision for all of them, then their
    // weights: independent chains that run beside each other.
    float top[GT];
    bool past = false;
#pragma unroll
    for (int u = 0; u < GT; ++u) {
      top[u] = -INFINITY;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (DT != DFLASH_BF16) s[u][kb][i] *= ks[kb][i];
          if (!all) s[u][kb][i] = (who[kb][i] >> node[u]) & 1u ? s[u][kb][i] : -INFINITY;
          top[u] = fmaxf(top[u], s[u][kb][i]);
        }
    }
#pragma unroll
    for (int u = 0; u < GT; ++u) {
      top[u] = quarter_max(top[u]);
      // The sums keep the maximum they were built with until a row's passes it
      // by 2^8: weights up to 256 are as exact as those up to 1.
      past = past || (top[u] - m[u]) * cs > 8.f;
    }
    if (__any(past)) {
#pragma unroll
      for (int u = 0; u < GT; ++u) {
        const float next = fmaxf(m[u], top[u]), keep = m[u] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((m[u] - next) * cs);
        m[u] = next;
        l[u] *= keep;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          in_accumulators<GT * kBlocks >= 32>(o[u][b]);
          o[u][b] *= keep;
          in_accumulators<GT * kBlocks >= 32>(o[u][b]);
        }
      }
    }
    bf16x8_t pf[GT];
#pragma unroll
    for (int u = 0; u < GT; ++u) {
      const float base = m[u] == -INFINITY ? 0.f : m[u] * cs;
      float sum = 0.f, p[8];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = __builtin_amdgcn_exp2f(DT == DFLASH_BF16 ? fmaf(s[u][kb][i], cs, -base) : s[u][kb][i] - base);
          sum += e;
          float x = DT == DFLASH_BF16 ? e : e * vs[kb][i];
          // 0 * NaN: the scale of a key that other rows see
          if (DT != DFLASH_BF16 && !all) x = (who[kb][i] >> node[u]) & 1u ? x : 0.f;
          p[4 * kb + i] = x;
        }
      l[u] += sum;
      // weights rounded to bf16 (half a step, 2^-8 of each), l sums them unrounded
      const u32x4 pw = {pack_bf16(p[0], p[1]), pack_bf16(p[2], p[3]), pack_bf16(p[4], p[5]), pack_bf16(p[6], p[7])};
      pf[u] = __builtin_bit_cast(bf16x8_t, pw);
    }
#pragma unroll
    for (int b0 = 0; b0 < kBlocks; b0 += kGroup) {
      if (b0) read_group(b0);
#pragma unroll
      for (int b = 0; b < kGroup; ++b) {
        bf16x8_t vf;
        if constexpr (DT == DFLASH_BF16) vf = __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(vr2[b][0], vr2[b][kPieces - 1], 0, 1, 2, 3));
        else vf = codes_to_bf16<DT>((uint32_t)vr2[b][0][0], (uint32_t)vr2[b][0][1]);
#pragma unroll
        for (int u = 0; u < GT; ++u) o[u][b0 + b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pf[u], o[u][b0 + b], 0, 0, 0);
      }
    }
  };

  // Iteration i multiplies step i, issues the direct loads of step i + 2,
  // writes the scales of step i + 2 and the addresses of step i + 3, and looks
  // up the pages of step i + 4.
  const int load_row = lane / S::kChunks, load_slot = lane % S::kChunks;
  auto look_up = [&](int i) {
    asm volatile("" ::: "memory");
    put_scale(i + 2);
    find_row(i + 3);
    find_page(i + 4);
    asm volatile("" ::: "memory");
  };
  auto load = [&](int i) {
    __builtin_amdgcn_s_waitcnt((0 << 8) | (7 << 4) | 15 | (3 << 14));   // this step's reads of the stage are done
    asm volatile("" ::: "memory");
    unsigned char* stage = stages + (i & 1) * 2 * S::kTile;
    int64_t from[S::kLoads];
#pragma unroll
    for (int x = 0; x < S::kLoads; ++x) from[x] = row_at[((i + 2) & 3) * 32 + x * (1024 / kRB) + load_row];
#pragma unroll
    for (int x = 0; x < S::kLoads; ++x) {
      const int r = x * (1024 / kRB) + load_row;
      __builtin_amdgcn_global_load_lds((const void*)(c.k + from[x] + ((load_slot ^ S::k_swizzle(r)) << 4)),
                                       (lds_void_t*)(stage + x * 1024), 16, 0, 0);
      __builtin_amdgcn_global_load_lds((const void*)(c.v + from[x] + ((load_slot ^ S::v_swizzle(r)) << 4)),
                                       (lds_void_t*)(stage + S::kTile + x * 1024), 16, 0, 0);
    }
  };
  auto shift = [&]() {
    vis0 = vis1;
    vis1 = vis2;
    vis2 = vis3;
    all0 = all1;
    all1 = all2;
    all2 = all3;
  };
  // Past the last step the same number of loads takes row 0 of the pool: at the
  // loop's top, on every path, all but the last 2 kLoads loads are waited for.
  if (t0 < t1) {
    for (int i = t0 - 4; i < t0 - 2; ++i) {
      wait_vm<0>();
      look_up(i);
      shift();
    }
    wait_vm<0>();
    look_up(t0 - 2);
    load(t0 - 2);
    shift();
    wait_vm<2 * S::kLoads>();
    look_up(t0 - 1);
    load(t0 - 1);
    shift();
    for (int i = t0; i < t1; ++i) {
      wait_vm<2 * S::kLoads>();
      // What was looked up is here, and no use of it moves before the wait.  (The
      // compiler joins a wait with the one that it would put at the next
      // instruction, of which direct loads in flight make a wait for everything.)
      asm volatile("s_nop 0");
      asm volatile("" : "+v"(a_page), "+v"(a_bits));
      look_up(i);
      products(i, vis0, all0);
      load(i);
      shift();
    }
  }
  wait_vm<0>();

  // --- the waves of the workgroup ---
  __syncthreads();                                 // the sets are cleared, the stages free
  if (seen) atomicOr(&node_sets[0], seen);
  if (bad) atomicOr(&node_sets[1], bad);
  float* sums = reinterpret_cast<float*>(st_smem);            // [wave][16 rows][D], then [wave][16] (m, l)
  float2* stats = reinterpret_cast<float2*>(sums + waves * 16 * D);
  float* part = lists.parts + (int64_t)w * part_floats(GT, D);
#pragma unroll 1
  for (int u0 = 0; u0 < GT; ++u0) {
    if (u0) __syncthreads();
#pragma unroll
    for (int u = 0; u < GT; ++u) {                // registers are named at compile time
      if (u != u0) continue;
      const float all = quarter_sum(l[u]);
      if (g16 == 0) stats[wave * 16 + l16] = make_float2(m[u] == -INFINITY ? -INFINITY : m[u] * cs, all);
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
        *reinterpret_cast<float4*>(sums + (wave * 16 + l16) * D + 16 * b + 4 * g16) = make_float4(o[u][b][0], o[u][b][1], o[u][b][2], o[u][b][3]);
    }
    __syncthreads();
    for (int x = tid; x < min(16, rows - 16 * u0) * (D / 4); x += 64 * waves) {
      const int h = x / (D / 4), d = x % (D / 4) * 4, f_row = 16 * u0 + h;
      float top = -INFINITY;
      // (as many reads as waves at most, so that they go out at once)
#pragma unroll
      for (int i = 0; i < S::kWaves; ++i) top = fmaxf(top, stats[min(i, waves - 1) * 16 + h].x);
      float all = 0.f, f[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < S::kWaves; ++i) {
        const int j = min(i, waves - 1);
        const float2 ml = stats[j * 16 + h];
        const float keep = ml.x == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(ml.x - top);   // without keys l and O are 0
        const float4 v = *reinterpret_cast<const float4*>(sums + (j * 16 + h) * D + d);
        all += i < waves ? ml.y * keep : 0.f;
        f[0] += i < waves ? v.x * keep : 0.f;
        f[1] += i < waves ? v.y * keep : 0.f;
        f[2] += i < waves ? v.z * keep : 0.f;
        f[3] += i < waves ? v.w * keep : 0.f;
      }
      if (splits == 1) {
        const int my_node = per_group.div(f_row);
        const bool sees = (node_sets[0] >> my_node) & 1u, broken = (node_sets[1] >> my_node) & 1u;
        const float inv = broken ? __builtin_nanf("") : sees ? 1.f / all : 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] *= inv;
        if (DT != DFLASH_I8 && !broken) {
          bool odd = false;
#pragma unroll
          for (int i = 0; i < 4; ++i) odd = odd || !isfinite(f[i]);
          if (odd) atomicOr((unsigned long long*)&odd_rows, 1ull << f_row);
          // a node that sees nothing
          if (!sees) f[0] = f[1] = f[2] = f[3] = 0.f;
        }
        *reinterpret_cast<uint2*>(a.out + ((t.row0 + my_node) * a.n_q_heads + (int64_t)head * group + (f_row - my_node * group)) * D + d) =
            make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
      } else {
        *reinterpret_cast<float4*>(part + f_row * D + d) = make_float4(f[0], f[1], f[2], f[3]);
        if (d == 0) *reinterpret_cast<float2*>(part + 16 * GT * D + 2 * f_row) = make_float2(top, all);
      }
    }
  }
  if (splits > 1) {
    if (tid == 0) {
      part[16 * GT * (D + 2)] = __uint_as_float(node_sets[0]);
      part[16 * GT * (D + 2) + 1] = __uint_as_float(node_sets[1]);
    }
    return;
  }
  if constexpr (DT != DFLASH_I8) {
    __syncthreads();                               // the results are written, which a row alone replaces
    uint64_t odd = odd_rows;
    for (int i = 0; odd; odd &= odd - 1, ++i) {
      if (i % waves != wave) continue;
      const int f_row = __builtin_ctzll(odd), my_node = per_group.div(f_row);
      if ((node_sets[0] >> my_node) & 1u) alone<DT, D>(a, t, my_node, head, head * group + (f_row - my_node * group));
    }
  }
}

// Joins the splits of a tile in their order; a workgroup takes 1024 elements.
template <int DT, int D, int GT>
__global__ void __launch_bounds__(kThreads) sparse_tile_join_kernel(SparseArgs a, Lists lists, FastDiv per_group, int nodes, int per_req, int splits) {
  constexpr int kPieces = 16 * GT * D / 1024, kRows = 1024 / D;
  __shared__ uint32_t odd_rows;                    // of this workgroup's
  const int group = per_group.d, tid = threadIdx.x;
  const uint32_t item = blockIdx.x / kPieces, tiles = (uint32_t)a.c.n_req * (uint32_t)per_req;
  const int head = (int)(item / tiles), row_at = (int)(blockIdx.x % kPieces) * kRows;
  Tile t;
  if (!tile_at(a, (int)(item % tiles), nodes, per_req, t) || row_at >= t.nt * group) return;
  if (tid == 0) odd_rows = 0;
  __syncthreads();
  const int f_row = row_at + tid / (D / 4), d = tid % (D / 4) * 4;
  const int64_t size = part_floats(GT, D);
  const float* part = lists.parts + (int64_t)item * splits * size;
  uint32_t seen = 0, bad = 0;
  if (f_row < t.nt * group) {
    float top = -INFINITY, l = 0.f, f[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int i = 0; i < splits; ++i) {
      const float2 ml = *reinterpret_cast<const float2*>(part + i * size + 16 * GT * D + 2 * f_row);
      const float4 v = *reinterpret_cast<const float4*>(part + i * size + f_row * D + d);
      seen |= __float_as_uint(part[i * size + 16 * GT * (D + 2)]);
      bad |= __float_as_uint(part[i * size + 16 * GT * (D + 2) + 1]);
      const float next = fmaxf(top, ml.x);
      const float w1 = top == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(top - next);
      const float w2 = ml.x == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(ml.x - next);
      top = next;
      l = l * w1 + ml.y * w2;
      f[0] = f[0] * w1 + v.x * w2;
      f[1] = f[1] * w1 + v.y * w2;
      f[2] = f[2] * w1 + v.z * w2;
      f[3] = f[3] * w1 + v.w * w2;
    }
    const int my_node = per_group.div(f_row);
    const bool sees = (seen >> my_node) & 1u, broken = (bad >> my_node) & 1u;
    const float inv = broken ? __builtin_nanf("") : sees ? 1.f / l : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] *= inv;
    if (DT != DFLASH_I8 && !broken) {
      bool odd = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) odd = odd || !isfinite(f[i]);
      if (odd && sees) atomicOr(&odd_rows, 1u << (f_row - row_at));
      if (!sees) f[0] = f[1] = f[2] = f[3] = 0.f;
    }
    *reinterpret_cast<uint2*>(a.out + ((t.row0 + my_node) * a.n_q_heads + (int64_t)head * group + (f_row - my_node * group)) * D + d) =
        make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
  }
  if constexpr (DT != DFLASH_I8) {
    __syncthreads();                               // the results are written, which a row alone replaces
    uint32_t odd = odd_rows;
    for (int i = 0; odd; odd &= odd - 1, ++i) {
      if (i % (kThreads / 64) != tid >> 6) continue;
      const int r = row_at + __builtin_ctz(odd), my_node = per_group.div(r);
      alone<DT, D>(a, t, my_node, head, head * group + (r - my_node * group));
    }
  }
}

template <int DT, int D, int GT>
hipError_t run(const SparseArgs& a, const TilePlan& plan, hipStream_t s) {
  using S = SparseShape<DT, D>;
  const KvView& c = a.c;
  const FastDiv per_group = FastDiv::make(a.n_q_heads / c.n_kv_heads);
  const Lists lists(a.workspace, c.n_rows, c.n_kv_heads, a.n_take, c.head_dim);
  const int64_t tiles = (int64_t)c.n_req * plan.per_req, items = tiles * c.n_kv_heads;
  sparse_union_kernel<<<(unsigned)items, kUnionThreads, (size_t)c.table_width * 4, s>>>(a, lists, plan.nodes, plan.per_req);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // Keys of a tile: the union is as long as its nodes' pages differ, taken for
  // twice a node's.  (One request of 16 nodes, 64 pages each out of 128: by one
  // node's pages 37 us, twice 35, four times 36; out of 1024 pages 77, 58, 49.)
  const int64_t keys = (int64_t)a.n_take * std::min(plan.nodes, 2) * c.page_size + c.page_size + a.max_nodes;
  const Spread x = spread<S>(items, GT, keys, kMaxTileParts);
  const int splits = x.splits;
  sparse_tile_kernel<DT, D, GT><<<(unsigned)(items * splits), 64 * x.waves, x.waves * S::kWaveLds, s>>>(a, lists, per_group, plan.nodes, plan.per_req, splits);
  if ((e = hipGetLastError()) != hipSuccess || splits == 1) return e;
  sparse_tile_join_kernel<DT, D, GT><<<(unsigned)(items * (16 * GT * D / 1024)), kThreads, 0, s>>>(a, lists, per_group, plan.nodes, plan.per_req, splits);
  return hipGetLastError();
}
template <int DT, int D>
hipError_t run_tiles(const SparseArgs& a, const TilePlan& plan, hipStream_t s) {
  if (plan.row_tiles == 1) return run<DT, D, 1>(a, plan, s);
  if constexpr (D < 256) {
    if (plan.row_tiles == 4) return run<DT, D, 4>(a, plan, s);
  }
  return run<DT, D, 2>(a, plan, s);
}
template <int DT>
hipError_t run_dim(const SparseArgs& a, const TilePlan& plan, hipStream_t s) {
  if (a.c.head_dim == 64) return run_tiles<DT, 64>(a, plan, s);
  if (a.c.head_dim == 128) return run_tiles<DT, 128>(a, plan, s);
  return run_tiles<DT, 256>(a, plan, s);
}

}  // namespace

// Rows go together where a request may have several and a tile holds at least
// two of them; the rest of the conditions bound what that takes: the words in
// LDS, the lists, and workgroups without rows where few requests are as long as
// max_nodes.
TilePlan sparse_tile_plan(const KvView& c, int64_t n_rows, int32_t n_take, int32_t max_nodes, int32_t n_q_heads) {
  const int group = n_q_heads / c.n_kv_heads, most = std::min(kMaxTileNodes, max_rows(c.head_dim) / group);
  TilePlan p{};
  if (max_nodes < 2 || most < 2 || c.table_width > kMaxBlocks) return p;
  p.per_req = (max_nodes + most - 1) / most;
  p.nodes = (max_nodes + p.per_req - 1) / p.per_req;
  const int row_tiles = (p.nodes * group + 15) / 16;
  p.row_tiles = row_tiles > 2 ? 4 : row_tiles;
  p.use = (int64_t)c.n_req * p.per_req <= 2 * n_rows && (size_t)n_rows * c.n_kv_heads * n_take * sizeof(uint2) <= kMaxLists;
  return p;
}

size_t sparse_tile_bytes(const KvView& c, int64_t n_rows, int32_t n_take, int32_t n_q_heads) {
  return Lists(nullptr, n_rows, c.n_kv_heads, n_take, c.head_dim).bytes;
}

hipError_t launch_sparse_tiles(const SparseArgs& a, const TilePlan& plan, hipStream_t stream) {
  if (a.c.dtype == DFLASH_BF16) return run_dim<DFLASH_BF16>(a, plan, stream);
  if (a.c.dtype == DFLASH_E4M3) return run_dim<DFLASH_E4M3>(a, plan, stream);
  return run_dim<DFLASH_I8>(a, plan, stream);
}

}  // namespace dflash
