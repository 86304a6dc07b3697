// Attention of query rows over chosen pages of a paged cache.
//
// A row and kv head (an item) has its own list of pages, so that only the
// group's query heads, up to 16 to a tile, share keys: the work is a gather
// bound by the memory that holds the pages.  Each wave walks a share of the
// item's line of keys (the chosen pages, the tail behind the last full page,
// the nodes) 32 keys a step, all by itself, without barriers:
//
//   S^T = K Q^T        v_mfma_f32_16x16x32_bf16, a lane holds 8 scores of one head
//   running maximum, p = 2^(s - m), running sum          in registers
//   O^T += V^T P^T     the same lane's p, packed to bf16, are the operand as they lie
//
// K and V come by 16-byte direct global -> LDS loads, whole rows in order, into
// two stages of the wave; their chunks are swizzled so that neither product's
// reads collide on banks, and V is read transposed (ds_read_b64_tr).  A step's
// rows are looked up by a lane each over five iterations: block and mask, page,
// address and scale, loads, products.  Every wait is for loads of the iteration
// before, or older.
//
// Keys that the row does not see have score -inf, weight 0 and a row of V that
// is zeroed in LDS, whatever the cache holds.  Waves join through LDS, and where
// an item is split over workgroups (few rows), a second kernel joins their
// partial sums in a fixed order.
//
// Measured: 128 single rows over 64 pages of 32 each, 8 kv heads of 128, 64 query
// heads, e4m3 (541 MB): 103 to 105 us, 5.2 TB/s, more than a copy of 2 GB reaches
// on the same card.  One row over 32 pages of 64, bf16 (8.4 MB): 11.8 us and 3.9 for
// the join.  Its 65 steps are two to a wave, and the way to them is what takes the
// time: lengths and list, then four rounds of look-ups that each wait for the last.
#include "sparse_core.h"

namespace dflash {
namespace {

// Partials of one call at most, and so their part of the workspace.
constexpr int kMaxParts = 1024;

// A row, a kv head and 16 GT of its group's heads.  Rows are neighbours.
struct Item {
  int head, tile;
  int64_t row;
};
__device__ __forceinline__ Item item_of(uint32_t i, uint32_t n_rows, int tiles) {
  Item it;
  it.tile = (int)(i % (uint32_t)tiles);
  i /= (uint32_t)tiles;
  it.head = (int)(i / n_rows);
  it.row = i - (uint32_t)it.head * n_rows;
  return it;
}

struct Part {                                     // what a split item leaves: [heads][D] O, then (m, l) of each head,
  __host__ __device__ static int64_t floats(int group, int d) { return ((int64_t)group * (d + 2) + 7) / 4 * 4; }   // then whether it saw anything
};

template <int DT, int D, int GT>
__global__ void __launch_bounds__((SparseShape<DT, D>::kThreads), (GT * D <= 128 ? 2 : 1))
    sparse_attention_kernel(SparseArgs a, int all_heads, int tiles, int splits) {
  using S = SparseShape<DT, D>;
  constexpr int kRB = S::kRB, kOps = D / 32, kBlocks = D / 16;
  extern __shared__ __align__(16) unsigned char sa_smem[];
  const KvView& c = a.c;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = blockDim.x >> 6;
  const int l16 = lane & 15, g16 = lane >> 4, l32 = lane & 31;
  // rows of one kv head are neighbours on one XCD: a request's share pages
  const uint32_t w = xcd_contiguous(blockIdx.x, gridDim.x);
  const int split = (int)(w % (uint32_t)splits);
  const Item it = item_of(w / (uint32_t)splits, (uint32_t)c.n_rows, tiles);
  const int head = it.head, h0 = it.tile * 16 * GT, group = min(all_heads - h0, 16 * GT);   // its query heads
  const int64_t row = it.row;
  const int32_t* chosen = a.blocks + ((int64_t)row * c.n_kv_heads + head) * a.n_take;
  int32_t named[4];                                // the first 256 entries, while the request is looked up
  if (a.n_take > 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) named[i] = chosen[min(lane + 64 * i, a.n_take - 1)];
  }
  RowOf at;
  if (!row_of(c, row, a.max_nodes, at)) return;     // padding: the whole workgroup
  const int32_t req = at.req;
  const int node = (int)(row - at.first);
  if (node >= a.max_nodes) return;
  const int n = (int)min(min(at.end, c.n_rows) - at.first, (int64_t)a.max_nodes);
  const int32_t start = max(at.start, 0);
  const bool over = (int64_t)start + n > min((int64_t)kMaxLen, (int64_t)c.table_width * c.page_size);
  const int32_t full = kv_blocks(c, start);                 // blocks that may be chosen
  const int32_t* table = c.table + req * c.table_stride;
  const uint32_t* mask = a.mask ? reinterpret_cast<const uint32_t*>(a.mask + (int64_t)row * a.mask_words) : nullptr;

  // the line: entries up to the last that names a block, the tail, the nodes
  int used = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (lane + 64 * i < a.n_take && named[i] >= 0 && named[i] < full) used = lane + 64 * i + 1;
  for (int i = 256 + lane; i < a.n_take; i += 64) {
    const int32_t b = chosen[i];
    if (b >= 0 && b < full) used = i + 1;
  }
  used = over ? 0 : (int)wave_max_u32((uint32_t)used);
  const int32_t chosen_keys = used * c.page_size, tail = start - full * c.page_size;
  const int32_t rest = over ? 0 : tail + (a.mask ? n : node + 1);
  const int64_t steps = ((int64_t)chosen_keys + rest + 31) / 32, slots = (int64_t)splits * waves, me = split * waves + wave;
  const int t0 = __builtin_amdgcn_readfirstlane((int)(steps * me / slots)), t1 = __builtin_amdgcn_readfirstlane((int)(steps * (me + 1) / slots));

  unsigned char* stages = sa_smem + wave * S::kWaveStages;
  unsigned char* ring = sa_smem + waves * S::kWaveStages + wave * S::kRing;
  int64_t* row_at = reinterpret_cast<int64_t*>(ring + S::kRowsAt);
  float* scales = reinterpret_cast<float*>(ring + S::kScalesAt);
  // log2(e) and the softmax scale; an 8-bit cache carries it in K's scales
  const float c2 = a.scale * 1.44269504088896340736f, cs = DT == DFLASH_BF16 ? c2 : 1.f;

  // queries, in the order K's chunks have in the product; heads past the group repeat its last
  bf16x8_t qf[GT][kOps];
#pragma unroll
  for (int t = 0; t < GT; ++t) {
    const int h = min(16 * t + l16, group - 1);
    const uint16_t* qp = a.q + row * a.q_row + ((int64_t)head * all_heads + h0 + h) * a.q_head;
#pragma unroll
    for (int o = 0; o < kOps; ++o) {
      const int d = DT == DFLASH_BF16 ? 32 * o + 8 * g16 : 64 * (o / 2) + 16 * g16 + 8 * (o & 1);
      qf[t][o] = __builtin_bit_cast(bf16x8_t, ld16(qp + d));
    }
  }

  f32x4_t o[GT][kBlocks];
  float m[GT], l[GT];                              // l over this lane's keys only
#pragma unroll
  for (int t = 0; t < GT; ++t) {
    m[t] = -INFINITY;
    l[t] = 0.f;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) o[t][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
  bool bad = over && sees_any(a, row, head, full, tail, n), seen = bad;

  // Two values to choose from, not two places of the arguments to load one from.
  uint64_t k_scales = reinterpret_cast<uint64_t>(c.k_scale), v_scales = reinterpret_cast<uint64_t>(c.v_scale);
  asm volatile("" : "+s"(k_scales), "+s"(v_scales));
  const unsigned char* row_scales = reinterpret_cast<const unsigned char*>(lane < 32 ? k_scales : v_scales);

  // --- looking up: lanes 0 .. 31 and 32 .. 63 both hold the step's 32 keys ---
  // Every look-up is the same loads on every path, whose values stay in the
  // registers that they came to until the next iteration uses them: so nothing
  // waits for the direct loads in flight.  Keys that are none load what is there.
  int32_t a_block = 0, a_before = -1, a_rest = 0, a_off = 0, a_bit = 0, b_page = -1, b_off = 0;
  uint32_t a_word = 0, vis0 = 0, vis1 = 0, vis2 = 0, vis3 = 0;
  bool a_ok = false, a_chosen = false, a_masked = false, a_first = false, b_ok = false, c_ok = false;

  auto find_block = [&](int step) {
    const int64_t x = (int64_t)step * 32 + l32;
    a_ok = step < t1 && x < (int64_t)chosen_keys + rest;
    a_chosen = a_ok && x < chosen_keys;
    const int32_t y = a_ok && !a_chosen ? (int32_t)(x - chosen_keys) : 0;   // among the rest
    const int32_t p = a_chosen ? (int32_t)x : full * c.page_size + y, d = c.per_page.div(p);
    a_off = p - d * c.page_size;
    a_rest = d;
    a_first = d == 0;
    const int32_t* from = a_chosen ? chosen + d : table;
    a_block = from[0];
    a_before = (a_chosen && !a_first ? from - 1 : from)[0];
    if (mask) {
      a_masked = a_ok && !a_chosen && y >= tail;
      a_bit = a_masked ? (y - tail) & 31 : 0;
      a_word = mask[a_masked ? (y - tail) >> 5 : 0];
    }
  };
  auto find_page = [&]() {
    const bool named = a_block >= 0 && a_block < full && (a_first || a_block > a_before);
    b_ok = a_ok && (!a_chosen || named) && (!a_masked || ((a_word >> a_bit) & 1u));
    b_off = a_off;
    b_page = table[b_ok ? (a_chosen ? a_block : a_rest) : 0];   // within the table: start + n is
  };
  auto find_row = [&](int step) {
    const bool held = b_page >= 0 && b_page < c.n_pages;
    bad = bad || __any(b_ok && !held);
    c_ok = b_ok && held;
    const int64_t id = c_ok ? b_page : 0;
    const int32_t at = c_ok ? head * c.page_size + b_off : 0;
    vis3 = (uint32_t)__ballot(c_ok);
    if (lane < 32) row_at[(step & 3) * 32 + lane] = id * c.page_bytes + (int64_t)at * kRB;
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
  // V's transposed reads: lane i of 16 addresses 8 bytes of a row, and gets column i of 4 (8-bit: 8) rows
  const int vr = DT == DFLASH_BF16 ? 4 * g16 + (l16 >> 2) : 16 * (l16 >> 3) + 4 * g16 + ((l16 >> 1) & 3);
  const int vx = (DT == DFLASH_BF16 ? (l16 >> 1) & 1 : 0) ^ S::v_swizzle(vr);
  const int vbase = vr * kRB + (l16 & 1) * 8;

  auto products = [&](int step, uint32_t vis) {
    unsigned char* stage = stages + (step & 1) * 2 * S::kTile;
    if (DT != DFLASH_I8 && vis != ~0u) {
      // 0 times an infinity or NaN: rows that are not seen become zeros
      for (int x = lane; x < S::kTile / 16; x += 64)
        if (!((vis >> (x / S::kChunks)) & 1u)) st16(stage + S::kTile + x * 16, u32x4{0, 0, 0, 0});
      wave_order();
    }
    // All of K's operands, scales and masks are read before the first product,
    // and V's while the scores become weights: one wave to a SIMD has nobody to
    // fill its waits.
    u32x4 kf[2][kRB / 64];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int i = 0; i < kRB / 64; ++i) kf[kb][i] = ld16(stage + (16 * kb + l16) * kRB + (((4 * i + g16) ^ kx) << 4));
    float ks[2][4], vs[2][4];                      // s[t][kb][i]: key 16 kb + 4 g16 + i, row 16 t + l16
    if constexpr (DT != DFLASH_BF16) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ks[kb][i] = scales[(step & 3) * 64 + 16 * kb + 4 * g16 + i];
          vs[kb][i] = scales[(step & 3) * 64 + 32 + 16 * kb + 4 * g16 + i];
        }
    }
    __builtin_amdgcn_sched_barrier(0);
    f32x4_t s[GT][2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
      for (int t = 0; t < GT; ++t) s[t][kb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < kRB / 64; ++i) {
        const u32x4 x = kf[kb][i];
        if constexpr (DT == DFLASH_BF16) {
#pragma unroll
          for (int t = 0; t < GT; ++t)
            s[t][kb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, x), qf[t][i], s[t][kb], 0, 0, 0);
        } else {
          const bf16x8_t lo = codes_to_bf16<DT>(x[0], x[1]), hi = codes_to_bf16<DT>(x[2], x[3]);
#pragma unroll
          for (int t = 0; t < GT; ++t) {
            s[t][kb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, qf[t][2 * i], s[t][kb], 0, 0, 0);
            s[t][kb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, qf[t][2 * i + 1], s[t][kb], 0, 0, 0);
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
    const uint32_t mine = vis >> (4 * g16);          // bit 16 kb + i
    bf16x8_t pf[GT];
#pragma unroll
    for (int t = 0; t < GT; ++t) {
      float top = -INFINITY;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (DT != DFLASH_BF16) s[t][kb][i] *= ks[kb][i];
          s[t][kb][i] = (mine >> (16 * kb + i)) & 1u ? s[t][kb][i] : -INFINITY;
          top = fmaxf(top, s[t][kb][i]);
        }
      top = quarter_max(top);
      // The sums keep the maximum they were built with until a row's passes it
      // by 2^8: weights up to 256 are as exact as those up to 1.
      if (__any((top - m[t]) * cs > 8.f)) {
        const float next = fmaxf(m[t], top), keep = m[t] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((m[t] - next) * cs);
        m[t] = next;
        l[t] *= keep;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          in_accumulators<GT * kBlocks >= 32>(o[t][b]);
          o[t][b] *= keep;
          in_accumulators<GT * kBlocks >= 32>(o[t][b]);
        }
      }
      const float base = m[t] == -INFINITY ? 0.f : m[t] * cs;
      float sum = 0.f, p[8];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = __builtin_amdgcn_exp2f(DT == DFLASH_BF16 ? fmaf(s[t][kb][i], cs, -base) : s[t][kb][i] - base);
          sum += e;
          p[4 * kb + i] = DT == DFLASH_BF16 ? e : e * vs[kb][i];
        }
      l[t] += sum;
      // weights rounded to bf16 (half a step, 2^-8 of each): the product with
      // V is bf16 x bf16 on the matrix cores; l sums them unrounded
      const u32x4 pw = {pack_bf16(p[0], p[1]), pack_bf16(p[2], p[3]), pack_bf16(p[4], p[5]), pack_bf16(p[6], p[7])};
      pf[t] = __builtin_bit_cast(bf16x8_t, pw);
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
        for (int t = 0; t < GT; ++t) o[t][b0 + b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pf[t], o[t][b0 + b], 0, 0, 0);
      }
    }
  };

  // Iteration i multiplies step i, issues the direct loads of step i + 2,
  // writes the scales of step i + 2 and the addresses of step i + 3, and looks
  // up the pages of step i + 4 and the blocks of step i + 5.
  const int load_row = lane / S::kChunks, load_slot = lane % S::kChunks;
  auto look_up = [&](int i) {
    wave_order();
    put_scale(i + 2);
    find_row(i + 3);
    find_page();
    find_block(i + 5);
    wave_order();
  };
  auto load = [&](int i) {
    __builtin_amdgcn_s_waitcnt((0 << 8) | (7 << 4) | 15 | (3 << 14));   // this step's reads of the stage are done
    wave_order();
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
  };
  // Past the last step the same number of loads takes row 0 of the pool: at the
  // loop's top, on every path, all but the last 2 kLoads loads are waited for.
  if (t0 < t1) {
    for (int i = t0 - 5; i < t0 - 2; ++i) {
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
      asm volatile("" : "+v"(a_block), "+v"(a_before), "+v"(a_word), "+v"(b_page));
      look_up(i);
      seen = seen || vis0;
      products(i, vis0);
      load(i);
      shift();
    }
  }
  wait_vm<0>();

  // --- the waves of the workgroup ---
  seen = __syncthreads_or(seen || bad);                      // a position without a page is seen too
  float* sums = reinterpret_cast<float*>(sa_smem);           // [wave][16 heads][D], then [wave][16] (m, l)
  float2* stats = reinterpret_cast<float2*>(sums + waves * 16 * D);
  bad = __syncthreads_or(bad);
#pragma unroll 1
  for (int t = 0; t < GT; ++t) {
    if (t) __syncthreads();
#pragma unroll
    for (int u = 0; u < GT; ++u) {                // registers are named at compile time
      if (u != t) continue;
      const float all = quarter_sum(l[u]);
      if (g16 == 0) stats[wave * 16 + l16] = make_float2(m[u] == -INFINITY ? -INFINITY : m[u] * cs, bad ? __builtin_nanf("") : all);
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
        *reinterpret_cast<float4*>(sums + (wave * 16 + l16) * D + 16 * b + 4 * g16) = make_float4(o[u][b][0], o[u][b][1], o[u][b][2], o[u][b][3]);
    }
    __syncthreads();
    const int heads = min(16, group - 16 * t);
    for (int x = tid; x < heads * (D / 4); x += 64 * waves) {
      const int h = x / (D / 4), d = x % (D / 4) * 4;
      float top = -INFINITY;
      // (as many reads as waves at most, so that they go out at once)
#pragma unroll
      for (int i = 0; i < S::kWaves; ++i) top = fmaxf(top, stats[min(i, waves - 1) * 16 + h].x);
      float all = 0.f, f[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < S::kWaves; ++i) {
        const int j = min(i, waves - 1);
        const float2 ml = stats[j * 16 + h];
        const float keep = ml.x == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(ml.x - top);   // without keys l and O are 0, or NaN
        const float4 v = *reinterpret_cast<const float4*>(sums + (j * 16 + h) * D + d);
        all += i < waves ? ml.y * keep : 0.f;
        f[0] += i < waves ? v.x * keep : 0.f;
        f[1] += i < waves ? v.y * keep : 0.f;
        f[2] += i < waves ? v.z * keep : 0.f;
        f[3] += i < waves ? v.w * keep : 0.f;
      }
      const int out_head = 16 * t + h;
      if (splits == 1) {
        const float inv = seen ? 1.f / all : 0.f;
        *reinterpret_cast<uint2*>(a.out + ((int64_t)row * a.n_q_heads + (int64_t)head * all_heads + h0 + out_head) * D + d) =
            make_uint2(pack_bf16(f[0] * inv, f[1] * inv), pack_bf16(f[2] * inv, f[3] * inv));
      } else {
        float* part = static_cast<float*>(a.workspace) + (int64_t)w * Part::floats(min(all_heads, 16 * GT), D);
        *reinterpret_cast<float4*>(part + out_head * D + d) = make_float4(f[0], f[1], f[2], f[3]);
        if (d == 0) *reinterpret_cast<float2*>(part + group * D + 2 * out_head) = make_float2(top, all);
        if (x == 0 && t == 0) part[group * (D + 2)] = seen ? 1.f : 0.f;
      }
    }
  }
}

// Joins the splits of an item in their order; a workgroup takes 1024 elements.
template <int D, int GT>
__global__ void __launch_bounds__(256) sparse_join_kernel(SparseArgs a, int all_heads, int tiles, int splits, int pieces) {
  const KvView& c = a.c;
  const uint32_t item = blockIdx.x / (uint32_t)pieces;
  const Item it = item_of(item, (uint32_t)c.n_rows, tiles);
  const int h0 = it.tile * 16 * GT, group = min(all_heads - h0, 16 * GT);
  RowOf at;
  if (!row_of(c, it.row, a.max_nodes, at) || it.row - at.first >= a.max_nodes) return;
  const int x = ((int)(blockIdx.x - item * (uint32_t)pieces) * 256 + (int)threadIdx.x) * 4, h = x / D, d = x % D;
  if (h >= group) return;
  const int64_t size = Part::floats(min(all_heads, 16 * GT), D);
  const float* part = static_cast<const float*>(a.workspace) + (int64_t)item * splits * size;
  float top = -INFINITY, l = 0.f, f[4] = {0.f, 0.f, 0.f, 0.f}, seen = 0.f;
#pragma unroll 4
  for (int i = 0; i < splits; ++i) {
    const float2 ml = *reinterpret_cast<const float2*>(part + i * size + group * D + 2 * h);
    const float4 v = *reinterpret_cast<const float4*>(part + i * size + h * D + d);
    seen += part[i * size + group * (D + 2)];
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
  const float inv = seen > 0.f ? 1.f / l : 0.f;
  *reinterpret_cast<uint2*>(a.out + (it.row * a.n_q_heads + (int64_t)it.head * all_heads + h0 + h) * D + d) =
      make_uint2(pack_bf16(f[0] * inv, f[1] * inv), pack_bf16(f[2] * inv, f[3] * inv));
}

template <int DT, int D, int GT>
hipError_t run(const SparseArgs& a, hipStream_t s) {
  using S = SparseShape<DT, D>;
  const int group = a.n_q_heads / a.c.n_kv_heads, tiles = (group + 16 * GT - 1) / (16 * GT);
  const int64_t items = a.c.n_rows * a.c.n_kv_heads * tiles;
  const int64_t keys = (int64_t)a.n_take * a.c.page_size + a.c.page_size + a.max_nodes;
  const Spread x = spread<S>(items, GT, keys, kMaxParts);
  const int splits = x.splits;
  sparse_attention_kernel<DT, D, GT><<<(unsigned)(items * splits), 64 * x.waves, x.waves * S::kWaveLds, s>>>(a, group, tiles, splits);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
  const int pieces = (std::min(group, 16 * GT) * D + 1023) / 1024;
  sparse_join_kernel<D, GT><<<(unsigned)(items * pieces), 256, 0, s>>>(a, group, tiles, splits, pieces);
  return hipGetLastError();
}
template <int DT, int D>
hipError_t run_group(const SparseArgs& a, hipStream_t s) {
  const int group = a.n_q_heads / a.c.n_kv_heads;
  if (group <= 16) return run<DT, D, 1>(a, s);
  // heads of 256 have no registers for four tiles: a second workgroup reads the
  // keys again
  if (group <= 32 || D == 256) return run<DT, D, 2>(a, s);
  if constexpr (D < 256) return run<DT, D, 4>(a, s);
}
template <int DT>
hipError_t run_dim(const SparseArgs& a, hipStream_t s) {
  if (a.c.head_dim == 64) return run_group<DT, 64>(a, s);
  if (a.c.head_dim == 128) return run_group<DT, 128>(a, s);
  return run_group<DT, 256>(a, s);
}

}  // namespace

size_t sparse_attention_bytes(const KvView& c, int64_t n_rows, int32_t n_take, int32_t max_nodes, int32_t n_q_heads) {
  const size_t rows = ((size_t)kMaxParts * Part::floats(n_q_heads / c.n_kv_heads, c.head_dim) * sizeof(float) + 255) / 256 * 256;
  return max_nodes == 1 ? rows : std::max(rows, sparse_tile_bytes(c, n_rows, n_take, n_q_heads));
}

hipError_t launch_sparse_attention(const SparseArgs& a, hipStream_t stream) {
  const TilePlan plan = sparse_tile_plan(a.c, a.c.n_rows, a.n_take, a.max_nodes, a.n_q_heads);
  if (plan.use) return launch_sparse_tiles(a, plan, stream);
  if (a.c.dtype == DFLASH_BF16) return run_dim<DFLASH_BF16>(a, stream);
  if (a.c.dtype == DFLASH_E4M3) return run_dim<DFLASH_E4M3>(a, stream);
  return run_dim<DFLASH_I8>(a, stream);
}

}  // namespace dflash
