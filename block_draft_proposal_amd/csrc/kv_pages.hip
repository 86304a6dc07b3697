// Page tables, the counts of a pool's pages, and the copies of whole pages.
//
// Planning reads the counts once, in chunks of 1024 pages, and the tables'
// entries that change.  Everything that is shared is an integer sum or a
// minimum, so that no result depends on an order; which page goes where comes
// from ranks (the i-th free page, the i-th held page from the top), whose sums
// over chunks one workgroup makes between two launches.  The steps of a call
// are launches of their own: a launch is what makes one step's writes visible
// to all of the next.  Where one workgroup holds pool and tables, a call is one.
//
// Planning moves little and is bound by latency: its floor is the launches.
// Measured: 512 requests in a pool of half a million pages, a resize 18 us (let go
// 4.9, count 2.7, plan 4.2, give 6.5), a fork 10, a compact's planning 23 (128
// requests, 32768 pages); 32 requests in a small pool 4 to 6 us a call.  Copies of
// pages stream: 0.53 GB, read and written in 192 us, 5.6 TB/s.
#include <algorithm>

#include "kv_pages.h"

namespace dflash {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 4 * kThreads;              // pages of a workgroup: 4 neighbours to a thread
constexpr int kPlanThreads = 1024;

// --- the workspace ---

struct Plan {                                     // a resize's decision
  int32_t pages;                                  // free pages that it gives; 0 where nobody grows
  int32_t grow;                                   // whether requests grow
};
struct Grant {                                    // what a request gets
  int32_t begin;                                  // rank of its first free page
  int32_t has;                                    // entries that it holds before
  int32_t copy;                                   // index among the copies, or -1
};
struct Claim {                                    // growing requests whose partly filled last page this is
  int32_t count, first;
};

constexpr size_t up256(size_t n) { return (n + 255) / 256 * 256; }
inline int64_t chunks_of(int64_t n_pages) { return (n_pages + kChunk - 1) / kChunk; }

struct Space {
  Plan* plan;
  int2* per_chunk;                                // (free, held) pages of each chunk, then the sums before it
  Grant* grants;                                  // resize
  Claim* claims;                                  // resize: by page
  int32_t* saved_lens;                            // fork
  int32_t* saved;                                 // fork: [n_req][table_width]
  int2* moves;                                    // compact: (held from the top, free from the bottom)
  size_t bytes;
  Space(void* base, int64_t n_pages, int32_t n_req, int32_t width) {
    unsigned char* p = static_cast<unsigned char*>(base);
    plan = reinterpret_cast<Plan*>(p);
    per_chunk = reinterpret_cast<int2*>(p + 256);
    const size_t shared = 256 + up256((size_t)(chunks_of(n_pages) + 1) * sizeof(int2));
    unsigned char* own = p + shared;
    grants = reinterpret_cast<Grant*>(own);
    const size_t grant_bytes = up256((size_t)n_req * sizeof(Grant));
    claims = reinterpret_cast<Claim*>(own + grant_bytes);
    const size_t resize = grant_bytes + up256((size_t)n_pages * sizeof(Claim));
    saved_lens = reinterpret_cast<int32_t*>(own);
    const size_t lens_bytes = up256((size_t)n_req * 4);
    saved = reinterpret_cast<int32_t*>(own + lens_bytes);
    const size_t fork = lens_bytes + up256((size_t)n_req * width * 4);
    moves = reinterpret_cast<int2*>(own);
    const size_t compact = up256((size_t)(n_pages / 2 + 1) * sizeof(int2));
    bytes = shared + (resize > fork ? (resize > compact ? resize : compact) : fork > compact ? fork : compact);
  }
};

// --- ranks within a chunk ---

// The counts of 4 neighbouring pages, 1 past the last page: neither free nor,
// where `held` asks below, held.
struct Four {
  int32_t refs[4];
};
__device__ __forceinline__ Four load_four(const PagesView& v, int64_t p) {
  typedef int32_t i32x4_t __attribute__((ext_vector_type(4), aligned(4)));
  Four f;
  if (p + 4 <= v.n_pages) {
    const i32x4_t x = *reinterpret_cast<const i32x4_t*>(v.refs + p);
#pragma unroll
    for (int i = 0; i < 4; ++i) f.refs[i] = x[i];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f.refs[i] = p + i < v.n_pages ? v.refs[p + i] : -1;
  }
  return f;
}

// Inclusive sums along a wave.
__device__ __forceinline__ uint64_t wave_scan_u64(uint64_t x) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint64_t y = (uint64_t)__shfl_up((unsigned long long)x, o, 64);
    if (lane >= o) x += y;
  }
  return x;
}
// Exclusive sums along the workgroup of N threads, and the total.
template <int N>
__device__ __forceinline__ uint64_t group_scan(uint64_t x, uint64_t& total) {
  __shared__ uint64_t sums[N / 64];
  const int wave = threadIdx.x >> 6;
  const uint64_t scan = wave_scan_u64(x);
  __syncthreads();                                // the last call's sums have been read
  if ((threadIdx.x & 63) == 63) sums[wave] = scan;
  __syncthreads();
  uint64_t before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < N / 64; ++i) {
    if (i < wave) before += sums[i];
    total += sums[i];
  }
  return before + scan - x;
}

// The chunk's pages with the property before the thread's four, and in all.
template <class F>
__device__ __forceinline__ int32_t chunk_ranks(const Four& f, const F& has, int32_t& total) {
  uint64_t n = 0, all;
#pragma unroll
  for (int i = 0; i < 4; ++i) n += has(f.refs[i]);
  const int32_t before = (int32_t)group_scan<kThreads>(n, all);
  total = (int32_t)all;
  return before;
}
struct IsFree {
  __device__ __forceinline__ bool operator()(int32_t r) const { return r == 0; }
};
struct IsHeld {
  __device__ __forceinline__ bool operator()(int32_t r) const { return r > 0; }
};

// --- resize ---

// What request r does; has < 0: nothing.
struct Change {
  int32_t has, needs;
  bool part;                                      // it grows, and its last page is partly filled
};
__device__ __forceinline__ Change change_of(const PagesView& v, const int32_t* want, int r) {
  const int32_t len = v.lens[r], to = want[r];
  Change c;
  c.has = v.entries(len);
  c.needs = v.entries(to);
  if (c.needs < 0) c.has = -1;
  c.part = c.has > 0 && to > len && len != c.has * (int64_t)v.page_size;
  return c;
}

// A page's count changes by `by` for every request of a group that lets it go or
// takes it.  Requests that share a prefix follow one another and hold the same
// page in the same column: a thread adds up what neighbours do to one page (512
// samples of 64 prompts, pages of 16 and 8 to a page: let go 5.0 us and forked
// 7.6, an atomic for each entry 7.7 and 12.9).
struct Tally {
  int32_t page = -1, by = 0;
  __device__ __forceinline__ void flush(const PagesView& v) {
    if (by) atomicAdd(v.refs + page, by);
    by = 0;
  }
  __device__ __forceinline__ void add(const PagesView& v, int32_t p, int32_t n) {
    if (!v.in_pool(p)) return;
    if (p != page) {
      flush(v);
      page = p;
    }
    by += n;
  }
};
constexpr int kGroup = 4;                         // requests of a workgroup

// Pages of requests that shrink are let go; the claims of those that grow are
// cleared.  `parts` workgroups to kGroup requests.
__global__ void __launch_bounds__(kThreads) resize_release_kernel(PagesView v, const int32_t* want, Claim* claims, int parts) {
  const int r0 = blockIdx.x / parts * kGroup, part = blockIdx.x % parts, n = min(kGroup, v.n_req - r0);
  __shared__ int32_t from[kGroup], to[kGroup];    // the entries that each lets go
  if ((int)threadIdx.x < n) {
    const int r = r0 + (int)threadIdx.x;
    const Change c = change_of(v, want, r);
    from[threadIdx.x] = c.has < 0 ? 0 : c.needs;
    to[threadIdx.x] = c.has < 0 ? 0 : c.has;
    if (part == 0 && c.part) {
      const int32_t page = v.table[r * v.table_stride + c.has - 1];
      if (v.in_pool(page)) claims[page] = Claim{0, 0x7fffffff};
    }
  }
  __syncthreads();
  int32_t first = 0x7fffffff, last = 0;
  for (int i = 0; i < n; ++i) {
    if (from[i] >= to[i]) continue;
    first = min(first, from[i]);
    last = max(last, to[i]);
  }
  for (int64_t j = first + (int64_t)part * kThreads + threadIdx.x; j < last; j += (int64_t)parts * kThreads) {
    Tally tally;
    int32_t page[kGroup];
#pragma unroll
    for (int i = 0; i < kGroup; ++i) page[i] = i < n && j >= from[i] && j < to[i] ? v.table[(r0 + i) * v.table_stride + j] : -1;
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      if (i >= n || j < from[i] || j >= to[i]) continue;
      tally.add(v, page[i], -1);
      v.table[(r0 + i) * v.table_stride + j] = -1;
    }
    tally.flush(v);
  }
}

// Workgroups below `chunks` count a chunk's free pages (and held ones, for
// compact); those behind enter the claims of 256 requests each.
__global__ void __launch_bounds__(kThreads) count_kernel(PagesView v, const int32_t* want, Claim* claims, int2* per_chunk, int chunks) {
  if ((int)blockIdx.x < chunks) {
    const Four f = load_four(v, (int64_t)blockIdx.x * kChunk + 4 * threadIdx.x);
    uint64_t x = 0, total;
#pragma unroll
    for (int i = 0; i < 4; ++i) x += (uint64_t)(f.refs[i] == 0) | (uint64_t)(f.refs[i] > 0) << 32;
    group_scan<kThreads>(x, total);
    if (threadIdx.x == 0) per_chunk[blockIdx.x] = make_int2((int)(uint32_t)total, (int)(total >> 32));
    return;
  }
  const int64_t r = ((int64_t)blockIdx.x - chunks) * kThreads + threadIdx.x;
  if (r >= v.n_req) return;
  const Change c = change_of(v, want, (int)r);
  if (!c.part) return;
  const int32_t page = v.table[r * v.table_stride + c.has - 1];
  if (!v.in_pool(page)) return;
  atomicAdd(&claims[page].count, 1);
  atomicMin(&claims[page].first, (int)r);
}

// The sums before each chunk, in place; the totals go to per_chunk[chunks].
__device__ __forceinline__ int2 scan_chunks(int2* per_chunk, int chunks) {
  uint64_t run = 0;
  for (int c0 = 0; c0 < chunks; c0 += kPlanThreads) {
    const int c = c0 + (int)threadIdx.x;
    uint64_t x = 0, total;
    if (c < chunks) x = (uint32_t)per_chunk[c].x | (uint64_t)(uint32_t)per_chunk[c].y << 32;
    const uint64_t before = run + group_scan<kPlanThreads>(x, total);
    if (c < chunks) per_chunk[c] = make_int2((int)(uint32_t)before, (int)(before >> 32));
    run += total;
  }
  if (threadIdx.x == 0) per_chunk[chunks] = make_int2((int)(uint32_t)run, (int)(run >> 32));
  return make_int2((int)(uint32_t)run, (int)(run >> 32));
}

__global__ void __launch_bounds__(kPlanThreads) resize_plan_kernel(PagesView v, const int32_t* want, Space s, int chunks, int32_t* counts) {
  const int2 pool = scan_chunks(s.per_chunk, chunks);
  uint64_t pages = 0, copies = 0;                 // up to 2^20 requests of up to 2^31 entries
  for (int r0 = 0; r0 < v.n_req; r0 += kPlanThreads) {
    const int r = r0 + (int)threadIdx.x;
    Change c{-1, 0, false};
    uint64_t more = 0;
    bool copy = false;
    if (r < v.n_req) {
      c = change_of(v, want, r);
      if (c.part) {
        const int32_t page = v.table[r * v.table_stride + c.has - 1];
        if (v.in_pool(page)) {
          const int32_t refs = v.refs[page];
          const Claim claim = s.claims[page];
          copy = refs > 1 && !(claim.count == refs && claim.first == r);
        }
      }
      if (c.has >= 0 && c.needs > c.has) more = (uint64_t)(c.needs - c.has);
    }
    uint64_t all;
    // pages in the low 52 bits (1024 requests: below 2^42), copies above
    const uint64_t before = group_scan<kPlanThreads>((more + copy) | (uint64_t)copy << 52, all);
    if (r < v.n_req) {
      const uint64_t begin = pages + (before & ((1ull << 52) - 1));
      // beyond the pool's size nothing is given, whatever the number
      s.grants[r] = Grant{(int32_t)min(begin, (uint64_t)0x7fffffff), c.has, copy ? (int32_t)(copies + (before >> 52)) : -1};
    }
    pages += all & ((1ull << 52) - 1);
    copies += all >> 52;
  }
  if (threadIdx.x == 0) {
    const bool enough = pages <= (uint64_t)(uint32_t)pool.x;
    *s.plan = Plan{enough ? (int32_t)pages : 0, enough};
    counts[0] = enough ? (int32_t)copies : 0;
    counts[1] = enough ? 0 : (int32_t)min(pages - (uint64_t)(uint32_t)pool.x, (uint64_t)0x7fffffff);
  }
}

// The last of grants [lo, hi) that begins at or before `rank`, where the first does.
__device__ __forceinline__ int grant_of(const Grant* grants, int lo, int hi, int32_t rank) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (grants[mid].begin <= rank) lo = mid; else hi = mid;
  }
  return lo;
}

// Each free page of a rank below plan.pages goes to the request whose share it
// lies in.  The shares lie in LDS: all of them, or those of the requests that a
// chunk's pages go to, which have neighbouring ranks (512 requests, a pool of half
// a million pages: 6 us; the chunk's requests searched for in memory 7, each page's
// 22).  Workgroups behind the chunks set the lengths.
constexpr int kShares = 2048;
__global__ void __launch_bounds__(kThreads) resize_assign_kernel(PagesView v, const int32_t* want, Space s, int chunks, int32_t* copies) {
  __shared__ Grant shares[kShares];
  __shared__ int ends[2];
  const Plan plan = *s.plan;
  if ((int)blockIdx.x >= chunks) {
    const int64_t r = ((int64_t)blockIdx.x - chunks) * kThreads + threadIdx.x;
    if (r >= v.n_req || s.grants[r].has < 0) return;
    const int32_t to = want[r];
    if (plan.grow || to < v.lens[r]) v.lens[r] = to;
    return;
  }
  const int32_t first = s.per_chunk[blockIdx.x].x;
  if (first >= plan.pages) return;
  const int64_t base = (int64_t)blockIdx.x * kChunk + 4 * threadIdx.x;
  const Four f = load_four(v, base);
  const bool all = v.n_req <= kShares;
  if (all)
    for (int i = threadIdx.x; i < v.n_req; i += kThreads) shares[i] = s.grants[i];
  int32_t total, rank = first + chunk_ranks(f, IsFree(), total);   // behind its barriers the shares are there
  if (total == 0) return;
  int r0 = 0, n = v.n_req;
  if (!all) {
    if (threadIdx.x < 2)
      ends[threadIdx.x] = grant_of(s.grants, 0, v.n_req, threadIdx.x ? min(first + total, plan.pages) - 1 : first);
    __syncthreads();
    r0 = ends[0];
    n = ends[1] - r0 + 1;
    if (n <= kShares) {
      for (int i = threadIdx.x; i < n; i += kThreads) shares[i] = s.grants[r0 + i];
      __syncthreads();
    }
  }
  const bool held = n <= kShares;
  int r = -1;
  int32_t next = 0;                               // where the share behind r's begins
  Grant g;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (f.refs[i] != 0) continue;
    if (rank >= plan.pages) continue;
    const int32_t page = (int32_t)(base + i);
    if (r < 0 || rank >= next) {
      r = held ? r0 + grant_of(shares, 0, n, rank) : grant_of(s.grants, r0, r0 + n, rank);
      g = held ? shares[r - r0] : s.grants[r];
      next = r + 1 >= r0 + n ? 0x7fffffff : held ? shares[r + 1 - r0].begin : s.grants[r + 1].begin;
    }
    int32_t* row = v.table + r * v.table_stride;
    int32_t at = rank - g.begin;
    if (g.copy >= 0) {
      if (at == 0) {
        const int32_t old = row[g.has - 1];
        row[g.has - 1] = page;
        copies[2 * (int64_t)g.copy] = old;
        copies[2 * (int64_t)g.copy + 1] = page;
        atomicSub(v.refs + old, 1);
      }
      --at;
    }
    if (at >= 0) row[g.has + at] = page;
    v.refs[page] = 1;
    ++rank;
  }
}

// --- fork ---

// The row that row r becomes (r: none, it stays; -1: empty).
__device__ __forceinline__ int fork_source(const PagesView& v, const int32_t* parents, const int32_t* lens, int r) {
  const int32_t p = parents[r];
  if (p < 0) return -1;
  if (p >= v.n_req || v.entries(lens[p]) < 0) return r;
  return p;
}

__global__ void __launch_bounds__(kThreads) fork_save_kernel(PagesView v, const int32_t* parents, Space s, int parts) {
  const int r = blockIdx.x / parts, part = blockIdx.x - r * parts;
  const int32_t len = v.lens[r];
  if (part == 0 && threadIdx.x == 0) s.saved_lens[r] = len;
  if (fork_source(v, parents, v.lens, r) == r) return;   // stays, and is read where it is
  const int32_t has = v.entries(len);
  const int32_t* row = v.table + r * v.table_stride;
  int32_t* to = s.saved + (int64_t)r * v.table_width;
  for (int64_t j = (int64_t)part * kThreads + threadIdx.x; j < has; j += (int64_t)parts * kThreads) to[j] = row[j];
}

__global__ void __launch_bounds__(kThreads) fork_apply_kernel(PagesView v, const int32_t* parents, Space s, int parts) {
  const int r0 = blockIdx.x / parts * kGroup, part = blockIdx.x % parts, n = min(kGroup, v.n_req - r0);
  __shared__ int32_t has[kGroup], needs[kGroup];  // entries before and after; both 0 where the row stays
  __shared__ const int32_t* source[kGroup];
  if ((int)threadIdx.x < n) {
    const int i = threadIdx.x, r = r0 + i, from = fork_source(v, parents, s.saved_lens, r);
    has[i] = needs[i] = 0;
    source[i] = nullptr;
    if (from != r) {
      has[i] = max(v.entries(s.saved_lens[r]), 0);
      if (from >= 0) {
        needs[i] = v.entries(s.saved_lens[from]);
        source[i] = fork_source(v, parents, s.saved_lens, from) == from ? v.table + from * v.table_stride
                                                                        : s.saved + (int64_t)from * v.table_width;
      }
      if (part == 0) v.lens[r] = from < 0 ? 0 : s.saved_lens[from];
    }
  }
  __syncthreads();
  int32_t most = 0;
  for (int i = 0; i < n; ++i) most = max(most, max(has[i], needs[i]));
  for (int64_t j = (int64_t)part * kThreads + threadIdx.x; j < most; j += (int64_t)parts * kThreads) {
    Tally gone, come;
    int32_t old[kGroup], now[kGroup];
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      old[i] = i < n && j < has[i] ? v.table[(r0 + i) * v.table_stride + j] : -1;
      now[i] = i < n && j < needs[i] ? source[i][j] : -1;
    }
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      if (i >= n || j >= max(has[i], needs[i]) || (old[i] == now[i] && j < has[i])) continue;
      gone.add(v, old[i], -1);
      come.add(v, now[i], 1);
      v.table[(r0 + i) * v.table_stride + j] = now[i];
    }
    gone.flush(v);
    come.flush(v);
  }
}

// --- compact ---

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(Space s, int chunks, int32_t* counts) {
  const int2 pool = scan_chunks(s.per_chunk, chunks);
  if (threadIdx.x == 0) {
    counts[0] = 0;
    counts[1] = pool.y;
  }
}

// moves[i]: the i-th held page from the top and the i-th free one from the bottom.
__global__ void __launch_bounds__(kThreads) compact_list_kernel(PagesView v, Space s, int chunks, int32_t max_moves, int32_t* page_map) {
  const int2 first = s.per_chunk[blockIdx.x], pool = s.per_chunk[chunks];
  const int32_t most = min(max_moves, min(pool.x, pool.y));
  const int64_t base = (int64_t)blockIdx.x * kChunk + 4 * threadIdx.x;
  const Four f = load_four(v, base);
  int32_t total;
  int32_t up = first.x + chunk_ranks(f, IsFree(), total), down = pool.y - 1 - (first.y + chunk_ranks(f, IsHeld(), total));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t page = base + i;
    if (page >= v.n_pages) continue;
    page_map[page] = f.refs[i] == 0 ? -1 : (int32_t)page;
    if (f.refs[i] == 0) {
      if (up < most) s.moves[up].y = (int32_t)page;
      ++up;
    } else if (f.refs[i] > 0) {
      if (down < most) s.moves[down].x = (int32_t)page;
      --down;
    }
  }
}

__global__ void __launch_bounds__(kThreads) compact_move_kernel(PagesView v, Space s, int chunks, int32_t max_moves, int32_t* page_map,
                                                                int32_t* copies, int32_t* counts) {
  const int2 pool = s.per_chunk[chunks];
  const int32_t most = min(max_moves, min(pool.x, pool.y));
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= most) return;
  const int2 m = s.moves[i];
  if (m.x <= m.y) return;                         // sources fall and targets rise: from here on none moves
  copies[2 * i] = m.x;
  copies[2 * i + 1] = m.y;
  page_map[m.x] = m.y;
  v.refs[m.y] = v.refs[m.x];
  v.refs[m.x] = 0;
  bool last = i + 1 >= most;
  if (!last) {
    const int2 next = s.moves[i + 1];
    last = next.x <= next.y;
  }
  if (last) counts[0] = (int32_t)(i + 1);
}

__global__ void __launch_bounds__(kThreads) compact_tables_kernel(PagesView v, const int32_t* page_map, int parts) {
  const int r = blockIdx.x / parts, part = blockIdx.x - r * parts;
  const int32_t has = v.entries(v.lens[r]);
  int32_t* row = v.table + r * v.table_stride;
  for (int64_t j = (int64_t)part * kThreads + threadIdx.x; j < has; j += (int64_t)parts * kThreads) {
    const int32_t page = row[j];
    if (!v.in_pool(page)) continue;
    const int32_t to = page_map[page];
    if (to >= 0 && to != page) row[j] = to;
  }
}

// --- small pools and tables: a call is one workgroup, whose steps are apart by
// barriers instead of launches ---

constexpr int kSmallThreads = 1024;
constexpr int kSmallPages = 8192;                 // counts, claims and free pages lie in LDS
constexpr int kSmallRequests = kSmallThreads;     // one thread each
constexpr int64_t kSmallEntries = 32768;          // of all tables: 32 to a thread; in LDS for fork

// This thread's pages are [lo, hi): neighbours, so that sums along the
// workgroup are ranks.
struct Own {
  int lo, hi;
};
__device__ __forceinline__ Own own_pages(const PagesView& v) {
  const int each = (v.n_pages + kSmallThreads - 1) / kSmallThreads;
  return Own{min((int)threadIdx.x * each, v.n_pages), min(((int)threadIdx.x + 1) * each, v.n_pages)};
}

__global__ void __launch_bounds__(kSmallThreads) small_resize_kernel(PagesView v, const int32_t* want, int32_t* copies, int32_t* counts) {
  extern __shared__ int32_t small_lds[];
  int32_t* refs = small_lds;
  int32_t* growing = refs + v.n_pages;            // requests that grow into the page
  int32_t* first = growing + v.n_pages;           // the first of them; then the free pages in order
  __shared__ int32_t has[kSmallRequests], needs[kSmallRequests], begin[kSmallRequests];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n_waves = kSmallThreads / 64;
  Change c{-1, 0, false};
  if (tid < v.n_req) c = change_of(v, want, tid);
  has[tid] = c.has;
  needs[tid] = c.needs;
  for (int p = tid; p < v.n_pages; p += kSmallThreads) {
    refs[p] = v.refs[p];
    growing[p] = 0;
    first[p] = 0x7fffffff;
  }
  __syncthreads();
  for (int r = wave; r < v.n_req; r += n_waves) {
    if (has[r] < 0) continue;
    int32_t* row = v.table + r * v.table_stride;
    for (int j = needs[r] + lane; j < has[r]; j += 64) {
      const int32_t page = row[j];
      if (v.in_pool(page)) atomicSub(refs + page, 1);
      row[j] = -1;
    }
  }
  int32_t last = -1;                              // the request's partly filled last page
  if (c.part) {
    last = v.table[tid * v.table_stride + c.has - 1];
    if (v.in_pool(last)) {
      atomicAdd(growing + last, 1);
      atomicMin(first + last, tid);
    } else {
      last = -1;
    }
  }
  __syncthreads();
  const bool copy = last >= 0 && refs[last] > 1 && !(growing[last] == refs[last] && first[last] == tid);
  const uint64_t more = (uint64_t)(c.has >= 0 && c.needs > c.has ? c.needs - c.has : 0) + copy;
  const Own own = own_pages(v);
  uint64_t n_free = 0;
  for (int p = own.lo; p < own.hi; ++p) n_free += refs[p] == 0;
  uint64_t free_all, all;
  uint64_t rank = group_scan<kSmallThreads>(n_free, free_all);
  const uint64_t before = group_scan<kSmallThreads>(more | (uint64_t)copy << 52, all);   // the claims have been read by now
  const uint64_t pages = all & ((1ull << 52) - 1);
  const bool enough = pages <= free_all;
  if (tid == 0) {
    counts[0] = enough ? (int32_t)(all >> 52) : 0;
    counts[1] = enough ? 0 : (int32_t)min(pages - free_all, (uint64_t)0x7fffffff);
  }
  if (enough) {
    for (int p = own.lo; p < own.hi; ++p)
      if (refs[p] == 0) first[rank++] = p;
    begin[tid] = (int32_t)(before & 0xffffffffu) + copy;
  }
  __syncthreads();
  if (enough) {
    if (copy) {
      const int32_t page = first[begin[tid] - 1];
      const int64_t i = (int64_t)(before >> 52);
      copies[2 * i] = last;
      copies[2 * i + 1] = page;
      v.table[tid * v.table_stride + c.has - 1] = page;
      atomicSub(refs + last, 1);
      refs[page] = 1;
    }
    for (int r = wave; r < v.n_req; r += n_waves) {
      if (has[r] < 0) continue;
      int32_t* row = v.table + r * v.table_stride;
      for (int j = has[r] + lane; j < needs[r]; j += 64) {
        const int32_t page = first[begin[r] + j - has[r]];
        row[j] = page;
        refs[page] = 1;
      }
    }
  }
  if (c.has >= 0) {
    const int32_t to = want[tid];
    if (enough || to < v.lens[tid]) v.lens[tid] = to;
  }
  __syncthreads();
  for (int p = tid; p < v.n_pages; p += kSmallThreads) v.refs[p] = refs[p];
}

__global__ void __launch_bounds__(kSmallThreads) small_fork_kernel(PagesView v, const int32_t* parents) {
  extern __shared__ int32_t small_lds[];          // the tables as they were
  __shared__ int32_t lens[kSmallRequests];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n_waves = kSmallThreads / 64;
  if (tid < v.n_req) lens[tid] = v.lens[tid];
  __syncthreads();
  for (int r = wave; r < v.n_req; r += n_waves) {
    const int32_t has = v.entries(lens[r]);
    const int32_t* row = v.table + r * v.table_stride;
    for (int j = lane; j < has; j += 64) small_lds[r * v.table_width + j] = row[j];
  }
  __syncthreads();
  for (int r = wave; r < v.n_req; r += n_waves) {
    const int from = fork_source(v, parents, lens, r);
    if (from == r) continue;
    const int32_t has = max(v.entries(lens[r]), 0), needs = from < 0 ? 0 : v.entries(lens[from]);
    int32_t* row = v.table + r * v.table_stride;
    for (int j = lane; j < max(has, needs); j += 64) {
      const int32_t old = j < has ? small_lds[r * v.table_width + j] : -1;
      const int32_t now = j < needs ? small_lds[from * v.table_width + j] : -1;
      if (old != now || j >= has) {
        if (v.in_pool(old)) atomicSub(v.refs + old, 1);
        if (v.in_pool(now)) atomicAdd(v.refs + now, 1);
        row[j] = now;
      }
    }
    if (lane == 0) v.lens[r] = from < 0 ? 0 : lens[from];
  }
}

__global__ void __launch_bounds__(kSmallThreads) small_compact_kernel(PagesView v, int32_t max_moves, int32_t* page_map, int32_t* copies,
                                                                      int32_t* counts) {
  extern __shared__ int32_t small_lds[];
  int32_t* refs = small_lds;
  int32_t* sources = refs + v.n_pages;            // held pages from the top; then the map
  int32_t* targets = sources + v.n_pages;         // free pages from the bottom
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n_waves = kSmallThreads / 64;
  for (int p = tid; p < v.n_pages; p += kSmallThreads) refs[p] = v.refs[p];
  __syncthreads();
  const Own own = own_pages(v);
  uint64_t x = 0, all;                            // free pages, and held ones above
  for (int p = own.lo; p < own.hi; ++p) x += (uint64_t)(refs[p] == 0) | (uint64_t)(refs[p] > 0) << 32;
  const uint64_t before = group_scan<kSmallThreads>(x, all);
  const int n_free = (int)(uint32_t)all, n_held = (int)(all >> 32), most = min(max_moves, min(n_free, n_held));
  int up = (int)(uint32_t)before, down = n_held - 1 - (int)(before >> 32);
  for (int p = own.lo; p < own.hi; ++p) {
    if (refs[p] == 0) targets[up++] = p;
    else if (refs[p] > 0) sources[down--] = p;
  }
  __syncthreads();
  // sources fall and targets rise: the pairs that move come first
  int from[kSmallPages / 2 / kSmallThreads], to[kSmallPages / 2 / kSmallThreads], moves = 0;
#pragma unroll
  for (int k = 0; k < kSmallPages / 2 / kSmallThreads; ++k) {
    const int i = k * kSmallThreads + tid;
    from[k] = to[k] = -1;
    if (i < most && sources[i] > targets[i]) {
      from[k] = sources[i];
      to[k] = targets[i];
      ++moves;
      copies[2 * i] = from[k];
      copies[2 * i + 1] = to[k];
    }
  }
  uint64_t n_moves;
  group_scan<kSmallThreads>((uint64_t)moves, n_moves);   // and the lists have been read by now
  if (tid == 0) {
    counts[0] = (int32_t)n_moves;
    counts[1] = n_held;
  }
  int32_t* map = sources;
  for (int p = tid; p < v.n_pages; p += kSmallThreads) map[p] = refs[p] == 0 ? -1 : p;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kSmallPages / 2 / kSmallThreads; ++k) {
    if (from[k] < 0) continue;
    map[from[k]] = to[k];
    refs[to[k]] = refs[from[k]];
    refs[from[k]] = 0;
  }
  __syncthreads();
  for (int p = tid; p < v.n_pages; p += kSmallThreads) {
    page_map[p] = map[p];
    v.refs[p] = refs[p];
  }
  for (int r = wave; r < v.n_req; r += n_waves) {
    const int32_t has = v.entries(v.lens[r]);
    int32_t* row = v.table + r * v.table_stride;
    for (int j = lane; j < has; j += 64) {
      const int32_t page = row[j];
      if (!v.in_pool(page)) continue;
      if (map[page] >= 0 && map[page] != page) row[j] = map[page];
    }
  }
}

// --- copies of whole pages ---

// K and V go in pieces of kPiece bytes, 4 x 16 bytes to a thread, all loaded
// before the first is stored; a pair's last unit is the small arrays.
constexpr int kPiece = 4 * 16 * kThreads;

struct PageArrays {
  unsigned char* base[4];                         // k_scale, v_scale, bounds' codes and scales; null: none
  int64_t stride[4], bytes[4];
};

__device__ __forceinline__ void copy_bytes(unsigned char* to, const unsigned char* from, int64_t n) {
  if ((((uintptr_t)to | (uintptr_t)from | (uintptr_t)n) & 15) == 0) {
    for (int64_t i = threadIdx.x * 16; i < n; i += 16 * kThreads) st16(to + i, ld16(from + i));
  } else {
    for (int64_t i = threadIdx.x; i < n; i += kThreads) to[i] = from[i];
  }
}

__global__ void __launch_bounds__(kThreads) copy_pages_kernel(KvView c, PageArrays small, const int32_t* copies, int64_t max_copies,
                                                              const int32_t* counts, int64_t row_bytes, int32_t pieces) {
  const int64_t n = counts ? min((int64_t)max(counts[0], 0), max_copies) : max_copies;
  const int32_t units = 2 * pieces + 1;           // of a pair
  for (int64_t u = blockIdx.x; u < n * units; u += gridDim.x) {
    const int64_t pair = u / units;
    const int32_t unit = (int32_t)(u - pair * units);
    const int64_t from = copies[2 * pair], to = copies[2 * pair + 1];
    if (from < 0 || from >= c.n_pages || to < 0 || to >= c.n_pages || from == to) continue;
    if (unit < 2 * pieces) {
      unsigned char* base = unit < pieces ? c.k : c.v;
      const int64_t at = (int64_t)(unit < pieces ? unit : unit - pieces) * kPiece + threadIdx.x * 16;
      const unsigned char* src = base + from * c.page_bytes + at;
      unsigned char* dst = base + to * c.page_bytes + at;
      u32x4 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (at + i * 16 * kThreads < row_bytes) w[i] = ld16_nt(src + i * 16 * kThreads);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (at + i * 16 * kThreads < row_bytes) st16_nt(dst + i * 16 * kThreads, w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (small.base[i]) copy_bytes(small.base[i] + to * small.stride[i], small.base[i] + from * small.stride[i], small.bytes[i]);
    }
  }
}

// Workgroups to `each` requests: enough of them for the chip where there are
// few, and no more than a row's entries can use.
int parts_of(const PagesView& v, int each) {
  const int by_width = (int)(((int64_t)v.table_width + kThreads - 1) / kThreads);
  const int by_req = std::max(1, 1024 / std::max(1, (v.n_req + each - 1) / each));
  return std::min(by_width, by_req);
}
unsigned groups_of(const PagesView& v) { return (unsigned)((v.n_req + kGroup - 1) / kGroup); }
// One launch where one workgroup is enough: beams of 4 x 8 requests, resize
// 5.6 us and the steps apart 15.0.
bool small_tables(const PagesView& v) {
  return v.n_req <= kSmallRequests && (int64_t)v.n_req * v.table_width <= kSmallEntries;
}
bool small_pool(const PagesView& v) { return v.n_pages <= kSmallPages && small_tables(v); }
size_t small_bytes(const PagesView& v) { return (size_t)v.n_pages * 12; }
unsigned request_groups(const PagesView& v) { return (unsigned)((v.n_req + kThreads - 1) / kThreads); }

}  // namespace

size_t kv_pages_workspace(int64_t n_pages, int32_t n_req, int32_t table_width) {
  return Space(nullptr, n_pages, n_req, table_width).bytes;
}

hipError_t launch_kv_resize(const PagesView& v, const int32_t* want, int32_t* copies, int32_t* counts, void* workspace,
                            hipStream_t stream) {
  if (small_pool(v)) {
    small_resize_kernel<<<1, kSmallThreads, small_bytes(v), stream>>>(v, want, copies, counts);
    return hipGetLastError();
  }
  const Space s(workspace, v.n_pages, v.n_req, v.table_width);
  const int chunks = (int)chunks_of(v.n_pages), parts = parts_of(v, kGroup);
  const unsigned groups = request_groups(v);
  hipError_t e;
  if (v.n_req > 0) {                              // without requests the call still sets counts
    resize_release_kernel<<<groups_of(v) * (unsigned)parts, kThreads, 0, stream>>>(v, want, s.claims, parts);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  count_kernel<<<chunks + groups, kThreads, 0, stream>>>(v, want, s.claims, s.per_chunk, chunks);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  resize_plan_kernel<<<1, kPlanThreads, 0, stream>>>(v, want, s, chunks, counts);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  resize_assign_kernel<<<chunks + groups, kThreads, 0, stream>>>(v, want, s, chunks, copies);
  return hipGetLastError();
}

hipError_t launch_kv_fork(const PagesView& v, const int32_t* parents, void* workspace, hipStream_t stream) {
  if (small_tables(v)) {
    small_fork_kernel<<<1, kSmallThreads, (size_t)v.n_req * v.table_width * 4, stream>>>(v, parents);
    return hipGetLastError();
  }
  const Space s(workspace, v.n_pages, v.n_req, v.table_width);
  const int parts = parts_of(v, 1), group_parts = parts_of(v, kGroup);
  fork_save_kernel<<<(unsigned)v.n_req * parts, kThreads, 0, stream>>>(v, parents, s, parts);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  fork_apply_kernel<<<groups_of(v) * (unsigned)group_parts, kThreads, 0, stream>>>(v, parents, s, group_parts);
  return hipGetLastError();
}

hipError_t launch_kv_compact(const PagesView& v, int32_t* page_map, int32_t* copies, int64_t max_copies,
                             int32_t* counts, void* workspace, hipStream_t stream) {
  const int32_t max_moves = (int32_t)std::min<int64_t>(max_copies, v.n_pages / 2);
  if (small_pool(v)) {
    small_compact_kernel<<<1, kSmallThreads, small_bytes(v), stream>>>(v, max_moves, page_map, copies, counts);
    return hipGetLastError();
  }
  const Space s(workspace, v.n_pages, v.n_req, v.table_width);
  const int chunks = (int)chunks_of(v.n_pages);
  count_kernel<<<chunks, kThreads, 0, stream>>>(v, nullptr, nullptr, s.per_chunk, chunks);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  compact_plan_kernel<<<1, kPlanThreads, 0, stream>>>(s, chunks, counts);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  compact_list_kernel<<<chunks, kThreads, 0, stream>>>(v, s, chunks, max_moves, page_map);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (max_moves > 0) {
    compact_move_kernel<<<(unsigned)((max_moves + kThreads - 1) / kThreads), kThreads, 0, stream>>>(v, s, chunks, max_moves, page_map, copies, counts);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (v.n_req > 0) {
    const int parts = parts_of(v, 1);
    compact_tables_kernel<<<(unsigned)v.n_req * parts, kThreads, 0, stream>>>(v, page_map, parts);
    e = hipGetLastError();
  }
  return e;
}

hipError_t launch_kv_copy_pages(const KvView& c, const dflash_page_bounds* bounds, const int32_t* copies,
                                int64_t max_copies, const int32_t* counts, hipStream_t stream) {
  const int64_t rows = (int64_t)c.n_kv_heads * c.page_size, row_bytes = rows * c.head_dim * (c.dtype == DFLASH_BF16 ? 2 : 1);
  PageArrays small{};
  if (c.k_scale) {
    small.base[0] = c.k_scale;
    small.base[1] = c.v_scale;
    small.stride[0] = small.stride[1] = c.scale_page_bytes;
    small.bytes[0] = small.bytes[1] = rows;
  }
  if (bounds) {
    small.base[2] = reinterpret_cast<unsigned char*>(bounds->codes);
    small.base[3] = bounds->scale;
    small.stride[2] = small.bytes[2] = (int64_t)c.n_kv_heads * 2 * c.head_dim;
    small.stride[3] = small.bytes[3] = c.n_kv_heads;
  }
  const int32_t pieces = (int32_t)((row_bytes + kPiece - 1) / kPiece);
  const int64_t units = max_copies * (2 * (int64_t)pieces + 1);
  copy_pages_kernel<<<(unsigned)std::min<int64_t>(units, 4096), kThreads, 0, stream>>>(c, small, copies, max_copies, counts, row_bytes, pieces);
  return hipGetLastError();
}

}  // namespace dflash
