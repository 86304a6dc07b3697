// The least and the greatest key of each channel of the pages that have become
// full, 8 bits outwards.
//
// A wave takes one (page, kv head): its rows are one contiguous run, of which
// a lane reads 16 bytes of every (64 / lanes of a row)-th row and keeps the
// extremes of its channels in registers; lanes of the same channels join at the
// end.  The keys are read once and the kernel is bound by that stream: 64 ragged
// prompts of up to 8192 positions, 8 heads of 128 in e4m3 (285 MB) 61 to 65 us,
// 4.4 TB/s; the pages that a step of 256 requests fills 6.4 us, latency.
#include <type_traits>

#include "kv_sparse.h"

namespace dflash {
namespace {

constexpr int kThreads = 256;

// The values of 16 bytes of a row.
template <int DT>
struct Sixteen {
  static constexpr int kN = DT == DFLASH_BF16 ? 8 : 16;
  __device__ static __forceinline__ void get(u32x4 w, float scale, float (&x)[kN]) {
    if constexpr (DT == DFLASH_BF16) {
      unpack16(w, x);
    } else if constexpr (DT == DFLASH_E4M3) {
      // conversion and scale (a power of two) in one instruction for two codes
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const auto lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[i], scale, false);
        const auto hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[i], scale, true);
        x[4 * i] = lo[0];
        x[4 * i + 1] = lo[1];
        x[4 * i + 2] = hi[0];
        x[4 * i + 3] = hi[1];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float f[4];
        unpack_codes<DT>(w[i], f);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[4 * i + j] = f[j] * scale;
      }
    }
  }
};

// x * 2^-e rounded outwards.  The product is exact unless it falls below
// 2^-126, where rounding to a whole number must not see a zero.
__device__ __forceinline__ int outward(float x, float inv, bool up) {
  const float p = x * inv;
  if (up) return x > 0.f ? max((int)ceilf(p), 1) : (int)ceilf(p);
  return x < 0.f ? min((int)floorf(p), -1) : (int)floorf(p);
}

// The lane `n` places back in its row of 16.
template <int N>
__device__ __forceinline__ float row_ror(float x) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), 0x120 + N, 0xf, 0xf, false));
}
// x[] of the lanes with the same lane % LANES, combined.  The first kLeft
// entries are the result: with 32 lanes to a row, half of a lane's channels,
// its half of the wave's; with fewer, a quarter of them, its row of 16's.
template <int LANES, int N, class F>
__device__ __forceinline__ void join_rows(float (&x)[N], const F& f) {
  if constexpr (LANES <= 8) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = f(x[i], row_ror<8>(x[i]));
  }
  if constexpr (LANES <= 4) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = f(x[i], row_ror<4>(x[i]));
  }
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x[i]), __float_as_uint(x[i + N / 2]), false, false);
    x[i] = f(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  if constexpr (LANES <= 16) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x[i]), __float_as_uint(x[i + N / 4]), false, false);
      x[i] = f(__uint_as_float(r[0]), __uint_as_float(r[1]));
    }
  }
}

// The pages that request r's positions have filled up.
struct Filled {
  int32_t first, count;
};
__device__ __forceinline__ Filled filled_of(const KvView& c, const int32_t* end, int r) {
  const int32_t from = max(c.start[r], 0), to = end[r];
  const int32_t first = kv_blocks(c, from);
  return Filled{first, to > from ? kv_blocks(c, to) - first : 0};
}

// All requests' (page, kv head) pairs form a line that the waves share evenly:
// prompts of any lengths, or the few pages of a step.  With more requests than
// kLine, each has a workgroup of its own.
constexpr int kLine = 2048;

template <int DT, int D>
__global__ void __launch_bounds__(kThreads) kv_bounds_kernel(KvView c, int8_t* codes, uint8_t* scale, const int32_t* end) {
  constexpr int kRB = D * (DT == DFLASH_BF16 ? 2 : 1), kLanes = kRB / 16, kRows = 64 / kLanes, kN = Sixteen<DT>::kN;
  constexpr int kBatch = 8;                       // loads of a lane in flight
  __shared__ int64_t ends[kLine];                 // of the requests' parts of the line
  __shared__ int64_t sums[kThreads / 64];
  const int lane = threadIdx.x & 63, part = lane % kLanes, sub = lane / kLanes;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), heads = c.n_kv_heads;
  int req, last;                                  // the wave's requests
  int64_t task, stop;                             // its share: of the line, or of its request
  const bool line = c.n_req <= kLine;
  if (line) {
    int64_t run = 0;
    for (int r0 = 0; r0 < c.n_req; r0 += kThreads) {
      const int r = r0 + (int)threadIdx.x;
      int64_t x = r < c.n_req ? (int64_t)filled_of(c, end, r).count * heads : 0;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int64_t y = __shfl_up(x, o, 64);
        if (lane >= o) x += y;
      }
      if (r0) __syncthreads();
      if (lane == 63) sums[wave] = x;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kThreads / 64; ++i) {
        if (i < wave) x += sums[i];
      }
      if (r < c.n_req) ends[r] = run + x;
#pragma unroll
      for (int i = 0; i < kThreads / 64; ++i) run += sums[i];
    }
    __syncthreads();
    const int64_t w = (int64_t)blockIdx.x * (kThreads / 64) + wave, waves = (int64_t)gridDim.x * (kThreads / 64);
    task = run / waves * w + run % waves * w / waves;
    stop = run / waves * (w + 1) + run % waves * (w + 1) / waves;
    if (task >= stop) return;
    int lo = -1, hi = c.n_req - 1;                // the first request that ends behind the task
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (ends[mid] > task) hi = mid; else lo = mid;
    }
    req = hi;
    last = c.n_req;
  } else {
    req = blockIdx.x;
    last = req + 1;
    task = wave;
    stop = (int64_t)filled_of(c, end, req).count * heads;
    if (task >= stop) return;
  }
  const int step = line ? 1 : kThreads / 64;
  Filled filled = filled_of(c, end, req);
  int64_t before = line && req ? ends[req - 1] : 0;
  int32_t head = 0, next_head = 0;
  // the next page, looked up a task ahead
  auto look_up = [&]() -> int32_t {
    while (line && task >= ends[req] && req + 1 < last) {
      before = ends[req];
      filled = filled_of(c, end, ++req);
    }
    const int64_t x = task - before;
    const int32_t b = (int32_t)(x / heads);
    next_head = (int32_t)(x - (int64_t)b * heads);
    return c.table[(int64_t)req * c.table_stride + filled.first + b];
  };
  int32_t next_id = look_up();
  for (bool more = true; more;) {
    const int32_t id = next_id;
    head = next_head;
    task += step;
    more = task < stop;
    if (more) next_id = look_up();
    if (id < 0 || id >= c.n_pages) continue;
    const unsigned char* rows = c.k + (int64_t)id * c.page_bytes + (int64_t)head * c.page_size * kRB + part * 16;
    const uint8_t* row_scale = DT == DFLASH_BF16 ? nullptr : c.k_scale + (int64_t)id * c.scale_page_bytes + (int64_t)head * c.page_size;
    float low[kN], high[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      low[i] = INFINITY;
      high[i] = -INFINITY;
    }
    bool odd = false;                             // a row's scale is NaN
    for (int r0 = 0; r0 < c.page_size; r0 += kRows * kBatch) {
      u32x4 w[kBatch];
      uint32_t byte[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {          // past the page's end the last row once more
        const int r = min(r0 + sub + i * kRows, c.page_size - 1);
        w[i] = ld16_nt(rows + (int64_t)r * kRB);
        byte[i] = DT == DFLASH_BF16 ? 127 : row_scale[r];
      }
      // two rows at a time: minimum and maximum of three, which keep a NaN
#pragma unroll
      for (int i = 0; i < kBatch; i += 2) {
        float x[kN], y[kN];
        odd = odd || byte[i] == 255u || byte[i + 1] == 255u;
        Sixteen<DT>::get(w[i], DT == DFLASH_BF16 ? 1.f : kv_scale_value(byte[i]), x);
        Sixteen<DT>::get(w[i + 1], DT == DFLASH_BF16 ? 1.f : kv_scale_value(byte[i + 1]), y);
#pragma unroll
        for (int j = 0; j < kN; ++j) {
          low[j] = __builtin_elementwise_minimum(__builtin_elementwise_minimum(low[j], x[j]), y[j]);
          high[j] = __builtin_elementwise_maximum(__builtin_elementwise_maximum(high[j], x[j]), y[j]);
        }
      }
    }
    // the largest magnitude by its bits, which order as the values do; those of
    // an infinity or a NaN are the largest
    uint32_t top = odd ? 0x7fffffffu : 0u;
#pragma unroll
    for (int i = 0; i < kN; ++i) top = max(top, max(__float_as_uint(low[i]) & 0x7fffffffu, __float_as_uint(high[i]) & 0x7fffffffu));
    top = wave_max_u32(top);
    const bool finite = top < 0x7f800000u;
    // 127 = 1.984375 * 2^6: the carry out of the mantissa takes the next
    // exponent where the largest magnitude's mantissa is above that
    const uint32_t byte = finite ? (uint32_t)max((int)((top + 0x1ffffu) >> 23) - 6, 27) : 255u;
    const float inv = __uint_as_float((254u - min(byte, 253u)) << 23);
    // Lanes of the same channels join.  Between the wave's halves, and between
    // rows of 16 lanes, a pair of registers changes places so that one of them
    // has one channel's two values and the other the other's: each step leaves
    // half as many registers, and at the end a lane has its share of the row.
    join_rows<kLanes>(low, [](float x, float y) { return fminf(x, y); });
    join_rows<kLanes>(high, [](float x, float y) { return fmaxf(x, y); });
    constexpr int kLeft = kLanes == 32 ? kN / 2 : kN / 4;
    if (kLanes >= 16 || (lane & 15) < kLanes) {
      const int at = part * kN + (kLanes == 32 ? lane >> 5 : lane >> 4) * kLeft;
      int8_t* out = codes + ((int64_t)id * c.n_kv_heads + head) * 2 * D + at;
      uint64_t lo = 0, hi = 0;
      if (finite) {
#pragma unroll
        for (int i = 0; i < kLeft; ++i) {
          lo |= (uint64_t)((uint32_t)outward(low[i], inv, false) & 255u) << (8 * i);
          hi |= (uint64_t)((uint32_t)outward(high[i], inv, true) & 255u) << (8 * i);
        }
      }
      typedef std::conditional_t<kLeft == 8, uint64_t, std::conditional_t<kLeft == 4, uint32_t, uint16_t>> Word;
      *reinterpret_cast<Word*>(out) = (Word)lo;
      *reinterpret_cast<Word*>(out + D) = (Word)hi;
    }
    if (lane == 0) scale[(int64_t)id * c.n_kv_heads + head] = (uint8_t)byte;
  }
}

template <int DT>
hipError_t bounds_dt(const KvView& c, int8_t* codes, uint8_t* scale, const int32_t* end, hipStream_t s) {
  // As many workgroups as run at once: 64 prompts 63 us and a step of 256
  // requests 6.3; half as many 75 and 5.8, twice as many 65 and 9.2.
  const unsigned grid = c.n_req <= kLine ? 1024u : (unsigned)c.n_req;
  if (c.head_dim == 64) kv_bounds_kernel<DT, 64><<<grid, kThreads, 0, s>>>(c, codes, scale, end);
  else if (c.head_dim == 128) kv_bounds_kernel<DT, 128><<<grid, kThreads, 0, s>>>(c, codes, scale, end);
  else kv_bounds_kernel<DT, 256><<<grid, kThreads, 0, s>>>(c, codes, scale, end);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_bounds(const KvView& c, int8_t* codes, uint8_t* scale, const int32_t* end, hipStream_t stream) {
  if (c.dtype == DFLASH_BF16) return bounds_dt<DFLASH_BF16>(c, codes, scale, end, stream);
  if (c.dtype == DFLASH_E4M3) return bounds_dt<DFLASH_E4M3>(c, codes, scale, end, stream);
  return bounds_dt<DFLASH_I8>(c, codes, scale, end, stream);
}

}  // namespace dflash
