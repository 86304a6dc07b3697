// The least and the greatest key of each channel of the pages that have become
// full, 8 bits outwards.
//
// A wave takes one (page, kv head): its rows are one contiguous run, of which
// a lane reads 16 bytes of every (64 / lanes of a row)-th row and keeps the
// extremes of its channels in registers; lanes of the same channels join at the
// end.  The keys are read once and the kernel is bound by that stream.
#include <algorithm>

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

template <int DT, int D>
__global__ void __launch_bounds__(kThreads) kv_bounds_kernel(KvView c, int8_t* codes, uint8_t* scale, const int32_t* end, int parts) {
  constexpr int kRB = D * (DT == DFLASH_BF16 ? 2 : 1), kLanes = kRB / 16, kRows = 64 / kLanes, kN = Sixteen<DT>::kN;
  constexpr int kBatch = 4;                       // loads of a lane in flight
  const int lane = threadIdx.x & 63, part = lane % kLanes, sub = lane / kLanes;
  const int req = blockIdx.x / parts, slice = blockIdx.x - req * parts;
  const int32_t from = max(c.start[req], 0), to = end[req];
  if (to <= from) return;
  const int32_t first = kv_blocks(c, from), count = kv_blocks(c, to) - first;
  const int64_t tasks = (int64_t)count * c.n_kv_heads;
  const int32_t* table = c.table + req * c.table_stride;
  for (int64_t task = (int64_t)slice * (kThreads / 64) + (threadIdx.x >> 6); task < tasks; task += (int64_t)parts * (kThreads / 64)) {
    const int32_t b = (int32_t)(task / c.n_kv_heads), head = (int32_t)(task - (int64_t)b * c.n_kv_heads);
    const int32_t id = table[first + b];
    if (id < 0 || id >= c.n_pages) continue;
    const unsigned char* rows = c.k + (int64_t)id * c.page_bytes + (int64_t)head * c.page_size * kRB + part * 16;
    const uint8_t* row_scale = DT == DFLASH_BF16 ? nullptr : c.k_scale + (int64_t)id * c.scale_page_bytes + (int64_t)head * c.page_size;
    float low[kN], high[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      low[i] = INFINITY;
      high[i] = -INFINITY;
    }
    uint32_t top = 0;                             // the largest magnitude's bits; of an infinity or NaN the largest of all
    for (int r0 = sub; r0 < c.page_size; r0 += kRows * kBatch) {
      u32x4 w[kBatch];
      uint32_t byte[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {          // past the page's end the last row once more
        const int r = min(r0 + i * kRows, c.page_size - 1);
        w[i] = ld16_nt(rows + (int64_t)r * kRB);
        byte[i] = DT == DFLASH_BF16 ? 127 : row_scale[r];
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        float x[kN];
        Sixteen<DT>::get(w[i], DT == DFLASH_BF16 ? 1.f : kv_scale_value(byte[i]), x);
#pragma unroll
        for (int j = 0; j < kN; ++j) {
          low[j] = fminf(low[j], x[j]);
          high[j] = fmaxf(high[j], x[j]);
          top = max(top, __float_as_uint(x[j]) & 0x7fffffffu);
        }
      }
    }
#pragma unroll
    for (int o = kLanes; o < 64; o <<= 1)
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        low[i] = fminf(low[i], __shfl_xor(low[i], o, 64));
        high[i] = fmaxf(high[i], __shfl_xor(high[i], o, 64));
      }
    top = wave_max_u32(top);
    const bool finite = top < 0x7f800000u;
    // 127 = 1.984375 * 2^6: the carry out of the mantissa takes the next
    // exponent where the largest magnitude's mantissa is above that
    const uint32_t byte = finite ? (uint32_t)max((int)((top + 0x1ffffu) >> 23) - 6, 27) : 255u;
    const float inv = __uint_as_float((254u - min(byte, 253u)) << 23);
    if (sub == 0) {
      uint32_t lo[kN / 4], hi[kN / 4];
#pragma unroll
      for (int i = 0; i < kN / 4; ++i) {
        lo[i] = hi[i] = 0;
        if (finite) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            lo[i] |= ((uint32_t)outward(low[4 * i + j], inv, false) & 255u) << (8 * j);
            hi[i] |= ((uint32_t)outward(high[4 * i + j], inv, true) & 255u) << (8 * j);
          }
        }
      }
      uint32_t* out = reinterpret_cast<uint32_t*>(codes + ((int64_t)id * c.n_kv_heads + head) * 2 * D) + part * (kN / 4);
#pragma unroll
      for (int i = 0; i < kN / 4; ++i) {
        out[i] = lo[i];
        out[D / 4 + i] = hi[i];
      }
    }
    if (lane == 0) scale[(int64_t)id * c.n_kv_heads + head] = (uint8_t)byte;
  }
}

template <int DT>
hipError_t bounds_dt(const KvView& c, int8_t* codes, uint8_t* scale, const int32_t* end, hipStream_t s) {
  // workgroups to a request: enough for the chip where there are few of them,
  // and no more than the table's pages can use
  const int64_t tasks = (int64_t)c.table_width * c.n_kv_heads;
  const int parts = (int)std::max<int64_t>(1, std::min<int64_t>((tasks + kThreads / 64 - 1) / (kThreads / 64), 4096 / c.n_req));
  const unsigned grid = (unsigned)c.n_req * (unsigned)parts;
  if (c.head_dim == 64) kv_bounds_kernel<DT, 64><<<grid, kThreads, 0, s>>>(c, codes, scale, end, parts);
  else if (c.head_dim == 128) kv_bounds_kernel<DT, 128><<<grid, kThreads, 0, s>>>(c, codes, scale, end, parts);
  else kv_bounds_kernel<DT, 256><<<grid, kThreads, 0, s>>>(c, codes, scale, end, parts);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_bounds(const KvView& c, int8_t* codes, uint8_t* scale, const int32_t* end, hipStream_t stream) {
  if (c.dtype == DFLASH_BF16) return bounds_dt<DFLASH_BF16>(c, codes, scale, end, stream);
  if (c.dtype == DFLASH_E4M3) return bounds_dt<DFLASH_E4M3>(c, codes, scale, end, stream);
  return bounds_dt<DFLASH_I8>(c, codes, scale, end, stream);
}

}  // namespace dflash
