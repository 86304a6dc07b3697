// Rows of K and V into and out of the paged cache, and the commit of an
// accepted path.
//
// All three are streams: write reads 2 (4) bytes an element and stores 1 or 2,
// read does the reverse, commit copies a few rows.  A wave holds 512
// elements, 8 to a lane: 8 (head_dim 64), 4 (128) or 2 (256) rows of
// consecutive tokens of one kv head, which are neighbours in a page, so its
// cache side is one contiguous run and its dense side whole 128- to 512-byte
// rows.  A thread finds its token's request, page and slot once and then
// takes kUnits (kv head, K or V) pairs, all loads issued before the first is
// used.
//
// Measured: 64 ragged prompts of up to 2048 rows, 8 heads of 128, bf16 into
// e4m3 (403 MB read and written) 74 us, 5.4 TB/s; 16 contexts of up to 8192
// back in bf16 (407 MB) 73 us, 5.6 TB/s; a copy of 2 GiB runs at 6.0.  The
// blocks of 32 requests are written in 3.1 us and a path is committed in 3.2,
// 256 requests' in 7.0: latency.
#include "kv_cache.h"

namespace dflash {
namespace {

constexpr int kThreads = 256;

struct RowPlace {
  int64_t page;
  int32_t slot;
};

// A lane's 8 elements of a row of LPR * 8: lane `part` takes 8 consecutive ones
// of a bf16 dense row, and of an fp32 one 4 in either half, so that each of
// its two 16-byte accesses is part of one run (int8 to fp32, 16 ragged
// requests of up to 4096 rows x 8 heads of 128: 71 to 78 us, with 8 consecutive
// 142; fp32 to e4m3, 64 of up to 1024: 70 us, with 8 consecutive 78).
template <int DENSE, int LPR>
__device__ __forceinline__ int first_of(int part) { return DENSE == DFLASH_F32 ? part * 4 : part * 8; }
template <int DENSE, int LPR>
__device__ __forceinline__ int second_of(int part) { return DENSE == DFLASH_F32 ? LPR * 4 + part * 4 : part * 8 + 4; }

// They are loaded from a dense row and widened to fp32.
template <int SRC, int LPR>
struct Eight;
template <int LPR>
struct Eight<DFLASH_BF16, LPR> {
  u32x4 w;
  __device__ __forceinline__ void load(const void* p, int64_t at, int part) { w = ld16_nt((const uint16_t*)p + at + part * 8); }
  __device__ __forceinline__ void get(float (&x)[8]) const { unpack16(w, x); }
};
template <int LPR>
struct Eight<DFLASH_F32, LPR> {
  u32x4 w0, w1;
  __device__ __forceinline__ void load(const void* p, int64_t at, int part) {
    w0 = ld16_nt((const float*)p + at + first_of<DFLASH_F32, LPR>(part));
    w1 = ld16_nt((const float*)p + at + second_of<DFLASH_F32, LPR>(part));
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    float a[4], b[4];
    unpack16(w0, a);
    unpack16(w1, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = a[i];
      x[4 + i] = b[i];
    }
  }
};

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
// Stores to the cache; NT passes the hardware's caches by.
template <bool NT, class T>
__device__ __forceinline__ void put(void* p, T v) {
  if constexpr (NT) __builtin_nontemporal_store(v, reinterpret_cast<T*>(p));
  else *reinterpret_cast<T*>(p) = v;
}

// LPR lanes of 8 elements hold one row.  grid.x covers the batch's rows,
// grid.y the (kv head, K or V) pairs in groups of UNITS.
template <int SRC, int DT, int LPR, int UNITS>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(KvView c, KvRows in) {
  constexpr int kRows = kThreads / LPR, kWaveRows = 64 / LPR;
  const int64_t t0 = (int64_t)blockIdx.x * kRows + (threadIdx.x >> 6) * kWaveRows;
  const int64_t t = t0 + (threadIdx.x & 63) / LPR;
  const int part = threadIdx.x % LPR;
  int32_t req = 0, slot = 0;
  int64_t pos = 0, page = 0;
  bool live = kv_row_position(c, t0, t, req, pos);
  if (live) live = kv_locate(c, c.table + req * c.table_stride, pos, page, slot);
  if (!live) return;                              // whole rows: the lanes of a row leave together
  const int units = 2 * c.n_kv_heads, u0 = blockIdx.y * UNITS;
  Eight<SRC, LPR> e[UNITS];
  // Large batches are not in the caches any more when they are read.  Whole
  // runs of 128 bytes and more pass them by (64 ragged prompts of up to 2048
  // rows x 8 heads of 128, e4m3 from bf16: 75 us, through them 82; bf16 103 and
  // 109), shorter ones would cost (64 int8: 23.5 and 22.2), and fp32 rows'
  // halves do not care (69.5 and 70.5).
  constexpr bool kNt = UNITS > 1 && SRC == DFLASH_BF16 && (DT == DFLASH_BF16 || LPR >= 16);
  const int first = first_of<SRC, LPR>(part), second = second_of<SRC, LPR>(part);
#pragma unroll
  for (int i = 0; i < UNITS; ++i) {
    const int u = min(u0 + i, units - 1), h = u >> 1;
    if (u & 1) e[i].load(in.v, t * in.v_row + h * in.v_head, part);
    else e[i].load(in.k, t * in.k_row + h * in.k_head, part);
  }
#pragma unroll
  for (int i = 0; i < UNITS; ++i) {
    const int u = u0 + i, h = u >> 1;
    if (u >= units) break;
    float x[8];
    e[i].get(x);
    const int64_t row = (int64_t)h * c.page_size + slot;
    unsigned char* page_at = ((u & 1) ? c.v : c.k) + page * c.page_bytes;
    if constexpr (DT == DFLASH_BF16) {
      if constexpr (SRC == DFLASH_BF16) {
        put<kNt>(page_at + (row * (LPR * 8) + first) * 2, e[i].w);   // no rounding: the bits as they are
      } else {
        u32x4 w;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = f32_to_bf16_rne(x[2 * j]) | (f32_to_bf16_rne(x[2 * j + 1]) << 16);
        put<kNt>(page_at + (row * (LPR * 8) + first) * 2, u32x2{w[0], w[1]});
        put<kNt>(page_at + (row * (LPR * 8) + second) * 2, u32x2{w[2], w[3]});
      }
    } else {
      // the largest magnitude by its bits, which order as the values do; an
      // infinity or NaN has the largest
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(x[j]) & 0x7fffffffu);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o, 64));
      const bool finite = top < 0x7f800000u;
      // 448 = 1.75 * 2^8, 127 = 1.984375 * 2^6: the carry out of the mantissa
      // takes the next exponent where amax's mantissa is above the type's top
      constexpr uint32_t carry = DT == DFLASH_E4M3 ? 0x1fffffu : 0x1ffffu;
      constexpr int down = DT == DFLASH_E4M3 ? 8 : 6;
      const int byte = finite ? max((int)((top + carry) >> 23) - down, 27) : 255;
      const float inv = finite ? __uint_as_float((uint32_t)(254 - byte) << 23) : 0.f;   // 2^-e
      uint32_t lo = 0, hi = 0;
      if (finite) {
        if constexpr (DT == DFLASH_E4M3) {
          int a = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * inv, x[1] * inv, 0, false);
          lo = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[2] * inv, x[3] * inv, a, true);
          int b = __builtin_amdgcn_cvt_pk_fp8_f32(x[4] * inv, x[5] * inv, 0, false);
          hi = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[6] * inv, x[7] * inv, b, true);
        } else {
          // adding 1.5 * 2^23 rounds to an integer, ties to even, whose two's
          // complement is then in the sum's low bits
          uint32_t r[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) r[j] = __float_as_uint(x[j] * inv + 12582912.f) & 255u;
          lo = r[0] | (r[1] << 8) | (r[2] << 16) | (r[3] << 24);
          hi = r[4] | (r[5] << 8) | (r[6] << 16) | (r[7] << 24);
        }
      }
      if constexpr (SRC == DFLASH_BF16) {
        put<kNt>(page_at + row * (LPR * 8) + first, u32x2{lo, hi});
      } else {
        put<kNt>(page_at + row * (LPR * 8) + first, lo);
        put<kNt>(page_at + row * (LPR * 8) + second, hi);
      }
      if (part == 0) ((u & 1) ? c.v_scale : c.k_scale)[page * c.scale_page_bytes + row] = (uint8_t)byte;
    }
  }
}

template <int DST, int DT, int LPR, int UNITS>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(KvView c, void* k_out, void* v_out) {
  constexpr int kRows = kThreads / LPR, kWaveRows = 64 / LPR, D = LPR * 8;
  const int64_t t0 = (int64_t)blockIdx.x * kRows + (threadIdx.x >> 6) * kWaveRows;
  const int64_t t = t0 + (threadIdx.x & 63) / LPR;
  const int part = threadIdx.x % LPR;
  int32_t req = 0, slot = 0;
  int64_t pos = 0, page = 0;
  if (!kv_row_position(c, t0, t, req, pos)) return;
  const bool held = kv_locate(c, c.table + req * c.table_stride, pos, page, slot);   // else page 0, slot 0 is read
  const int first = first_of<DST, LPR>(part), second = second_of<DST, LPR>(part);
  const int units = 2 * c.n_kv_heads, u0 = blockIdx.y * UNITS;
  u32x4 w[UNITS];
  uint32_t byte[UNITS];
#pragma unroll
  for (int i = 0; i < UNITS; ++i) {
    const int u = min(u0 + i, units - 1), h = u >> 1;
    const int64_t row = (int64_t)h * c.page_size + slot;
    const unsigned char* page_at = ((u & 1) ? c.v : c.k) + page * c.page_bytes;
    if constexpr (DT == DFLASH_BF16) {
      if constexpr (DST == DFLASH_BF16) {
        w[i] = ld16_nt(page_at + (row * D + first) * 2);
      } else {
        const u32x2 a = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(page_at + (row * D + first) * 2));
        const u32x2 b = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(page_at + (row * D + second) * 2));
        w[i] = u32x4{a[0], a[1], b[0], b[1]};
      }
      byte[i] = 127;
    } else {
      if constexpr (DST == DFLASH_BF16) {
        const u32x2 a = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(page_at + row * D + first));
        w[i][0] = a[0];
        w[i][1] = a[1];
      } else {
        w[i][0] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(page_at + row * D + first));
        w[i][1] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(page_at + row * D + second));
      }
      byte[i] = ((u & 1) ? c.v_scale : c.k_scale)[page * c.scale_page_bytes + row];
    }
  }
#pragma unroll
  for (int i = 0; i < UNITS; ++i) {
    const int u = u0 + i, h = u >> 1;
    if (u >= units) break;
    float x[8];
    if constexpr (DT == DFLASH_BF16) {
      unpack16(w[i], x);
    } else {
      const float scale = kv_scale_value(byte[i]);
      float a[4], b[4];
      unpack_codes<DT>(w[i][0], a);
      unpack_codes<DT>(w[i][1], b);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = a[j] * scale;
        x[4 + j] = b[j] * scale;
      }
    }
    if (!held) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = __builtin_nanf("");
    }
    const int64_t at = (t * c.n_kv_heads + h) * D;
    void* out = (u & 1) ? v_out : k_out;
    if constexpr (DST == DFLASH_BF16) {
      u32x4 o;
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = pack_bf16(x[2 * j], x[2 * j + 1]);
      if (DT == DFLASH_BF16 && held) o = w[i];    // no arithmetic: the bits as they are
      st16_nt((uint16_t*)out + at + first, o);
    } else {
      st16_nt((float*)out + at + first, u32x4{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])});
      st16_nt((float*)out + at + second, u32x4{__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7])});
    }
  }
}

// One wave moves one (request, kv head, K or V): CPR lanes of 16 bytes hold a
// row, 64 / CPR path entries go at a time, all loaded before any is stored.
// In place that is safe: a later entry's source start + paths[i] >= start + i
// lies behind every destination of the entries before it.
template <int CPR>
__global__ void __launch_bounds__(kThreads) kv_commit_kernel(KvView c, const int32_t* paths, int64_t path_stride,
                                                             int32_t path_width, const int32_t* path_lens) {
  constexpr int kRows = 64 / CPR;
  const int lane = threadIdx.x & 63, part = lane % CPR, units = 2 * c.n_kv_heads;
  const int64_t job = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  if (job >= (int64_t)c.n_req * units) return;
  const int32_t req = (int32_t)(job / units), u = (int32_t)(job - (int64_t)req * units), h = u >> 1;
  const int n = min(path_lens[req], path_width);
  const int64_t start = c.start[req];
  const int32_t* table = c.table + req * c.table_stride;
  unsigned char* base = (u & 1) ? c.v : c.k;
  uint8_t* scales = (u & 1) ? c.v_scale : c.k_scale;
  for (int i0 = 0; i0 < n; i0 += kRows) {
    const int i = i0 + lane / CPR;
    int64_t from = 0, to = 0;
    int32_t from_slot = 0, to_slot = 0;
    bool live = i < n;
    if (live) {
      const int32_t node = paths[req * path_stride + i];
      live = node > i && kv_locate(c, table, start + node, from, from_slot) &&
             kv_locate(c, table, start + i, to, to_slot);
    }
    u32x4 w = {0, 0, 0, 0};
    uint8_t s = 0;
    const int64_t src = (int64_t)h * c.page_size + from_slot, dst = (int64_t)h * c.page_size + to_slot;
    if (live) {
      w = ld16(base + from * c.page_bytes + src * (CPR * 16) + part * 16);
      if (scales && part == 0) s = scales[from * c.scale_page_bytes + src];
    }
    __builtin_amdgcn_s_waitcnt(0);                // every lane's loads are done before any lane stores
    asm volatile("" ::: "memory");
    if (live) {
      st16(base + to * c.page_bytes + dst * (CPR * 16) + part * 16, w);
      if (scales && part == 0) scales[to * c.scale_page_bytes + dst] = s;
    }
    asm volatile("" ::: "memory");
  }
}

// (kv head, K or V) pairs per thread: 4 keep enough loads in flight for the
// stream (64 ragged prompts into e4m3: 75 us, with 2 93, with 1 137, with 8
// 76; read back 74, 90, 162, 73); 1 where the batch is too small to fill the
// chip with 4 (32 blocks of 16: 3.5 us, with 4 4.1).
inline int units_for(int64_t n_rows, int lpr, int n_kv_heads) {
  const int64_t wgs = (n_rows * lpr + kThreads - 1) / kThreads * ((2 * n_kv_heads + 3) / 4);
  return wgs >= 1024 ? 4 : 1;
}

template <int SRC, int DT, int LPR>
hipError_t write_lpr(const KvView& c, const KvRows& in, hipStream_t s) {
  const unsigned gx = (unsigned)((c.n_rows * LPR + kThreads - 1) / kThreads);
  const unsigned units = 2u * c.n_kv_heads;
  if (units_for(c.n_rows, LPR, c.n_kv_heads) == 4)
    kv_write_kernel<SRC, DT, LPR, 4><<<dim3(gx, (units + 3) / 4), kThreads, 0, s>>>(c, in);
  else
    kv_write_kernel<SRC, DT, LPR, 1><<<dim3(gx, units), kThreads, 0, s>>>(c, in);
  return hipGetLastError();
}
template <int SRC, int DT>
hipError_t write_dt(const KvView& c, const KvRows& in, hipStream_t s) {
  if (c.head_dim == 64) return write_lpr<SRC, DT, 8>(c, in, s);
  if (c.head_dim == 128) return write_lpr<SRC, DT, 16>(c, in, s);
  return write_lpr<SRC, DT, 32>(c, in, s);
}
template <int SRC>
hipError_t write_src(const KvView& c, const KvRows& in, hipStream_t s) {
  if (c.dtype == DFLASH_BF16) return write_dt<SRC, DFLASH_BF16>(c, in, s);
  if (c.dtype == DFLASH_E4M3) return write_dt<SRC, DFLASH_E4M3>(c, in, s);
  return write_dt<SRC, DFLASH_I8>(c, in, s);
}

template <int DST, int DT, int LPR>
hipError_t read_lpr(const KvView& c, void* k, void* v, hipStream_t s) {
  const unsigned gx = (unsigned)((c.n_rows * LPR + kThreads - 1) / kThreads);
  const unsigned units = 2u * c.n_kv_heads;
  if (units_for(c.n_rows, LPR, c.n_kv_heads) == 4)
    kv_read_kernel<DST, DT, LPR, 4><<<dim3(gx, (units + 3) / 4), kThreads, 0, s>>>(c, k, v);
  else
    kv_read_kernel<DST, DT, LPR, 1><<<dim3(gx, units), kThreads, 0, s>>>(c, k, v);
  return hipGetLastError();
}
template <int DST, int DT>
hipError_t read_dt(const KvView& c, void* k, void* v, hipStream_t s) {
  if (c.head_dim == 64) return read_lpr<DST, DT, 8>(c, k, v, s);
  if (c.head_dim == 128) return read_lpr<DST, DT, 16>(c, k, v, s);
  return read_lpr<DST, DT, 32>(c, k, v, s);
}
template <int DST>
hipError_t read_dst(const KvView& c, void* k, void* v, hipStream_t s) {
  if (c.dtype == DFLASH_BF16) return read_dt<DST, DFLASH_BF16>(c, k, v, s);
  if (c.dtype == DFLASH_E4M3) return read_dt<DST, DFLASH_E4M3>(c, k, v, s);
  return read_dt<DST, DFLASH_I8>(c, k, v, s);
}

}  // namespace

hipError_t launch_kv_write(const KvView& c, const KvRows& in, hipStream_t stream) {
  return in.dtype == DFLASH_BF16 ? write_src<DFLASH_BF16>(c, in, stream) : write_src<DFLASH_F32>(c, in, stream);
}

hipError_t launch_kv_read(const KvView& c, void* k_out, void* v_out, int32_t dtype, hipStream_t stream) {
  return dtype == DFLASH_BF16 ? read_dst<DFLASH_BF16>(c, k_out, v_out, stream)
                              : read_dst<DFLASH_F32>(c, k_out, v_out, stream);
}

hipError_t launch_kv_commit(const KvView& c, const int32_t* paths, int64_t path_stride, int32_t path_width,
                            const int32_t* path_lens, hipStream_t stream) {
  const int64_t jobs = (int64_t)c.n_req * 2 * c.n_kv_heads;
  const unsigned g = (unsigned)((jobs + kThreads / 64 - 1) / (kThreads / 64));
  const int row_bytes = c.head_dim * (c.dtype == DFLASH_BF16 ? 2 : 1);
  switch (row_bytes) {
    case 64: kv_commit_kernel<4><<<g, kThreads, 0, stream>>>(c, paths, path_stride, path_width, path_lens); break;
    case 128: kv_commit_kernel<8><<<g, kThreads, 0, stream>>>(c, paths, path_stride, path_width, path_lens); break;
    case 256: kv_commit_kernel<16><<<g, kThreads, 0, stream>>>(c, paths, path_stride, path_width, path_lens); break;
    default: kv_commit_kernel<32><<<g, kThreads, 0, stream>>>(c, paths, path_stride, path_width, path_lens); break;
  }
  return hipGetLastError();
}

}  // namespace dflash
