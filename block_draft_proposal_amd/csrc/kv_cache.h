// The paged KV cache as the kernels see it: row addressing, the 8-bit number
// formats and the host-side launchers of the operators on it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "dflash_kv.h"

namespace dflash {

// t / d for 0 <= t < 2^31 and 1 <= d <= 2^16, as one 32 x 32 -> 64 product:
// with l = ceil(log2 d) and mul = ceil(2^(31 + l) / d) < 2^32, the quotient is
// floor(t mul / 2^(31 + l)) exactly (mul d exceeds 2^(31 + l) by less than
// d <= 2^l, which t < 2^31 cannot carry past the next multiple).
struct FastDiv {
  uint32_t mul = 0;
  int32_t shift = 0, d = 1;
  __host__ static FastDiv make(int32_t d) {
    int l = 0;
    while ((1 << l) < d) ++l;
    FastDiv f;
    f.shift = 31 + l;
    f.mul = (uint32_t)((((uint64_t)1 << f.shift) + (uint64_t)d - 1) / (uint64_t)d);
    f.d = d;
    return f;
  }
  __host__ __device__ int32_t div(int32_t t) const { return (int32_t)(((uint64_t)(uint32_t)t * mul) >> shift); }
};

struct KvView {
  unsigned char* k;
  unsigned char* v;
  uint8_t* k_scale;
  uint8_t* v_scale;
  int64_t page_bytes;         // from a page to the next
  int64_t scale_page_bytes;
  int64_t n_pages;
  int32_t page_size, n_kv_heads, head_dim, dtype;
  FastDiv per_page;           // division by page_size
  const int32_t* table;
  int64_t table_stride;
  int32_t table_width, n_req;
  const int32_t* start;
  const int32_t* offsets;
  int64_t n_rows;
};

// Page and slot of position pos of a request whose table row is `row`; false
// (and no read past the table) where the position has no page in the pool.
__device__ __forceinline__ bool kv_locate(const KvView& c, const int32_t* row, int64_t pos, int64_t& page,
                                          int32_t& slot) {
  page = 0;
  slot = 0;
  if (pos < 0 || pos > 0x7fffffff) return false;
  const int32_t idx = c.per_page.div((int32_t)pos);
  if (idx >= c.table_width) return false;
  const int32_t id = row[idx];
  if (id < 0 || id >= c.n_pages) return false;
  page = id;
  slot = (int32_t)pos - idx * c.page_size;
  return true;
}

// The request that row t of a ragged batch belongs to and the row's position;
// false for padding.  t0 is the first row of the wave (uniform): a 64-ary
// search of offsets finds its request, two steps for up to 4096 requests, and
// later rows of the wave walk on from there.
__device__ __forceinline__ bool kv_row_position(const KvView& c, int64_t t0, int64_t t, int32_t& req, int64_t& pos) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = c.n_req;                       // the largest r in [lo, lo + n) with offsets[r] <= t0
  while (n > 1) {
    const int step = (n + 63) >> 6;
    const int r = lo + lane * step;
    const bool at_or_before = lane * step < n && c.offsets[r] <= t0;
    const uint64_t b = __ballot(at_or_before);
    const int i = b ? 63 - __builtin_clzll(b) : 0;
    n = min(step, n - i * step);
    lo += i * step;
  }
  req = lo;
  if (t >= c.n_rows) return false;
  int64_t first = c.offsets[req], end = c.offsets[req + 1];
  while (t >= end && req + 1 < c.n_req) {
    ++req;
    first = end;
    end = c.offsets[req + 1];
  }
  if (t < first || t >= end) return false;
  pos = (int64_t)c.start[req] + (t - first);
  return true;
}

// A scale byte's value: 2^(b - 127), NaN for 255 (b = 0: 2^-127, subnormal).
__device__ __forceinline__ float kv_scale_value(uint32_t b) {
  const uint32_t bits = b == 255u ? 0x7fc00000u : b == 0u ? 0x00400000u : b << 23;
  return __uint_as_float(bits);
}

// Two fp32 as packed bf16, each rounded to nearest even (a lower in the word).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{a, b}), bf16x2_t));
}

// The 4 elements of a word of e4m3 or int8 codes.
template <int DT>
__device__ __forceinline__ void unpack_codes(uint32_t w, float (&o)[4]) {
  if constexpr (DT == DFLASH_E4M3) {
    o[0] = __builtin_amdgcn_cvt_f32_fp8((int)w, 0);
    o[1] = __builtin_amdgcn_cvt_f32_fp8((int)w, 1);
    o[2] = __builtin_amdgcn_cvt_f32_fp8((int)w, 2);
    o[3] = __builtin_amdgcn_cvt_f32_fp8((int)w, 3);
  } else {
    o[0] = (float)(int8_t)(w & 255u);
    o[1] = (float)(int8_t)((w >> 8) & 255u);
    o[2] = (float)(int8_t)((w >> 16) & 255u);
    o[3] = (float)(int8_t)(w >> 24);
  }
}

// ---------------------------------------------------------------------------
// Host-side launchers (each returns hipSuccess or the launch error)
// ---------------------------------------------------------------------------
struct KvRows {               // strided rows of K and V outside the cache
  const void* k;
  const void* v;
  int64_t k_row, k_head, v_row, v_head;   // strides in elements
  int32_t dtype;
};
hipError_t launch_kv_write(const KvView& c, const KvRows& in, hipStream_t stream);
hipError_t launch_kv_read(const KvView& c, void* k_out, void* v_out, int32_t dtype, hipStream_t stream);
hipError_t launch_kv_commit(const KvView& c, const int32_t* paths, int64_t path_stride, int32_t path_width,
                            const int32_t* path_lens, hipStream_t stream);

struct TreeArgs {
  KvView c;
  const uint16_t* q;
  int64_t q_row, q_head;      // strides in elements
  int32_t n_q_heads;
  const uint64_t* mask;       // null: a chain
  int32_t mask_words, max_nodes;
  float scale;
  uint16_t* out;
  void* workspace;
};
size_t tree_attention_bytes(const KvView& c, int32_t n_req, int32_t max_nodes, int32_t n_q_heads);
hipError_t launch_tree_attention(const TreeArgs& a, hipStream_t stream);

}  // namespace dflash
