// What the attention kernels over a paged cache share: operands of the matrix
// instructions from codes, transposed reads, and joins across a wave's halves.
#pragma once

#include "kv_cache.h"

namespace dflash {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef int i32x2_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void lds_void_t;

// Lengths beyond this, or beyond the page table, have no positions: such a
// request takes one step, whatever its length claims to be, and is NaN.
constexpr int kMaxLen = 0x7fffffff - (1 << 17);

// Waits until at most N vector memory accesses are in flight.
template <int N>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
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

}  // namespace dflash
