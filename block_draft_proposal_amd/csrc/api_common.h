// What the files of the C ABI share: the calling thread's error string and
// the checks every entry point makes.  Defined in api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "dflash.h"

namespace dflash {

// Sets the calling thread's error message and returns `code`.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears it and returns DFLASH_OK.
int ok();
int launch_status(hipError_t e, const char* what);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int elem_bytes(int32_t dtype) { return dtype == DFLASH_BF16 ? 2 : 4; }
inline bool dtype_ok(int32_t dtype) { return dtype == DFLASH_F32 || dtype == DFLASH_BF16; }
inline hipStream_t as_hip(dflash_stream_t s) { return reinterpret_cast<hipStream_t>(s); }
inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

}  // namespace dflash
