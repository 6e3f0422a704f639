// Host-side argument checks shared by the C ABI's source files.
#pragma once

#include "common.h"

namespace staple {

inline int elem_bytes(int32_t dt) { return dt == STAPLE_BF16 ? 2 : 4; }
inline bool valid_dtype(int32_t dt) { return dt == STAPLE_BF16 || dt == STAPLE_F32; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline hipStream_t S(void* s) { return static_cast<hipStream_t>(s); }

}  // namespace staple

#define REQUIRE(cond)                                   \
  do {                                                  \
    if (!(cond)) return STAPLE_ERR_INVALID_ARGUMENT;    \
  } while (0)

#define HIPCALL(expr)                                   \
  do {                                                  \
    if ((expr) != hipSuccess) return STAPLE_ERR_HIP;    \
  } while (0)

#define GET_ERR(var)                                    \
  int* var = device_error_word();                       \
  if (var == nullptr) return STAPLE_ERR_HIP
