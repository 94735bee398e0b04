// host_checks.h -- argument checks shared by the C entry points (host.cu, host_cache.cu).
#pragma once

#include "internal.h"

#define TA_EXPORT extern "C" __attribute__((visibility("default")))

namespace triattn {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline bool valid_dtype(int d) { return d == TA_F32 || d == TA_F16 || d == TA_BF16; }

inline int dtype_bytes(int d) { return d == TA_F32 ? 4 : (d == TA_E4M3 ? 1 : 2); }

// Head-dimension rules: 16-bit inputs D % 8 == 0 and D <= 256; fp32 D % 4 == 0 and D <= 256.
inline bool supported_d(int dtype, int D) {
    if (D > 256) return false;
    return dtype == TA_F32 ? (D % 4 == 0) : (D % 8 == 0);
}

}  // namespace triattn
