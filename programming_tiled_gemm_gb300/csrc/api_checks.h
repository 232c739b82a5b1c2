// Argument checks that the entry points of the linear layers and of what stands around them share
// (not installed).
#pragma once

#include "internal.h"

namespace gemm_gb300 {

constexpr int64_t kLim32 = 0x7fffffffLL - 1024;  // the kernels index sizes in 32 bits

inline bool is_16(int dtype) { return dtype == GEMM_BF16 || dtype == GEMM_F16; }
inline int size_of(int dtype) { return dtype == GEMM_F32 ? 4 : 2; }
inline bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// A matrix of `rows` rows of `cols` used elements: null or a leading dimension below the
// row's length is refused, unless there is nothing to access.
inline bool bad_matrix(const void* p, int64_t rows, int64_t cols, int64_t ld)
{
    if (rows == 0 || cols == 0) return false;
    return !p || ld < cols || ld > kLim32;
}

// TMA and 16-byte vector operands: aligned base, row stride a multiple of 16 bytes.
inline bool bad_rows16(const void* p, int64_t rows, int64_t cols, int64_t ld)
{
    return rows > 0 && cols > 0 && (misaligned(p, 16) || ld % 8 != 0);
}

inline bool known_dtype(int d) { return d == GEMM_F32 || is_16(d); }

// Logs a refusal.
inline int told(const char* what, int rc)
{
    if (rc != GEMM_OK) glog("%s refused: %s (%d)", what, gemm_status_string(rc), rc);
    return rc;
}

}  // namespace gemm_gb300
