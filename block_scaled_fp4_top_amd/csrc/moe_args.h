// Argument checks shared by the C entry points of the operators around the
// layer (sort, dispatch, combine, 8-bit integer products).
#pragma once

#include <stdarg.h>
#include <stdio.h>

#include "moe_internal.h"
#include "moe_kernels.h"

namespace moe {

inline int reject(int code, const char* fmt, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return report_error(code, buf);
}

inline int launched(hipError_t e, const char* where) {
    return e == hipSuccess ? MOE_OK : reject(MOE_ERR_HIP, "%s: %s", where, hipGetErrorString(e));
}

inline bool is_aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Whether two buffers share bytes (an empty one shares none).
inline bool overlap(const void* p, size_t n, const void* q, size_t m) {
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
    return p && q && n && m && a < b + m && b < a + n;
}

inline int dtype_bytes(int dtype) { return dtype == MOE_DT_FP32 ? 4 : 2; }
inline bool dtype_ok(int dtype) { return dtype >= MOE_DT_BF16 && dtype <= MOE_DT_FP32; }

// Bytes from a matrix's first element to behind its last one.
inline size_t extent(int64_t rows, int64_t stride, int64_t cols, int bytes) {
    return rows > 0 ? ((size_t)(rows - 1) * (size_t)stride + (size_t)cols) * (size_t)bytes : 0;
}

}  // namespace moe
