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

// Routes, rows of a quantizer, rows of a product: a launch has at most 2^32
// threads, of which a row may take 256.
constexpr int64_t kMaxRows = 1 << 23;

// `rows` pieces of `width` bytes, `stride` bytes apart.
struct Bytes {
    const void* p;
    int64_t rows, stride, width;
};
inline Bytes flat(const void* p, int64_t n) { return Bytes{p, 1, 0, n}; }
inline Bytes matrix(const void* p, int64_t rows, int64_t stride, int64_t cols, int bytes) {
    return Bytes{p, rows, stride * bytes, cols * bytes};
}

// Whether two buffers share bytes (an empty one shares none). Columns of one
// matrix that lie apart do not; other buffers whose extents cross are taken to.
inline bool overlap(const Bytes& a, const Bytes& b) {
    if (!a.p || !b.p || a.rows < 1 || b.rows < 1 || a.width < 1 || b.width < 1) return false;
    const uintptr_t p = (uintptr_t)a.p, q = (uintptr_t)b.p;
    if (p >= q + (uintptr_t)((b.rows - 1) * b.stride + b.width) || q >= p + (uintptr_t)((a.rows - 1) * a.stride + a.width))
        return false;
    const int64_t s = a.rows > 1 ? a.stride : b.stride;
    if (s > 0 && (a.rows == 1 || a.stride == s) && (b.rows == 1 || b.stride == s)) {
        const int64_t d = (((int64_t)(q - p)) % s + s) % s;  // column of b's rows in a's
        return !(d >= a.width && d + b.width <= s);
    }
    return true;
}

inline int dtype_bytes(int dtype) { return dtype == MOE_DT_FP32 ? 4 : 2; }
inline bool dtype_ok(int dtype) { return dtype >= MOE_DT_BF16 && dtype <= MOE_DT_FP32; }

}  // namespace moe
