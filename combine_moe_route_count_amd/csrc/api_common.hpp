// api_common.hpp - what the C ABI layers (api.cpp, api_train.cpp,
// api_experts.cpp) share: the calling thread's last error, workspace carving and the
// checks of buffers.
// Not part of the public ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "moe_route.h"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace moe {

// Records the calling thread's last error (moe_last_error) and returns status.
int fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
inline int hip_fail(hipError_t e, const char* where) {
    return fail(MOE_ERR_HIP, "%s: %s", where, hipGetErrorString(e));
}

constexpr int64_t kMaxRows = INT32_MAX;

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

inline bool quantized(moe_dtype d) { return d == MOE_FP8_E4M3 || d == MOE_FP4_E2M1; }

// Workspace carving: 256-byte aligned pieces, one after the other.
struct Carve {
    size_t total = 0;
    size_t take(size_t bytes) {
        const size_t at = total;
        total += align256(bytes);
        return at;
    }
};

int check_ws(void* ws, size_t ws_bytes, size_t need);
int check_rows_ptr(const void* p, int64_t rows, const char* name);
int check_H(int64_t H, bool quantized_rows);

inline bool is_float(moe_dtype d) { return d == MOE_BF16 || d == MOE_F32; }

inline int64_t float_bytes(moe_dtype d) { return d == MOE_F32 ? 4 : 2; }

inline int check_float(moe_dtype d, const char* name) {
    if (is_float(d)) return MOE_OK;
    return fail(MOE_ERR_INVALID_ARG, "%s dtype must be MOE_BF16 or MOE_F32", name);
}

inline int check_elems(const void* p, int64_t n, size_t align, const char* name) {
    if (n > 0 && !p) return fail(MOE_ERR_INVALID_ARG, "%s is NULL", name);
    if (p && !aligned(p, align))
        return fail(MOE_ERR_INVALID_ARG, "%s is not %zu-byte aligned", name, align);
    return MOE_OK;
}

// out and in must not share bytes.
inline int check_apart(const void* out, int64_t out_bytes, const char* out_name, const void* in,
                int64_t in_bytes, const char* in_name) {
    if (!out || !in || out_bytes <= 0 || in_bytes <= 0) return MOE_OK;
    const uintptr_t a = (uintptr_t)out, b = (uintptr_t)in;
    if (a < b + (uintptr_t)in_bytes && b < a + (uintptr_t)out_bytes)
        return fail(MOE_ERR_INVALID_ARG, "%s overlaps %s", out_name, in_name);
    return MOE_OK;
}

inline int check_row_count(int64_t rows, const char* name) {
    if (rows < 0 || rows > kMaxRows)
        return fail(MOE_ERR_INVALID_ARG, "%s must be in [0, 2^31-1]", name);
    return MOE_OK;
}

}  // namespace moe

#define MOE_TRY(expr)                 \
    do {                              \
        const int st_ = (expr);       \
        if (st_ != MOE_OK) return st_; \
    } while (0)

#define MOE_HIP(expr, where)                  \
    do {                                      \
        const hipError_t e_ = (expr);         \
        if (e_ != hipSuccess) return moe::hip_fail(e_, where); \
    } while (0)
