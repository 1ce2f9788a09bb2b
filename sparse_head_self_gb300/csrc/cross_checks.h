// What the C ABI's files share: messages and the checks of arguments that several
// calls have.
#pragma once

#include <cstdarg>
#include <cstdio>
#include <string>

#include "cross.h"

namespace fibatt {

inline std::string fmt(const char *f, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, f);
    vsnprintf(buf, sizeof buf, f, ap);
    va_end(ap);
    return buf;
}

inline fibatt_status invalid(const std::string &m) { return set_error(FIBATT_ERR_INVALID_ARG, m); }
inline fibatt_status unsupported(const std::string &m) { return set_error(FIBATT_ERR_UNSUPPORTED, m); }
inline bool off(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

inline fibatt_status check_type(int D, fibatt_dtype t) {
    if (D != kHeadDim) return unsupported(fmt("head dim %d unsupported (only %d)", D, kHeadDim));
    if (t != FIBATT_F32 && t != FIBATT_BF16) return unsupported(fmt("unknown dtype %d", (int)t));
    return FIBATT_OK;
}

inline fibatt_status check_ptr(const void *p, const char *name, size_t a = 16) {
    if (!p) return invalid(fmt("%s is NULL", name));
    if (off(p, a)) return invalid(fmt("%s is not %zu-byte aligned", name, a));
    return FIBATT_OK;
}

inline int64_t size_of(fibatt_dtype t) { return t == FIBATT_F32 ? 4 : 2; }

// A head tensor of B sequences, H heads and N rows; `out`: the call writes it.
inline fibatt_status check_heads(const fibatt_heads *v, const char *name, fibatt_dtype t, int B, int H, int N, bool out) {
    if (!v) return invalid(fmt("%s is NULL", name));
    if (fibatt_status st = check_ptr(v->ptr, name)) return st;
    const int64_t strides[3] = {v->stride_b, v->stride_h, v->stride_n};
    const int sizes[3] = {B, H, N};
    for (int i = 0; i < 3; ++i) {
        if (strides[i] < 0 || strides[i] > (int64_t)1 << 38 || strides[i] * size_of(t) % 16)
            return invalid(fmt("%s: stride %lld is not a multiple of 16 bytes in [0, 2^38]", name, (long long)strides[i]));
        if (i == 2 && N > 1 && strides[i] == 0) return invalid(fmt("%s: rows with a stride of 0", name));
        if (out && sizes[i] > 1 && strides[i] < kHeadDim)
            return invalid(fmt("%s is written, but a stride of %lld lets its rows overlap", name, (long long)strides[i]));
    }
    return FIBATT_OK;
}

}  // namespace fibatt
