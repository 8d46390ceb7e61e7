// dr_rows.h -- host-side checks of strided row tensors, alignment and workspaces,
// shared by the entry points that take them (not part of the public interface).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "deltarule.h"
#include "dr_host.h"

namespace dr {

inline size_t elem_size(int dtype) { return dtype == DR_F32 ? 4 : 2; }

// A strided argument of n[0] x n[1] x n[2] rows of `d` channels.
struct Rows {
    const char* name;
    const void* p;
    dr_strides s;
    int64_t n[3];
    int64_t d;
    int dtype;
};

inline bool rows_empty(const Rows& r) { return r.n[0] == 0 || r.n[1] == 0 || r.n[2] == 0 || r.d == 0; }

// Strides: not negative, and (vec) whole 16-byte pieces.  A dimension of one
// has no stride.
inline dr_status check_strides(const Rows& r, bool vec) {
    const int64_t s[3] = {r.s.b, r.s.h, r.s.t};
    const int64_t unit = 16 / (int64_t)elem_size(r.dtype);
    for (int i = 0; i < 3; ++i) {
        if (r.n[i] <= 1) continue;
        if (s[i] < 0) return fail(DR_ERR_SHAPE, "%s has a negative stride (%lld)", r.name, (long long)s[i]);
        if (vec && s[i] % unit)
            return fail(DR_ERR_ALIGN, "%s: stride %lld is not a multiple of 16 bytes", r.name, (long long)s[i]);
        if (vec && i == 2 && s[i] > ((int64_t)1 << 23))
            return fail(DR_ERR_UNSUPPORTED, "%s: tokens %lld elements apart, at most 2^23 are supported", r.name,
                        (long long)s[i]);
        if (s[i] > ((int64_t)1 << 48) / (r.n[i] - 1))
            return fail(DR_ERR_SHAPE, "%s: stride %lld too large", r.name, (long long)s[i]);
    }
    return DR_OK;
}

// An output's rows must not share memory: taken by size, every stride reaches
// behind what the smaller ones cover.
inline dr_status check_rows_apart(const Rows& r) {
    if (rows_empty(r)) return DR_OK;
    int64_t s[3] = {r.s.b, r.s.h, r.s.t}, n[3] = {r.n[0], r.n[1], r.n[2]};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (s[j] < s[i]) {
                std::swap(s[i], s[j]);
                std::swap(n[i], n[j]);
            }
    int64_t extent = r.d;
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) continue;
        if (s[i] < extent) return fail(DR_ERR_UNSUPPORTED, "%s: its strides make rows overlap", r.name);
        extent += (n[i] - 1) * s[i];
    }
    return DR_OK;
}

inline Span rows_span(const Rows& r) {
    if (!r.p || rows_empty(r)) return {nullptr, 0, r.name};
    int64_t last = r.d;
    const int64_t s[3] = {r.s.b, r.s.h, r.s.t};
    for (int i = 0; i < 3; ++i)
        if (r.n[i] > 1) last += (r.n[i] - 1) * s[i];
    return {r.p, (size_t)last * elem_size(r.dtype), r.name};
}

inline dr_status check_workspace(size_t need, const void* ws, size_t bytes) {
    if (!need) return DR_OK;
    if (!ws) return fail(DR_ERR_WORKSPACE, "workspace is NULL, %zu bytes needed", need);
    if (bytes < need) return fail(DR_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", bytes, need);
    return DR_OK;
}

inline dr_status check_aligned(const Span* t, int n) {
    for (int i = 0; i < n; ++i)
        if (t[i].p && !aligned16(t[i].p)) return fail(DR_ERR_ALIGN, "%s is not 16-byte aligned", t[i].name);
    return DR_OK;
}

// Read and written one element at a time.
inline dr_status check_elements(const void* p, size_t elem, const char* name) {
    if ((uintptr_t)p % elem) return fail(DR_ERR_ALIGN, "%s is not %zu-byte aligned", name, elem);
    return DR_OK;
}

inline dr_status hip_status(hipError_t e, const char* what) {
    return e == hipSuccess ? DR_OK : fail(DR_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

}  // namespace dr
