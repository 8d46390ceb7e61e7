// dr_host.h -- host-side helpers of the C ABI: the error text, argument spans
// and overlap checks (not part of the public interface).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "deltarule.h"

namespace dr {

// Sets the calling thread's error text and returns s.
dr_status fail(dr_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
inline bool valid_dtype(int x) { return x == DR_F32 || x == DR_BF16; }

// A tensor argument as a byte range (p may be NULL: an absent tensor).
struct Span {
    const void* p;
    size_t bytes;
    const char* name;
};

// Every output in `outs` must be disjoint from every input in `ins` and from
// the other outputs, except that output alias_out may be input alias_in
// exactly (the same address and size: the in-place state carry); any other
// overlap is an error.
dr_status check_disjoint(const Span* outs, int nout, const Span* ins, int nin, const void* alias_out = nullptr,
                         const void* alias_in = nullptr);

}  // namespace dr
