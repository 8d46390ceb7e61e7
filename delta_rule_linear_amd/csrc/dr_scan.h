// dr_scan.h -- the gated linear recurrence's kernels (dr_scan.hip forward and
// one token, dr_scan_bwd.hip the backward).
//
//   h_t = a_t h_{t-1} + c(a_t) x_t      a = e^g or sigmoid(g);  c = 1, 1 - a, sqrt(1 - a^2)
//
// a is carried in two parts, hi + lo, where it is near one: rounded to 24 bits it
// would be off by 2^-25, and a memory of 1 / (1 - a) tokens multiplies that.  1 - a
// is made directly (-expm1(g), sigmoid(-g)), and hi = 1 - (1 - a) rounded, lo what
// that left over.
#pragma once

#include <hip/hip_runtime.h>

#include "dr_device.h"
#include "dr_internal.h"
#include "dr_octet.h"
#include "dr_seqops.h"

namespace dr {

enum { kGsLog = 0, kGsLogit = 1 };
enum { kGsPlain = 0, kGsBlend = 1, kGsUnit = 2 };

struct GsFactor {
    float hi, lo;   // a
    float rest;     // 1 - a
};

template <int DEC>
__device__ __forceinline__ GsFactor gs_factor(float g) {
    constexpr float kLog2e = 1.44269504088896340736f;
    GsFactor o;
    bool near;
    float far;
    if constexpr (DEC == kGsLog) {
        // expm1 by its series where |g| < 0.4 (the next term, g^9 / 9!, is below
        // 2^-28 of g), else e^g - 1
        const float e = __builtin_amdgcn_exp2f(g * kLog2e);
        float q = 1.f / 40320.f;
        q = __builtin_fmaf(q, g, 1.f / 5040.f);
        q = __builtin_fmaf(q, g, 1.f / 720.f);
        q = __builtin_fmaf(q, g, 1.f / 120.f);
        q = __builtin_fmaf(q, g, 1.f / 24.f);
        q = __builtin_fmaf(q, g, 1.f / 6.f);
        q = __builtin_fmaf(q, g, 0.5f);
        near = __builtin_fabsf(g) < 0.4f;
        o.rest = near ? -__builtin_fmaf(g * g, q, g) : 1.f - e;
        far = e;
    } else {
        const float e = __builtin_amdgcn_exp2f(-kLog2e * __builtin_fabsf(g));
        const float big = __builtin_amdgcn_rcpf(1.f + e), little = e * big;
        near = g > 0.f;
        o.rest = near ? little : big;
        far = little;
        if (g != g) far = o.rest = g;
    }
    const float hi = 1.f - o.rest;
    o.hi = near ? hi : far;
    o.lo = near ? (1.f - hi) - o.rest : 0.f;
    return o;
}

// c(a), the factor of the input.
template <int INP>
__device__ __forceinline__ float gs_input(const GsFactor& f) {
    if constexpr (INP == kGsPlain) return 1.f;
    if constexpr (INP == kGsBlend) return f.rest;
    return __builtin_amdgcn_sqrtf(f.rest * (1.f + f.hi));
}

// a h + b
__device__ __forceinline__ float gs_apply(float hi, float lo, float h, float b) {
    return __builtin_fmaf(hi, h, __builtin_fmaf(lo, h, b));
}
// (hi, lo) <- a (hi, lo)
__device__ __forceinline__ void gs_times(float& hi, float& lo, float ahi, float alo) {
    const float p = hi * ahi;
    lo = __builtin_fmaf(hi, ahi, -p) + __builtin_fmaf(hi, alo, lo * ahi);
    hi = p;
}

// Eight values to and from LDS (32-byte aligned there).
__device__ __forceinline__ void gs_put(float* to, const float (&x)[8]) {
    reinterpret_cast<float4*>(to)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(to)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void gs_get(const float* from, float (&x)[8]) {
    const float4 a = reinterpret_cast<const float4*>(from)[0], b = reinterpret_cast<const float4*>(from)[1];
    x[0] = a.x;
    x[1] = a.y;
    x[2] = a.z;
    x[3] = a.w;
    x[4] = b.x;
    x[5] = b.y;
    x[6] = b.z;
    x[7] = b.w;
}

}  // namespace dr
