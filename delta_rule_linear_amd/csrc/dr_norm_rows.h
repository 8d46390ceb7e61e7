// dr_norm_rows.h -- what the norms' kernels share: sums over the lanes of a row, the
// statistics' divisions and roots, and where a row is.
#pragma once

#include <hip/hip_runtime.h>

#include "dr_device.h"
#include "dr_layernorm.h"

namespace dr {

constexpr int kLnThreads = 256;

// Sums of two values over the lanes of a row, in every one of them.  Rows of
// several waves add their waves' sums through LDS; `turn` alternates between two
// places, so that one barrier a time is enough.
template <int LPR>
__device__ __forceinline__ void ln_sum2(float& x, float& y, float2* red, int& turn) {
    x = group_sum<(LPR < 32 ? LPR : 32)>(x);
    y = group_sum<(LPR < 32 ? LPR : 32)>(y);
    if constexpr (LPR >= 64) {
        x += __shfl_xor(x, 32);
        y += __shfl_xor(y, 32);
    }
    if constexpr (LPR > 64) {
        const int wave = threadIdx.x >> 6;
        float2* at = red + 4 * turn;
        turn ^= 1;
        if ((threadIdx.x & 63) == 0) at[wave] = make_float2(x, y);
        __syncthreads();
        if constexpr (LPR == 128) {
            const float2 p = at[wave & ~1], q = at[wave | 1];
            x = p.x + q.x;
            y = p.y + q.y;
        } else {
            x = (at[0].x + at[1].x) + (at[2].x + at[3].x);
            y = (at[0].y + at[1].y) + (at[2].y + at[3].y);
        }
    }
}
template <int LPR>
__device__ __forceinline__ float ln_sum(float x, float2* red, int& turn) {
    float y = 0.f;
    ln_sum2<LPR>(x, y, red, turn);
    return x;
}

// s / D to the nearest (one correction of s times the rounded 1 / D), so that a
// row of one value has that value as its mean.
__device__ __forceinline__ float ln_div(float s, float D, float inv) {
    const float q = s * inv;
    const float c = __builtin_fmaf(__builtin_fmaf(-q, D, s), inv, q);
    return __builtin_isfinite(q) ? c : q;
}
// 1 / sqrt(v): the hardware's estimate and one Newton step; zero, infinity, NaN
// and values whose products would be subnormal take the plain form.
__device__ __forceinline__ float ln_rsqrt(float v) {
    if (!(v > 1e-30f && v < 1e30f)) return 1.f / sqrtf(v);
    const float y = __builtin_amdgcn_rsqf(v);
    return y * __builtin_fmaf(-0.5f * v * y, y, 1.5f);
}

// Row r of a group.
template <typename Args>
__device__ __forceinline__ void ln_row(const Args& a, unsigned g, unsigned r, unsigned& b, unsigned& h, unsigned& l) {
    const unsigned q = r / (unsigned)a.L;
    l = r - q * (unsigned)a.L;
    if (a.per_head) {
        b = q;
        h = g;
    } else {
        b = q / (unsigned)a.H;
        h = q - b * (unsigned)a.H;
    }
}
__device__ __forceinline__ int64_t ln_at(const LnRows& s, unsigned b, unsigned h, unsigned l) {
    return b * s.b + h * s.h + l * s.t;
}

}  // namespace dr
