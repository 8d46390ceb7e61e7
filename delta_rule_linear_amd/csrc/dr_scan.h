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

// ---------------------------------------------------------------- long sequences
// With few sequences each tile of a sequence has a workgroup of its own.  A workgroup
// draws its tile from a counter, tiles in the order that the state passes them, so
// that the tiles before its own belong to workgroups that already run.  It publishes
// the map of its tile, h -> A h + B for each channel, before it waits for anything;
// then it takes the maps of the tiles before it, in their order (the same one every
// time), back to the last tile whose number is a multiple of kGsGroup, whose state at
// the start is published as well.  So no wait goes on without end: maps depend on
// nothing, and the state at a group's start on earlier tiles only.
//
// A map is one 64-bit word (A in the low half, B in the high one), a state another,
// so that a word is whole when it is there at all; until then it is kGsAbsent, which
// launch_gs_clear writes first.  Between tiles A is rounded to 24 bits, which costs half a
// rounding of the state per tile.
constexpr uint64_t kGsAbsent = ~(uint64_t)0;

__device__ __forceinline__ void gs_publish(uint64_t* to, float a, float b) {
    uint64_t v = ((uint64_t)__float_as_uint(b) << 32) | __float_as_uint(a);
    if (v == kGsAbsent) v = 0x7fc000007fc00000u;   // two NaN of the one kind that means "not there"
    __hip_atomic_store(to, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t gs_peek(const uint64_t* from) {
    return __hip_atomic_load(from, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The state that tile `seg` starts with, for one channel: maps [seg][128] and the
// groups' states [group][128] of its column.
__device__ __forceinline__ float gs_wait(const uint64_t* maps, const uint64_t* states, int seg) {
    const int group = seg / kGsGroup, n = seg - group * kGsGroup;
    // all words at once; where there are fewer maps, the last one again
    uint64_t m[kGsGroup];
    bool all;
    do {
#pragma unroll
        for (int i = 0; i < kGsGroup - 1; ++i) m[i] = gs_peek(maps + (size_t)(group * kGsGroup + max(min(i, n - 1), 0)) * kGsTile);
        m[kGsGroup - 1] = gs_peek(states + (size_t)group * kGsTile);
        all = group == 0 || m[kGsGroup - 1] != kGsAbsent;
#pragma unroll
        for (int i = 0; i < kGsGroup - 1; ++i) all = all && (i >= n || m[i] != kGsAbsent);
        if (!all) __builtin_amdgcn_s_sleep(1);
    } while (!all);
    if (group == 0) m[kGsGroup - 1] = 0;   // the first tile's map holds what came in
    float h = __uint_as_float((unsigned)m[kGsGroup - 1]);
#pragma unroll
    for (int i = 0; i < kGsGroup - 1; ++i)
        if (i < n) h = __builtin_fmaf(__uint_as_float((unsigned)m[i]), h, __uint_as_float((unsigned)(m[i] >> 32)));
    return h;
}

// Which tile a workgroup has.
__device__ __forceinline__ unsigned gs_draw(unsigned* counter, unsigned* lds) {
    if (threadIdx.x == 0) *lds = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    return *lds;
}

// Joins a tile's runs, [k][128] maps in LDS, for channel c; the state each run starts
// with takes the place of its B.  FWD: runs from the first to the last.
template <bool FWD>
__device__ __forceinline__ float gs_join(const float* shH, const float* shL, float* shB, int ntg, int c, float h) {
#pragma unroll 4
    for (int i = 0; i < ntg; ++i) {
        const int at = (FWD ? i : ntg - 1 - i) * kGsTile + c;
        const float start = h;
        h = gs_apply(shH[at], shL[at], h, shB[at]);
        shB[at] = start;
    }
    return h;
}
// The same through the other workgroups: `first` is what the first tile starts with.
template <bool FWD>
__device__ __forceinline__ float gs_join_far(const GsArgs& a, const float* shH, const float* shL, float* shB, int c,
                                             unsigned col, int seg, float first) {
    float H = 1.f, L = 0.f, B = 0.f;
#pragma unroll 4
    for (int i = 0; i < a.groups; ++i) {
        const int at = (FWD ? i : a.groups - 1 - i) * kGsTile + c;
        B = gs_apply(shH[at], shL[at], B, shB[at]);
        gs_times(H, L, shH[at], shL[at]);
    }
    uint64_t* maps = a.maps + (size_t)col * a.nseg * kGsTile + c;
    uint64_t* states = a.states + (size_t)col * ((a.nseg + kGsGroup - 1) / kGsGroup) * kGsTile + c;
    float h = first;
    if (seg == 0) {
        // what comes in is part of the first tile's map, so that nobody else reads it
        if (a.nseg > 1) gs_publish(maps, 0.f, gs_apply(H, L, h, B));
    } else {
        if (seg + 1 < a.nseg) gs_publish(maps + (size_t)seg * kGsTile, H + L, B);
        h = gs_wait(maps, states, seg);
        if (seg % kGsGroup == kGsGroup - 1 && seg + 1 < a.nseg)
            gs_publish(states + (size_t)(seg / kGsGroup + 1) * kGsTile, gs_apply(H, L, h, B), 0.f);
    }
    return gs_join<FWD>(shH, shL, shB, a.groups, c, h);
}

}  // namespace dr
