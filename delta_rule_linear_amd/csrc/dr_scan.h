// dr_scan.h -- the gated linear recurrence's kernels (dr_scan.hip forward and
// one token, dr_scan_bwd.hip the backward).
//
//   h_t = a_t h_{t-1} + c(a_t) x_t      a = e^g or sigmoid(g);  c = 1, 1 - a, sqrt(1 - a^2)
//
// a is carried in two parts, hi + lo, where it is near one: rounded to 24 bits it
// would be off by 2^-25, and a memory of 1 / (1 - a) tokens multiplies that.  1 - a
// is made directly (-expm1(g), sigmoid(-g)); hi is a rounded, and lo = (1 - hi) - (1 - a).
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
        const bool near = __builtin_fabsf(g) < 0.4f;
        o.rest = near ? -__builtin_fmaf(g * g, q, g) : 1.f - e;
        const float hi = 1.f - o.rest;
        o.hi = near ? hi : e;
        o.lo = near ? (1.f - hi) - o.rest : 0.f;
    } else {
        const float e = __builtin_amdgcn_exp2f(-kLog2e * __builtin_fabsf(g));
        const float big = __builtin_amdgcn_rcpf(1.f + e), little = e * big;
        const bool near = g > 0.f;
        o.rest = near ? little : big;
        o.hi = near ? big : little;
        o.lo = near ? (1.f - big) - little : 0.f;
    }
    return o;
}

// The gate of a token that changes nothing (a = 1 exactly).
template <int DEC, bool F32>
__device__ __forceinline__ void gs_stay(Oct<F32>& g) {
    constexpr unsigned one = DEC == kGsLog ? 0u : F32 ? 0x7f800000u : 0x7f807f80u;
#pragma unroll
    for (int i = 0; i < (F32 ? 8 : 4); ++i) g.w[i] = one;
}
template <bool F32>
__device__ __forceinline__ void gs_zero(Oct<F32>& x) {
#pragma unroll
    for (int i = 0; i < (F32 ? 8 : 4); ++i) x.w[i] = 0u;
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
// launch_gs_clear writes first.  Between tiles A is rounded to 24 bits, which costs
// half a rounding of the state per tile.
//
// kGsGroup tiles are a group, as many groups a block.  The last tile of a group
// publishes the group's map, as soon as it has the others' maps, and the last one of
// a block the state behind it.  A tile takes up to kGsGroup - 1 maps of each kind, and
// the state is handed on once per block: about 0.85 us each time (one state for every 8 tiles
// of 64 tokens held 65536 tokens up for 109 us).
constexpr uint64_t kGsAbsent = ~(uint64_t)0;

__device__ __forceinline__ void gs_publish(uint64_t* to, float a, float b) {
    uint64_t v = ((uint64_t)__float_as_uint(b) << 32) | __float_as_uint(a);
    if (v == kGsAbsent) v = 0x7fc000007fc00000u;   // two NaN of the one kind that means "not there"
    __hip_atomic_store(to, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t gs_peek(const uint64_t* from) {
    return __hip_atomic_load(from, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// n words (fewer than kGsGroup, 128 apart) once all are there; all are asked for at
// once, where there are fewer the last one again.
__device__ __forceinline__ void gs_wait(const uint64_t* from, int n, uint64_t (&m)[kGsGroup - 1]) {
    bool all = n == 0;
    while (!all) {
#pragma unroll
        for (int i = 0; i < kGsGroup - 1; ++i) m[i] = gs_peek(from + (size_t)min(i, n - 1) * kGsTile);
        all = true;
#pragma unroll
        for (int i = 0; i < kGsGroup - 1; ++i) all = all && m[i] != kGsAbsent;
        if (!all) __builtin_amdgcn_s_sleep(1);
    }
}
__device__ __forceinline__ float gs_through(const uint64_t (&m)[kGsGroup - 1], int n, float h) {
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
    const int ngroup = (a.nseg + kGsGroup - 1) / kGsGroup, nblock = (ngroup + kGsGroup - 1) / kGsGroup;
    uint64_t* maps = a.maps + (size_t)col * (a.nseg + ngroup + nblock) * kGsTile + c;
    uint64_t* gmaps = maps + (size_t)a.nseg * kGsTile;
    uint64_t* states = gmaps + (size_t)ngroup * kGsTile;
    const int group = seg / kGsGroup, n = seg - group * kGsGroup, block = group / kGsGroup, q = group - block * kGsGroup;
    const bool more = seg + 1 < a.nseg;
    float h = first, A = H + L;
    if (seg == 0) {
        // what comes in is part of the first tile's map, so that nobody else reads it
        B = gs_apply(H, L, first, B);
        A = 0.f;
        gs_publish(maps, A, B);
    } else {
        if (more) gs_publish(maps + (size_t)seg * kGsTile, A, B);
        uint64_t m[kGsGroup - 1], g[kGsGroup - 1];
        gs_wait(maps + (size_t)group * kGsGroup * kGsTile, n, m);
        if (n == kGsGroup - 1 && more) {
            float ga = A, gb = gs_through(m, n, 0.f);
#pragma unroll
            for (int i = 0; i < kGsGroup - 1; ++i) ga *= __uint_as_float((unsigned)m[i]);
            gs_publish(gmaps + (size_t)group * kGsTile, ga, __builtin_fmaf(A, gb, B));
        }
        gs_wait(gmaps + (size_t)block * kGsGroup * kGsTile, q, g);
        h = 0.f;   // the first block's first map holds what came in
        if (block) {
            uint64_t s;
            while ((s = gs_peek(states + (size_t)block * kGsTile)) == kGsAbsent) __builtin_amdgcn_s_sleep(1);
            h = __uint_as_float((unsigned)s);
        }
        h = gs_through(m, n, gs_through(g, q, h));
        if (n == kGsGroup - 1 && q == kGsGroup - 1 && more)
            gs_publish(states + (size_t)(block + 1) * kGsTile, __builtin_fmaf(A, h, B), 0.f);
    }
    return gs_join<FWD>(shH, shL, shB, a.groups, c, h);
}

}  // namespace dr
