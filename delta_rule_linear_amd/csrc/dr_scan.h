// dr_scan.h -- what the gated linear recurrence's kernels share (dr_scan.hip forward and
// one token, dr_scan_bwd.hip the backward).
//
//   h_t = a_t h_{t-1} + c(a_t) x_t      a = e^g or sigmoid(g);  c = 1, 1 - a, sqrt(1 - a^2)
//
// Where a is near one, a h is made as h - (1 - a) h with 1 - a taken directly
// (-expm1(g), sigmoid(-g)): a rounded to 24 bits would be off by 2^-25, and a memory
// of 1 / (1 - a) tokens multiplies that.  Elsewhere a itself is used, so that strong
// decays are exact relative to themselves.
//
// An infinite h stays infinite under every decay, of 0 too: what a tile does to it must not
// depend on how its tokens' decays multiply.  The forms above make NaN of it (infinity
// minus infinity, or 0 times it), and NaN stays.  So the forward looks at what comes out, in
// the places where few values show it, and where that is odd goes through it once more in
// forms that take any h (`all` in their names).  The backward does not: its gradients are
// infinite or NaN from there on (looking cost it up to a tenth of its time).
#pragma once

#include <hip/hip_runtime.h>

#include "dr_device.h"
#include "dr_internal.h"
#include "dr_octet.h"
#include "dr_seqops.h"

namespace dr {

enum { kGsLog = 0, kGsLogit = 1 };
enum { kGsPlain = 0, kGsBlend = 1, kGsUnit = 2 };

// a = one + part: where a is near one, `one` is 1 and part = a - 1, its sign bit set (of
// zero too); elsewhere `one` is 0 and part = a, its sign bit clear.  rest = 1 - a.
struct GsFactor {
    float part, rest;
};
// All bits set where `part` says that a is near one.
__device__ __forceinline__ int gs_near(float part) { return __float_as_int(part) >> 31; }
__device__ __forceinline__ float gs_masked(int mask, float x) { return __int_as_float(mask & __float_as_int(x)); }
__device__ __forceinline__ float gs_select(int mask, float x, float y) {
    return __int_as_float((mask & __float_as_int(x)) | (~mask & __float_as_int(y)));
}

// e^x within 3 + |x| / 20 units of 2^-24 of itself (one of the exponential's last place, one
// rounding, and ln 2 in 24 bits): the product with log2 e is rounded, which alone would be
// 64 units at x = 87; what that left out, x - p ln 2, is added (2 x 16384 x 2048 92.4 -> 94.6
// us, backward 174.0 -> 174.6).  GROWS: x may be positive.
template <bool GROWS>
__device__ __forceinline__ float gs_exp(float x) {
    if (!GROWS) x = __builtin_elementwise_maximum(x, -104.f);   // e^x is 0 there; NaN stays
    const float p = x * 1.44269504088896340736f, e = __builtin_amdgcn_exp2f(p);
    const float r = __builtin_fmaf(-p, 0.69314718055994530942f, x);
    // where e is 0 or infinite it stays
    return __builtin_fmaf(e, !GROWS || __builtin_fabsf(p) < 128.f ? r : 0.f, e);
}

template <int DEC>
__device__ __forceinline__ GsFactor gs_factor(float g) {
    GsFactor o;
    if constexpr (DEC == kGsLog) {
        // expm1 by its series for -0.4 < g <= -0 (the next term, g^9 / 9!, is below
        // 2^-28 of g), e^g elsewhere
        const float e = gs_exp<true>(g);
        float q = 1.f / 40320.f;
        q = __builtin_fmaf(q, g, 1.f / 5040.f);
        q = __builtin_fmaf(q, g, 1.f / 720.f);
        q = __builtin_fmaf(q, g, 1.f / 120.f);
        q = __builtin_fmaf(q, g, 1.f / 24.f);
        q = __builtin_fmaf(q, g, 1.f / 6.f);
        q = __builtin_fmaf(q, g, 0.5f);
        q = __builtin_fmaf(g * g, q, g);
        // as integers, negative floats grow with their size, and positive ones are larger
        // (of -0 the series is +0, whose sign has to be set)
        o.part = __float_as_int(g) < __float_as_int(-0.4f) ? -__builtin_fabsf(q) : e;
        o.rest = gs_masked(~gs_near(o.part), 1.f) - o.part;
    } else {
        const float e = gs_exp<false>(-__builtin_fabsf(g));
        const float big = __builtin_amdgcn_rcpf(1.f + e), little = e * big;
        o.part = gs_select(0x7fffffff, little, __int_as_float(~__float_as_int(g)));
        o.rest = gs_select(gs_near(o.part), little, big);
    }
    return o;
}
__device__ __forceinline__ float gs_decay(const GsFactor& f) {
    const int near = gs_near(f.part);
    return gs_masked(near, 1.f) + f.part;
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
    // 1 - a^2 = (1 - a) (2 - (1 - a)), scaled: the root takes no subnormal numbers
    return __builtin_amdgcn_sqrtf(f.rest * __builtin_fmaf(f.rest, -0x1p64f, 0x1p65f)) * 0x1p-32f;
}

// a h + b
__device__ __forceinline__ float gs_step(float part, float h, float b) {
    return gs_masked(gs_near(part), h) + __builtin_fmaf(part, h, b);
}

// What a step makes of any h; s is what gs_step makes of it.
__device__ __forceinline__ float gs_stay_infinite(float part, float h, float b, float s) {
    return __builtin_isinf(h) ? h + __builtin_fmaf(part, 0.f, b) : s;   // NaN of a NaN decay
}

// The same value, of which the compiler knows nothing: what it made of it elsewhere is made
// again here instead of kept in registers.
__device__ __forceinline__ float gs_fresh(float x) {
    asm volatile("" : "+v"(x));
    return x;
}

// Whether the wave has a value that is infinite or NaN, or from 2^100 on, whose sums with
// others could be.
__device__ __forceinline__ bool gs_odd_here(float x) { return !(__builtin_fabsf(x) < 0x1p100f); }
__device__ __forceinline__ bool gs_odd(float x) {
    return __builtin_expect(__builtin_amdgcn_ballot_w64(gs_odd_here(x)) != 0, 0);
}

// The map of several tokens, h -> (one + part) h + b, one again 0 or 1.
struct GsMap {
    float one, part, b;
};
__device__ __forceinline__ float gs_apply(const GsMap& m, float h) {
    return __builtin_fmaf(m.one, h, __builtin_fmaf(m.part, h, m.b));
}
__device__ __forceinline__ float gs_apply_all(const GsMap& m, float h) {
    return gs_stay_infinite(m.part, h, m.b, gs_apply(m, h));
}
// A decay that has become strong over several tokens is held as it is, so that it is
// exact relative to itself (1 + part is exact from -1 to -1/2).
__device__ __forceinline__ void gs_settle(float& one, float& part) {
    const bool strong = part < -0.5f;
    part = strong ? 1.f + part : part;
    one = strong ? 0.f : one;
}
// first m, then n; settled or, if little follows, not
__device__ __forceinline__ GsMap gs_pair(const GsMap& m, const GsMap& n) {
    return {m.one * n.one, __builtin_fmaf(m.part, n.part, __builtin_fmaf(m.one, n.part, m.part * n.one)), gs_apply(n, m.b)};
}
__device__ __forceinline__ GsMap gs_then(const GsMap& m, const GsMap& n) {
    GsMap r = gs_pair(m, n);
    gs_settle(r.one, r.part);
    return r;
}
__device__ __forceinline__ float gs_four_all(const GsMap (&m)[4], float h) {
#pragma unroll
    for (int i = 0; i < 4; ++i) h = gs_apply_all(m[i], h);
    return h;
}
// Four, by two.  Of four decays that are near one (over 1/2) 1/16 at least is left, which is
// early enough for settling.
__device__ __forceinline__ GsMap gs_four(const GsMap (&m)[4]) {
    GsMap r = gs_pair(gs_pair(m[0], m[1]), gs_pair(m[2], m[3]));
    gs_settle(r.one, r.part);
    return r;
}
// one token's, and first m, then a token
__device__ __forceinline__ GsMap gs_token(float part, float b) { return {gs_masked(gs_near(part), 1.f), part, b}; }
__device__ __forceinline__ GsMap gs_then(const GsMap& m, float part, float b) {
    const int near = gs_near(part);
    return {gs_masked(near, m.one), __builtin_fmaf(m.part, part, __builtin_fmaf(m.one, part, gs_masked(near, m.part))),
            gs_step(part, m.b, b)};
}
// A map's decay as a token's, in one word.
__device__ __forceinline__ float gs_word(const GsMap& m) {
    return __int_as_float(__float_as_int(m.part) | (__float_as_int(m.one) << 2 & (int)0x80000000));   // a bit of 1.0
}

// ---------------------------------------------------------------- tiles
// A workgroup has 64 channels of a tile of tokens, a thread eight channels of a run of
// them; eight threads have the channels of a run, a wave the channels of eight runs.
// Every thread makes its run's map.  A wave joins its eight runs, one channel a lane
// (through LDS that is its own, [run][64]), and leaves its map for the other waves
// behind the one barrier that a tile needs; from the state that the tile starts with
// every lane then follows the waves before its own.
struct GsLds {
    float *one, *part, *b;   // [runs][64], a wave's own
    float* start;            // [waves][64], a wave's own: what it starts with
    float* waves;            // twice [3][waves][64]: the waves' maps, used in turn
    float* back;             // [3][waves][64]: maps of earlier tiles
    int n;                   // waves
};
constexpr int kGsWaves = 4;   // of a full workgroup
inline unsigned gs_lds_bytes(int runs) { return (3 * runs + 10 * (runs / 8)) * kGsTile * 4; }
__device__ __forceinline__ GsLds gs_lds(float* p) {
    GsLds l;
    l.n = blockDim.x >> 6;
    l.one = p;
    l.part = l.one + 8 * l.n * kGsTile;
    l.b = l.part + 8 * l.n * kGsTile;
    l.start = l.b + 8 * l.n * kGsTile;
    l.waves = l.start + l.n * kGsTile;
    l.back = l.waves + 6 * l.n * kGsTile;
    return l;
}

// What a wave writes to LDS it reads in the same order; only the compiler has to keep to it.
__device__ __forceinline__ void gs_wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ void gs_put4(float* to, float x, float y, float z, float w) {
    *reinterpret_cast<float4*>(to) = make_float4(x, y, z, w);
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

// A thread's runs, put where its wave joins them.
__device__ __forceinline__ int gs_own() { return (threadIdx.x >> 3) * kGsTile + (threadIdx.x & 7) * 8; }
__device__ __forceinline__ void gs_put_runs(const GsLds& l, GsMap (&run)[8]) {
    // a run is short enough for this to be late enough: four tokens' decays that are near
    // one (over 1/2) make 1/16 at least
#pragma unroll
    for (int e = 0; e < 8; ++e) gs_settle(run[e].one, run[e].part);
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
        gs_put4(l.one + gs_own() + e, run[e].one, run[e + 1].one, run[e + 2].one, run[e + 3].one);
        gs_put4(l.part + gs_own() + e, run[e].part, run[e + 1].part, run[e + 2].part, run[e + 3].part);
        gs_put4(l.b + gs_own() + e, run[e].b, run[e + 1].b, run[e + 2].b, run[e + 3].b);
    }
}

// A wave's runs joined, channel `c` = the lane: each run's map becomes that of the runs
// before it in the wave, and the wave's map goes to the others.  FWD: runs, and waves,
// from the first to the last.  Returns whether the wave's map is odd: then some of them are
// not as they should be, and the runs, with any b, are joined once more by ALL.
template <bool FWD, bool ALL = false>
__device__ __forceinline__ bool gs_join(const GsLds& l, int turn) {
    const int tid = threadIdx.x, wave = tid >> 6, c = tid & 63;
    gs_wave_fence();
    GsMap all{1.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int k = (wave * 8 + (FWD ? i : 7 - i)) * kGsTile + c;
        const GsMap m{l.one[k], l.part[k], l.b[k]};
        l.one[k] = all.one;
        l.part[k] = all.part;
        l.b[k] = all.b;
        const float before = all.b;
        all = gs_then(all, m);
        if (ALL) all.b = gs_apply_all(m, before);
    }
    float* w = l.waves + (turn * 3 * l.n + wave) * kGsTile + c;
    w[0] = all.one;
    w[l.n * kGsTile] = all.part;
    w[2 * l.n * kGsTile] = all.b;
    return gs_odd(all.b);
}
// Behind the barrier: wave `i`'s map, in the order that the state passes them.
template <bool FWD>
__device__ __forceinline__ GsMap gs_wave_map(const GsLds& l, int turn, int i, int c) {
    const float* w = l.waves + (turn * 3 * l.n + (FWD ? i : l.n - 1 - i)) * kGsTile + c;
    return {w[0], w[l.n * kGsTile], w[2 * l.n * kGsTile]};
}
// The states that a thread's run starts with, in s, from what the tile starts with (h, of
// the lane's channel).  Returns what it ends with; odd is set if the wave has odd states.
template <bool FWD>
__device__ __forceinline__ float gs_starts(const GsLds& l, int turn, float h, float (&s)[8], bool* odd = nullptr) {
    const int tid = threadIdx.x, wave = tid >> 6, c = tid & 63;
    const float start = h;
    float mine = h;
#pragma unroll
    for (int i = 0; i < kGsWaves; ++i) {
        if (i >= l.n) break;
        if ((FWD ? i : l.n - 1 - i) == wave) mine = h;
        h = gs_apply(gs_wave_map<FWD>(l, turn, i, c), h);
    }
    const bool all = FWD && gs_odd(h);
    if (all) {
        *odd = true;
        h = start;
        for (int i = 0; i < l.n; ++i) {
            if ((FWD ? i : l.n - 1 - i) == wave) mine = h;
            h = gs_apply_all(gs_wave_map<FWD>(l, turn, i, c), h);
        }
    }
    l.start[wave * kGsTile + c] = mine;
    gs_wave_fence();
    float one[8], part[8], b[8];
    const int at = gs_own();
    gs_get(l.one + at, one);
    gs_get(l.part + at, part);
    gs_get(l.b + at, b);
    gs_get(l.start + wave * kGsTile + (tid & 7) * 8, s);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const GsMap m{one[e], part[e], b[e]};
        s[e] = all ? gs_apply_all(m, s[e]) : gs_apply(m, s[e]);
    }
    return h;
}

// ---------------------------------------------------------------- long sequences
// With few sequences each tile of a column (64 channels of a sequence) has a workgroup
// of its own.  A workgroup draws its tile from its column's counter, tiles in the order
// that the state passes them, so that the tiles before its own belong to workgroups
// that already run.  (One counter for all columns hands out a number every 15 ns: 8192
// tiles took 124 us.)  It publishes the map of its tile, h -> A h + B for each channel,
// before it waits for anything; then it takes the maps of the kGsBack tiles before it
// and the state that the first of those starts with, and publishes the state that it
// starts with itself.  The distance is always the same, and so are the bits.  No wait
// goes on without end: maps depend on nothing, and states on earlier tiles.
//
// kGsBack: about as many tiles of a column as are on the chip at once, so that the
// state is there as a rule and only the maps of tiles that run side by side are waited
// for, once.  (Maps joined over groups of 8 tiles and blocks of 8 groups need fewer
// words, but three such round trips of 1.5 us and more.)
//
// A map is one 64-bit word (A in the low half, held as a token's, B in the high one), a
// state another, so that a word is whole when it is there at all; until then it is
// kGsAbsent, which launch_gs_clear writes first.  (A rounded to 24 bits would be off by the
// same in every tile of an even decay: 7e-5 of the state at a memory of 1e6 tokens.)
constexpr uint64_t kGsAbsent = ~(uint64_t)0;
constexpr int kGsBack = 16;

__device__ __forceinline__ void gs_publish(uint64_t* to, float a, float b) {
    uint64_t v = ((uint64_t)__float_as_uint(b) << 32) | __float_as_uint(a);
    if (v == kGsAbsent) v = 0x7fc000007fc00000u;   // two NaN of the one kind that means "not there"
    __hip_atomic_store(to, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t gs_peek(const uint64_t* from) {
    return __hip_atomic_load(from, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float gs_low(uint64_t m) { return __uint_as_float((unsigned)m); }
__device__ __forceinline__ float gs_high(uint64_t m) { return __uint_as_float((unsigned)(m >> 32)); }

// Draws a tile of the column (thread 0).  Counters start at -1, as everything that
// launch_gs_clear writes.
__device__ __forceinline__ unsigned gs_draw(const GsArgs& a, unsigned col) {
    return __hip_atomic_fetch_add(a.counters + (size_t)col * kGsCounter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1u;
}

// The column of the i-th workgroup of a row of tiles.  Workgroups go to the eight dies in
// turn; neighbouring columns, whose channels lie side by side in memory, go to the same
// one where the row is a multiple of eight (2 x 16384 x 2048 103 -> 91 us, backward 193
// -> 171).
__device__ __forceinline__ unsigned gs_column(const GsArgs& a, unsigned i) {
    return a.padded % 8 ? i : i % 8 * (a.padded / 8) + i / 8;
}

// The state that tile `seg` of a column starts with, for the lane's channel, by four
// waves, behind the barrier after gs_join; `first` is what the first tile starts with.
// Each wave takes a quarter of the maps before the tile.
template <bool FWD>
__device__ __forceinline__ float gs_far(const GsArgs& a, const GsLds& l, unsigned col, int seg, float first) {
    constexpr int N = kGsBack / kGsWaves;
    const int tid = threadIdx.x, c = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    uint64_t* maps = a.maps + (size_t)col * a.nseg * 2 * kGsTile;
    uint64_t* states = maps + (size_t)a.nseg * kGsTile;
    if (wave == 0 && seg + 1 < a.nseg) {
        GsMap w[kGsWaves];
#pragma unroll
        for (int i = 0; i < kGsWaves; ++i) w[i] = gs_wave_map<FWD>(l, 0, i, c);
        const GsMap all = gs_four(w);
        // what comes in is part of the first tile's map, so that nobody else reads it
        float b = all.b;
        if (seg == 0 || (FWD && gs_odd(b))) {
            // one after the other: for the channels that need it, so that others keep their bits
            const float whole = gs_four_all(w, seg ? 0.f : first);
            b = seg == 0 || gs_odd_here(b) ? whole : b;
        }
        gs_publish(maps + (size_t)seg * kGsTile + c, seg ? gs_word(all) : 0.f, b);
    }
    if (seg == 0) return first;
    const int from = seg - kGsBack + wave * N;               // this wave's maps: from .. from + N - 1
    const bool state = wave == 0 && seg > kGsBack;
    GsMap all{1.f, 0.f, 0.f};
    if (from + N > 0) {
        // one lane looks for the word that comes last, as a rule
        const uint64_t* at = maps + (int64_t)from * kGsTile;
        if (c == 0)
            while (gs_peek(at + (N - 1) * kGsTile) == kGsAbsent) __builtin_amdgcn_s_sleep(2);
        uint64_t m[N], h = 0;
        for (;;) {
            bool there = true;
#pragma unroll
            for (int i = 0; i < N; ++i) m[i] = gs_peek(at + (from + i < 0 ? N - 1 : i) * kGsTile + c);
            if (state) h = gs_peek(states + (size_t)(seg - kGsBack) * kGsTile + c);
#pragma unroll
            for (int i = 0; i < N; ++i) there = there && m[i] != kGsAbsent;
            if (there && h != kGsAbsent) break;
            __builtin_amdgcn_s_sleep(2);
        }
        GsMap t[N];
#pragma unroll
        for (int i = 0; i < N; ++i) t[i] = from + i < 0 ? all : gs_token(gs_low(m[i]), gs_high(m[i]));
        all = gs_four(t);
        // the first of all starts with 0: its map holds what came in
        if (wave == 0) all.b = gs_apply(all, gs_low(h));
    }
    float* back = l.back + wave * kGsTile + c;
    back[0] = all.b;
    back[kGsWaves * kGsTile] = all.one;
    back[2 * kGsWaves * kGsTile] = all.part;
    __syncthreads();
    float s = l.back[c];   // the first wave's, which begins with the state
#pragma unroll
    for (int i = 1; i < kGsWaves; ++i) {
        const float* m = l.back + i * kGsTile + c;
        s = gs_apply({m[kGsWaves * kGsTile], m[2 * kGsWaves * kGsTile], m[0]}, s);
    }
    if (FWD && gs_odd(s)) {
        // the words are all there
        float whole = seg > kGsBack ? gs_low(gs_peek(states + (size_t)(seg - kGsBack) * kGsTile + c)) : 0.f;
        for (int i = max(0, seg - kGsBack); i < seg; ++i) {
            const uint64_t m = gs_peek(maps + (size_t)i * kGsTile + c);
            whole = gs_apply_all(gs_token(gs_low(m), gs_high(m)), whole);
        }
        s = gs_odd_here(s) ? whole : s;
    }
    if (wave == 0 && seg + kGsBack < a.nseg) gs_publish(states + (size_t)seg * kGsTile + c, s, 0.f);
    return s;
}

// n / d by a product: d's divider from the host (dr_seqops.h).
__device__ __forceinline__ unsigned gs_divide(unsigned n, const GsDivide& d) {
    return (unsigned)(((uint64_t)n * d.factor) >> d.shift);
}

}  // namespace dr
