// dr_scan.hip -- the gated linear recurrence: forward over sequences and one token.
//
// Memory bounds it: x and the gate are read once, and what is made of them stays in
// registers until the state that a tile starts with is known (dr_scan.h).
//
// Measured: 2 x 16384 x 2048 bf16, sigmoid gates, unit inputs, 95 us for 403 MB (4.25
// TB/s; a large copy reaches 5.2), the vector units busy for 86% of it; 1 x 65536 x 200
// fp32 69.5 us for 157 MB, with two rounds of tiles that wait for each other; 33 x 992 x
// 2048, where a workgroup walks each column, 116 us for 402 MB; one token for 256 x 2048
// states 4 us.
//
// kGsRun is 4 by count, not by a timing of this form: 8 tokens do not fit the registers of
// four waves per SIMD, 2 double the joining.

#include "dr_scan.h"

namespace dr {

// FAR: one tile of a long sequence, drawn; else whole sequences, tile by tile.  The latter
// does not fit the 128 registers of four waves per SIMD: 33 x 992 x 2048 took 147 to 180 us
// with some of them spilled, at three waves 116.
template <bool FX, bool FG, int DEC, int INP, bool SMALL, bool FAR>
__global__ __launch_bounds__(256, FAR ? 4 : 3) void gs_fwd_kernel(GsArgs a) {
    constexpr int T = kGsRun;
    extern __shared__ __align__(16) float lds[];
    __shared__ unsigned drawn;
    const int tid = threadIdx.x, lane = tid & 7, tg = tid >> 3, span = a.groups * T;
    const GsLds l = gs_lds(lds);
    const int xs = a.x_f32 ? 4 : 2, gs = a.g_f32 ? 4 : 2, os = a.out_f32 ? 4 : 2;
    const unsigned xt = (unsigned)a.sx.t * xs, gt = (unsigned)a.sg.t * gs, ot = (unsigned)a.so.t * os;
    Oct<FX> x[T];
    Oct<FG> g[T];
    auto load_row = [&](unsigned col, int seg, int i, Oct<FX>& x, Oct<FG>& g) {
        const unsigned b = gs_divide(col, a.by_tiles), ct = col - b * a.tiles;
        const OctPlace pl = oct_place(ct * 8 + lane, a.C);
        const int t0 = seg * span, last = a.L - 1 - t0;
        // rows of the tile by 32-bit offsets from its first
        const char* xb = (const char*)a.x + (b * a.sx.b + t0 * a.sx.t) * xs;
        const char* gb = (const char*)a.g + (b * a.sg.b + t0 * a.sg.t) * gs;
        const unsigned r = min(tg * T + i, last);
        oct_load<FX, SMALL>(xb + r * xt, a.x_f32, pl.at, a.C, x);
        oct_load<FG, SMALL>(gb + r * gt, a.g_f32, pl.at, a.C, g);
    };
    auto load = [&](unsigned col, int seg) {
#pragma unroll
        for (int i = 0; i < T; ++i) load_row(col, seg, i, x[i], g[i]);
    };
    unsigned first = blockIdx.x, seg0 = 0;
    if constexpr (FAR) {
        // workgroups start in their order as a rule: the rows of the tile that would then be
        // this one's are asked for before the tile is known
        seg0 = gs_divide(blockIdx.x, a.by_columns);
        first = gs_column(a, blockIdx.x - seg0 * a.padded);
        if (first >= a.columns) return;
        const unsigned ticket = tid == 0 ? gs_draw(a, first) : 0;
        load(first, seg0);
        if (tid == 0) drawn = ticket;
        __syncthreads();
        const unsigned mine = __builtin_amdgcn_readfirstlane(drawn);
        if (mine != seg0) load(first, mine);
        seg0 = mine;
    }
    for (unsigned col = first; col < a.columns; col += gridDim.x) {
        const unsigned b = gs_divide(col, a.by_tiles), ct = col - b * a.tiles;
        const OctPlace pl = oct_place(ct * 8 + lane, a.C);
        float h = 0.f;   // the state between tiles, of the lane's channel
        if (a.h0 && seg0 == 0)
            h = a.h0[(size_t)b * a.C + oct_channel<SMALL>(ct * 8 + ((tid & 63) >> 3), tid & 7, a.C)];
        for (int seg = seg0; seg < a.nseg; ++seg) {
            const int t0 = seg * span, last = a.L - 1 - t0, turn = FAR ? 0 : seg & 1;
            if (!FAR) load(col, seg);
            if (span > last + 1) {
                // behind the last token the map is the identity
#pragma unroll
                for (int i = 0; i < T; ++i)
                    if (tg * T + i > last) {
                        gs_stay<DEC>(g[i]);
                        gs_zero(x[i]);
                    }
            }
            float part[T][8], in[T][8];
            GsMap run[8];
#pragma unroll
            for (int i = 0; i < T; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const GsFactor f = gs_factor<DEC>(oct_value(g[i], e));
                    part[i][e] = f.part;
                    in[i][e] = gs_fresh(gs_input<INP>(f) * oct_value(x[i], e));
                    run[e] = i == 0 ? gs_token(f.part, in[i][e]) : gs_then(run[e], f.part, in[i][e]);
                }
            gs_put_runs(l, run);
            bool odd = gs_join<true>(l, turn);
            if (odd) {
                // b is infinite as the sum of the inputs is, under any decay but NaN
                GsMap again[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float sum = 0.f;
#pragma unroll
                    for (int i = 0; i < T; ++i) {
                        const float p = gs_fresh(part[i][e]);
                        again[e] = i == 0 ? gs_token(p, in[i][e]) : gs_then(again[e], p, in[i][e]);
                        sum += in[i][e];
                    }
                    again[e].b = __builtin_isfinite(again[e].b) ? again[e].b : __builtin_fmaf(again[e].part, 0.f, sum);
                }
                gs_put_runs(l, again);
                gs_join<true, true>(l, turn);
            }
            asm volatile("" : "+v"(h));   // what comes in is read before anything goes out: both may be one tensor
            __syncthreads();
            if constexpr (FAR) h = gs_far<true>(a, l, col, seg, h);
            float s[8];
            h = gs_starts<true>(l, turn, h, s, &odd);
            char* ob = (char*)a.out + (b * a.so.b + t0 * a.so.t) * os;
            auto store = [&](int i) {
                if (tg * T + i <= last && pl.own) oct_store<SMALL>(ob + (tg * T + i) * ot, a.out_f32, pl, s);
                if (tg * T + i == last && pl.own && a.last) oct_store<SMALL>(a.last + (size_t)b * a.C, true, pl, s);
            };
            if (!odd) {
#pragma unroll
                for (int i = 0; i < T; ++i) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) s[e] = gs_step(gs_fresh(part[i][e]), s[e], in[i][e]);
                    store(i);
                }
            } else {
                // token by token from their rows again: few instructions, and no registers, for
                // what hardly ever runs
                Oct<FX> xi;
                Oct<FG> gi;
#pragma unroll 1
                for (int i = 0; i < T; ++i) {
                    if (tg * T + i > last) break;
                    load_row(col, seg, i, xi, gi);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const GsFactor f = gs_factor<DEC>(oct_value(gi, e));
                        const float before = s[e], bi = gs_input<INP>(f) * oct_value(xi, e);
                        s[e] = gs_stay_infinite(f.part, before, bi, gs_step(f.part, before, bi));
                    }
                    store(i);
                }
            }
            if constexpr (FAR) break;
        }
        if constexpr (FAR) break;
        __syncthreads();   // the waves' maps are read before the next column's come
    }
}

// A call's counters, maps and states, before its tiles are drawn.
__global__ __launch_bounds__(256) void gs_clear_kernel(uint64_t* p, size_t n) {
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) p[i] = kGsAbsent;
}

hipError_t launch_gs_clear(const GsArgs& a, int slot, hipStream_t st) {
    const size_t blocks = (a.words + 255) / 256;
    return launch_k(slot, gs_clear_kernel, dim3((unsigned)(blocks < 2048 ? blocks : 2048)), dim3(256), 0, st,
                    (uint64_t*)a.counters, a.words);
}

// One token: h <- a h + c x, and h in the output's type.  A lane has eight channels
// of a state; one at the end of a row reads its neighbour's channels too, which
// that one may have written by then, and uses none of them.
template <bool FX, bool FG, int DEC, int INP, bool SMALL>
__global__ __launch_bounds__(256) void gs_step_kernel(GsArgs a) {
    const unsigned per = ((unsigned)a.C + 7) / 8;
    const size_t n = (size_t)a.B * per;
    const int xs = a.x_f32 ? 4 : 2, gs = a.g_f32 ? 4 : 2, os = a.out_f32 ? 4 : 2;
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) {
        const size_t b = i / per, row = b * a.C;
        const OctPlace pl = oct_place((int)(i - b * per), a.C);
        Oct<FX> x;
        Oct<FG> g;
        Oct<true> s;
        oct_load<FX, SMALL>((const char*)a.x + row * xs, a.x_f32, pl.at, a.C, x);
        oct_load<FG, SMALL>((const char*)a.g + row * gs, a.g_f32, pl.at, a.C, g);
        oct_load<true, SMALL>(a.last + row, true, pl.at, a.C, s);
        float h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const GsFactor f = gs_factor<DEC>(oct_value(g, e));
            const float before = oct_value(s, e), in = gs_input<INP>(f) * oct_value(x, e);
            h[e] = gs_stay_infinite(f.part, before, in, gs_step(f.part, before, in));
        }
        oct_store<SMALL>(a.last + row, true, pl, h);
        oct_store<SMALL>((char*)a.out + row * os, a.out_f32, pl, h);
    }
}

template <bool FX, bool FG, int DEC, int INP, bool SMALL>
static hipError_t gs_launch(const GsArgs& a, bool step, int slot, hipStream_t st) {
    if (step) {
        const size_t n = (size_t)a.B * (((unsigned)a.C + 7) / 8), blocks = (n + 255) / 256;
        return launch_k(slot, gs_step_kernel<FX, FG, DEC, INP, SMALL>, dim3((unsigned)(blocks < 65536 ? blocks : 65536)),
                        dim3(256), 0, st, a);
    }
    if (a.maps) {
        const hipError_t e = launch_gs_clear(a, slot, st);
        if (e != hipSuccess) return e;
        return launch_k(slot, gs_fwd_kernel<FX, FG, DEC, INP, SMALL, true>, dim3(a.padded * a.nseg), dim3(256),
                        gs_lds_bytes(32), st, a);
    }
    return launch_k(slot, gs_fwd_kernel<FX, FG, DEC, INP, SMALL, false>, dim3(a.columns < 65536 ? a.columns : 65536), dim3(8 * a.groups),
                    gs_lds_bytes(a.groups), st, a);
}

template <int DEC, int INP>
static hipError_t gs_launch_types(const GsArgs& a, bool step, int slot, hipStream_t st) {
    if (a.C < 8) return gs_launch<true, true, DEC, INP, true>(a, step, slot, st);
    if (a.x_f32) return gs_launch<true, true, DEC, INP, false>(a, step, slot, st);
    return a.g_f32 ? gs_launch<false, true, DEC, INP, false>(a, step, slot, st)
                   : gs_launch<false, false, DEC, INP, false>(a, step, slot, st);
}

template <int DEC>
static hipError_t gs_launch_inputs(const GsArgs& a, bool step, int slot, hipStream_t st) {
    if (a.inputs == kGsPlain) return gs_launch_types<DEC, kGsPlain>(a, step, slot, st);
    if (a.inputs == kGsBlend) return gs_launch_types<DEC, kGsBlend>(a, step, slot, st);
    return gs_launch_types<DEC, kGsUnit>(a, step, slot, st);
}

hipError_t launch_gs_fwd(const GsArgs& a, int slot, hipStream_t st) {
    return a.logit ? gs_launch_inputs<kGsLogit>(a, false, slot, st) : gs_launch_inputs<kGsLog>(a, false, slot, st);
}
hipError_t launch_gs_step(const GsArgs& a, int slot, hipStream_t st) {
    return a.logit ? gs_launch_inputs<kGsLogit>(a, true, slot, st) : gs_launch_inputs<kGsLog>(a, true, slot, st);
}

}  // namespace dr
