// dr_scan_bwd.hip -- the gated linear recurrence's backward.
//
//   d_t = dh_t + e_{t+1},  e_t = a_t d_t (e_{L+1}: the last state's gradient),  dh0 = e_1
//   dx_t = c d_t
//   dg_t = d_t (h_{t-1} + c'(a) x_t) da/dg:   c' = 0, -1, -a / c;   da/dg = a, or a (1 - a)
//
// The same walk as the forward's, over the tokens backwards, with e as the state.
// h is the forward's output as it was kept: nothing is run forwards again.
//
// Measured: 2 x 16384 x 2048 bf16, sigmoid gates, blended inputs, 174 us for 805 MB (4.65
// TB/s), the vector units busy for 67% of it; 33 x 992 x 2048 bf16, unit inputs, where a
// workgroup walks each column, 232 us for 802 MB, two waves per SIMD (up to 237
// registers).

#include "dr_scan.h"

namespace dr {

template <bool FX, bool FG, bool FH, bool FD, int DEC, int INP, bool SMALL, bool FAR>
__global__ __launch_bounds__(256) void gs_bwd_kernel(GsArgs a) {
    constexpr int T = kGsRun;
    extern __shared__ __align__(16) float lds[];
    __shared__ unsigned drawn;
    const int tid = threadIdx.x, lane = tid & 7, tg = tid >> 3, span = a.groups * T;
    const GsLds l = gs_lds(lds);
    const int xs = a.x_f32 ? 4 : 2, gs = a.g_f32 ? 4 : 2, hs = a.h_f32 ? 4 : 2, ds = a.dh_f32 ? 4 : 2,
              os = a.out_f32 ? 4 : 2;
    const unsigned xt = (unsigned)a.sx.t * xs, gt = (unsigned)a.sg.t * gs, ht = (unsigned)a.sh.t * hs,
                   dt = (unsigned)a.sdh.t * ds, ot = (unsigned)a.so.t * os, got = (unsigned)a.sdg.t * os;
    Oct<FX> x[T];
    Oct<FG> g[T];
    Oct<FH> hp[T];   // the states before the run's tokens
    Oct<FD> d[T];
    // tiles in the order that the gradient passes them: the last tokens first
    auto load = [&](unsigned col, int seg) {
        const unsigned b = gs_divide(col, a.by_tiles), ct = col - b * a.tiles;
        const OctPlace pl = oct_place(ct * 8 + lane, a.C);
        const int t0 = (a.nseg - 1 - seg) * span, last = a.L - 1 - t0;
        const char* xb = (const char*)a.x + (b * a.sx.b + t0 * a.sx.t) * xs;
        const char* gb = (const char*)a.g + (b * a.sg.b + t0 * a.sg.t) * gs;
        const char* hb = (const char*)a.h + (b * a.sh.b + t0 * a.sh.t) * hs;
        const char* db = (const char*)a.dh + (b * a.sdh.b + t0 * a.sdh.t) * ds;
#pragma unroll
        for (int i = 0; i < T; ++i) {
            const unsigned r = min(tg * T + i, last);
            oct_load<FG, SMALL>(gb + r * gt, a.g_f32, pl.at, a.C, g[i]);
            oct_load<FD, SMALL>(db + r * dt, a.dh_f32, pl.at, a.C, d[i]);
        }
#pragma unroll
        for (int i = 0; i < T; ++i) {
            const unsigned r = min(tg * T + i, last);
            // the row before; the first token's comes from h0
            oct_load<FH, SMALL>(t0 + r ? hb + ((int64_t)(r * ht) - ht) : hb, a.h_f32, pl.at, a.C, hp[i]);
            if (INP != kGsPlain) oct_load<FX, SMALL>(xb + r * xt, a.x_f32, pl.at, a.C, x[i]);
        }
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
        if (a.dlast && seg0 == 0)
            h = a.dlast[(size_t)b * a.C + oct_channel<SMALL>(ct * 8 + ((tid & 63) >> 3), tid & 7, a.C)];
        for (int seg = seg0; seg < a.nseg; ++seg) {
            const int t0 = (a.nseg - 1 - seg) * span, last = a.L - 1 - t0, turn = FAR ? 0 : seg & 1;
            if (!FAR) load(col, seg);
            if (span > last + 1) {
                // behind the last token nothing changes the gradient
#pragma unroll
                for (int i = 0; i < T; ++i)
                    if (tg * T + i > last) {
                        gs_stay<DEC>(g[i]);
                        gs_zero(d[i]);
                    }
            }
            GsMap run[8];
#pragma unroll
            for (int i = T - 1; i >= 0; --i)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    // e -> a (e + dh)
                    const GsFactor f = gs_factor<DEC>(oct_value(g[i], e));
                    const float in = gs_step(f.part, oct_value(d[i], e), 0.f);
                    run[e] = i == T - 1 ? gs_token(f.part, in) : gs_then(run[e], f.part, in);
                }
            gs_put_runs(l, run);
            gs_join<false>(l, turn);
            asm volatile("" : "+v"(h));   // what comes in is read before anything goes out: both may be one tensor
            __syncthreads();
            if constexpr (FAR) h = gs_far<false>(a, l, col, seg, h);
            float s[8];
            h = gs_starts<false>(l, turn, h, s);
            char* ob = (char*)a.out + (b * a.so.b + t0 * a.so.t) * os;
            char* gob = (char*)a.dg + (b * a.sdg.b + t0 * a.sdg.t) * os;
            // the factors are made again: kept, they would take the registers of a second
            // workgroup
#pragma unroll
            for (int i = 0; i < T; ++i) oct_forget(g[i]);
#pragma unroll
            for (int i = T - 1; i >= 0; --i) {
                float dx[8], dg[8], h0[8];
                const bool start = t0 + tg * T + i == 0;
                if (start) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        h0[e] = a.h0 ? a.h0[(size_t)b * a.C + (SMALL ? min(e, a.C - 1) : pl.at + e)] : 0.f;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const GsFactor f = gs_factor<DEC>(oct_value(g[i], e));
                    const float sum = oct_value(d[i], e) + s[e], c = gs_input<INP>(f), decay = gs_decay(f);
                    float before = start ? h0[e] : oct_value(hp[i], e);
                    if constexpr (INP == kGsBlend) before -= oct_value(x[i], e);
                    if constexpr (INP == kGsUnit) {
                        // c = 0 where a = 1: the square root has no slope there, and the
                        // input's part is left out
                        const float k = c > 0.f ? decay * __builtin_amdgcn_rcpf(c) : 0.f;
                        before = __builtin_fmaf(-k, oct_value(x[i], e), before);
                    }
                    dx[e] = c * sum;
                    dg[e] = sum * before * (DEC == kGsLog ? decay : decay * f.rest);
                    s[e] = gs_step(f.part, sum, 0.f);
                }
                if (tg * T + i <= last && pl.own) {
                    oct_store<SMALL>(ob + (tg * T + i) * ot, a.out_f32, pl, dx);
                    oct_store<SMALL>(gob + (tg * T + i) * got, a.out_f32, pl, dg);
                    if (start && a.last) oct_store<SMALL>(a.last + (size_t)b * a.C, true, pl, s);
                }
            }
            if constexpr (FAR) break;
        }
        if constexpr (FAR) break;
        __syncthreads();   // the waves' maps are read before the next column's come
    }
}

template <bool FX, bool FG, bool FH, bool FD, int DEC, int INP, bool SMALL>
static hipError_t gs_launch(const GsArgs& a, int slot, hipStream_t st) {
    if (a.maps) {
        const hipError_t e = launch_gs_clear(a, slot, st);
        if (e != hipSuccess) return e;
        return launch_k(slot, gs_bwd_kernel<FX, FG, FH, FD, DEC, INP, SMALL, true>, dim3(a.padded * a.nseg), dim3(256),
                        gs_lds_bytes(32), st, a);
    }
    return launch_k(slot, gs_bwd_kernel<FX, FG, FH, FD, DEC, INP, SMALL, false>, dim3(a.columns < 65536 ? a.columns : 65536), dim3(8 * a.groups),
                    gs_lds_bytes(a.groups), st, a);
}

template <bool FX, bool FG, int DEC, int INP>
static hipError_t gs_launch_grads(const GsArgs& a, int slot, hipStream_t st) {
    if (a.h_f32)
        return a.dh_f32 ? gs_launch<FX, FG, true, true, DEC, INP, false>(a, slot, st)
                        : gs_launch<FX, FG, true, false, DEC, INP, false>(a, slot, st);
    return a.dh_f32 ? gs_launch<FX, FG, false, true, DEC, INP, false>(a, slot, st)
                    : gs_launch<FX, FG, false, false, DEC, INP, false>(a, slot, st);
}

template <int DEC, int INP>
static hipError_t gs_launch_types(const GsArgs& a, int slot, hipStream_t st) {
    if (a.C < 8) return gs_launch<true, true, true, true, DEC, INP, true>(a, slot, st);
    if (a.x_f32) return gs_launch_grads<true, true, DEC, INP>(a, slot, st);
    return a.g_f32 ? gs_launch_grads<false, true, DEC, INP>(a, slot, st)
                   : gs_launch_grads<false, false, DEC, INP>(a, slot, st);
}

template <int DEC>
static hipError_t gs_launch_inputs(const GsArgs& a, int slot, hipStream_t st) {
    if (a.inputs == kGsPlain) return gs_launch_types<DEC, kGsPlain>(a, slot, st);
    if (a.inputs == kGsBlend) return gs_launch_types<DEC, kGsBlend>(a, slot, st);
    return gs_launch_types<DEC, kGsUnit>(a, slot, st);
}

hipError_t launch_gs_bwd(const GsArgs& a, int slot, hipStream_t st) {
    return a.logit ? gs_launch_inputs<kGsLogit>(a, slot, st) : gs_launch_inputs<kGsLog>(a, slot, st);
}

}  // namespace dr
