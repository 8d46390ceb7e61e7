// dr_scan_bwd.hip -- the gated linear recurrence's backward.
//
//   d_t = dh_t + e_{t+1},  e_t = a_t d_t (e_{L+1}: the last state's gradient),  dh0 = e_1
//   dx_t = c d_t
//   dg_t = d_t (h_{t-1} + c'(a) x_t) da/dg:   c' = 0, -1, -a / c;   da/dg = a, or a (1 - a)
//
// The same walk as the forward's, over the tokens backwards, with e as the state.
// h is the forward's output as it was kept: nothing is run forwards again.

#include "dr_scan.h"

namespace dr {

constexpr int kRunBwd = 4;

template <bool FX, bool FG, bool FH, bool FD, int DEC, int INP, bool SMALL, bool FAR>
__global__ __launch_bounds__(256) void gs_bwd_kernel(GsArgs a) {
    constexpr int T = kRunBwd;
    extern __shared__ float lds[];
    __shared__ unsigned drawn;
    const int ntg = a.groups, tid = threadIdx.x, lane = tid & 15, tg = tid >> 4;
    float* carry = lds;
    float* shH = carry + kGsTile;
    float* shL = shH + ntg * kGsTile;
    float* shB = shL + ntg * kGsTile;
    const unsigned nct = ((unsigned)a.C + kGsTile - 1) / kGsTile;
    const int xs = a.x_f32 ? 4 : 2, gs = a.g_f32 ? 4 : 2, hs = a.h_f32 ? 4 : 2, ds = a.dh_f32 ? 4 : 2,
              os = a.out_f32 ? 4 : 2, span = ntg * T;
    // tiles in the order that the gradient passes them: the last tokens first
    const unsigned tile = FAR ? gs_draw(a.counter, &drawn) : 0;
    const int seg = FAR ? (int)(tile / a.columns) : 0;
    for (unsigned col = FAR ? tile - seg * a.columns : blockIdx.x; col < a.columns; col += gridDim.x) {
        const unsigned b = col / nct, ct = col - b * nct;
        const OctPlace pl = oct_place(ct * 16 + lane, a.C);
        if (!FAR || seg == 0)
            for (int c = tid; c < kGsTile; c += blockDim.x)
                carry[c] = a.dlast ? a.dlast[(size_t)b * a.C + oct_channel<SMALL>(ct * 16 + (c >> 3), c & 7, a.C)] : 0.f;
        const char* xb = (const char*)a.x + b * a.sx.b * xs;
        const char* gb = (const char*)a.g + b * a.sg.b * gs;
        const char* hb = (const char*)a.h + b * a.sh.b * hs;
        const char* db = (const char*)a.dh + b * a.sdh.b * ds;
        char* ob = (char*)a.out + b * a.so.b * os;
        char* gob = (char*)a.dg + b * a.sdg.b * os;
        for (int t0 = FAR ? (a.nseg - 1 - seg) * span : (a.L - 1) / span * span; t0 >= 0; t0 -= span) {
            const int t = t0 + tg * T;
            Oct<FX> x[T];
            Oct<FG> g[T];
            Oct<FH> h[T];   // the states before the run's tokens
            Oct<FD> d[T];
#pragma unroll
            for (int i = 0; i < T; ++i) {
                const int64_t r = min(t + i, a.L - 1);
                oct_load<FG, SMALL>(gb + r * a.sg.t * gs, a.g_f32, pl.at, a.C, g[i]);
                oct_load<FD, SMALL>(db + r * a.sdh.t * ds, a.dh_f32, pl.at, a.C, d[i]);
            }
#pragma unroll
            for (int i = 0; i < T; ++i) {
                const int64_t r = min(t + i, a.L - 1), p = max(r - 1, (int64_t)0);
                oct_load<FH, SMALL>(hb + p * a.sh.t * hs, a.h_f32, pl.at, a.C, h[i]);
                if (INP != kGsPlain) oct_load<FX, SMALL>(xb + r * a.sx.t * xs, a.x_f32, pl.at, a.C, x[i]);
            }
            if (t0 + span > a.L) {
                // behind the last token nothing changes the gradient
#pragma unroll
                for (int i = 0; i < T; ++i)
                    if (t + i >= a.L) {
                        gs_stay<DEC>(g[i]);
                        gs_zero(d[i]);
                    }
            }
            float H[8], Lo[8], B[8];
#pragma unroll
            for (int i = T - 1; i >= 0; --i)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const GsFactor f = gs_factor<DEC>(oct_value(g[i], e));
                    const float hi = f.hi, lo = f.lo, dh = oct_value(d[i], e);
                    if (i == T - 1) {
                        H[e] = hi;
                        Lo[e] = lo;
                        B[e] = gs_apply(hi, lo, dh, 0.f);
                    } else {
                        gs_times(H[e], Lo[e], hi, lo);
                        B[e] = gs_apply(hi, lo, dh + B[e], 0.f);
                    }
                }
            gs_put(shH + tg * kGsTile + lane * 8, H);
            gs_put(shL + tg * kGsTile + lane * 8, Lo);
            gs_put(shB + tg * kGsTile + lane * 8, B);
            __syncthreads();
            for (int c = tid; c < kGsTile; c += blockDim.x) {
                if constexpr (FAR) carry[c] = gs_join_far<false>(a, shH, shL, shB, c, col, seg, carry[c]);
                else carry[c] = gs_join<false>(shH, shL, shB, ntg, c, carry[c]);
            }
            __syncthreads();
            float s[8];
            gs_get(shB + tg * kGsTile + lane * 8, s);
#pragma unroll
            for (int i = T - 1; i >= 0; --i) {
                float dx[8], dg[8], first[8];
                const bool start = t + i == 0;
                if (start) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        first[e] = a.h0 ? a.h0[(size_t)b * a.C + (SMALL ? min(e, a.C - 1) : pl.at + e)] : 0.f;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const GsFactor f = gs_factor<DEC>(oct_value(g[i], e));
                    const float dt = oct_value(d[i], e) + s[e];
                    const float c = gs_input<INP>(f);
                    float before = start ? first[e] : oct_value(h[i], e);
                    if constexpr (INP == kGsBlend) before -= oct_value(x[i], e);
                    if constexpr (INP == kGsUnit) {
                        // c = 0 where a = 1: the square root has no slope there, and the
                        // input's part is left out
                        const float k = c > 0.f ? f.hi * __builtin_amdgcn_rcpf(c) : 0.f;
                        before = __builtin_fmaf(-k, oct_value(x[i], e), before);
                    }
                    dx[e] = c * dt;
                    dg[e] = dt * before * (DEC == kGsLog ? f.hi : f.hi * f.rest);
                    s[e] = gs_apply(f.hi, f.lo, dt, 0.f);
                }
                if (t + i < a.L && pl.own) {
                    oct_store<SMALL>(ob + (int64_t)(t + i) * a.so.t * os, a.out_f32, pl, dx);
                    oct_store<SMALL>(gob + (int64_t)(t + i) * a.sdg.t * os, a.out_f32, pl, dg);
                }
            }
            if constexpr (FAR) break;
            __syncthreads();
        }
        if (a.last && (!FAR || seg + 1 == a.nseg))
            for (int c = tid; c < kGsTile; c += blockDim.x) {
                const OctPlace p = oct_place(ct * 16 + (c >> 3), a.C);
                if (oct_own<SMALL>(p, c & 7)) a.last[(size_t)b * a.C + p.at + (c & 7)] = carry[c];
            }
        if constexpr (FAR) break;
        __syncthreads();
    }
}

template <bool FX, bool FG, bool FH, bool FD, int DEC, int INP, bool SMALL>
static hipError_t gs_launch(const GsArgs& a, int slot, hipStream_t st) {
    const unsigned lds = (1 + 3 * a.groups) * kGsTile * 4;
    if (a.nseg > 1) {
        const hipError_t e = launch_gs_clear(a, slot, st);
        if (e != hipSuccess) return e;
        return launch_k(slot, gs_bwd_kernel<FX, FG, FH, FD, DEC, INP, SMALL, true>, dim3(a.columns * a.nseg),
                        dim3(16 * a.groups), lds, st, a);
    }
    return launch_k(slot, gs_bwd_kernel<FX, FG, FH, FD, DEC, INP, SMALL, false>,
                    dim3(a.columns < 65536 ? a.columns : 65536), dim3(16 * a.groups), lds, st, a);
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
