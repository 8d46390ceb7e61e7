// dr_scan.hip -- the gated linear recurrence: forward over sequences and one token.
//
// A workgroup has 128 channels of a sequence and walks its tokens in tiles.  Of a
// tile every thread has a run of kRun tokens for eight channels: it makes the run's
// own map h -> A h + B, 128 threads join the runs' maps along the tile, one channel
// each, and every thread then runs its tokens from the state that it starts with.
// The inputs are read once, and held in registers between the two.

#include "dr_scan.h"

namespace dr {

constexpr int kRun = 4;

int gs_run(bool) { return kRun; }

// FAR: a tile of a long sequence (dr_scan.h), else whole sequences, tile by tile.
template <bool FX, bool FG, int DEC, int INP, bool SMALL, bool FAR>
__global__ __launch_bounds__(256) void gs_fwd_kernel(GsArgs a) {
    constexpr int T = kRun;
    extern __shared__ float lds[];
    __shared__ unsigned drawn;
    const int ntg = a.groups, tid = threadIdx.x, lane = tid & 15, tg = tid >> 4, span = ntg * T;
    float* carry = lds;                        // [128] the state between tiles
    float* shH = carry + kGsTile;              // [ntg][128] the runs' maps: A in two parts, B
    float* shL = shH + ntg * kGsTile;
    float* shB = shL + ntg * kGsTile;          // then the state that each run starts with
    const unsigned nct = ((unsigned)a.C + kGsTile - 1) / kGsTile;
    const int xs = a.x_f32 ? 4 : 2, gs = a.g_f32 ? 4 : 2, os = a.out_f32 ? 4 : 2;
    const unsigned tile = FAR ? gs_draw(a.counter, &drawn) : 0;
    const int seg = FAR ? (int)(tile / a.columns) : 0;
    for (unsigned col = FAR ? tile - seg * a.columns : blockIdx.x; col < a.columns; col += gridDim.x) {
        const unsigned b = col / nct, ct = col - b * nct;
        const OctPlace pl = oct_place(ct * 16 + lane, a.C);
        if (!FAR || seg == 0)
            for (int c = tid; c < kGsTile; c += blockDim.x)
                carry[c] = a.h0 ? a.h0[(size_t)b * a.C + oct_channel<SMALL>(ct * 16 + (c >> 3), c & 7, a.C)] : 0.f;
        const char* xb = (const char*)a.x + b * a.sx.b * xs;
        const char* gb = (const char*)a.g + b * a.sg.b * gs;
        char* ob = (char*)a.out + b * a.so.b * os;
        for (int t0 = FAR ? seg * span : 0; t0 < a.L; t0 += span) {
            const int t = t0 + tg * T;
            Oct<FX> x[T];
            Oct<FG> g[T];
#pragma unroll
            for (int i = 0; i < T; ++i) {
                const int64_t r = min(t + i, a.L - 1);
                oct_load<FX, SMALL>(xb + r * a.sx.t * xs, a.x_f32, pl.at, a.C, x[i]);
                oct_load<FG, SMALL>(gb + r * a.sg.t * gs, a.g_f32, pl.at, a.C, g[i]);
            }
            if (t0 + span > a.L) {
                // behind the last token the map is the identity
#pragma unroll
                for (int i = 0; i < T; ++i)
                    if (t + i >= a.L) {
                        gs_stay<DEC>(g[i]);
                        gs_zero(x[i]);
                    }
            }
            float hi[T][8], lo[T][8], in[T][8], H[8], Lo[8], B[8];
#pragma unroll
            for (int i = 0; i < T; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const GsFactor f = gs_factor<DEC>(oct_value(g[i], e));
                    hi[i][e] = f.hi;
                    lo[i][e] = f.lo;
                    in[i][e] = gs_input<INP>(f) * oct_value(x[i], e);
                    if (i == 0) {
                        H[e] = hi[i][e];
                        Lo[e] = lo[i][e];
                        B[e] = in[i][e];
                    } else {
                        gs_times(H[e], Lo[e], hi[i][e], lo[i][e]);
                        B[e] = gs_apply(hi[i][e], lo[i][e], B[e], in[i][e]);
                    }
                }
            gs_put(shH + tg * kGsTile + lane * 8, H);
            gs_put(shL + tg * kGsTile + lane * 8, Lo);
            gs_put(shB + tg * kGsTile + lane * 8, B);
            __syncthreads();
            for (int c = tid; c < kGsTile; c += blockDim.x) {
                if constexpr (FAR) carry[c] = gs_join_far<true>(a, shH, shL, shB, c, col, seg, carry[c]);
                else carry[c] = gs_join<true>(shH, shL, shB, ntg, c, carry[c]);
            }
            __syncthreads();
            float s[8];
            gs_get(shB + tg * kGsTile + lane * 8, s);
#pragma unroll
            for (int i = 0; i < T; ++i) {
#pragma unroll
                for (int e = 0; e < 8; ++e) s[e] = gs_apply(hi[i][e], lo[i][e], s[e], in[i][e]);
                if (t + i < a.L && pl.own)
                    oct_store<SMALL>(ob + (int64_t)(t + i) * a.so.t * os, a.out_f32, pl, s);
            }
            if constexpr (FAR) break;
            __syncthreads();   // the starts are read before the next tile's maps come
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

// The words of a call's maps and states, before its tiles are drawn.
__global__ __launch_bounds__(256) void gs_clear_kernel(uint64_t* p, size_t n, unsigned* counter) {
    if (blockIdx.x == 0 && threadIdx.x == 0) *counter = 0;
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) p[i] = kGsAbsent;
}

hipError_t launch_gs_clear(const GsArgs& a, int slot, hipStream_t st) {
    const size_t blocks = (a.words + 255) / 256;
    return launch_k(slot, gs_clear_kernel, dim3((unsigned)(blocks < 2048 ? blocks : 2048)), dim3(256), 0, st, a.maps,
                    a.words, a.counter);
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
            h[e] = gs_apply(f.hi, f.lo, oct_value(s, e), gs_input<INP>(f) * oct_value(x, e));
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
    const unsigned lds = (1 + 3 * a.groups) * kGsTile * 4;
    if (a.nseg > 1) {
        const hipError_t e = launch_gs_clear(a, slot, st);
        if (e != hipSuccess) return e;
        return launch_k(slot, gs_fwd_kernel<FX, FG, DEC, INP, SMALL, true>, dim3(a.columns * a.nseg), dim3(16 * a.groups),
                        lds, st, a);
    }
    return launch_k(slot, gs_fwd_kernel<FX, FG, DEC, INP, SMALL, false>, dim3(a.columns < 65536 ? a.columns : 65536),
                    dim3(16 * a.groups), lds, st, a);
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
