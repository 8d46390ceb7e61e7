// dr_rmsnorm_bwd.hip -- the RMS norm's backward.
//
//   dx = ds + rstd (t - n mean(t n)),  n = s rstd,  t = dy w,  dw = sum over the rows of dy n
//
// with s the sum that the forward wrote (or its x), ds the gradient that reaches it
// by other ways.  s, dy and ds are read once, dx is written once; a workgroup stays
// with the rows of one weight, whose sums stay in registers until its end.  The
// workgroups' sums are added in a fixed order, and in fp64, by a second kernel.
//
// Measured: 8191 x 2048 bf16 with a gradient of the sum 27 us for 134 MB (4.9 TB/s), and
// 4 for the sums.

#include "dr_rmsnorm.h"

namespace dr {

// DS: a gradient of the sum is added (loaded in either type)
template <bool FX, bool FDY, int DS, bool TAIL, bool SMALL, int LPR, int VPT>
__global__ __launch_bounds__(kLnThreads) void rn_bwd_kernel(RnArgs a) {
    constexpr int RPB = kLnThreads / LPR, RU = rn_rows<VPT>();
    constexpr int NCOL = 8 * VPT * LPR;
    constexpr int PARTS = LPR <= 64 ? 4 : 1;
    constexpr bool FS = DS == 2 || SMALL;
    __shared__ float2 red[8];
    __shared__ float acc[PARTS][PARTS > 1 ? NCOL : 1];
    int turn = 0;
    const unsigned g = blockIdx.x % a.groups, blk = blockIdx.x / a.groups;
    const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
    const int xs = a.x_f32 ? 4 : 2, rs = a.r_f32 ? 4 : 2, ds = a.dy_f32 ? 4 : 2, ys = a.y_f32 ? 4 : 2;
    float w[VPT][8], dw[VPT][8];
    rn_weights<TAIL, SMALL, LPR>(a, g, lane, w);
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[v][e] = 0.f;
    const float D = (float)a.D, inv = 1.f / D;
    Oct<FX> nx[RU][VPT];
    Oct<FDY> ny[RU][VPT];
    Oct<FS> ns[DS ? RU : 1][DS ? VPT : 1];
    float nrstd[RU];
    int64_t nat[RU];
    auto fetch = [&](unsigned r0) {
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            unsigned b, h, l;
            ln_row(a, g, min(r0 + u * RPB + sub, a.rows - 1), b, h, l);
            nrstd[u] = a.rstd[((size_t)b * a.H + h) * a.L + l];
            nat[u] = ln_at(a.sy, b, h, l);
            const char* x = (const char*)a.x + ln_at(a.sx, b, h, l) * xs;
            const char* y = (const char*)a.dy + ln_at(a.sdy, b, h, l) * ds;
            const char* s = (const char*)a.r + (DS ? ln_at(a.sr, b, h, l) * rs : 0);
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const OctPlace p = rn_place<LPR>(lane, v, a.D);
                oct_load<FX, SMALL>(x, a.x_f32, p.at, a.D, nx[u][v]);
                oct_load<FDY, SMALL>(y, a.dy_f32, p.at, a.D, ny[u][v]);
                if constexpr (DS != 0) oct_load<FS, SMALL>(s, a.r_f32, p.at, a.D, ns[u][v]);
            }
        }
    };
    const unsigned step = a.blocks * (RPB * RU);
    if (rn_ahead<VPT>()) fetch(blk * (RPB * RU));
    for (unsigned r0 = blk * (RPB * RU); r0 < a.rows; r0 += step) {
        if (!rn_ahead<VPT>()) fetch(r0);
        Oct<FX> rx[RU][VPT];
        Oct<FDY> ry[RU][VPT];
        Oct<FS> rss[DS ? RU : 1][DS ? VPT : 1];
        float rstd[RU];
        int64_t at[RU];
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            rstd[u] = nrstd[u];
            at[u] = nat[u];
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                rx[u][v] = nx[u][v];
                ry[u][v] = ny[u][v];
                if constexpr (DS != 0) rss[u][v] = ns[u][v];
            }
        }
        if (rn_ahead<VPT>() && r0 + step < a.rows) fetch(r0 + step);
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            const bool ok = r0 + u * RPB + sub < a.rows;
            float n[VPT][8], t[VPT][8], s = 0.f;
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const OctPlace p = rn_place<LPR>(lane, v, a.D);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    n[v][e] = rn_value<TAIL, SMALL>(rx[u][v], p, e) * rstd[u];
                    const float dy = rn_value<TAIL, SMALL>(ry[u][v], p, e);
                    if (ok) dw[v][e] = __builtin_fmaf(dy, n[v][e], dw[v][e]);
                    t[v][e] = dy * w[v][e];
                    s = __builtin_fmaf(t[v][e], n[v][e], s);
                }
            }
            s = ln_div(ln_sum<LPR>(s, red, turn), D, inv);
            if (!ok) continue;
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const OctPlace p = rn_place<LPR>(lane, v, a.D);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    t[v][e] = rstd[u] * __builtin_fmaf(-n[v][e], s, t[v][e]);
                    if constexpr (DS != 0) t[v][e] += oct_value(rss[u][v], e);
                }
                if (p.own) oct_store<SMALL>((char*)a.y + at[u] * ys, a.y_f32, p, t[v]);
            }
        }
    }
    if (!a.part) return;
    float* part = a.part + ((size_t)g * a.blocks + blk) * a.D;
    if constexpr (PARTS == 1) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const OctPlace p = rn_place<LPR>(lane, v, a.D);
            if (p.own) oct_store<SMALL>(part, true, p, dw[v]);
        }
    } else {
        // over the rows of a wave by shuffles, then over the four waves through LDS
        const int wave = threadIdx.x / 64;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const OctPlace p = rn_place<LPR>(lane, v, a.D);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
#pragma unroll
                for (int d = LPR; d < 64; d <<= 1) dw[v][e] += __shfl_xor(dw[v][e], d);
                if ((threadIdx.x & 63) < LPR && oct_own<SMALL>(p, e)) acc[wave][p.at + e] = dw[v][e];
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < a.D; c += kLnThreads)
            part[c] = (acc[0][c] + acc[1][c]) + (acc[2][c] + acc[3][c]);
    }
}

// dw from the workgroups' sums, as the layer norm's: 32 columns per workgroup and
// turn, 32 threads for each column, in fp64; the grid is capped.
constexpr unsigned kRnSumGrid = 1u << 16;

__global__ __launch_bounds__(1024) void rn_sum_kernel(RnArgs a, unsigned tiles) {
    __shared__ double red[32][33];
    const unsigned cols = (unsigned)a.D, per = (cols + 31) / 32;
    const unsigned lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    for (unsigned tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const unsigned g = tile / per, c = (tile % per) * 32 + lane;
        double s = 0.0;
        if (c < cols) {
            const float* p = a.part + (size_t)g * a.blocks * cols + c;
#pragma unroll 8
            for (unsigned k = slice; k < a.blocks; k += 32) s += p[(size_t)k * cols];
        }
        if (tile != blockIdx.x) __syncthreads();   // the last turn's sums are read
        red[slice][lane] = s;
        __syncthreads();
        if (slice == 0 && c < cols) {
            s = 0.0;
#pragma unroll
            for (int k = 0; k < 32; ++k) s += red[k][lane];
            a.dw[(size_t)g * a.D + c] = (float)s;
        }
    }
}

template <bool FX, bool FDY, int DS, bool TAIL, bool SMALL, int LPR, int VPT>
static hipError_t rn_launch(const RnArgs& a, int slot, hipStream_t st) {
    return launch_k(slot, rn_bwd_kernel<FX, FDY, DS, TAIL, SMALL, LPR, VPT>, dim3(a.groups * a.blocks), dim3(kLnThreads),
                    0, st, a);
}

template <bool FX, bool FDY, int DS, bool TAIL>
static hipError_t rn_launch_shape(const RnArgs& a, int slot, hipStream_t st) {
    const LnShape s = rn_shape(a.D, (size_t)a.groups * a.rows);
    if (s.lanes == 8) return rn_launch<FX, FDY, DS, TAIL, false, 8, 1>(a, slot, st);
    if (s.lanes == 16) return rn_launch<FX, FDY, DS, TAIL, false, 16, 1>(a, slot, st);
    if (s.lanes == 32) return rn_launch<FX, FDY, DS, TAIL, false, 32, 1>(a, slot, st);
    if (s.lanes == 64) {
        if (s.vecs == 1) return rn_launch<FX, FDY, DS, TAIL, false, 64, 1>(a, slot, st);
        if (s.vecs == 2) return rn_launch<FX, FDY, DS, TAIL, false, 64, 2>(a, slot, st);
        return rn_launch<FX, FDY, DS, TAIL, false, 64, 4>(a, slot, st);
    }
    if (s.vecs == 1) return rn_launch<FX, FDY, DS, TAIL, false, 256, 1>(a, slot, st);
    if (s.vecs == 2) return rn_launch<FX, FDY, DS, TAIL, false, 256, 2>(a, slot, st);
    if (s.vecs == 4) return rn_launch<FX, FDY, DS, TAIL, false, 256, 4>(a, slot, st);
    return rn_launch<FX, FDY, DS, TAIL, false, 256, 8>(a, slot, st);
}

template <bool TAIL, bool FX, bool FDY>
static hipError_t rn_launch_sum(const RnArgs& a, int slot, hipStream_t st) {
    if (!a.r) return rn_launch_shape<FX, FDY, 0, TAIL>(a, slot, st);
    return a.r_f32 ? rn_launch_shape<FX, FDY, 2, TAIL>(a, slot, st) : rn_launch_shape<FX, FDY, 1, TAIL>(a, slot, st);
}

template <bool TAIL>
static hipError_t rn_launch_types(const RnArgs& a, int slot, hipStream_t st) {
    if (a.x_f32)
        return a.dy_f32 ? rn_launch_sum<TAIL, true, true>(a, slot, st) : rn_launch_sum<TAIL, true, false>(a, slot, st);
    return a.dy_f32 ? rn_launch_sum<TAIL, false, true>(a, slot, st) : rn_launch_sum<TAIL, false, false>(a, slot, st);
}

hipError_t launch_rn_bwd(const RnArgs& a, int slot, hipStream_t st) {
    hipError_t e;
    if (a.D < 8)
        e = a.r ? rn_launch<true, true, 2, false, true, 8, 1>(a, slot, st)
                : rn_launch<true, true, 0, false, true, 8, 1>(a, slot, st);
    else
        e = a.D % 8 ? rn_launch_types<true>(a, slot, st) : rn_launch_types<false>(a, slot, st);
    if (e == hipSuccess && a.part) {
        const unsigned tiles = a.groups * ((unsigned)(a.D + 31) / 32);   // at most 2^20 * 2^9
        e = launch_k(slot, rn_sum_kernel, dim3(tiles < kRnSumGrid ? tiles : kRnSumGrid), dim3(1024), 0, st, a, tiles);
    }
    return e;
}

}  // namespace dr
