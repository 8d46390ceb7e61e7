// dr_rmsnorm.hip -- root-mean-square norm of rows, with the residual's addition in
// front and, where asked, an output in 8 bits.
//
//   s = x + residual,  y = s rstd w,  rstd = 1 / sqrt(mean(s^2) + eps)
//   8 bits: scale = max(amax |y| / 448, 2^-126) of 128 columns or of the row, y / scale in e4m3
//
// Memory bounds it: x and the residual are read once into registers, the sum of
// squares, the blocks' largest values and both outputs come from there.  y is made
// from the sum as it is in fp32, before that is rounded to the residual's type.
// Every sum has a fixed order.
//
// Measured: 8191 x 2048 bf16 with a bf16 residual 26.5 us for 134 MB (5.1 TB/s; a large
// copy reaches 5.2); 16384 x 4096 with an fp32 residual to e4m3 136 us for 740 MB (5.45
// TB/s); one row of 2048 5.5 us.

#include "dr_rmsnorm.h"

namespace dr {

// A wave per row up to 2048 values, which takes no barrier; where there are fewer rows
// than the chip has places for waves, four waves per row of more than 512.
constexpr size_t kRnFewRows = 1024;

LnShape rn_shape(int D, size_t rows) {
    if (D <= 64) return {8, 1};
    if (D <= 128) return {16, 1};
    if (D <= 256) return {32, 1};
    if (D <= 512) return {64, 1};
    if (D <= 2048 && rows <= kRnFewRows) return {256, 1};
    if (D <= 1024) return {64, 2};
    if (D <= 2048) return {64, 4};
    if (D <= 4096) return {256, 2};
    if (D <= 8192) return {256, 4};
    return {256, 8};
}

int rn_pass_rows(int D, size_t rows) {
    const LnShape s = rn_shape(D, rows);
    return kLnThreads / s.lanes * (s.vecs == 1 ? rn_rows<1>() : rn_rows<2>());
}

// The largest of values over N lanes side by side, in every one of them.
template <int N>
__device__ __forceinline__ float rn_max(float x) {
    auto step = [](float v, float u) { return __builtin_fmaxf(v, u); };
#pragma unroll
    for (int d = 1; d < N && d < 64; d <<= 1) x = step(x, __shfl_xor(x, d));
    return x;
}

// Eight values in e4m3, each the nearest to y / scale: the quotient is y times the
// rounded 1 / scale with one correction.
__device__ __forceinline__ void rn_codes(const float (&y)[8], float scale, float inv, unsigned (&out)[2]) {
    float q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        q[e] = y[e] * inv;
        const float c = __builtin_fmaf(__builtin_fmaf(-q[e], scale, y[e]), inv, q[e]);
        q[e] = __builtin_isfinite(q[e]) ? c : q[e];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int p = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i], q[4 * i + 1], 0, false);
        p = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i + 2], q[4 * i + 3], p, true);
        out[i] = (unsigned)p;
    }
}

// RES: 0 no residual, 1 in bf16, 2 in fp32
template <bool FX, int RES, bool Q8, bool TAIL, bool SMALL, int LPR, int VPT>
__global__ __launch_bounds__(kLnThreads) void rn_fwd_kernel(RnArgs a) {
    constexpr int RPB = kLnThreads / LPR, RU = rn_rows<VPT>();
    constexpr bool FR = RES == 2 || SMALL;
    __shared__ float2 red[8];
    __shared__ float redm[2][4];
    int turn = 0, mturn = 0;
    const unsigned g = blockIdx.x % a.groups, blk = blockIdx.x / a.groups;
    const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
    const int xs = a.x_f32 ? 4 : 2, rs = a.r_f32 ? 4 : 2, ys = Q8 ? 1 : a.y_f32 ? 4 : 2;
    float w[VPT][8];
    rn_weights<TAIL, SMALL, LPR>(a, g, lane, w);
    const float D = (float)a.D, inv = 1.f / D;
    Oct<FX> nx[RU][VPT];
    Oct<FR> nr[RES ? RU : 1][RES ? VPT : 1];
    unsigned nb[RU], nh[RU], nl[RU];
    auto fetch = [&](unsigned r0) {
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            ln_row(a, g, min(r0 + u * RPB + sub, a.rows - 1), nb[u], nh[u], nl[u]);
            const char* x = (const char*)a.x + ln_at(a.sx, nb[u], nh[u], nl[u]) * xs;
            const char* r = (const char*)a.r + (RES ? ln_at(a.sr, nb[u], nh[u], nl[u]) * rs : 0);
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const OctPlace p = rn_place<LPR>(lane, v, a.D);
                oct_load<FX, SMALL>(x, a.x_f32, p.at, a.D, nx[u][v]);
                if constexpr (RES != 0) oct_load<FR, SMALL>(r, a.r_f32, p.at, a.D, nr[u][v]);
            }
        }
    };
    const unsigned step = a.blocks * (RPB * RU);
    if (rn_ahead<VPT>()) fetch(blk * (RPB * RU));
    for (unsigned r0 = blk * (RPB * RU); r0 < a.rows; r0 += step) {
        if (!rn_ahead<VPT>()) fetch(r0);
        float x[RU][VPT][8];
        unsigned b[RU], h[RU], l[RU];
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            b[u] = nb[u];
            h[u] = nh[u];
            l[u] = nl[u];
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const OctPlace p = rn_place<LPR>(lane, v, a.D);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[u][v][e] = rn_value<TAIL, SMALL>(nx[u][v], p, e);
                    if constexpr (RES != 0) x[u][v][e] += rn_value<TAIL, SMALL>(nr[u][v], p, e);
                }
            }
        }
        if (rn_ahead<VPT>() && r0 + step < a.rows) fetch(r0 + step);
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            float s = 0.f;
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int e = 0; e < 8; ++e) s = __builtin_fmaf(x[u][v][e], x[u][v][e], s);
            const float rstd = ln_rsqrt(ln_div(ln_sum<LPR>(s, red, turn), D, inv) + a.eps);
            const bool ok = r0 + u * RPB + sub < a.rows;
            const size_t at = ((size_t)b[u] * a.H + h[u]) * a.L + l[u];
            if (RES && ok) {
                char* to = (char*)a.total + ln_at(a.st, b[u], h[u], l[u]) * rs;
#pragma unroll
                for (int v = 0; v < VPT; ++v) {
                    const OctPlace p = rn_place<LPR>(lane, v, a.D);
                    if (p.own) oct_store<SMALL>(to, a.r_f32, p, x[u][v]);
                }
            }
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int e = 0; e < 8; ++e) x[u][v][e] = x[u][v][e] * rstd * w[v][e];
            char* y = (char*)a.y + ln_at(a.sy, b[u], h[u], l[u]) * ys;
            if constexpr (Q8) {
                float m[VPT];
#pragma unroll
                for (int v = 0; v < VPT; ++v) {
                    m[v] = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) m[v] = __builtin_fmaxf(m[v], __builtin_fabsf(x[u][v][e]));
                    m[v] = rn_max<(LPR < 16 ? LPR : 16)>(m[v]);
                }
                if (a.block == 0) {
                    // one scale for the row: over its lanes' vectors, its waves
#pragma unroll
                    for (int v = 1; v < VPT; ++v) m[0] = __builtin_fmaxf(m[0], m[v]);
#pragma unroll
                    for (int d = 16; d < LPR && d < 64; d <<= 1) m[0] = __builtin_fmaxf(m[0], __shfl_xor(m[0], d));
                    if constexpr (LPR > 64) {
                        if ((threadIdx.x & 63) == 0) redm[mturn][threadIdx.x >> 6] = m[0];
                        __syncthreads();
#pragma unroll
                        for (int i = 0; i < 4; ++i) m[0] = __builtin_fmaxf(m[0], redm[mturn][i]);
                        mturn ^= 1;
                    }
#pragma unroll
                    for (int v = 1; v < VPT; ++v) m[v] = m[0];
                }
                const int nblk = a.block ? (a.D + 127) / 128 : 1;
#pragma unroll
                for (int v = 0; v < VPT; ++v) {
                    const float scale = __builtin_fmaxf(ln_div(m[v], 448.f, 1.f / 448.f), 0x1p-126f);
                    unsigned code[2];
                    rn_codes(x[u][v], scale, 1.f / scale, code);
                    const OctPlace p = rn_place<LPR>(lane, v, a.D);
                    if (!ok || !p.own) continue;
                    const int k = a.block ? (lane + LPR * v) / 16 : 0;
                    if (a.block ? (lane & 15) == 0 : lane == 0 && v == 0) a.scale[at * nblk + k] = scale;
                    unsigned char* to = (unsigned char*)y + p.at;
                    if (!SMALL && p.own == 8) {
                        *reinterpret_cast<oct_u8x8*>(to) = oct_u8x8{code[0], code[1]};
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (oct_own<SMALL>(p, e)) to[e] = (unsigned char)(code[e / 4] >> (8 * (e % 4)));
                    }
                }
            } else if (ok) {
#pragma unroll
                for (int v = 0; v < VPT; ++v) {
                    const OctPlace p = rn_place<LPR>(lane, v, a.D);
                    if (p.own) oct_store<SMALL>(y, a.y_f32, p, x[u][v]);
                }
            }
            if (ok && lane == 0 && a.rstd_out) a.rstd_out[at] = rstd;
        }
    }
}

template <bool FX, int RES, bool Q8, bool TAIL, bool SMALL, int LPR, int VPT>
static hipError_t rn_launch(const RnArgs& a, int slot, hipStream_t st) {
    return launch_k(slot, rn_fwd_kernel<FX, RES, Q8, TAIL, SMALL, LPR, VPT>, dim3(a.groups * a.blocks), dim3(kLnThreads),
                    0, st, a);
}

template <bool FX, int RES, bool Q8, bool TAIL>
static hipError_t rn_launch_shape(const RnArgs& a, int slot, hipStream_t st) {
    const LnShape s = rn_shape(a.D, (size_t)a.groups * a.rows);
    if (s.lanes == 8) return rn_launch<FX, RES, Q8, TAIL, false, 8, 1>(a, slot, st);
    if (s.lanes == 16) return rn_launch<FX, RES, Q8, TAIL, false, 16, 1>(a, slot, st);
    if (s.lanes == 32) return rn_launch<FX, RES, Q8, TAIL, false, 32, 1>(a, slot, st);
    if (s.lanes == 64) {
        if (s.vecs == 1) return rn_launch<FX, RES, Q8, TAIL, false, 64, 1>(a, slot, st);
        if (s.vecs == 2) return rn_launch<FX, RES, Q8, TAIL, false, 64, 2>(a, slot, st);
        return rn_launch<FX, RES, Q8, TAIL, false, 64, 4>(a, slot, st);
    }
    if (s.vecs == 1) return rn_launch<FX, RES, Q8, TAIL, false, 256, 1>(a, slot, st);
    if (s.vecs == 2) return rn_launch<FX, RES, Q8, TAIL, false, 256, 2>(a, slot, st);
    if (s.vecs == 4) return rn_launch<FX, RES, Q8, TAIL, false, 256, 4>(a, slot, st);
    return rn_launch<FX, RES, Q8, TAIL, false, 256, 8>(a, slot, st);
}

template <bool Q8, bool TAIL>
static hipError_t rn_launch_types(const RnArgs& a, int slot, hipStream_t st) {
    if (a.x_f32)
        return a.r ? rn_launch_shape<true, 2, Q8, TAIL>(a, slot, st) : rn_launch_shape<true, 0, Q8, TAIL>(a, slot, st);
    if (!a.r) return rn_launch_shape<false, 0, Q8, TAIL>(a, slot, st);
    return a.r_f32 ? rn_launch_shape<false, 2, Q8, TAIL>(a, slot, st) : rn_launch_shape<false, 1, Q8, TAIL>(a, slot, st);
}

template <bool Q8>
static hipError_t rn_launch_width(const RnArgs& a, int slot, hipStream_t st) {
    if (a.D < 8)
        return a.r ? rn_launch<true, 2, Q8, false, true, 8, 1>(a, slot, st)
                   : rn_launch<true, 0, Q8, false, true, 8, 1>(a, slot, st);
    return a.D % 8 ? rn_launch_types<Q8, true>(a, slot, st) : rn_launch_types<Q8, false>(a, slot, st);
}

hipError_t launch_rn_fwd(const RnArgs& a, int slot, hipStream_t st) {
    return a.scale ? rn_launch_width<true>(a, slot, st) : rn_launch_width<false>(a, slot, st);
}

}  // namespace dr
