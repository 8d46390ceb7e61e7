// dr_layernorm.hip -- layer norm of rows and its backward pass.
//
//   y  = (x - mu) r w + b,  mu = mean(x),  r = 1 / sqrt(mean((x - mu)^2) + eps)
//   dx = r (t - mean(t) - n mean(t n)),  n = (x - mu) r,  t = dy w
//   dw = sum over the rows that share w of dy n,  db = the same sum of dy
//
// Both are bound by memory: x (and dy) are read once into registers, the
// statistics are taken from there (the variance around the mean, in a second
// pass over the registers), and the row is written once.  A row is held by 8 to
// 256 lanes, 8 values per lane and vector.  A workgroup stays with the rows of
// one weight, so that weight and bias, and in the backward the sums dw and db,
// stay in registers; the workgroups' sums are added in a fixed order, and in
// fp64, by a second kernel.  All other arithmetic is fp32.
//
// Measured: forward of 524288 rows of 128 bf16 (a weight for each of 16 heads,
// y token-major) 60 us for 272 MB, 4.5 TB/s (a large copy reaches 5.2); its
// backward 82 us for 403 MB, 4.9 TB/s, and 4.5 for the sums; 8191 x 2048 bf16
// backward 27 us for 110 MB (4.0 TB/s; 512 workgroups of 16 rows each have a
// start and an end) and 4.

#include <hip/hip_runtime.h>

#include "dr_device.h"
#include "dr_internal.h"
#include "dr_layernorm.h"

namespace dr {

constexpr int kLnThreads = 256;

LnShape ln_shape(int D) {
    // the least lanes that hold a row in 8 values each, up to the workgroup; then
    // more values per lane (a wave with 32 values per lane holds 2048 as well,
    // but the backward's 200 registers leave one wave per SIMD)
    if (D <= 64) return {8, 1};
    if (D <= 128) return {16, 1};
    if (D <= 256) return {32, 1};
    if (D <= 512) return {64, 1};
    if (D <= 1024) return {128, 1};
    if (D <= 2048) return {256, 1};
    if (D <= 4096) return {256, 2};
    if (D <= 8192) return {256, 4};
    return {256, 8};
}

// Rows are read and written W values at a time: 8 where every row starts at a
// multiple of 8 values and D is one, else 2 or 1.  Columns behind D are clamped
// when loading and left out when used, so that the loads of a row are all in
// flight at once: with a branch and a conversion for each, the backward of 286884
// x 100 bf16 took 172 us and that of 65536 x 501 232; now 42 (W = 2) and 58 (W =
// 1).  Column of value e of vector v of a lane: consecutive lanes take
// consecutive groups of W.
template <int W, int LPR>
__device__ __forceinline__ int ln_col(int lane, int v, int e) {
    return ((8 * v + e) / W * LPR + lane) * W + e % W;
}

// A lane's part of a row as loaded: 8 / W groups of W values, bf16 or fp32 bits
// (nothing waits for them until they are used).
template <int W, bool F32, int VPT>
struct LnRaw {
    static constexpr int WORDS = F32 ? 8 : W == 1 ? 8 : 4;
    unsigned v[VPT][WORDS];
};

template <int W, bool F32, int LPR, int VPT>
__device__ __forceinline__ void ln_fetch(const void* base, int64_t at, int D, int lane, LnRaw<W, F32, VPT>& r) {
    const char* row = (const char*)base + at * (F32 ? 4 : 2);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        if constexpr (W == 8) {
            const int c = ln_col<W, LPR>(lane, v, 0);
            uint4* to = reinterpret_cast<uint4*>(r.v[v]);
#pragma unroll
            for (int i = 0; i < (F32 ? 2 : 1); ++i) {
                to[i] = make_uint4(0u, 0u, 0u, 0u);
                if (c < D) to[i] = reinterpret_cast<const uint4*>(row + c * (F32 ? 4 : 2))[i];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; e += W) {
                const int c = min(ln_col<W, LPR>(lane, v, e), D - W);   // ln_values leaves out what is behind D
                if constexpr (F32 && W == 2) {
                    const uint2 x = *reinterpret_cast<const uint2*>(row + 4 * c);
                    r.v[v][e] = x.x;
                    r.v[v][e + 1] = x.y;
                } else if constexpr (F32) {
                    r.v[v][e] = *reinterpret_cast<const unsigned*>(row + 4 * c);
                } else if constexpr (W == 2) {
                    r.v[v][e / 2] = *reinterpret_cast<const unsigned*>(row + 2 * c);
                } else {
                    r.v[v][e] = *reinterpret_cast<const unsigned short*>(row + 2 * c);
                }
            }
        }
    }
}
template <int W, bool F32, int LPR, int VPT>
__device__ __forceinline__ void ln_values(const LnRaw<W, F32, VPT>& r, int D, int lane, float (&x)[VPT][8]) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            unsigned u;
            if constexpr (F32) u = r.v[v][e];
            else if constexpr (W == 1) u = r.v[v][e] << 16;
            else u = e % 2 ? r.v[v][e / 2] & 0xffff0000u : r.v[v][e / 2] << 16;
            x[v][e] = W == 8 || ln_col<W, LPR>(lane, v, e) < D ? __uint_as_float(u) : 0.f;
        }
    }
}

template <int W, int LPR, int VPT>
__device__ __forceinline__ void ln_store(void* to, bool f32, int64_t at, int D, int lane, const float (&x)[VPT][8]) {
    typedef float lnfw __attribute__((ext_vector_type(W)));
    typedef __bf16 lnbw __attribute__((ext_vector_type(W)));
    char* base = (char*)to;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
#pragma unroll
        for (int e0 = 0; e0 < 8; e0 += W) {
            const int c = ln_col<W, LPR>(lane, v, e0);
            if (c >= D) continue;
            lnfw f;
#pragma unroll
            for (int e = 0; e < W; ++e) f[e] = x[v][e0 + e];
            if (f32) *reinterpret_cast<lnfw*>(base + (at + c) * 4) = f;
            else *reinterpret_cast<lnbw*>(base + (at + c) * 2) = __builtin_convertvector(f, lnbw);
        }
    }
}

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
__device__ __forceinline__ void ln_row(const LnArgs& a, unsigned g, unsigned r, unsigned& b, unsigned& h, unsigned& l) {
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

// Rows of a lane group's pass.  The next pass's rows are loaded while one is
// computed, so that memory is never waited for by every workgroup at once; not
// where a row's 64 values per lane leave no registers for that (backward of 2048
// x 16384 bf16: 110 us, with it 166).
template <int VPT>
constexpr int ln_rows() { return VPT == 1 ? 2 : 1; }
template <int VPT>
constexpr bool ln_ahead() { return VPT < 8; }

template <int W, bool FX, int LPR, int VPT>
__global__ __launch_bounds__(kLnThreads) void ln_fwd_kernel(LnArgs a) {
    constexpr int RPB = kLnThreads / LPR, RU = ln_rows<VPT>();
    __shared__ float2 red[8];
    int turn = 0;
    // groups side by side: rows of the same tokens are near each other in a
    // token-major tensor
    const unsigned g = blockIdx.x % a.groups, blk = blockIdx.x / a.groups;
    const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
    float w[VPT][8], bs[VPT][8];
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = ln_col<W, LPR>(lane, v, e);
            w[v][e] = c < a.D ? (a.w ? a.w[(size_t)g * a.D + c] : 1.f) : 0.f;
            bs[v][e] = c < a.D && a.bias ? a.bias[(size_t)g * a.D + c] : 0.f;
        }
    const float D = (float)a.D, inv = 1.f / D;
    LnRaw<W, FX, VPT> raw[RU], next[RU];
    unsigned b[RU], h[RU], l[RU], nb[RU], nh[RU], nl[RU];
    auto fetch = [&](unsigned r0) {
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            ln_row(a, g, min(r0 + u * RPB + sub, a.rows - 1), nb[u], nh[u], nl[u]);
            ln_fetch<W, FX, LPR, VPT>(a.x, ln_at(a.sx, nb[u], nh[u], nl[u]), a.D, lane, next[u]);
        }
    };
    const unsigned step = a.blocks * (RPB * RU);
    if (ln_ahead<VPT>()) fetch(blk * (RPB * RU));
    for (unsigned r0 = blk * (RPB * RU); r0 < a.rows; r0 += step) {
        if (!ln_ahead<VPT>()) fetch(r0);
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            raw[u] = next[u];
            b[u] = nb[u];
            h[u] = nh[u];
            l[u] = nl[u];
        }
        if (ln_ahead<VPT>() && r0 + step < a.rows) fetch(r0 + step);
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            float x[VPT][8], s = 0.f;
            ln_values<W, FX, LPR>(raw[u], a.D, lane, x);
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int e = 0; e < 8; ++e) s += x[v][e];
            const float mean = ln_div(ln_sum<LPR>(s, red, turn), D, inv);
            s = 0.f;
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[v][e] = ln_col<W, LPR>(lane, v, e) < a.D ? x[v][e] - mean : 0.f;
                    s += x[v][e] * x[v][e];
                }
            const float rstd = ln_rsqrt(ln_div(ln_sum<LPR>(s, red, turn), D, inv) + a.eps);
            if (r0 + u * RPB + sub >= a.rows) continue;
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int e = 0; e < 8; ++e) x[v][e] = x[v][e] * rstd * w[v][e] + bs[v][e];
            ln_store<W, LPR, VPT>(a.y, a.y_f32, ln_at(a.sy, b[u], h[u], l[u]), a.D, lane, x);
            if (lane == 0) {
                const size_t at = ((size_t)b[u] * a.H + h[u]) * a.L + l[u];
                if (a.mean_out) a.mean_out[at] = mean;
                if (a.rstd_out) a.rstd_out[at] = rstd;
            }
        }
    }
}

template <int W, bool FX, bool FDY, int LPR, int VPT>
__global__ __launch_bounds__(kLnThreads) void ln_bwd_kernel(LnArgs a) {
    constexpr int RPB = kLnThreads / LPR, RU = ln_rows<VPT>();
    constexpr int NCOL = 8 * VPT * LPR;   // columns that the lanes of a row hold
    constexpr int PARTS = LPR <= 64 ? 4 : LPR == 128 ? 2 : 1;
    __shared__ float2 red[8];
    __shared__ float acc[PARTS][PARTS > 1 ? NCOL : 1];
    int turn = 0;
    const unsigned g = blockIdx.x % a.groups, blk = blockIdx.x / a.groups;
    const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
    float w[VPT][8], dw[VPT][8], db[VPT][8];
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = ln_col<W, LPR>(lane, v, e);
            w[v][e] = c < a.D ? (a.w ? a.w[(size_t)g * a.D + c] : 1.f) : 0.f;
            dw[v][e] = db[v][e] = 0.f;
        }
    const float D = (float)a.D, inv = 1.f / D;
    LnRaw<W, FX, VPT> rx[RU], nx[RU];
    LnRaw<W, FDY, VPT> ry[RU], ny[RU];
    float mean[RU], rstd[RU], nm[RU], nr[RU];
    int64_t at[RU], nat[RU];
    auto fetch = [&](unsigned r0) {
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            unsigned b, h, l;
            ln_row(a, g, min(r0 + u * RPB + sub, a.rows - 1), b, h, l);
            const size_t stat = ((size_t)b * a.H + h) * a.L + l;
            nm[u] = a.mean[stat];
            nr[u] = a.rstd[stat];
            nat[u] = ln_at(a.sy, b, h, l);
            ln_fetch<W, FX, LPR, VPT>(a.x, ln_at(a.sx, b, h, l), a.D, lane, nx[u]);
            ln_fetch<W, FDY, LPR, VPT>(a.dy, ln_at(a.sdy, b, h, l), a.D, lane, ny[u]);
        }
    };
    const unsigned step = a.blocks * (RPB * RU);
    if (ln_ahead<VPT>()) fetch(blk * (RPB * RU));
    for (unsigned r0 = blk * (RPB * RU); r0 < a.rows; r0 += step) {
        if (!ln_ahead<VPT>()) fetch(r0);
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            rx[u] = nx[u];
            ry[u] = ny[u];
            mean[u] = nm[u];
            rstd[u] = nr[u];
            at[u] = nat[u];
        }
        if (ln_ahead<VPT>() && r0 + step < a.rows) fetch(r0 + step);
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            const bool ok = r0 + u * RPB + sub < a.rows;
            float x[VPT][8], dy[VPT][8], s1 = 0.f, s2 = 0.f;
            ln_values<W, FX, LPR>(rx[u], a.D, lane, x);
            ln_values<W, FDY, LPR>(ry[u], a.D, lane, dy);
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[v][e] = (x[v][e] - mean[u]) * rstd[u];   // behind D: dy and w are zero there
                    if (ok) {
                        dw[v][e] += dy[v][e] * x[v][e];
                        db[v][e] += dy[v][e];
                    }
                    dy[v][e] *= w[v][e];
                    s1 += dy[v][e];
                    s2 += dy[v][e] * x[v][e];
                }
            ln_sum2<LPR>(s1, s2, red, turn);
            s1 = ln_div(s1, D, inv);
            s2 = ln_div(s2, D, inv);
            if (!ok) continue;
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int e = 0; e < 8; ++e) x[v][e] = rstd[u] * (dy[v][e] - s1 - x[v][e] * s2);
            ln_store<W, LPR, VPT>(a.y, a.y_f32, at[u], a.D, lane, x);
        }
    }
    if (!a.part) return;
    // the workgroup's sums: over the rows of a wave by shuffles, then over the
    // four waves through LDS
    float* part = a.part + ((size_t)g * a.blocks + blk) * 2 * a.D;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float(&s)[VPT][8] = k == 0 ? dw : db;
        if constexpr (PARTS == 1) {
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int c = ln_col<W, LPR>(lane, v, e);
                    if (c < a.D) part[(size_t)k * a.D + c] = s[v][e];
                }
        } else {
            const int at = threadIdx.x / (kLnThreads / PARTS);
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
#pragma unroll
                    for (int d = LPR; d < 64; d <<= 1) s[v][e] += __shfl_xor(s[v][e], d);
                    if (LPR >= 64 || (threadIdx.x & 63) < LPR) acc[at][ln_col<W, LPR>(lane, v, e)] = s[v][e];
                }
            __syncthreads();
            for (int c = threadIdx.x; c < a.D; c += kLnThreads) {
                float x = acc[0][c] + acc[1][c];
                if constexpr (PARTS == 4) x += acc[2][c] + acc[3][c];
                part[(size_t)k * a.D + c] = x;
            }
            __syncthreads();
        }
    }
}

// dw and db from the workgroups' sums: 32 columns per workgroup and turn; each of
// 32 threads per column adds every 32nd workgroup's sum, then the 32 are added, in
// fp64 (a sum of many rows is small against its terms).  The grid is capped (a
// launch holds fewer than 2^32 threads, which 65536 heads of 1024 columns pass);
// below the cap every workgroup has one turn.
constexpr unsigned kLnSumGrid = 1u << 16;

__global__ __launch_bounds__(1024) void ln_bwd_sum_kernel(LnArgs a, unsigned tiles) {
    __shared__ double red[32][33];
    const unsigned cols = 2 * (unsigned)a.D, per = (cols + 31) / 32;
    const unsigned lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    for (unsigned tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const unsigned g = tile / per;
        const unsigned c = (tile % per) * 32 + lane;
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
            if (c < (unsigned)a.D) {
                if (a.dw) a.dw[(size_t)g * a.D + c] = (float)s;
            } else if (a.db) {
                a.db[(size_t)g * a.D + c - a.D] = (float)s;
            }
        }
    }
}

__global__ __launch_bounds__(256) void ln_zero_kernel(float* p, size_t n) {
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) p[i] = 0.f;
}

int ln_pass_rows(int D) {
    const LnShape s = ln_shape(D);
    return kLnThreads / s.lanes * (s.vecs == 1 ? ln_rows<1>() : ln_rows<2>());
}

template <bool BWD, int W, bool FX, bool FDY, int LPR, int VPT>
static hipError_t ln_launch(const LnArgs& a, int slot, hipStream_t st) {
    const dim3 grid(a.groups * a.blocks);
    if constexpr (BWD) return launch_k(slot, ln_bwd_kernel<W, FX, FDY, LPR, VPT>, grid, dim3(kLnThreads), 0, st, a);
    else return launch_k(slot, ln_fwd_kernel<W, FX, LPR, VPT>, grid, dim3(kLnThreads), 0, st, a);
}

template <bool BWD, int W, bool FX, bool FDY>
static hipError_t ln_launch_shape(const LnArgs& a, int slot, hipStream_t st) {
    const LnShape s = ln_shape(a.D);
    if (s.lanes == 8) return ln_launch<BWD, W, FX, FDY, 8, 1>(a, slot, st);
    if (s.lanes == 16) return ln_launch<BWD, W, FX, FDY, 16, 1>(a, slot, st);
    if (s.lanes == 32) return ln_launch<BWD, W, FX, FDY, 32, 1>(a, slot, st);
    if (s.lanes == 64) return ln_launch<BWD, W, FX, FDY, 64, 1>(a, slot, st);
    if (s.lanes == 128) return ln_launch<BWD, W, FX, FDY, 128, 1>(a, slot, st);
    if (s.vecs == 1) return ln_launch<BWD, W, FX, FDY, 256, 1>(a, slot, st);
    if (s.vecs == 2) return ln_launch<BWD, W, FX, FDY, 256, 2>(a, slot, st);
    if (s.vecs == 4) return ln_launch<BWD, W, FX, FDY, 256, 4>(a, slot, st);
    return ln_launch<BWD, W, FX, FDY, 256, 8>(a, slot, st);
}

template <bool BWD, int W>
static hipError_t ln_launch_types(const LnArgs& a, int slot, hipStream_t st) {
    if constexpr (BWD) {
        if (a.x_f32)
            return a.dy_f32 ? ln_launch_shape<BWD, W, true, true>(a, slot, st)
                            : ln_launch_shape<BWD, W, true, false>(a, slot, st);
        return a.dy_f32 ? ln_launch_shape<BWD, W, false, true>(a, slot, st)
                        : ln_launch_shape<BWD, W, false, false>(a, slot, st);
    } else {
        return a.x_f32 ? ln_launch_shape<BWD, W, true, false>(a, slot, st)
                       : ln_launch_shape<BWD, W, false, false>(a, slot, st);
    }
}

template <bool BWD>
static hipError_t ln_launch_width(const LnArgs& a, int width, int slot, hipStream_t st) {
    if (width == 8) return ln_launch_types<BWD, 8>(a, slot, st);
    if (width == 2) return ln_launch_types<BWD, 2>(a, slot, st);
    return ln_launch_types<BWD, 1>(a, slot, st);
}

hipError_t launch_ln_fwd(const LnArgs& a, int width, int slot, hipStream_t st) {
    return ln_launch_width<false>(a, width, slot, st);
}

hipError_t launch_ln_bwd(const LnArgs& a, int width, int slot, hipStream_t st) {
    hipError_t e = ln_launch_width<true>(a, width, slot, st);
    if (e == hipSuccess && a.part) {
        const unsigned tiles = a.groups * ((unsigned)(2 * a.D + 31) / 32);   // at most 2^20 * 2^10
        e = launch_k(slot, ln_bwd_sum_kernel, dim3(tiles < kLnSumGrid ? tiles : kLnSumGrid), dim3(1024), 0, st, a, tiles);
    }
    return e;
}

hipError_t launch_ln_zero(float* p, size_t n, int slot, hipStream_t st) {
    const size_t blocks = (n + 255) / 256;
    return launch_k(slot, ln_zero_kernel, dim3((unsigned)(blocks < 1024 ? blocks : 1024)), dim3(256), 0, st, p, n);
}

}  // namespace dr
