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
// y token-major) 58 us for 272 MB, 4.7 TB/s (a large copy reaches 5.2); its
// backward 82 us for 403 MB, 4.9 TB/s, and 4.5 for the sums; 8191 x 2048 bf16
// backward 27 us for 101 MB (3.7 TB/s, of which four rows per workgroup and 256
// workgroups' start are a part) and 4.

#include <hip/hip_runtime.h>

#include "dr_device.h"
#include "dr_internal.h"
#include "dr_layernorm.h"

namespace dr {

typedef __bf16 lnbf8 __attribute__((ext_vector_type(8)));
typedef float lnf8 __attribute__((ext_vector_type(8)));

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

// Column of value e of vector v of a lane.  VEC: eight consecutive values;
// otherwise consecutive lanes take consecutive values.
template <bool VEC, int LPR>
__device__ __forceinline__ int ln_col(int lane, int v, int e) {
    return VEC ? 8 * (v * LPR + lane) + e : (8 * v + e) * LPR + lane;
}

// A lane's part of a row as loaded: bf16 or fp32 bits (VEC), or fp32 values.
template <bool VEC, bool F32, int VPT>
struct LnRaw {
    uint4 v[VPT][F32 || !VEC ? 2 : 1];
};

template <bool VEC, bool F32, int LPR, int VPT>
__device__ __forceinline__ void ln_fetch(const void* base, int64_t at, int D, int lane, LnRaw<VEC, F32, VPT>& r) {
    constexpr int W = F32 || !VEC ? 2 : 1;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        if constexpr (VEC) {
            const int c = ln_col<VEC, LPR>(lane, v, 0);
#pragma unroll
            for (int i = 0; i < W; ++i) {
                r.v[v][i] = make_uint4(0u, 0u, 0u, 0u);
                if (c < D) r.v[v][i] = reinterpret_cast<const uint4*>((const char*)base + (at + c) * (F32 ? 4 : 2))[i];
            }
        } else {
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = ln_col<VEC, LPR>(lane, v, e);
                x[e] = 0.f;
                if (c < D) x[e] = load1<F32>(base, (size_t)(at + c));
            }
            r.v[v][0] = __builtin_bit_cast(uint4, f32x4{x[0], x[1], x[2], x[3]});
            r.v[v][1] = __builtin_bit_cast(uint4, f32x4{x[4], x[5], x[6], x[7]});
        }
    }
}
template <bool VEC, bool F32, int VPT>
__device__ __forceinline__ void ln_values(const LnRaw<VEC, F32, VPT>& r, float (&x)[VPT][8]) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        if constexpr (VEC && !F32) {
            unpack_bf16x8(r.v[v][0], x[v]);
        } else {
            const f32x4 a = __builtin_bit_cast(f32x4, r.v[v][0]), b = __builtin_bit_cast(f32x4, r.v[v][1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[v][e] = a[e];
                x[v][4 + e] = b[e];
            }
        }
    }
}

template <bool VEC, int LPR, int VPT>
__device__ __forceinline__ void ln_store(void* to, bool f32, int64_t at, int D, int lane, const float (&x)[VPT][8]) {
    char* base = (char*)to;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        if constexpr (VEC) {
            const int c = ln_col<VEC, LPR>(lane, v, 0);
            if (c >= D) continue;
            lnf8 f;
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = x[v][e];
            if (f32) *reinterpret_cast<lnf8*>(base + (at + c) * 4) = f;
            else *reinterpret_cast<lnbf8*>(base + (at + c) * 2) = __builtin_convertvector(f, lnbf8);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = ln_col<VEC, LPR>(lane, v, e);
                if (c >= D) continue;
                if (f32) *reinterpret_cast<float*>(base + (at + c) * 4) = x[v][e];
                else *reinterpret_cast<__bf16*>(base + (at + c) * 2) = (__bf16)x[v][e];
            }
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
// computed, so that memory is never waited for by every workgroup at once.
template <int VPT>
constexpr int ln_rows() { return VPT == 1 ? 2 : 1; }

template <bool VEC, bool FX, int LPR, int VPT>
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
            const int c = ln_col<VEC, LPR>(lane, v, e);
            w[v][e] = c < a.D ? (a.w ? a.w[(size_t)g * a.D + c] : 1.f) : 0.f;
            bs[v][e] = c < a.D && a.bias ? a.bias[(size_t)g * a.D + c] : 0.f;
        }
    const float D = (float)a.D, inv = 1.f / D;
    LnRaw<VEC, FX, VPT> raw[RU], next[RU];
    unsigned b[RU], h[RU], l[RU], nb[RU], nh[RU], nl[RU];
    auto fetch = [&](unsigned r0) {
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            ln_row(a, g, min(r0 + u * RPB + sub, a.rows - 1), nb[u], nh[u], nl[u]);
            ln_fetch<VEC, FX, LPR, VPT>(a.x, ln_at(a.sx, nb[u], nh[u], nl[u]), a.D, lane, next[u]);
        }
    };
    const unsigned step = a.blocks * (RPB * RU);
    fetch(blk * (RPB * RU));
    for (unsigned r0 = blk * (RPB * RU); r0 < a.rows; r0 += step) {
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            raw[u] = next[u];
            b[u] = nb[u];
            h[u] = nh[u];
            l[u] = nl[u];
        }
        if (r0 + step < a.rows) fetch(r0 + step);
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            float x[VPT][8], s = 0.f;
            ln_values(raw[u], x);
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
                    x[v][e] = ln_col<VEC, LPR>(lane, v, e) < a.D ? x[v][e] - mean : 0.f;
                    s += x[v][e] * x[v][e];
                }
            const float rstd = ln_rsqrt(ln_div(ln_sum<LPR>(s, red, turn), D, inv) + a.eps);
            if (r0 + u * RPB + sub >= a.rows) continue;
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int e = 0; e < 8; ++e) x[v][e] = x[v][e] * rstd * w[v][e] + bs[v][e];
            ln_store<VEC, LPR, VPT>(a.y, a.y_f32, ln_at(a.sy, b[u], h[u], l[u]), a.D, lane, x);
            if (lane == 0) {
                const size_t at = ((size_t)b[u] * a.H + h[u]) * a.L + l[u];
                if (a.mean_out) a.mean_out[at] = mean;
                if (a.rstd_out) a.rstd_out[at] = rstd;
            }
        }
    }
}

template <bool VEC, bool FX, bool FDY, int LPR, int VPT>
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
            const int c = ln_col<VEC, LPR>(lane, v, e);
            w[v][e] = c < a.D ? (a.w ? a.w[(size_t)g * a.D + c] : 1.f) : 0.f;
            dw[v][e] = db[v][e] = 0.f;
        }
    const float D = (float)a.D, inv = 1.f / D;
    LnRaw<VEC, FX, VPT> rx[RU], nx[RU];
    LnRaw<VEC, FDY, VPT> ry[RU], ny[RU];
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
            ln_fetch<VEC, FX, LPR, VPT>(a.x, ln_at(a.sx, b, h, l), a.D, lane, nx[u]);
            ln_fetch<VEC, FDY, LPR, VPT>(a.dy, ln_at(a.sdy, b, h, l), a.D, lane, ny[u]);
        }
    };
    const unsigned step = a.blocks * (RPB * RU);
    fetch(blk * (RPB * RU));
    for (unsigned r0 = blk * (RPB * RU); r0 < a.rows; r0 += step) {
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            rx[u] = nx[u];
            ry[u] = ny[u];
            mean[u] = nm[u];
            rstd[u] = nr[u];
            at[u] = nat[u];
        }
        if (r0 + step < a.rows) fetch(r0 + step);
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            const bool ok = r0 + u * RPB + sub < a.rows;
            float x[VPT][8], dy[VPT][8], s1 = 0.f, s2 = 0.f;
            ln_values(rx[u], x);
            ln_values(ry[u], dy);
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
            ln_store<VEC, LPR, VPT>(a.y, a.y_f32, at[u], a.D, lane, x);
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
                    const int c = ln_col<VEC, LPR>(lane, v, e);
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
                    if (LPR >= 64 || (threadIdx.x & 63) < LPR) acc[at][ln_col<VEC, LPR>(lane, v, e)] = s[v][e];
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

// dw and db from the workgroups' sums: 32 columns per workgroup; each of 32
// threads per column adds every 32nd workgroup's sum, then the 32 are added, in
// fp64 (a sum of many rows is small against its terms).
__global__ __launch_bounds__(1024) void ln_bwd_sum_kernel(LnArgs a) {
    __shared__ double red[32][33];
    const unsigned cols = 2 * (unsigned)a.D, per = (cols + 31) / 32;
    const unsigned g = blockIdx.x / per;
    const unsigned lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const unsigned c = (blockIdx.x % per) * 32 + lane;
    double s = 0.0;
    if (c < cols) {
        const float* p = a.part + (size_t)g * a.blocks * cols + c;
#pragma unroll 8
        for (unsigned k = slice; k < a.blocks; k += 32) s += p[(size_t)k * cols];
    }
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

__global__ __launch_bounds__(256) void ln_zero_kernel(float* p, size_t n) {
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) p[i] = 0.f;
}

int ln_pass_rows(int D) {
    const LnShape s = ln_shape(D);
    return kLnThreads / s.lanes * (s.vecs == 1 ? ln_rows<1>() : ln_rows<2>());
}

template <bool BWD, bool VEC, bool FX, bool FDY, int LPR, int VPT>
static hipError_t ln_launch(const LnArgs& a, int slot, hipStream_t st) {
    const dim3 grid(a.groups * a.blocks);
    if constexpr (BWD) return launch_k(slot, ln_bwd_kernel<VEC, FX, FDY, LPR, VPT>, grid, dim3(kLnThreads), 0, st, a);
    else return launch_k(slot, ln_fwd_kernel<VEC, FX, LPR, VPT>, grid, dim3(kLnThreads), 0, st, a);
}

template <bool BWD, bool VEC, bool FX, bool FDY>
static hipError_t ln_launch_shape(const LnArgs& a, int slot, hipStream_t st) {
    const LnShape s = ln_shape(a.D);
    if (s.lanes == 8) return ln_launch<BWD, VEC, FX, FDY, 8, 1>(a, slot, st);
    if (s.lanes == 16) return ln_launch<BWD, VEC, FX, FDY, 16, 1>(a, slot, st);
    if (s.lanes == 32) return ln_launch<BWD, VEC, FX, FDY, 32, 1>(a, slot, st);
    if (s.lanes == 64) return ln_launch<BWD, VEC, FX, FDY, 64, 1>(a, slot, st);
    if (s.lanes == 128) return ln_launch<BWD, VEC, FX, FDY, 128, 1>(a, slot, st);
    if (s.vecs == 1) return ln_launch<BWD, VEC, FX, FDY, 256, 1>(a, slot, st);
    if (s.vecs == 2) return ln_launch<BWD, VEC, FX, FDY, 256, 2>(a, slot, st);
    if (s.vecs == 4) return ln_launch<BWD, VEC, FX, FDY, 256, 4>(a, slot, st);
    return ln_launch<BWD, VEC, FX, FDY, 256, 8>(a, slot, st);
}

template <bool BWD, bool VEC>
static hipError_t ln_launch_types(const LnArgs& a, int slot, hipStream_t st) {
    if constexpr (BWD) {
        if (a.x_f32)
            return a.dy_f32 ? ln_launch_shape<BWD, VEC, true, true>(a, slot, st)
                            : ln_launch_shape<BWD, VEC, true, false>(a, slot, st);
        return a.dy_f32 ? ln_launch_shape<BWD, VEC, false, true>(a, slot, st)
                        : ln_launch_shape<BWD, VEC, false, false>(a, slot, st);
    } else {
        return a.x_f32 ? ln_launch_shape<BWD, VEC, true, false>(a, slot, st)
                       : ln_launch_shape<BWD, VEC, false, false>(a, slot, st);
    }
}

hipError_t launch_ln_fwd(const LnArgs& a, bool vec, int slot, hipStream_t st) {
    return vec ? ln_launch_types<false, true>(a, slot, st) : ln_launch_types<false, false>(a, slot, st);
}

hipError_t launch_ln_bwd(const LnArgs& a, bool vec, int slot, hipStream_t st) {
    hipError_t e = vec ? ln_launch_types<true, true>(a, slot, st) : ln_launch_types<true, false>(a, slot, st);
    if (e == hipSuccess && a.part) {
        const unsigned per = (unsigned)(2 * a.D + 31) / 32;
        e = launch_k(slot, ln_bwd_sum_kernel, dim3(a.groups * per), dim3(1024), 0, st, a);
    }
    return e;
}

hipError_t launch_ln_zero(float* p, size_t n, int slot, hipStream_t st) {
    const size_t blocks = (n + 255) / 256;
    return launch_k(slot, ln_zero_kernel, dim3((unsigned)(blocks < 1024 ? blocks : 1024)), dim3(256), 0, st, p, n);
}

}  // namespace dr
