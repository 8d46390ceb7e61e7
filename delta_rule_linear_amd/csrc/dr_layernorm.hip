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
// stay in registers; the workgroups' sums are added in a fixed order by a
// second kernel.  All arithmetic is fp32.

#include <hip/hip_runtime.h>

#include "dr_device.h"
#include "dr_internal.h"
#include "dr_layernorm.h"

namespace dr {

typedef __bf16 lnbf8 __attribute__((ext_vector_type(8)));
typedef float lnf8 __attribute__((ext_vector_type(8)));

constexpr int kLnThreads = 256;

LnShape ln_shape(int D) {
    // the least lanes that hold a row in 8 values each, up to a wave; then
    // more values per lane; wider rows take the whole workgroup
    if (D <= 64) return {8, 1};
    if (D <= 128) return {16, 1};
    if (D <= 256) return {32, 1};
    if (D <= 512) return {64, 1};
    if (D <= 1024) return {64, 2};
    if (D <= 2048) return {64, 4};
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

template <bool VEC, int LPR, int VPT>
__device__ __forceinline__ void ln_load(const void* base, bool f32, int64_t at, int D, int lane, float (&x)[VPT][8]) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        if constexpr (VEC) {
            const int c = ln_col<VEC, LPR>(lane, v, 0);
            if (c < D) {
                if (f32) load_n<true, 8>(base, (size_t)(at + c), x[v]);
                else load_n<false, 8>(base, (size_t)(at + c), x[v]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[v][e] = 0.f;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = ln_col<VEC, LPR>(lane, v, e);
                x[v][e] = 0.f;
                if (c < D) x[v][e] = f32 ? load1<true>(base, (size_t)(at + c)) : load1<false>(base, (size_t)(at + c));
            }
        }
    }
}

template <bool VEC, int LPR, int VPT>
__device__ __forceinline__ void ln_store(void* base, bool f32, int64_t at, int D, int lane, const float (&x)[VPT][8]) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        if constexpr (VEC) {
            const int c = ln_col<VEC, LPR>(lane, v, 0);
            if (c >= D) continue;
            lnf8 f;
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = x[v][e];
            if (f32) *reinterpret_cast<lnf8*>((float*)base + at + c) = f;
            else *reinterpret_cast<lnbf8*>((__bf16*)base + at + c) = __builtin_convertvector(f, lnbf8);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = ln_col<VEC, LPR>(lane, v, e);
                if (c >= D) continue;
                if (f32) ((float*)base)[at + c] = x[v][e];
                else ((__bf16*)base)[at + c] = (__bf16)x[v][e];
            }
        }
    }
}

// Sum over the lanes of a row, in every one of them.  red: one float per wave.
template <int LPR>
__device__ __forceinline__ float ln_sum(float x, float* red) {
#pragma unroll
    for (int d = 1; d < (LPR < 64 ? LPR : 64); d <<= 1) x += __shfl_xor(x, d);
    if constexpr (LPR > 64) {
        __syncthreads();   // the last sum has been read
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
        __syncthreads();
        x = (red[0] + red[1]) + (red[2] + red[3]);
    }
    return x;
}

// Row r of a group: its index among the statistics and its strided offset.
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

// Rows that a lane group has in flight: short rows leave room for several.
template <int VPT>
constexpr int ln_rows_fwd() { return VPT == 1 ? 4 : VPT == 2 ? 2 : 1; }
template <int VPT>
constexpr int ln_rows_bwd() { return VPT == 1 ? 2 : 1; }

template <bool VEC, int LPR, int VPT>
__global__ __launch_bounds__(kLnThreads) void ln_fwd_kernel(LnArgs a) {
    constexpr int RPB = kLnThreads / LPR, RU = ln_rows_fwd<VPT>();   // rows at a time, and in flight of each
    __shared__ float red[4];
    const unsigned g = blockIdx.x / a.blocks, blk = blockIdx.x % a.blocks;
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
    const float rD = (float)a.D;
    for (unsigned r0 = blk * (RPB * RU); r0 < a.rows; r0 += a.blocks * (RPB * RU)) {
        float x[RU][VPT][8];
        unsigned b[RU], h[RU], l[RU];
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            const unsigned r = r0 + u * RPB + sub;
            ln_row(a, g, r < a.rows ? r : a.rows - 1, b[u], h[u], l[u]);
            ln_load<VEC, LPR, VPT>(a.x, a.x_f32, b[u] * a.sx.b + h[u] * a.sx.h + l[u] * a.sx.t, a.D, lane, x[u]);
        }
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            float s = 0.f;
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int e = 0; e < 8; ++e) s += x[u][v][e];
            const float mean = ln_sum<LPR>(s, red) / rD;
            s = 0.f;
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[u][v][e] = ln_col<VEC, LPR>(lane, v, e) < a.D ? x[u][v][e] - mean : 0.f;
                    s += x[u][v][e] * x[u][v][e];
                }
            const float rstd = 1.f / sqrtf(ln_sum<LPR>(s, red) / rD + a.eps);
            if (r0 + u * RPB + sub >= a.rows) continue;
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int e = 0; e < 8; ++e) x[u][v][e] = x[u][v][e] * rstd * w[v][e] + bs[v][e];
            ln_store<VEC, LPR, VPT>(a.y, a.y_f32, b[u] * a.sy.b + h[u] * a.sy.h + l[u] * a.sy.t, a.D, lane, x[u]);
            if (lane == 0) {
                const size_t at = ((size_t)b[u] * a.H + h[u]) * a.L + l[u];
                if (a.mean_out) a.mean_out[at] = mean;
                if (a.rstd_out) a.rstd_out[at] = rstd;
            }
        }
    }
}

template <bool VEC, int LPR, int VPT>
__global__ __launch_bounds__(kLnThreads) void ln_bwd_kernel(LnArgs a) {
    constexpr int RPB = kLnThreads / LPR, RU = ln_rows_bwd<VPT>();
    constexpr int NCOL = 8 * VPT * LPR;   // columns that the lanes of a row hold
    __shared__ float red[4];
    __shared__ float acc[LPR <= 64 ? 4 : 1][LPR <= 64 ? NCOL : 1];
    const unsigned g = blockIdx.x / a.blocks, blk = blockIdx.x % a.blocks;
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
    const float rD = (float)a.D;
    for (unsigned r0 = blk * (RPB * RU); r0 < a.rows; r0 += a.blocks * (RPB * RU)) {
        float x[RU][VPT][8], dy[RU][VPT][8], mean[RU], rstd[RU];
        unsigned b[RU], h[RU], l[RU];
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            const unsigned r = r0 + u * RPB + sub;
            ln_row(a, g, r < a.rows ? r : a.rows - 1, b[u], h[u], l[u]);
            const size_t at = ((size_t)b[u] * a.H + h[u]) * a.L + l[u];
            mean[u] = a.mean[at];
            rstd[u] = a.rstd[at];
            ln_load<VEC, LPR, VPT>(a.x, a.x_f32, b[u] * a.sx.b + h[u] * a.sx.h + l[u] * a.sx.t, a.D, lane, x[u]);
            ln_load<VEC, LPR, VPT>(a.dy, a.dy_f32, b[u] * a.sdy.b + h[u] * a.sdy.h + l[u] * a.sdy.t, a.D, lane, dy[u]);
        }
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            const bool ok = r0 + u * RPB + sub < a.rows;
            float s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[u][v][e] = (x[u][v][e] - mean[u]) * rstd[u];   // behind D: dy and w are zero there
                    if (ok) {
                        dw[v][e] += dy[u][v][e] * x[u][v][e];
                        db[v][e] += dy[u][v][e];
                    }
                    dy[u][v][e] *= w[v][e];
                    s1 += dy[u][v][e];
                    s2 += dy[u][v][e] * x[u][v][e];
                }
            s1 = ln_sum<LPR>(s1, red) / rD;
            s2 = ln_sum<LPR>(s2, red) / rD;
            if (!ok) continue;
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int e = 0; e < 8; ++e) x[u][v][e] = rstd[u] * (dy[u][v][e] - s1 - x[u][v][e] * s2);
            ln_store<VEC, LPR, VPT>(a.y, a.y_f32, b[u] * a.sy.b + h[u] * a.sy.h + l[u] * a.sy.t, a.D, lane, x[u]);
        }
    }
    if (!a.part) return;
    // the workgroup's sums: over the rows of a wave by shuffles, then over the
    // four waves through LDS
    float* part = a.part + ((size_t)g * a.blocks + blk) * 2 * a.D;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float(&s)[VPT][8] = k == 0 ? dw : db;
        if constexpr (LPR > 64) {
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int c = ln_col<VEC, LPR>(lane, v, e);
                    if (c < a.D) part[(size_t)k * a.D + c] = s[v][e];
                }
        } else {
            const int wave = threadIdx.x >> 6;
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
#pragma unroll
                    for (int d = LPR; d < 64; d <<= 1) s[v][e] += __shfl_xor(s[v][e], d);
                    if ((threadIdx.x & 63) < LPR) acc[wave][ln_col<VEC, LPR>(lane, v, e)] = s[v][e];
                }
            __syncthreads();
            for (int c = threadIdx.x; c < a.D; c += kLnThreads)
                part[(size_t)k * a.D + c] = (acc[0][c] + acc[1][c]) + (acc[2][c] + acc[3][c]);
            __syncthreads();
        }
    }
}

// dw and db from the workgroups' sums: 32 columns per workgroup; each of 32
// threads per column adds every 32nd workgroup's sum, then the 32 are added.
__global__ __launch_bounds__(1024) void ln_bwd_sum_kernel(LnArgs a) {
    __shared__ float red[32][33];
    const unsigned cols = 2 * (unsigned)a.D, per = (cols + 31) / 32;
    const unsigned g = blockIdx.x / per;
    const unsigned lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const unsigned c = (blockIdx.x % per) * 32 + lane;
    float s = 0.f;
    if (c < cols) {
        const float* p = a.part + (size_t)g * a.blocks * cols + c;
#pragma unroll 8
        for (unsigned k = slice; k < a.blocks; k += 32) s += p[(size_t)k * cols];
    }
    red[slice][lane] = s;
    __syncthreads();
    if (slice == 0 && c < cols) {
        s = 0.f;
#pragma unroll
        for (int k = 0; k < 32; ++k) s += red[k][lane];
        if (c < (unsigned)a.D) {
            if (a.dw) a.dw[(size_t)g * a.D + c] = s;
        } else if (a.db) {
            a.db[(size_t)g * a.D + c - a.D] = s;
        }
    }
}

__global__ __launch_bounds__(256) void ln_zero_kernel(float* p, size_t n) {
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) p[i] = 0.f;
}

int ln_pass_rows(int D, bool bwd) {
    const LnShape s = ln_shape(D);
    const int rows = bwd ? (s.vecs == 1 ? ln_rows_bwd<1>() : ln_rows_bwd<2>())
                         : (s.vecs == 1 ? ln_rows_fwd<1>() : s.vecs == 2 ? ln_rows_fwd<2>() : ln_rows_fwd<4>());
    return kLnThreads / s.lanes * rows;
}

template <bool BWD, bool VEC, int LPR, int VPT>
static hipError_t ln_launch(const LnArgs& a, int slot, hipStream_t st) {
    const dim3 grid(a.groups * a.blocks);
    if constexpr (BWD) return launch_k(slot, ln_bwd_kernel<VEC, LPR, VPT>, grid, dim3(kLnThreads), 0, st, a);
    else return launch_k(slot, ln_fwd_kernel<VEC, LPR, VPT>, grid, dim3(kLnThreads), 0, st, a);
}

template <bool BWD, bool VEC>
static hipError_t ln_launch_shape(const LnArgs& a, int slot, hipStream_t st) {
    const LnShape s = ln_shape(a.D);
    if (s.lanes == 8) return ln_launch<BWD, VEC, 8, 1>(a, slot, st);
    if (s.lanes == 16) return ln_launch<BWD, VEC, 16, 1>(a, slot, st);
    if (s.lanes == 32) return ln_launch<BWD, VEC, 32, 1>(a, slot, st);
    if (s.lanes == 64) {
        if (s.vecs == 1) return ln_launch<BWD, VEC, 64, 1>(a, slot, st);
        if (s.vecs == 2) return ln_launch<BWD, VEC, 64, 2>(a, slot, st);
        return ln_launch<BWD, VEC, 64, 4>(a, slot, st);
    }
    if (s.vecs == 2) return ln_launch<BWD, VEC, 256, 2>(a, slot, st);
    if (s.vecs == 4) return ln_launch<BWD, VEC, 256, 4>(a, slot, st);
    return ln_launch<BWD, VEC, 256, 8>(a, slot, st);
}

hipError_t launch_ln_fwd(const LnArgs& a, bool vec, int slot, hipStream_t st) {
    return vec ? ln_launch_shape<false, true>(a, slot, st) : ln_launch_shape<false, false>(a, slot, st);
}

hipError_t launch_ln_bwd(const LnArgs& a, bool vec, int slot, hipStream_t st) {
    hipError_t e = vec ? ln_launch_shape<true, true>(a, slot, st) : ln_launch_shape<true, false>(a, slot, st);
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
