// dr_conv.hip -- the short causal convolution of each channel, its backward and one
// token.
//
//   z_t = bias + sum_j w_j x_{t-W+1+j},   y_t = z_t, or z_t sigmoid(z_t)
//   dz_t = dy_t act'(z_t),  dx_t = sum_j w_j dz_{t+W-1-j},  dw_j = sum_t dz_t x_{t-W+1+j},  db = sum_t dz_t
//
// The tokens before the first are the state's W - 1 rows.  A thread has eight
// channels of a run of tokens, the last W rows in registers and the next ones loaded
// ahead; 16 lanes have 128 channels of a token side by side, a workgroup 16 runs, of
// one sequence or several.  Both passes read x (and dy) once, but for the W - 1 rows
// between two runs, and write once: memory bounds them.
//
// Measured: forward of 2 x 16384 x 2048 bf16, W = 4, a slice of wider rows, 62 us for 268
// MB (4.4 TB/s; a large copy reaches 5.2); its backward 93 us for 403 MB (4.3), with two
// waves per SIMD (243 registers: taps, their sums, and the rows of x and dz).

#include <hip/hip_runtime.h>

#include "dr_device.h"
#include "dr_internal.h"
#include "dr_octet.h"
#include "dr_seqops.h"

namespace dr {

constexpr int kScThreads = 256;
constexpr int kScTile = 128;    // channels of a workgroup

// Tokens loaded ahead, a multiple of W: the last W rows are kept in turn in the same
// registers, and in a loop of so many tokens each has its place.
constexpr int sc_ahead(int W) { return W == 2 ? 4 : W; }
int sc_run(int W) { return sc_ahead(W); }

__device__ __forceinline__ float sc_sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504088896340736f * z));
}
// z sigmoid(z); the bound makes it 0 for -infinity (a NaN comes through the sigmoid)
__device__ __forceinline__ float sc_silu(float z) { return __builtin_fmaxf(z, -1e4f) * sc_sigmoid(z); }
// its slope, s (1 + z (1 - s)), with bounds as above for both infinities
__device__ __forceinline__ float sc_slope(float z) {
    const float s = sc_sigmoid(z);
    return s * __builtin_fmaf(__builtin_amdgcn_fmed3f(z, -1e4f, 1e4f), 1.f - s, 1.f);
}

// The rows of a run, one after the other; behind the last one that one again.  They are
// loaded as read once: the outputs stay in the last-level cache instead, for who comes
// next (2 x 16384 x 2048 67 -> 62 us, backward 101 -> 95, then 93).
template <bool F32, bool SMALL>
struct ScRows {
    const char* p;
    int64_t step;
    int left;   // rows behind this one
    __device__ __forceinline__ void next(bool f32, int at, int C, Oct<F32>& r) {
        oct_load<F32, SMALL, true>(p, f32, at, C, r);
        p += left > 0 ? step : 0;
        --left;
    }
};

// Row t of x, of the state's rows before the first token, or zeros.
template <bool FX, bool SMALL>
__device__ __forceinline__ void sc_row(const ScArgs& a, const char* xb, unsigned b, int t, int at, float (&x)[8]) {
    const int xs = a.x_f32 ? 4 : 2;
    Oct<FX> r;
    if (t >= 0) {
        oct_load<FX, SMALL>(xb + (int64_t)t * a.sx.t * xs, a.x_f32, at, a.C, r);
    } else if (a.state) {
        oct_load<FX, SMALL>((const char*)a.state + ((size_t)b * (a.W - 1) + (a.W - 1 + t)) * a.C * xs, a.x_f32, at, a.C, r);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 0.f;
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = oct_value(r, e);
}

template <bool FX, int W, bool SMALL>
__global__ __launch_bounds__(kScThreads) void sc_fwd_kernel(ScArgs a) {
    constexpr int U = sc_ahead(W);
    const int lane = threadIdx.x & 15, sub = threadIdx.x >> 4;
    const unsigned nct = ((unsigned)a.C + kScTile - 1) / kScTile;
    const unsigned per = ((unsigned)a.L + a.run - 1) / a.run;   // runs of a sequence
    const int xs = a.x_f32 ? 4 : 2, ys = a.y_f32 ? 4 : 2;
    for (size_t item = blockIdx.x; item < (size_t)a.tiles * nct; item += gridDim.x) {
        const unsigned ct = (unsigned)(item % nct), run = (unsigned)(item / nct) * 16 + sub;
        const unsigned b = run / per, t0 = (run - b * per) * a.run;
        const OctPlace pl = oct_place(ct * 16 + lane, a.C);
        const char* xb = (const char*)a.x + b * a.sx.b * xs;
        if (b < (unsigned)a.B) {
            const int n = min(a.run, a.L - (int)t0);
            float w[W][8], bias[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = SMALL ? min(e, a.C - 1) : pl.at + e;
#pragma unroll
                for (int j = 0; j < W; ++j) w[j][e] = a.w[(size_t)c * W + j];
                bias[e] = a.bias ? a.bias[c] : 0.f;
            }
            float past[W][8];   // row t in past[(t - t0) % W]
#pragma unroll
            for (int j = 1; j < W; ++j) sc_row<FX, SMALL>(a, xb, b, (int)t0 - W + j, pl.at, past[j]);
            ScRows<FX, SMALL> rows{xb + t0 * a.sx.t * xs, a.sx.t * xs, n - 1};
            char* y = (char*)a.y + (b * a.sy.b + t0 * a.sy.t) * ys;
            Oct<FX> x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) rows.next(a.x_f32, pl.at, a.C, x[u]);
            for (int i = 0; i < n; i += U) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float z[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        past[u % W][e] = oct_value(x[u], e);
                        z[e] = bias[e];
#pragma unroll
                        for (int j = 0; j < W; ++j) z[e] = __builtin_fmaf(w[j][e], past[(u + 1 + j) % W][e], z[e]);
                        if (a.silu) z[e] = sc_silu(z[e]);
                    }
                    if (i + U < n) rows.next(a.x_f32, pl.at, a.C, x[u]);
                    if (i + u < n && pl.own) oct_store<SMALL>(y, a.y_f32, pl, z);
                    y += a.sy.t * ys;
                }
            }
        }
        if (b < (unsigned)a.B && t0 == 0 && a.state_out) {
            // the last W - 1 rows; the only thread that reads the state writes it, so that
            // both may be one tensor
            float s[W - 1][8];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) sc_row<FX, SMALL>(a, xb, b, a.L - (W - 1) + j, pl.at, s[j]);
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
                if (pl.own)
                    oct_store<SMALL>((char*)a.state_out + ((size_t)b * (W - 1) + j) * a.C * xs, a.x_f32, pl, s[j]);
        }
    }
}

template <bool FX, int W, bool SMALL>
__global__ __launch_bounds__(kScThreads) void sc_step_kernel(ScArgs a) {
    const unsigned per = ((unsigned)a.C + 7) / 8;
    const size_t n = (size_t)a.B * per;
    const int xs = a.x_f32 ? 4 : 2, ys = a.y_f32 ? 4 : 2;
    for (size_t i = (size_t)blockIdx.x * kScThreads + threadIdx.x; i < n; i += (size_t)gridDim.x * kScThreads) {
        const size_t b = i / per;
        const OctPlace pl = oct_place((int)(i - b * per), a.C);
        char* st = (char*)a.state_out + b * (W - 1) * a.C * xs;
        float z[8], row[8];
        Oct<FX> r[W];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) oct_load<FX, SMALL>(st + (size_t)j * a.C * xs, a.x_f32, pl.at, a.C, r[j]);
        oct_load<FX, SMALL>((const char*)a.x + b * a.C * xs, a.x_f32, pl.at, a.C, r[W - 1]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = SMALL ? min(e, a.C - 1) : pl.at + e;
            z[e] = a.bias ? a.bias[c] : 0.f;
#pragma unroll
            for (int j = 0; j < W; ++j) z[e] = __builtin_fmaf(a.w[(size_t)c * W + j], oct_value(r[j], e), z[e]);
            if (a.silu) z[e] = sc_silu(z[e]);
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
#pragma unroll
            for (int e = 0; e < 8; ++e) row[e] = oct_value(r[j + 1], e);
            oct_store<SMALL>(st + (size_t)j * a.C * xs, a.x_f32, pl, row);
        }
        oct_store<SMALL>((char*)a.y + b * a.C * ys, a.y_f32, pl, z);
    }
}

// dz of the run's tokens and of the W - 1 behind it (made again by the next run);
// dx_t = sum_j w_j dz_{t+W-1-j} is whole once dz_{t+W-1} is in.  Places behind the last
// token, which stand for its row again, have dz = 0 and are no part of the sums: a product
// with 0 would make NaN of an infinity that is in their windows.
//
// Two waves per SIMD (256 registers) for bf16 up to W = 4 (an earlier form 95 us, with one
// wave 118; now 93); fp32, which would spill, does not gain (109, 105).
template <bool FX, bool FD, int W, bool SMALL>
__global__ __launch_bounds__(kScThreads, W <= 4 && !FX ? 2 : 1) void sc_bwd_kernel(ScArgs a) {
    constexpr int U = sc_ahead(W);
    __shared__ float red[16][kScTile];
    const int lane = threadIdx.x & 15, sub = threadIdx.x >> 4;
    const unsigned nct = ((unsigned)a.C + kScTile - 1) / kScTile;
    const unsigned per = ((unsigned)a.L + a.run - 1) / a.run;
    const unsigned ct = blockIdx.x % nct, blk = blockIdx.x / nct;
    const int xs = a.x_f32 ? 4 : 2, ds = a.dy_f32 ? 4 : 2, ys = a.y_f32 ? 4 : 2;
    const OctPlace pl = oct_place(ct * 16 + lane, a.C);
    float w[W][8], bias[8], dw[W][8], db[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int c = SMALL ? min(e, a.C - 1) : pl.at + e;
#pragma unroll
        for (int j = 0; j < W; ++j) {
            w[j][e] = a.w[(size_t)c * W + j];
            dw[j][e] = 0.f;
        }
        bias[e] = a.bias ? a.bias[c] : 0.f;
        db[e] = 0.f;
    }
    for (unsigned tile = blk; tile < a.tiles; tile += a.blocks) {
        const unsigned run = tile * 16 + sub, b = run / per;
        if (b >= (unsigned)a.B) continue;
        const char* xb = (const char*)a.x + b * a.sx.b * xs;
        const int t0 = (int)((run - b * per) * a.run), rest = a.L - t0, n = min(a.run, rest);
        float past[W][8], dz[W][8];   // rows t of x and dz in [(t - t0) % W]
#pragma unroll
        for (int j = 1; j < W; ++j) sc_row<FX, SMALL>(a, xb, b, t0 - W + j, pl.at, past[j]);
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) dz[j][e] = 0.f;
        ScRows<FX, SMALL> rx{xb + t0 * a.sx.t * xs, a.sx.t * xs, rest - 1};
        ScRows<FD, SMALL> ry{(const char*)a.dy + (b * a.sdy.b + t0 * a.sdy.t) * ds, a.sdy.t * ds, rest - 1};
        // the row of dx that is whole W - 1 tokens later; from the first token on also the
        // state's rows
        char* ob = (char*)a.y + (b * a.sy.b + ((int64_t)t0 - (W - 1)) * a.sy.t) * ys;
        Oct<FX> x[U];
        Oct<FD> y[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            rx.next(a.x_f32, pl.at, a.C, x[u]);
            ry.next(a.dy_f32, pl.at, a.C, y[u]);
        }
        // token t0 + i, at place u of the U
        auto token = [&](int u, int i, bool sums) {
            const bool in = i < rest;
            float s[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                past[u % W][e] = oct_value(x[u], e);
                float g = oct_value(y[u], e);
                if (a.silu) {
                    float z = bias[e];
#pragma unroll
                    for (int j = 0; j < W; ++j) z = __builtin_fmaf(w[j][e], past[(u + 1 + j) % W][e], z);
                    g *= sc_slope(z);
                }
                g = in ? g : 0.f;
                dz[u % W][e] = g;
                s[e] = 0.f;
#pragma unroll
                for (int j = 0; j < W; ++j) s[e] = __builtin_fmaf(w[j][e], dz[(u + W - j) % W][e], s[e]);
            }
            if (sums && in) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
#pragma unroll
                    for (int j = 0; j < W; ++j)
                        dw[j][e] = __builtin_fmaf(dz[u % W][e], past[(u + 1 + j) % W][e], dw[j][e]);
                    db[e] += dz[u % W][e];
                }
            }
            const int r = i - (W - 1);   // of the run
            if ((r >= 0 || t0 == 0) && r < n && pl.own) {
                const int j = t0 + r + W - 1 - a.L;   // its place in the final state
                if (j >= 0 && a.dstate_in) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        s[e] += a.dstate_in[((size_t)b * (W - 1) + j) * a.C + (SMALL ? min(e, a.C - 1) : pl.at + e)];
                }
                if (r >= 0) oct_store<SMALL>(ob, a.y_f32, pl, s);
                else if (a.dstate) oct_store<SMALL>(a.dstate + ((size_t)b * (W - 1) + (W - 1 + r)) * a.C, true, pl, s);
            }
            ob += a.sy.t * ys;
        };
        int i = 0;
        for (; i < n; i += U) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                token(u, i + u, true);
                rx.next(a.x_f32, pl.at, a.C, x[u]);
                ry.next(a.dy_f32, pl.at, a.C, y[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < W - 1; ++u) token(u, i + u, false);
    }
    if (!a.part) return;
    float* part = a.part + (size_t)blk * a.C * (W + 1);
#pragma unroll
    for (int j = 0; j <= W; ++j) {
#pragma unroll
        for (int e = 0; e < 8; ++e) red[sub][lane * 8 + e] = j < W ? dw[j < W ? j : 0][e] : db[e];
        __syncthreads();
        if (threadIdx.x < kScTile) {
            const int e = threadIdx.x & 7;
            const OctPlace p = oct_place(ct * 16 + (threadIdx.x >> 3), a.C);
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) s += red[i][threadIdx.x];
            if (oct_own<SMALL>(p, e)) part[(size_t)j * a.C + p.at + e] = s;
        }
        __syncthreads();
    }
}

// dw and db from the workgroups' sums, in fp64: 32 channels' sums per workgroup, 8
// threads for each.
__global__ __launch_bounds__(256) void sc_sum_kernel(ScArgs a) {
    __shared__ double red[8][33];
    const size_t cols = (size_t)a.C * (a.W + 1);
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    for (size_t tile = blockIdx.x; tile * 32 < cols; tile += gridDim.x) {
        const size_t c = tile * 32 + lane;
        double s = 0.0;
        if (c < cols)
            for (unsigned k = slice; k < a.blocks; k += 8) s += a.part[k * cols + c];
        __syncthreads();
        red[slice][lane] = s;
        __syncthreads();
        if (slice == 0 && c < cols) {
            s = 0.0;
#pragma unroll
            for (int i = 0; i < 8; ++i) s += red[i][lane];
            const int j = (int)(c / a.C);
            const size_t ch = c - (size_t)j * a.C;
            if (j < a.W) {
                if (a.dw) a.dw[ch * a.W + j] = (float)s;
            } else if (a.db) {
                a.db[ch] = (float)s;
            }
        }
    }
}

enum { kScFwd, kScBwd, kScStep };

template <bool FX, bool FD, int W, bool SMALL, int OP>
static hipError_t sc_launch(const ScArgs& a, int slot, hipStream_t st) {
    const size_t nct = ((size_t)a.C + kScTile - 1) / kScTile;
    if constexpr (OP == kScFwd) {
        const size_t n = a.tiles * nct;
        return launch_k(slot, sc_fwd_kernel<FX, W, SMALL>, dim3((unsigned)(n < (1u << 20) ? n : 1u << 20)), dim3(kScThreads),
                        0, st, a);
    } else if constexpr (OP == kScBwd) {
        return launch_k(slot, sc_bwd_kernel<FX, FD, W, SMALL>, dim3((unsigned)(a.blocks * nct)), dim3(kScThreads), 0, st, a);
    } else {
        const size_t n = (size_t)a.B * (((unsigned)a.C + 7) / 8), blocks = (n + kScThreads - 1) / kScThreads;
        return launch_k(slot, sc_step_kernel<FX, W, SMALL>, dim3((unsigned)(blocks < 65536 ? blocks : 65536)),
                        dim3(kScThreads), 0, st, a);
    }
}

template <int W, int OP>
static hipError_t sc_launch_type(const ScArgs& a, int slot, hipStream_t st) {
    if (a.C < 8) return sc_launch<true, true, W, true, OP>(a, slot, st);
    if constexpr (OP == kScBwd) {
        if (a.x_f32 && a.dy_f32) return sc_launch<true, true, W, false, OP>(a, slot, st);
        if (a.x_f32) return sc_launch<true, false, W, false, OP>(a, slot, st);
        if (a.dy_f32) return sc_launch<false, true, W, false, OP>(a, slot, st);
        return sc_launch<false, false, W, false, OP>(a, slot, st);
    } else {
        return a.x_f32 ? sc_launch<true, true, W, false, OP>(a, slot, st) : sc_launch<false, false, W, false, OP>(a, slot, st);
    }
}

template <int OP>
static hipError_t sc_launch_width(const ScArgs& a, int slot, hipStream_t st) {
    switch (a.W) {
        case 2: return sc_launch_type<2, OP>(a, slot, st);
        case 3: return sc_launch_type<3, OP>(a, slot, st);
        case 4: return sc_launch_type<4, OP>(a, slot, st);
        case 5: return sc_launch_type<5, OP>(a, slot, st);
        case 6: return sc_launch_type<6, OP>(a, slot, st);
        case 7: return sc_launch_type<7, OP>(a, slot, st);
        default: return sc_launch_type<8, OP>(a, slot, st);
    }
}

// n 16-bit values copied, or zeroed.
__global__ __launch_bounds__(256) void seq_copy_kernel(uint16_t* to, const uint16_t* from, size_t n) {
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) to[i] = from ? from[i] : 0;
}

hipError_t launch_seq_copy(void* to, const void* from, size_t bytes, int slot, hipStream_t st) {
    const size_t n = bytes / 2, blocks = (n + 255) / 256;
    return launch_k(slot, seq_copy_kernel, dim3((unsigned)(blocks < 1024 ? blocks : 1024)), dim3(256), 0, st, (uint16_t*)to,
                    (const uint16_t*)from, n);
}

hipError_t launch_sc_fwd(const ScArgs& a, int slot, hipStream_t st) { return sc_launch_width<kScFwd>(a, slot, st); }
hipError_t launch_sc_step(const ScArgs& a, int slot, hipStream_t st) { return sc_launch_width<kScStep>(a, slot, st); }

hipError_t launch_sc_bwd(const ScArgs& a, int slot, hipStream_t st) {
    hipError_t e = sc_launch_width<kScBwd>(a, slot, st);
    if (e == hipSuccess && a.part) {
        const size_t tiles = ((size_t)a.C * (a.W + 1) + 31) / 32;
        e = launch_k(slot, sc_sum_kernel, dim3((unsigned)(tiles < 65536 ? tiles : 65536)), dim3(256), 0, st, a);
    }
    return e;
}

}  // namespace dr
