// dr_linattn_kernel.h -- the chunked kernel of linear attention with a decay
// per head, for bf16 inputs (dr_linattn.hip) and fp32 inputs (dr_linattn32.hip).
//
// Mathematics.  With g the running sum of log alpha, S_t = a_t S_{t-1} + k_t v_t^T
// and o_t = S_t^T q_t give, for a 64-token chunk that starts from state S,
//   o_i = e^{g_i} S^T q_i + sum_{j <= i} e^{g_i - g_j} (q_i . k_j) v_j
//   S  <- e^{g_63} S + sum_j e^{g_63 - g_j} k_j v_j^T,
// and the gradients of q, k and v have the same form with the roles exchanged
// and, for k and v, the tokens taken backwards (LaPass in dr_linattn.h names
// them x, y, z).  Backwards, a row's u is the sum of log alpha over the tokens
// behind it, without its own: the exclusive running sum.
//
// Layout.  One workgroup walks the chunks of one segment of one sequence for
// 32 columns of z per wave.  A wave keeps its Dx x 32 state in accumulator
// registers of the 32x32 matrix ops.  A lane of an accumulator holds rows
// 8 b + 4 h + j (b, j < 4; h the half of the wave) of one column; taken as an
// operand with that row order as the contraction's order, the same registers
// feed the next product, so neither the state nor the 64 x 64 matrix of
// products x . y passes through LDS: x and y rows are read from LDS in that
// order.  Products that contract over tokens read y and z transposed
// (ds_read_b64_tr_b16 for bf16).
//
// Precision.  bf16 inputs are operands as they are.  fp32 quantities that meet
// them are split into bf16 terms: the decayed z of the state update into three
// (24 significant bits: the state is as exact as in fp32), the state and the
// decayed products of the output into NT = 3 where the output is kept in fp32
// or feeds the gate's gradient, else 2 (16 bits, below the output's own
// rounding to bf16).  fp32 inputs use the fp32 matrix ops throughout.  Running
// sums of log alpha are fp64; differences are taken between hi + lo float
// pairs, so a long or strong decay loses nothing to cancellation.  log alpha
// below -256 / log2(e) counts as that (its e^ is 0 in fp32 either way), so a
// decay of exactly zero (log alpha = -inf) resets the state.
#pragma once

#include <hip/hip_runtime.h>

#include "dr_device.h"
#include "dr_internal.h"
#include "dr_lds.h"
#include "dr_linattn.h"

namespace dr {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Swizzle of the 16-byte pieces of a row of RB bytes.  Row reads take the same
// piece of 16 or 32 consecutive rows, transposing reads 64 consecutive bytes of
// four consecutive rows: the low two bits of the row go to the piece's upper
// bits (four rows fall on different quarters of the banks), the next two to
// its lower bits.
template <int RB>
__device__ __forceinline__ int la_swz(int r) {
    if constexpr (RB >= 256) return ((r & 3) << 2) | ((r >> 2) & 3);
    else if constexpr (RB == 128) return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
    else return 0;
}

template <typename T>
struct LaFrag;   // eight contraction values of one row or column
template <>
struct LaFrag<__bf16> {
    uint4 v;
};
template <>
struct LaFrag<float> {
    float v[8];
};

// fp32 values as an operand: NT bf16 terms, or themselves
template <typename T, int NT>
struct LaTerms {
    uint4 t[NT];
};
template <int NT>
struct LaTerms<float, NT> {
    float v[8];
};

// The constants of la_rest, kept in scalar registers: bf16 pairs (-1, 0) and
// (0, -1), as (low, high) halves.
struct LaNeg {
    unsigned lo, hi;
};
__device__ __forceinline__ LaNeg la_neg() {
    LaNeg c{0x0000bf80u, 0xbf800000u};
    asm volatile("" : "+s"(c.lo), "+s"(c.hi));
    return c;
}
__device__ __forceinline__ unsigned la_pack(float a, float b) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 f = {a, b};
    return __builtin_bit_cast(unsigned, __builtin_convertvector(f, bf16x2));
}
// What two values rounded to the bf16 pair p leave: a - p.lo and b - p.hi, as
// dot products of p with (-1, 0) and (0, -1), one instruction each and exact.
__device__ __forceinline__ void la_rest(unsigned p, const LaNeg& c, float& a, float& b) {
    const bf16x2 h = __builtin_bit_cast(bf16x2, p);
    a = __builtin_amdgcn_fdot2_f32_bf16(h, __builtin_bit_cast(bf16x2, c.lo), a, false);
    b = __builtin_amdgcn_fdot2_f32_bf16(h, __builtin_bit_cast(bf16x2, c.hi), b, false);
}

template <typename T, int NT>
__device__ __forceinline__ LaTerms<T, NT> la_split(float (&x)[8], const LaNeg& c) {
    LaTerms<T, NT> r;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int e = 0; e < 8; ++e) r.v[e] = x[e];
    } else {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            unsigned w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                w[e] = la_pack(x[2 * e], x[2 * e + 1]);
                if (n + 1 < NT) la_rest(w[e], c, x[2 * e], x[2 * e + 1]);
            }
            r.t[n] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    return r;
}

__device__ __forceinline__ f32x16 la_mfma(const uint4& a, const uint4& b, const f32x16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}
__device__ __forceinline__ f32x16 la_mfma(const float (&a)[8], const float (&b)[8], f32x16 c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], c, 0, 0, 0);
    return c;
}
// c += a b, a or b split into terms (smallest first, so that they are not lost)
template <int NT>
__device__ __forceinline__ f32x16 la_mma(const LaTerms<__bf16, NT>& a, const LaFrag<__bf16>& b, f32x16 c) {
#pragma unroll
    for (int n = NT - 1; n >= 0; --n) c = la_mfma(a.t[n], b.v, c);
    return c;
}
template <int NT>
__device__ __forceinline__ f32x16 la_mma(const LaFrag<__bf16>& a, const LaTerms<__bf16, NT>& b, f32x16 c) {
#pragma unroll
    for (int n = NT - 1; n >= 0; --n) c = la_mfma(a.v, b.t[n], c);
    return c;
}
template <int NT>
__device__ __forceinline__ f32x16 la_mma(const LaTerms<float, NT>& a, const LaFrag<float>& b, f32x16 c) {
    return la_mfma(a.v, b.v, c);
}
template <int NT>
__device__ __forceinline__ f32x16 la_mma(const LaFrag<float>& a, const LaTerms<float, NT>& b, f32x16 c) {
    return la_mfma(a.v, b.v, c);
}
template <typename T>
__device__ __forceinline__ f32x16 la_mma(const LaFrag<T>& a, const LaFrag<T>& b, f32x16 c) {
    return la_mfma(a.v, b.v, c);
}

// Row `row`, contraction values 16 m + 8 (e / 4) + 4 h + (e % 4), e < 8.  bf16
// tiles that are read so hold the four 8-byte quads of each 16 values in the
// order 0, 2, 1, 3 (la_stage), so that this is one 16-byte read.
template <typename T, int RB>
__device__ __forceinline__ LaFrag<T> la_row(const lchar* tile, int row, int m, int h) {
    LaFrag<T> f;
    const lchar* r = tile + row * RB;
    const int s = la_swz<RB>(row);
    if constexpr (sizeof(T) == 2) {
        f.v = lds_ld<uint4>(r + 16 * ((2 * m + h) ^ s));
    } else {
        const f32x4 a = lds_ld<f32x4>(r + 16 * ((4 * m + h) ^ s));
        const f32x4 b = lds_ld<f32x4>(r + 16 * ((4 * m + 2 + h) ^ s));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f.v[j] = a[j];
            f.v[4 + j] = b[j];
        }
    }
    return f;
}

// Column c0 + lane % 32, rows 16 m + 8 (e / 4) + 4 h + (e % 4), e < 8.  QUADS:
// the tile is in la_row's order.
template <typename T, int RB, bool QUADS>
__device__ __forceinline__ LaFrag<T> la_col(const lchar* tile, int m, int c0, int lane) {
    LaFrag<T> f;
    const int h = lane >> 5;
    if constexpr (sizeof(T) == 2) {
        const int i = lane & 15, g = (lane >> 4) & 1;
        const int piece = (c0 >> 3) + 2 * g + (QUADS ? i & 1 : (i >> 1) & 1);
        const int sub = 8 * (QUADS ? (i >> 1) & 1 : i & 1);
        uint2 w[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int row = 16 * m + 8 * q + 4 * h + (i >> 2);
            w[q] = lds_tr4(tile + row * RB + 16 * (piece ^ la_swz<RB>(row)) + sub);
        }
        f.v = make_uint4(w[0].x, w[0].y, w[1].x, w[1].y);
    } else {
        const int col = c0 + (lane & 31);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int row = 16 * m + 8 * (e >> 2) + 4 * h + (e & 3);
            f.v[e] = lds_ld<float>(tile + row * RB + 16 * ((col >> 2) ^ la_swz<RB>(row)) + 4 * (col & 3));
        }
    }
    return f;
}

template <typename T>
__device__ __forceinline__ void la_floats(const LaFrag<T>& f, float (&x)[8]) {
    if constexpr (sizeof(T) == 2) {
        unpack_bf16x8(f.v, x);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = f.v[e];
    }
}

// A value that the compiler takes as new here, so that what follows from it is
// computed in the loop and not held in registers across it.
__device__ __forceinline__ int la_fresh(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

// 64 x PPR 16-byte pieces of a chunk's rows (in the pass's order) into
// registers.  A thread takes the same piece of rows row0 + i STEP; `base` (the
// chunk's first token, the same for all lanes) moves by STEP rows at a time and
// `off` is the thread's own part, so that the addresses are a scalar base and
// one 32-bit offset.  Rows behind the last token and (ok) pieces behind the
// width are zero.
template <int N, int PPR, int NTHR>
__device__ __forceinline__ void la_fetch(uint4 (&r)[N], const char* base, int64_t row_bytes, unsigned off, bool rev,
                                         int rows, bool ok, int tid) {
    constexpr int STEP = NTHR / PPR;
    const int row0 = tid / PPR;
    if (rows >= 64) {
        if (ok) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                r[i] = *reinterpret_cast<const uint4*>(base + (rev ? 64 - (i + 1) * STEP : i * STEP) * row_bytes + off);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int row = row0 + i * STEP;
            r[i] = make_uint4(0u, 0u, 0u, 0u);
            if (ok && (rev ? 63 - row : row) < rows)
                r[i] = *reinterpret_cast<const uint4*>(base + (rev ? 64 - (i + 1) * STEP : i * STEP) * row_bytes + off);
        }
    }
}
// The thread's part of la_fetch's addresses.
template <int PPR, int NTHR>
__device__ __forceinline__ unsigned la_offset(int64_t row_bytes, bool rev, int tid) {
    constexpr int STEP = NTHR / PPR;
    const int row0 = tid / PPR;
    return (unsigned)(rev ? STEP - 1 - row0 : row0) * (unsigned)row_bytes + 16 * (tid % PPR);
}
template <int N, int PPR, int NTHR, bool QUADS>
__device__ __forceinline__ void la_stage(lchar* tile, const uint4 (&r)[N], int tid) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int row = tid / PPR + i * (NTHR / PPR), p = tid % PPR;
        const int s = la_swz<PPR * 16>(row);
        if constexpr (QUADS) {
            lds_st(tile + row * (PPR * 16) + 16 * ((p & ~1) ^ s) + 8 * (p & 1), make_uint2(r[i].x, r[i].y));
            lds_st(tile + row * (PPR * 16) + 16 * ((p | 1) ^ s) + 8 * (p & 1), make_uint2(r[i].z, r[i].w));
        } else {
            lds_st(tile + row * (PPR * 16) + 16 * (p ^ s), r[i]);
        }
    }
}

// One step of a running sum on DPP moves: x plus the value that CTRL brings
// (zero where it brings none).
template <int CTRL, int ROWS>
__device__ __forceinline__ double la_scan_step(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const unsigned lo = __builtin_amdgcn_update_dpp(0, (int)(unsigned)u, CTRL, ROWS, 0xF, false);
    const unsigned hi = __builtin_amdgcn_update_dpp(0, (int)(unsigned)(u >> 32), CTRL, ROWS, 0xF, false);
    return x + __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
// Running sum of x over the wave's lanes, each lane's own value included:
// shifts by 1, 2, 4 and 8 within rows of 16 lanes, then a row's sum to the
// next row (rows 1 and 3) and the lower half's to the upper half.
__device__ __forceinline__ double la_scan(double x) {
    x = la_scan_step<0x111, 0xF>(x);
    x = la_scan_step<0x112, 0xF>(x);
    x = la_scan_step<0x114, 0xF>(x);
    x = la_scan_step<0x118, 0xF>(x);
    x = la_scan_step<0x142, 0xA>(x);
    return la_scan_step<0x143, 0xC>(x);
}

// The decays of a chunk in LDS: u as hi + lo floats, e^u, e^{total - u}, and
// e^total; two buffers, the next chunk's made while this one's are read.
constexpr int kLaGateBytes = 4 * 64 * 4 + 16;

template <typename T, int DX, int NW, int NT, bool STATE>
constexpr int la_lds_bytes() {
    constexpr int y = 64 * DX * (int)sizeof(T), z = 64 * 32 * NW * (int)sizeof(T);
    return (STATE ? y + z : 2 * y + z + 64 * 64 * (int)sizeof(T) * (sizeof(T) == 2 ? NT : 1)) + 2 * kLaGateBytes;
}

// waves per SIMD that the registers are held to: two for bf16, one for fp32,
// whose tiles fill the LDS of a CU
template <typename T, int NW>
constexpr int la_waves() { return sizeof(T) == 2 && NW > 1 ? 2 : 1; }

template <typename T, int DX, int NW, int NT, bool STATE>
__global__ __launch_bounds__(64 * NW, (la_waves<T, NW>())) void la_kernel(LaArgs a) {
    constexpr int NTHR = 64 * NW;
    constexpr int EPP = 16 / (int)sizeof(T);         // elements per piece
    constexpr int PX = DX / EPP, PZ = 32 * NW / EPP; // pieces per row
    constexpr int RX = PX * 16, RZ = PZ * 16;        // bytes per row
    constexpr int RP = 64 * (int)sizeof(T);          // of the products x . y (each term)
    constexpr int NX = 64 * PX / NTHR, NZ = 64 * PZ / NTHR;
    constexpr int TX = DX / 32;                      // 32-row tiles of the state
    extern __shared__ __attribute__((aligned(16))) char smem[];
    lchar* const sY = (lchar*)smem;
    lchar* const sZ = sY + 64 * RX;
    lchar* const sG = sZ + 64 * RZ;
    lchar* const sX = sG + 2 * kLaGateBytes;         // not with STATE
    lchar* const sP = sX + 64 * RX;

    // Workgroups go to the eight XCDs in turn; consecutive work (the column
    // tiles of a sequence, heads that share rows) stays on one of them.
    const int per = (a.total + 7) / 8;
    int id = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
    if (id >= a.total || (int)(blockIdx.x >> 3) >= per) return;
    const int ct = id % a.ntile;
    id /= a.ntile;
    const int nseq = a.B * a.H;
    const int seq = id % nseq;
    id /= nseq;
    const int sg = id % a.nseg;
    const LaPass& ps = a.pass[id / a.nseg];
    const int b = seq / a.H, hd = seq % a.H;
    const bool rev = ps.rev != 0;
    // nothing starts from behind the last segment
    if (STATE && sg == (rev ? 0 : a.nseg - 1)) return;

    const int tid = threadIdx.x, lane0 = tid & 63;
    int lane = lane0, h = lane >> 5, l31 = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int zc0 = (ct * NW + wave) * kLaCols;      // the wave's first column
    const int Dx = ps.Dx, Dz = ps.Dz, L = a.L;
    const int px = Dx / EPP, pz = (Dz - ct * NW * kLaCols) / EPP;
    const char* gx = nullptr;
    if constexpr (!STATE)
        gx = (const char*)ps.x.p + sizeof(T) * (b * ps.x.b + (hd / ps.x.group) * ps.x.h);
    const char* gy = (const char*)ps.y.p + sizeof(T) * (b * ps.y.b + (hd / ps.y.group) * ps.y.h);
    const char* gz = (const char*)ps.z.p + sizeof(T) * (b * ps.z.b + (hd / ps.z.group) * ps.z.h + ct * NW * kLaCols);
    const int64_t bx = sizeof(T) * ps.x.t, by = sizeof(T) * ps.y.t, bz = sizeof(T) * ps.z.t;
    const float* la = a.la ? (a.la_head ? a.la + hd : a.la + (size_t)seq * L) : nullptr;
    const LaNeg neg = la_neg();

    // the state, from its start
    f32x16 S[TX];
    const float* start = nullptr;
    const size_t elems = (size_t)Dx * Dz;
    if constexpr (!STATE)
        start = a.nseg > 1 ? ps.seg + ((size_t)seq * a.nseg + sg) * elems : ps.start ? ps.start + seq * elems : nullptr;
    const int zc = zc0 + l31;
#pragma unroll
    for (int t = 0; t < TX; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) S[t][r] = 0.f;
    if (!STATE && start && zc < Dz) {
        if (ps.tr) {
            const float* s = start + (size_t)zc * Dx + 4 * h;
#pragma unroll
            for (int t = 0; t < TX; ++t)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (32 * t + 8 * q < Dx) {
                        const f32x4 v = *reinterpret_cast<const f32x4*>(s + 32 * t + 8 * q);
#pragma unroll
                        for (int j = 0; j < 4; ++j) S[t][4 * q + j] = v[j];
                    }
        } else {
            const float* s = start + (size_t)(4 * h) * Dz + zc;
#pragma unroll
            for (int t = 0; t < TX; ++t)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (32 * t + 8 * q < Dx) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) S[t][4 * q + j] = s[(32 * t + 8 * q + j) * Dz];
                    }
        }
    }

    const int c_lo = sg * a.cps, c_hi = min(a.NC, c_lo + a.cps);
    const int nc = c_hi - c_lo;
    const bool gate_wave = wave == NW - 1;
    double seg_total = 0.0;   // the gate wave's: the segment's sum of log2 alpha

    uint4 rx[STATE ? 1 : NX], ry[NX], rz[NZ];
    auto chunk = [&](int n) { return rev ? c_hi - 1 - n : c_lo + n; };
#pragma unroll
    for (int i = 0; i < NX; ++i) {
        if constexpr (!STATE) rx[i] = make_uint4(0u, 0u, 0u, 0u);
        ry[i] = make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < NZ; ++i) rz[i] = make_uint4(0u, 0u, 0u, 0u);
    const bool okx = tid % PX < px, okz = tid % PZ < pz;
    const unsigned fx = STATE ? 0 : la_offset<PX, NTHR>(bx, rev, tid), fy = la_offset<PX, NTHR>(by, rev, tid),
                   fz = la_offset<PZ, NTHR>(bz, rev, tid);
    auto fetch = [&](int n) {
        const int c = chunk(n), rows = L - 64 * c;
        if constexpr (!STATE) la_fetch<NX, PX, NTHR>(rx, gx + 64 * c * bx, bx, fx, rev, rows, okx, tid);
        la_fetch<NX, PX, NTHR>(ry, gy + 64 * c * by, by, fy, rev, rows, okx, tid);
        la_fetch<NZ, PZ, NTHR>(rz, gz + 64 * c * bz, bz, fz, rev, rows, okz, tid);
    };
    auto log_alpha = [&](int n) {
        const int t = 64 * chunk(n) + (rev ? 63 - lane0 : lane0);
        return la && t < L ? la[a.la_head ? 0 : t] : 0.f;
    };
    auto decays = [&](int n, float x) {
        lchar* g = sG + (n & 1) * kLaGateBytes;
        const double l2 = x < -177.445678f ? -256.0 : (double)x * 1.4426950408889634;
        const double s = la_scan(l2);
        const double total = __shfl(s, 63);
        const double u = rev ? s - l2 : s;
        const float uh = (float)u;
        lds_st(g + 4 * lane0, uh);
        lds_st(g + 256 + 4 * lane0, (float)(u - (double)uh));
        lds_st(g + 512 + 4 * lane0, __builtin_amdgcn_exp2f(uh));
        lds_st(g + 768 + 4 * lane0, __builtin_amdgcn_exp2f((float)(total - u)));
        if (lane0 == 0) lds_st(g + 1024, __builtin_amdgcn_exp2f((float)total));
        if constexpr (STATE) seg_total += total;
    };

    // the output rows of a chunk, stored while the next one is computed: a wait
    // for loads waits for every store before them too
    f32x16 O[2];           // O^T: the wave's columns by rows
    RawN<sizeof(T) == 4, 4> W[2][4];
    const bool dots = !STATE && ps.w.p != nullptr, out_bf16 = ps.out_bf16 != 0;
    char* const gout = STATE ? nullptr : (char*)ps.out + (out_bf16 ? 2 : 4) * (b * ps.ob + hd * ps.oh);
    const int64_t ot = ps.ot, wt = ps.w.t;
    const char* gw = dots ? (const char*)ps.w.p + sizeof(T) * (b * ps.w.b + (hd / ps.w.group) * ps.w.h) : nullptr;
    float* const gd = dots ? ps.dots + ((size_t)(zc0 / kLaCols) * nseq + seq) * L : nullptr;
    auto fetch_w = [&](int n) {
        const int c = chunk(n);
#pragma unroll
        for (int it = 0; it < 2; ++it) {
            const int row = 32 * it + l31, tl = rev ? 63 - row : row;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (64 * c + tl < L && zc0 + 8 * q < Dz)
                    W[it][q] = ld_rawn<sizeof(T) == 4, 4>(gw + 64 * c * wt * (int64_t)sizeof(T),
                                                          (unsigned)tl * (unsigned)wt + zc0 + 8 * q + 4 * h);
        }
    };
    auto store = [&](int n) {
        const int c = chunk(n);
#pragma unroll
        for (int it = 0; it < 2; ++it) {
            const int row = 32 * it + l31, tl = rev ? 63 - row : row;
            const bool ok = 64 * c + tl < L;
            const unsigned at = (unsigned)tl * (unsigned)ot + zc0 + 4 * h;
            if (out_bf16) {
                char* base = gout + 64 * c * ot * 2;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (ok && zc0 + 8 * q < Dz)
                        *reinterpret_cast<uint2*>(base + 2 * (at + 8 * q)) =
                            make_uint2(la_pack(O[it][4 * q], O[it][4 * q + 1]), la_pack(O[it][4 * q + 2], O[it][4 * q + 3]));
            } else {
                char* base = gout + 64 * c * ot * 4;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (ok && zc0 + 8 * q < Dz)
                        *reinterpret_cast<f32x4*>(base + 4 * (at + 8 * q)) =
                            f32x4{O[it][4 * q], O[it][4 * q + 1], O[it][4 * q + 2], O[it][4 * q + 3]};
            }
            if (dots) {
                float dot = 0.f;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float w4[4];
                    cvt_rawn<sizeof(T) == 4, 4>(W[it][q], w4);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (ok && zc0 + 8 * q < Dz) dot += O[it][4 * q + j] * w4[j];
                }
                dot += __shfl_xor(dot, 32);
                if (ok && h == 0 && zc0 < Dz) gd[64 * c + tl] = dot;
            }
        }
    };
    fetch(0);
    if (gate_wave) decays(0, log_alpha(0));

    for (int n = 0; n < nc; ++n) {
        const lchar* g = sG + (n & 1) * kLaGateBytes;
        if (n) lds_barrier();   // the last chunk's tiles are done with
        if constexpr (!STATE) la_stage<NX, PX, NTHR, sizeof(T) == 2>(sX, rx, tid);
        la_stage<NX, PX, NTHR, sizeof(T) == 2>(sY, ry, tid);
        la_stage<NZ, PZ, NTHR, false>(sZ, rz, tid);
        lds_barrier();
        lane = la_fresh(lane0);
        h = lane >> 5;
        l31 = lane & 31;
        float next_la = 0.f;
        if constexpr (!STATE)
            if (n) store(n - 1);
        if (n + 1 < nc) {
            fetch(n + 1);
            if (gate_wave) next_la = log_alpha(n + 1);
        }
        if constexpr (!STATE)
            if (dots) fetch_w(n);

        const f32x16 zero = {};
        if constexpr (!STATE) {
            // the products x . y of 32 x 32 tiles (i, j) = (0,0), (1,0), (1,1), times their decays, into LDS
            for (int k = wave; k < 3; k += NW) {
                const int it = (k + 1) >> 1, jt = k >> 1;
                f32x16 P = zero;
#pragma unroll
                for (int m = 0; m < DX / 16; ++m)
                    P = la_mma(la_row<T, RX>(sY, 32 * jt + l31, m, h), la_row<T, RX>(sX, 32 * it + l31, m, h), P);
                const int i = 32 * it + l31;
                const float ui = lds_ld<float>(g + 4 * i), wi = lds_ld<float>(g + 256 + 4 * i);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int j = 32 * jt + 8 * q + 4 * h;
                    const f32x4 uj = lds_ld<f32x4>(g + 4 * j), wj = lds_ld<f32x4>(g + 256 + 4 * j);
                    f32x4 v;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float d = (ui - uj[e]) + (wi - wj[e]);
                        const float x = P[4 * q + e] * __builtin_amdgcn_exp2f(d);
                        v[e] = j + e <= i ? x : 0.f;
                    }
                    if constexpr (sizeof(T) == 2) {
                        // la_row's order of quads: j / 4 = 4 (j / 16) + 2 (q % 2) + h
                        lchar* at = sP + i * RP + 16 * ((4 * jt + (q & ~1) + h) ^ la_swz<RP>(i)) + 8 * (q & 1);
#pragma unroll
                        for (int term = 0; term < NT; ++term) {
                            const unsigned lo = la_pack(v[0], v[1]), hi = la_pack(v[2], v[3]);
                            lds_st(at + term * 64 * RP, make_uint2(lo, hi));
                            if (term + 1 < NT) {
                                float r0 = v[0], r1 = v[1], r2 = v[2], r3 = v[3];
                                la_rest(lo, neg, r0, r1);
                                la_rest(hi, neg, r2, r3);
                                v = f32x4{r0, r1, r2, r3};
                            }
                        }
                    } else {
                        lds_st(sP + i * RP + 16 * ((j >> 2) ^ la_swz<RP>(i)), v);
                    }
                }
            }
            // what the state at the chunk's start gives the rows
            LaFrag<T> x0 = la_row<T, RX>(sX, l31, 0, h), x1 = la_row<T, RX>(sX, 32 + l31, 0, h);
#pragma unroll
            for (int m = 0; m < DX / 16; ++m) {
                const LaFrag<T> c0 = x0, c1 = x1;
                if (m + 1 < DX / 16) {
                    x0 = la_row<T, RX>(sX, l31, m + 1, h);
                    x1 = la_row<T, RX>(sX, 32 + l31, m + 1, h);
                }
                float s8[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) s8[e] = S[m >> 1][8 * (m & 1) + e];
                const LaTerms<T, NT> st = la_split<T, NT>(s8, neg);
                O[0] = la_mma(st, c0, m ? O[0] : zero);
                O[1] = la_mma(st, c1, m ? O[1] : zero);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int it = 0; it < 2; ++it) {
                const float e = lds_ld<float>(g + 512 + 4 * (32 * it + l31));
#pragma unroll
                for (int r = 0; r < 16; ++r) O[it][r] *= e;
            }
        }
        const float decay = lds_ld<float>(g + 1024);
#pragma unroll
        for (int t = 0; t < TX; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) S[t][r] *= decay;
        if constexpr (!STATE) lds_barrier();   // the products are in LDS
        // rows 16 ks .. 16 ks + 15 of y and z: into the output's later rows, then into the state
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            const LaFrag<T> z = la_col<T, RZ, false>(sZ, ks, wave * kLaCols, lane);
            const int j0 = 16 * ks + 4 * h;   // the lane's rows: j0 + [0, 4) and j0 + 8 + [0, 4)
            if constexpr (!STATE) {
#pragma unroll
                for (int it = ks >> 1; it < 2; ++it) {
                    LaTerms<T, NT> pt;
                    if constexpr (sizeof(T) == 2) {
#pragma unroll
                        for (int term = 0; term < NT; ++term)
                            pt.t[term] = la_row<T, RP>(sP + term * 64 * RP, 32 * it + l31, ks, h).v;
                    } else {
                        const LaFrag<T> f = la_row<T, RP>(sP, 32 * it + l31, ks, h);
#pragma unroll
                        for (int e = 0; e < 8; ++e) pt.v[e] = f.v[e];
                    }
                    O[it] = la_mma(z, pt, O[it]);
                }
            }
            const f32x4 k0 = lds_ld<f32x4>(g + 768 + 4 * j0), k1 = lds_ld<f32x4>(g + 768 + 4 * j0 + 32);
            float z8[8];
            la_floats(z, z8);
#pragma unroll
            for (int e = 0; e < 8; ++e) z8[e] *= e < 4 ? k0[e & 3] : k1[e & 3];
            const LaTerms<T, 3> zt = la_split<T, 3>(z8, neg);
#pragma unroll
            for (int t = 0; t < TX; ++t)
                S[t] = la_mma(la_col<T, RX, sizeof(T) == 2>(sY, ks, 32 * t, lane), zt, S[t]);
        }
        if (gate_wave && n + 1 < nc) decays(n + 1, next_la);
    }
    if constexpr (!STATE) store(nc - 1);

    float* end = nullptr;
    if constexpr (STATE) {
        end = ps.seg + ((size_t)seq * a.nseg + sg) * elems;
        if (ct == 0 && gate_wave && lane == 0)
            ps.segdec[(size_t)seq * a.nseg + sg] = __builtin_amdgcn_exp2f((float)seg_total);
    } else if (ps.end && sg == (rev ? 0 : a.nseg - 1)) {
        end = ps.end + seq * elems;
    }
    if (end && zc < Dz) {
        const bool tr = ps.tr != 0;
        float* e = tr ? end + (size_t)zc * Dx + 4 * h : end + (size_t)(4 * h) * Dz + zc;
#pragma unroll
        for (int t = 0; t < TX; ++t)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int d = 32 * t + 8 * q;
                if (d >= Dx) continue;
                if (tr) {
                    *reinterpret_cast<f32x4*>(e + d) =
                        f32x4{S[t][4 * q], S[t][4 * q + 1], S[t][4 * q + 2], S[t][4 * q + 3]};
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) e[(d + j) * Dz] = S[t][4 * q + j];
                }
            }
    }
}

template <typename T, int DX, int NW, int NT, bool STATE>
hipError_t la_launch(const LaArgs& a, int slot, hipStream_t st) {
    auto kern = la_kernel<T, DX, NW, NT, STATE>;
    constexpr int lds = la_lds_bytes<T, DX, NW, NT, STATE>();
    if constexpr (lds > 65536) {
        const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
    }
    const unsigned grid = (unsigned)((a.total + 7) / 8 * 8);
    return launch_k(slot, kern, dim3(grid), dim3(64 * NW), lds, st, a);
}

template <typename T, int DX, int NT, bool STATE>
hipError_t la_launch_w(const LaArgs& a, int waves, int slot, hipStream_t st) {
    if (waves == 4) return la_launch<T, DX, 4, NT, STATE>(a, slot, st);
    if (waves == 2) return la_launch<T, DX, 2, NT, STATE>(a, slot, st);
    return la_launch<T, DX, 1, NT, STATE>(a, slot, st);
}

}  // namespace dr
