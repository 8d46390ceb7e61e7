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
// 16 columns of z per wave.  A wave keeps its Dx x 16 state in accumulator
// registers of the 16x16 matrix ops.  A lane of two stacked accumulators holds
// rows 4 g + j and 16 + 4 g + j (j < 4; g the 16-lane group) of one column;
// taken as an operand with that row order as the contraction's order, the same
// registers feed the next product, so the state never passes through LDS: x and
// y rows are staged there in that order.  The 64 x 64 matrix of products x . y
// is made once per workgroup, a 16 x 16 block or two per wave, and shared
// through LDS with its decays applied.  Products that contract over tokens read
// y and z transposed (ds_read_b64_tr_b16 for bf16).
//
// Why 16 columns and eight waves: the registers stay at 128, four waves per SIMD
// in two workgroups per CU.  32 columns per wave on the 32x32 ops read LDS half
// as often, but with two waves per SIMD the kernel took 187 us for the forward at
// B2 H16 L16384 d128 bf16, against 163 with four at the same stage.
//
// What bounds it, at that size: the forward's main pass takes 138 us for 570 MB
// (4.1 TB/s; a large copy reaches 5.2) and the state pass 66 us for 285 MB.  The
// main pass without its products took 110 us, so memory comes first, then the
// issue of vector and matrix instructions, which overlap only in part: 424 and 97
// per wave and chunk, a third of the former splitting fp32 values into bf16 terms.
// The backward's three passes (three terms, row dot products; 552 and 119) are
// bound by that issue: 470 us for 1.65 GB, and 530-640 where calls follow each
// other without a pause and the clock falls.  Where few workgroups run, a chunk
// is a chain of latencies: 3.1 us at d64 in a workgroup of four waves alone.
// Tried there without gain: two blocks of the products side by side, LDS reads
// ahead across steps, the decays made earlier in the chunk.
//
// Precision.  bf16 inputs are operands as they are.  fp32 quantities that meet
// them are split into bf16 terms: the decayed z of the state update into three
// (24 significant bits: the state is as exact as in fp32), the state and the
// decayed products of the output into NT = 3 where the output is kept in fp32
// or feeds the gate's gradient, else 2 (16 bits, below the output's own
// rounding to bf16).  fp32 inputs use the fp32 matrix ops throughout; 32 tokens
// are summed before they are added to the state (with the matrix ops adding to
// it product by product a state of 4096 tokens without a decay was off by 19
// units of 2^-24, now 3.8; H16 L4096 128 x 128 takes 108 us instead of 107).
// Running sums of log alpha are fp64; differences are taken between hi + lo float
// pairs, so a long or strong decay loses nothing to cancellation, and the
// exponentials that a state is scaled by take hi and lo (la_exp2; between two
// tokens of a chunk the difference is one float).  log alpha below -256 /
// log2(e) counts as that (its e^ is 0 in fp32 either way), so a
// decay of exactly zero (log alpha = -inf) resets the state.
#pragma once

#include <hip/hip_runtime.h>

#include "dr_device.h"
#include "dr_internal.h"
#include "dr_lds.h"
#include "dr_linattn.h"

namespace dr {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Swizzle of the 16-byte pieces of a row of RB bytes: piece p of row r lies at
// piece p ^ la_swz(r).  The 64 banks hold 256 bytes.
//   bf16: a transposing read takes 32 bytes of 16 rows, half a wave (rows r to
//   r + 7) at a time; a row read takes piece p of 16 rows for each lane group,
//   pieces p to p + 3 over the groups, in phases of 16 lanes: rows 0-3 and
//   12-15 of one group with rows 4-11 of the next, then the others.  The four
//   rows of a quad go to different quarters of the banks (r & 3: the piece's
//   upper bits, or where rows are shorter the rows themselves), and the quads to
//   pieces 0, 2, 3, 1 of a quarter, which serves both without a conflict.
//   fp32: a column read takes one row of each quad, so the quads go to
//   different quarters.
template <typename T, int RB>
__device__ __forceinline__ int la_swz(int r) {
    if constexpr (sizeof(T) == 4) return RB >= 256 ? r & 15 : (((r >> 2) & 1) << 2) | ((r >> 1) & 3);
    const int b0 = (r >> 2) & 1, b1 = (r >> 3) & 1;
    const int low = ((b0 ^ b1) << 1) | b1;
    if constexpr (RB >= 256) return ((r & 3) << 2) | low;
    else if constexpr (RB == 128) return (((r >> 1) & 1) << 2) | low;
    else return low;
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

// c += a b over 32 contraction values
__device__ __forceinline__ f32x4 la_mfma(const uint4& a, const uint4& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}
__device__ __forceinline__ f32x4 la_mfma(const float (&a)[8], const float (&b)[8], f32x4 c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
}
// Term n of a split operand, as a fragment; fp32 operands have one.
template <typename T, int NT>
__device__ __forceinline__ auto& la_term(const LaTerms<T, NT>& a, int n) {
    if constexpr (sizeof(T) == 4) return a.v;
    else return a.t[n];
}
// Terms that a product runs over (smallest first, so that they are not lost).
template <typename T, int NT>
constexpr int la_terms() { return sizeof(T) == 4 ? 1 : NT; }

// LDS addresses.  A lane's address in a tile is a value of its own (the tile's
// start, a multiple of its row bytes, included), the tile's step in the
// contraction flips bits of it (the swizzle is a flip too), and whole 16-row
// steps are the instruction's offset: one register and at most one instruction
// per read.
//
// Rows, contraction values 32 m + 16 (e / 4) + 4 g + (e % 4), e < 8, of row
// l15 (+ 16 per step).  QUADS: a bf16 tile that holds the eight 8-byte quads of
// each 32 values in the order 0, 4, 1, 5, 2, 6, 3, 7 (la_stage), so that a lane's
// values are one 16-byte read; else two.
template <typename T, int RB, bool QUADS>
__device__ __forceinline__ int la_row_at(int l15, int g) {
    const int s = la_swz<T, RB>(l15);
    if constexpr (sizeof(T) == 2 && !QUADS) return l15 * RB + 16 * ((g >> 1) ^ s) + 8 * (g & 1);
    else return l15 * RB + 16 * (g ^ s);
}
__device__ __forceinline__ lchar* la_lds(int at) { return (lchar*)(uintptr_t)(unsigned)at; }
__device__ __forceinline__ int la_lds_at(const lchar* p) { return (int)(uintptr_t)p; }

template <typename T, bool QUADS>
__device__ __forceinline__ LaFrag<T> la_row(int at, int m, int offset) {
    LaFrag<T> f;
    if constexpr (sizeof(T) == 2 && QUADS) {
        f.v = lds_ld<uint4>(la_lds(at ^ (64 * m)) + offset);
    } else if constexpr (sizeof(T) == 2) {
        const uint2 a = lds_ld<uint2>(la_lds(at ^ (64 * m)) + offset),
                    b = lds_ld<uint2>(la_lds(at ^ (64 * m + 32)) + offset);
        f.v = make_uint4(a.x, a.y, b.x, b.y);
    } else {
        const f32x4 a = lds_ld<f32x4>(la_lds(at ^ (128 * m)) + offset),
                    b = lds_ld<f32x4>(la_lds(at ^ (128 * m + 64)) + offset);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f.v[j] = a[j];
            f.v[4 + j] = b[j];
        }
    }
    return f;
}

// Columns 16 c + lane % 16, rows 32 m + 16 (e / 4) + 4 g + (e % 4), e < 8, of a
// tile in its own order: the four rows of a transposing read lie on different
// quarters of the banks and the lane groups' rows on both halves of a quarter
// (in the QUADS order a read would touch every other 8 bytes only).  fp32
// reads take one address per row of a quad (e % 4).
template <typename T, int RB>
__device__ __forceinline__ int la_col_at(int l15, int g, int j) {
    if constexpr (sizeof(T) == 2) {
        const int row = 4 * g + (l15 >> 2);
        return row * RB + 16 * (((l15 >> 1) & 1) ^ la_swz<T, RB>(row)) + 8 * (l15 & 1);
    } else {
        const int row = 4 * g + j;
        return row * RB + 16 * ((l15 >> 2) ^ la_swz<T, RB>(row)) + 4 * (l15 & 3);
    }
}
template <typename T>
struct LaColAt {
    int at[sizeof(T) == 2 ? 1 : 4];
};
template <typename T, int RB>
__device__ __forceinline__ LaFrag<T> la_col(const LaColAt<T>& a, int m, int c) {
    LaFrag<T> f;
    if constexpr (sizeof(T) == 2) {
        const lchar* p = la_lds(a.at[0] ^ (32 * c)) + 32 * m * RB;
        const uint2 x = lds_tr4(p), y = lds_tr4(p + 16 * RB);
        f.v = make_uint4(x.x, x.y, y.x, y.y);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f.v[e] = lds_ld<float>(la_lds(a.at[e & 3] ^ (64 * c)) + (32 * m + 16 * (e >> 2)) * RB);
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
// computed where it is used and not held in registers across the loop.
__device__ __forceinline__ int la_fresh(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

__device__ __forceinline__ int la_fresh_s(int x) {
    asm volatile("" : "+s"(x));
    return x;
}

// A product whose upper half no register is kept for.
__device__ __forceinline__ unsigned la_mul(unsigned a, unsigned b) { return (unsigned)la_fresh((int)(a * b)); }

// Global memory goes through buffer instructions: a scalar descriptor with the
// range of a chunk's rows and one 32-bit offset per access; reads outside the
// range give zeros and writes outside are dropped, so that rows behind the last
// token and columns behind the width (an offset of kLaOut or more) need no
// branches.  Only the offset in the vector register is checked, so everything
// that varies is in it.
constexpr unsigned kLaOut = 0x80000000u;   // behind every range (host: 64 rows span less)
typedef __amdgpu_buffer_rsrc_t LaRange;

__device__ __forceinline__ LaRange la_range(const void* p, int64_t offset, int rows, unsigned row_bytes, unsigned width) {
    const unsigned n = rows <= 0 ? 0u : (unsigned)((rows < 64 ? rows : 64) - 1) * row_bytes + width;
    return __builtin_amdgcn_make_buffer_rsrc((char*)p + offset, 0, (int)n, 0x00027000);
}

// 64 x PPR 16-byte pieces of a chunk's rows (in the pass's order): a thread
// takes piece tid % PPR of rows tid / PPR + i STEP.  flip: 63 for a pass that
// runs backwards, else 0.
template <int PPR, int NTHR>
__device__ __forceinline__ int la_offset(unsigned tid, unsigned row_bytes, int flip, int pieces) {
    constexpr unsigned STEP = NTHR / PPR;
    const unsigned p = tid % PPR, row = (tid / PPR) ^ (flip & (STEP - 1));
    return ((int)p < pieces ? 16 * p : kLaOut) + la_mul(row, row_bytes);
}
template <int N, int PPR, int NTHR>
__device__ __forceinline__ unsigned la_step(int i, unsigned row_bytes, int flip) {
    constexpr unsigned STEP = NTHR / PPR;
    return (flip ? N - 1 - i : i) * STEP * row_bytes;
}
template <int N, int PPR, int NTHR>
__device__ __forceinline__ void la_fetch(uint4 (&r)[N], LaRange range, unsigned off, unsigned row_bytes, int flip) {
#pragma unroll
    for (int i = 0; i < N; ++i)
        r[i] = __builtin_bit_cast(
            uint4, __builtin_amdgcn_raw_buffer_load_b128(range, off + la_step<N, PPR, NTHR>(i, row_bytes, flip), 0, 0));
}

// A thread's place in a tile: row tid / PPR, piece tid % PPR (QUADS: where the
// first half of the piece goes; the second half's place is 16 bytes away, a
// flip).  Rows STEP apart have the same swizzle where STEP is a multiple of 16.
template <typename T, int PPR, bool QUADS>
__device__ __forceinline__ int la_slot(unsigned tid, int rows) {
    const unsigned row = tid / PPR + rows, p = tid % PPR;
    const int s = la_swz<T, PPR * 16>(row);
    if constexpr (!QUADS) return row * (PPR * 16) + 16 * (p ^ s);
    return row * (PPR * 16) + 16 * (((p & ~3u) + 2 * (p & 1)) ^ s) + 8 * ((p >> 1) & 1);
}
template <typename T, int PPR, int NTHR, bool QUADS>
struct LaSlots {
    static constexpr int STEP = NTHR / PPR, N = STEP >= 16 ? 1 : 16 / STEP;
    int at[N];
    __device__ __forceinline__ LaSlots(const lchar* tile, unsigned tid) {
#pragma unroll
        for (int i = 0; i < N; ++i) at[i] = la_lds_at(tile) + la_slot<T, PPR, QUADS>(tid, i * STEP);
    }
    __device__ __forceinline__ int operator[](int i) const {
        return at[i % N] + i / N * (N * STEP) * (PPR * 16);
    }
};
template <typename T, int N, int PPR, int NTHR, bool QUADS>
__device__ __forceinline__ void la_stage(const uint4 (&r)[N], const LaSlots<T, PPR, NTHR, QUADS>& slot) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if constexpr (QUADS) {
            lds_st(la_lds(slot[i]), make_uint2(r[i].x, r[i].y));
            lds_st(la_lds(slot[i] ^ 16), make_uint2(r[i].z, r[i].w));
        } else {
            lds_st(la_lds(slot[i]), r[i]);
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

// The last lane's value.
__device__ __forceinline__ double la_last(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const unsigned lo = __builtin_amdgcn_readlane((int)(unsigned)u, 63);
    const unsigned hi = __builtin_amdgcn_readlane((int)(unsigned)(u >> 32), 63);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// 2^x to fp32: the hardware's 2^hi (one unit in the last place) times 2^lo, where
// x = hi + lo; hi alone would be off by up to |x| 2^-24 ln 2 (e^-75: 44 units of
// 2^-24).  Three per lane and chunk, in one wave: within 0.6% of the time.
__device__ __forceinline__ float la_exp2(double x) {
    const float hi = (float)x, lo = (float)(x - (double)hi);
    const float e = __builtin_amdgcn_exp2f(hi);
    return e * __builtin_fmaf(lo, 0.693147180559945f, 1.f);
}

// log alpha below -256 / log2(e) counts as that: its e^ is 0 in fp32.
constexpr float kLaZero = -177.445678f;

// The decays of a chunk in LDS: u as hi + lo floats, e^u, e^{total - u}, and
// e^total; two buffers, the next chunk's made while this one's are read.
constexpr int kLaGateBytes = 4 * 64 * 4 + 16;

template <typename T, int DX, int NW, int NT, bool STATE>
constexpr int la_lds_bytes() {
    constexpr int y = 64 * DX * (int)sizeof(T), z = 64 * kLaCols * NW * (int)sizeof(T);
    return (STATE ? y + z : 2 * y + z + 64 * 64 * (int)sizeof(T) * la_terms<T, NT>() + NW * 256) + 2 * kLaGateBytes;
}

// Waves per SIMD that the registers are held to: four for bf16 workgroups of
// eight waves, two of which share a CU; one for fp32 workgroups of two waves,
// whose tiles (88 KB at d_k 128) leave a CU to one of them (H16 L4096, 128 x 32:
// 76 us, with two and 67 registers spilled 94); else two, all that the tiles in
// LDS leave room for.
template <typename T, int NW>
constexpr int la_waves() { return sizeof(T) == 2 ? (NW == 8 ? 4 : 2) : NW == 2 ? 1 : 2; }

template <typename T, int DX, int NW, int NT, bool STATE>
__global__ __launch_bounds__(64 * NW, (la_waves<T, NW>())) void la_kernel(LaArgs a) {
    constexpr int NTHR = 64 * NW;
    constexpr int EPP = 16 / (int)sizeof(T);              // elements per piece
    constexpr int PX = DX / EPP, PZ = kLaCols * NW / EPP; // pieces per row
    constexpr int RX = PX * 16, RZ = PZ * 16;             // bytes per row
    constexpr int RP = 64 * (int)sizeof(T);               // of the products x . y (each term)
    constexpr int NX = 64 * PX / NTHR, NZ = 64 * PZ / NTHR;
    constexpr int TX = DX / 16;                           // 16-row tiles of the state
    constexpr int TERMS = la_terms<T, NT>();
    constexpr bool BF = sizeof(T) == 2;
    extern __shared__ __attribute__((aligned(512))) char smem[];
    lchar* const sY = (lchar*)smem;
    lchar* const sZ = sY + 64 * RX;
    lchar* const sX = sZ + 64 * RZ;                       // not with STATE
    lchar* const sP = sX + 64 * RX;                       // nor this
    lchar* const sG = STATE ? sX : sP + TERMS * 64 * RP;
    lchar* const sR = sG + 2 * kLaGateBytes;              // [NW][64] partial dot products

    // Workgroups go to the eight XCDs in turn; consecutive work (heads that share
    // rows) stays on one of them.
    const int per = (a.total + 7) / 8;
    int id = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
    if (id >= a.total || (int)(blockIdx.x >> 3) >= per) return;
    // The passes of one segment run side by side, so that what they share is
    // read from memory once; the segments are taken from the last, which the
    // state pass has left in the caches.
    const LaPass& ps = a.pass[id % a.npass];
    id /= a.npass;
    const int nseq = a.B * a.H;
    if constexpr (!STATE) id = nseq * a.nseg - 1 - id;
    const int seq = id % nseq;
    const int sg = id / nseq;
    const int b = seq / a.H, hd = seq % a.H;
    const bool rev = ps.rev != 0;
    // nothing starts from behind the last segment
    if (STATE && sg == (rev ? 0 : a.nseg - 1)) return;

    const unsigned tid = threadIdx.x;
    const int lane = tid & 63, g = lane >> 4, l15 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int zc0 = wave * kLaCols;     // the wave's first column
    const int Dx = ps.Dx, Dz = ps.Dz, L = a.L;
    const int px = Dx / EPP, pz = Dz / EPP;
    const char* gx = nullptr;
    if constexpr (!STATE)
        gx = (const char*)ps.x.p + sizeof(T) * (b * ps.x.b + (hd / ps.x.group) * ps.x.h);
    const char* gy = (const char*)ps.y.p + sizeof(T) * (b * ps.y.b + (hd / ps.y.group) * ps.y.h);
    const char* gz = (const char*)ps.z.p + sizeof(T) * (b * ps.z.b + (hd / ps.z.group) * ps.z.h);
    // bytes between rows (host: below 2^25) and of a row
    const unsigned bx = STATE ? 0u : (unsigned)(sizeof(T) * ps.x.t), by = (unsigned)(sizeof(T) * ps.y.t),
                   bz = (unsigned)(sizeof(T) * ps.z.t);
    const int flip = rev ? 63 : 0;
    const float* la = a.la ? (a.la_head ? a.la + hd : a.la + (size_t)seq * L) : nullptr;
    const LaNeg neg = la_neg();

    // the state, from its start
    f32x4 S[TX];
    const float* start = nullptr;
    const size_t elems = (size_t)Dx * Dz;
    if constexpr (!STATE)
        start = a.nseg > 1 ? ps.seg + ((size_t)seq * a.nseg + sg) * elems : ps.start ? ps.start + seq * elems : nullptr;
    const int zc = zc0 + l15;
#pragma unroll
    for (int t = 0; t < TX; ++t) S[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (!STATE && start && zc < Dz) {
        // rows 16 t + 4 g + j: Dx is a multiple of 8, so four rows are inside or outside together
        if (ps.tr) {
            const float* s = start + (size_t)zc * Dx + 4 * g;
#pragma unroll
            for (int t = 0; t < TX; ++t)
                if (16 * t + 4 * g < Dx) S[t] = *reinterpret_cast<const f32x4*>(s + 16 * t);
        } else {
            const float* s = start + (size_t)(4 * g) * Dz + zc;
#pragma unroll
            for (int t = 0; t < TX; ++t)
                if (16 * t + 4 * g < Dx)
#pragma unroll
                    for (int j = 0; j < 4; ++j) S[t][j] = s[(16 * t + j) * Dz];
        }
    }

    const int c_lo = sg * a.cps, c_hi = min(a.NC, c_lo + a.cps);
    const int nc = c_hi - c_lo;
    const bool gate_wave = wave == NW - 1;
    double seg_total = 0.0;   // the gate wave's: the segment's sum of log2 alpha

    uint4 rx[STATE ? 1 : NX], ry[NX], rz[NZ];
    auto chunk = [&](int n) { return rev ? c_hi - 1 - n : c_lo + n; };
    const LaSlots<T, PX, NTHR, false> slot_y(sY, tid);
    const LaSlots<T, PZ, NTHR, false> slot_z(sZ, tid);
    auto fetch = [&](int n) {
        const int c = chunk(n), rows = L - 64 * c;
        const unsigned t = la_fresh(tid);
        if constexpr (!STATE)
            la_fetch<NX, PX, NTHR>(rx, la_range(gx, (int64_t)(64 * c) * bx, rows, bx, Dx * sizeof(T)),
                                   la_offset<PX, NTHR>(t, bx, flip, px), bx, flip);
        la_fetch<NX, PX, NTHR>(ry, la_range(gy, (int64_t)(64 * c) * by, rows, by, Dx * sizeof(T)),
                               la_offset<PX, NTHR>(t, by, flip, px), by, flip);
        la_fetch<NZ, PZ, NTHR>(rz, la_range(gz, (int64_t)(64 * c) * bz, rows, bz, Dz * sizeof(T)),
                               la_offset<PZ, NTHR>(t, bz, flip, pz), bz, flip);
    };
    auto log_alpha = [&](int n) {
        const int t = 64 * chunk(n) + ((la_fresh(tid) & 63) ^ flip);
        return la && t < L ? la[a.la_head ? 0 : t] : 0.f;
    };
    auto decays = [&](int n, float x) {
        const int l = (la_fresh(tid) & 63);
        lchar* gt = sG + (n & 1) * kLaGateBytes + 4 * l;
        const double l2 = x < kLaZero ? -256.0 : (double)x * 1.4426950408889634;
        const double s = la_scan(l2);
        const double total = la_last(s);
        const double u = rev ? s - l2 : s;
        const float uh = (float)u;
        // a row behind the last token adds nothing to others: its u is beyond
        // every other row's and its e^{total - u} zero (where rows of an input
        // share memory, its loads are not zeros)
        const bool in = 64 * chunk(n) + (l ^ flip) < L;
        lds_st(gt, in ? uh : 1e30f);
        lds_st(gt + 256, (float)(u - (double)uh));
        lds_st(gt + 512, la_exp2(u));
        lds_st(gt + 768, in ? la_exp2(total - u) : 0.f);
        if (l == 0) lds_st(gt + 1024, la_exp2(total));
        if constexpr (STATE) seg_total += total;
    };

    // The output rows of a chunk are stored after the next chunk is staged: a
    // wait for loads waits for every store before them too.  bf16 rows leave
    // through the waves' own columns of z in LDS, as whole rows; fp32 rows as
    // the lanes hold them (64 bytes of a row per wave).
    f32x4 O[4];            // O^T: the wave's columns by rows 16 it + lane % 16
    typedef uint4 Pieces[BF ? NZ : 1];
    RawN<!BF, 4> W[4];
    const bool dots = !STATE && NT != 2 && ps.w.p != nullptr, out_bf16 = ps.out_bf16 != 0;
    const int osz = out_bf16 ? 2 : 4;
    const unsigned bo = (unsigned)(osz * ps.ot), bw = (unsigned)(sizeof(T) * ps.w.t);
    char* const gout = STATE ? nullptr : (char*)ps.out + osz * (b * ps.ob + hd * ps.oh);
    const char* gw = dots ? (const char*)ps.w.p + sizeof(T) * (b * ps.w.b + (hd / ps.w.group) * ps.w.h) : nullptr;
    float* const gd = dots ? ps.dots + (size_t)seq * L : nullptr;
    // the lane's four columns of row l15 (in the pass's order), in a tensor of
    // `size`-byte values, and the step to row 16 it + l15
    auto out_offset = [&](unsigned row_bytes, int size) {
        const int l = (la_fresh(tid) & 63), col = zc0 + 4 * (l >> 4);
        return (col < Dz ? (unsigned)(size * col) : kLaOut) + la_mul((l & 15) ^ (flip & 15), row_bytes);
    };
    auto out_step = [&](int it, unsigned row_bytes) { return 16u * (unsigned)(it ^ (flip & 3)) * row_bytes; };
    auto fetch_w = [&](int n) {
        const int c = chunk(n);
        const LaRange r = la_range(gw, (int64_t)(64 * c) * bw, L - 64 * c, bw, Dz * sizeof(T));
        const unsigned off = out_offset(bw, sizeof(T));
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            const unsigned at = off + out_step(it, bw);
            if constexpr (BF)
                W[it] = __builtin_bit_cast(RawN<!BF, 4>, __builtin_amdgcn_raw_buffer_load_b64(r, at, 0, 0));
            else
                W[it] = __builtin_bit_cast(RawN<!BF, 4>, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
        }
    };
    // the rows' dot products, per wave into LDS, then their sums.  A sum over
    // the four lane groups takes two exchanges of groups, each of which adds two
    // rows' halves at once and leaves them to a group each.
    auto dot_rows = [&]() {
        float dot[4];
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            float w4[4];
            cvt_rawn<!BF, 4>(W[it], w4);
            dot[it] = O[it][0] * w4[0];
#pragma unroll
            for (int j = 1; j < 4; ++j) dot[it] += O[it][j] * w4[j];
        }
        auto add = [](auto r) { return __uint_as_float(r[0]) + __uint_as_float(r[1]); };
#pragma unroll
        for (int it = 0; it < 4; it += 2)
            dot[it] = add(__builtin_amdgcn_permlane16_swap(__float_as_uint(dot[it]), __float_as_uint(dot[it + 1]), false,
                                                           false));
        dot[0] = add(__builtin_amdgcn_permlane32_swap(__float_as_uint(dot[0]), __float_as_uint(dot[2]), false, false));
        lds_st(sR + 256 * wave + 4 * (la_fresh(tid) & 63), dot[0]);   // group g: row 16 g + l15
    };
    auto store_dots = [&](int n) {
        if (tid >= 64) return;
        const int l = la_fresh(tid), t = 64 * chunk(n) + (l ^ flip);
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) x += lds_ld<float>(sR + 256 * w + 4 * l);
        if (t < L) gd[t] = x;
    };
    // at the end of a chunk: bf16 rows into LDS
    auto finish = [&]() {
        const int l = (la_fresh(tid) & 63), g = l >> 4, l15 = l & 15;
        if constexpr (BF) {
            if (out_bf16) {
                lchar* at = sZ + l15 * RZ + 16 * ((2 * wave + (g >> 1)) ^ la_swz<T, RZ>(l15)) + 8 * (g & 1);
#pragma unroll
                for (int it = 0; it < 4; ++it)
                    lds_st(at + 16 * it * RZ, make_uint2(la_pack(O[it][0], O[it][1]), la_pack(O[it][2], O[it][3])));
            }
        }
    };
    auto store = [&](int n, const Pieces& ro) {
        typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
        const int c = chunk(n), rows = L - 64 * c;
        const LaRange r = la_range(gout, (int64_t)(64 * c) * bo, rows, bo, Dz * osz);
        if (BF && out_bf16) {
            if constexpr (BF) {
                const unsigned off = la_offset<PZ, NTHR>(la_fresh(tid), bo, flip, pz);
#pragma unroll
                for (int i = 0; i < NZ; ++i)
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, ro[i]), r,
                                                           off + la_step<NZ, PZ, NTHR>(i, bo, flip), 0, 0);
            }
        } else {
            const unsigned off = out_offset(bo, osz);
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const unsigned at = off + out_step(it, bo);
                if (!BF && out_bf16) {
                    typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
                    const u32x2 v = {la_pack(O[it][0], O[it][1]), la_pack(O[it][2], O[it][3])};
                    __builtin_amdgcn_raw_buffer_store_b64(v, r, at, 0, 0);
                } else {
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, O[it]), r, at, 0, 0);
                }
            }
        }
    };
    const int ax0 = la_lds_at(sX) + la_row_at<T, RX, true>(l15, g), ap = la_lds_at(sP) + la_row_at<T, RP, true>(l15, g);
    LaColAt<T> ay0, az;
#pragma unroll
    for (int j = 0; j < (BF ? 1 : 4); ++j) {
        ay0.at[j] = la_lds_at(sY) + la_col_at<T, RX>(l15, g, j);
        az.at[j] = la_lds_at(sZ) + (la_col_at<T, RZ>(l15, g, j) ^ (2 * (int)sizeof(T) * 8 * wave));
    }
    fetch(0);
    if (gate_wave) decays(0, log_alpha(0));
    if constexpr (!STATE)   // the blocks above the diagonal stay zero
        for (unsigned i = tid; i < TERMS * 64 * RP / 16; i += NTHR) lds_st(sP + 16 * i, make_uint4(0u, 0u, 0u, 0u));

    for (int n = 0; n < nc; ++n) {
        const lchar* gt = sG + (n & 1) * kLaGateBytes;
        if (n) lds_barrier();   // the last chunk's tiles are done with
        Pieces ro;
        if constexpr (!STATE && BF)
#pragma unroll
            for (int i = 0; i < NZ; ++i) ro[i] = lds_ld<uint4>(la_lds(slot_z[i]));
        if constexpr (!STATE) la_stage(rx, LaSlots<T, PX, NTHR, BF>(sX, la_fresh(tid)));
        la_stage(ry, slot_y);
        la_stage(rz, slot_z);
        lds_barrier();
        if constexpr (!STATE)
            if (n) {
                store(n - 1, ro);
                if (dots) dot_rows();
            }
        float next_la = 0.f;
        if (n + 1 < nc) {
            fetch(n + 1);
            if (gate_wave) next_la = log_alpha(n + 1);
        }

        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        const float decay = lds_ld<float>(gt + 1024);
        if constexpr (!STATE) {
            const int ax = la_fresh(ax0);
            // 16 x 16 blocks (it, jt), jt <= it, of the products x . y, times their decays, into LDS
            for (int n = wave; n < 10; n += NW) {
                const int k = 2 * la_fresh_s(n), it = (0xFFA94 >> k) & 3, jt = (0xE4910 >> k) & 3;   // row by row
                const int l = (la_fresh(tid) & 63), g = l >> 4, l15 = l & 15;
                const int yrow = la_fresh(la_lds_at(sY) + la_row_at<T, RX, false>(l15, g) + 16 * jt * RX), xrow = la_fresh(ax + 16 * it * RX);
                f32x4 P = zero;
#pragma unroll
                for (int m = 0; m < DX / 32; ++m)
                    P = la_mfma(la_row<T, false>(yrow, m, 0).v, la_row<T, true>(xrow, m, 0).v, P);
                const lchar* ti = gt + la_fresh(4 * l15) + 64 * it;
                const lchar* tj = gt + la_fresh(16 * g) + 64 * jt;
                const float ui = lds_ld<float>(ti), wi = lds_ld<float>(ti + 256);
                const f32x4 uj = lds_ld<f32x4>(tj), wj = lds_ld<f32x4>(tj + 256);
                const int last = 16 * (it - jt) + l15 - 4 * g;   // of the lane's j that row i takes
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float d = (ui - uj[e]) + (wi - wj[e]);
                    const float x = P[e] * __builtin_amdgcn_exp2f(d);
                    v[e] = e <= last ? x : 0.f;
                }
                if constexpr (BF) {
                    // la_row's order of quads: 8-byte quad 4 (jt % 2) + g of 32 values
                    lchar* at = la_lds(la_fresh(ap) ^ (64 * (jt >> 1))) + 16 * it * RP + 8 * (jt & 1);
#pragma unroll
                    for (int term = 0; term < TERMS; ++term) {
                        const unsigned lo = la_pack(v[0], v[1]), hi = la_pack(v[2], v[3]);
                        lds_st(at + term * 64 * RP, make_uint2(lo, hi));
                        if (term + 1 < TERMS) {
                            la_rest(lo, neg, v[0], v[1]);
                            la_rest(hi, neg, v[2], v[3]);
                        }
                    }
                } else {
                    lds_st(la_lds(la_fresh(ap) ^ (64 * jt)) + 16 * it * RP, f32x4{v[0], v[1], v[2], v[3]});
                }
            }
            // what the state at the chunk's start gives the rows
#pragma unroll
            for (int m = 0; m < DX / 32; ++m) {
                float s8[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    s8[e] = S[2 * m + (e >> 2)][e & 3];
                    S[2 * m + (e >> 2)][e & 3] *= decay;   // here: the split takes the old one's register
                }
                const LaTerms<T, NT> st = la_split<T, NT>(s8, neg);
#pragma unroll
                for (int i0 = 0; i0 < 4; i0 += 2) {
                    LaFrag<T> x[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) x[i] = la_row<T, true>(ax, m, 16 * (i0 + i) * RX);
#pragma unroll
                    for (int term = TERMS - 1; term >= 0; --term)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            O[i0 + i] = la_mfma(la_term(st, term), x[i].v,
                                                m == 0 && term == TERMS - 1 ? zero : O[i0 + i]);
                }
                __builtin_amdgcn_sched_barrier(0);   // no more of x in registers at once
            }
            const lchar* eu = gt + 512 + 4 * (la_fresh(tid) & 15);
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const float e = lds_ld<float>(eu + 64 * it);
#pragma unroll
                for (int j = 0; j < 4; ++j) O[it][j] *= e;
            }
        }
        if constexpr (STATE) {
#pragma unroll
            for (int t = 0; t < TX; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) S[t][j] *= decay;
        } else {
            lds_barrier();   // the products are in LDS
        }
        if constexpr (!STATE)
            if (dots && n) store_dots(n - 1);
        LaColAt<T> ay;
#pragma unroll
        for (int j = 0; j < (BF ? 1 : 4); ++j) ay.at[j] = la_fresh(ay0.at[j]);
        const int g = (la_fresh(tid) & 63) >> 4;
        // rows 32 ks .. 32 ks + 31 of y and z: into the output's later rows, then into the state
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            const LaFrag<T> z = la_col<T, RZ>(az, ks, 0);
            if constexpr (!STATE) {
                const int pr = la_fresh(ap);
#pragma unroll
                for (int it = 2 * ks; it < 4; ++it) {
#pragma unroll
                    for (int term = TERMS - 1; term >= 0; --term)
                        O[it] = la_mfma(z.v, la_row<T, true>(pr, ks, term * 64 * RP + 16 * it * RP).v, O[it]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            const int j0 = 32 * ks + 4 * g;   // the lane's rows: j0 + [0, 4) and j0 + 16 + [0, 4)
            const f32x4 k0 = lds_ld<f32x4>(gt + 768 + 4 * j0), k1 = lds_ld<f32x4>(gt + 768 + 4 * j0 + 64);
            float z8[8];
            la_floats(z, z8);
#pragma unroll
            for (int e = 0; e < 8; ++e) z8[e] *= e < 4 ? k0[e & 3] : k1[e & 3];
            const LaTerms<T, 3> zt = la_split<T, 3>(z8, neg);
#pragma unroll
            for (int t0 = 0; t0 < TX; t0 += 2) {
                LaFrag<T> y[2];
#pragma unroll
                for (int t = 0; t < 2; ++t) y[t] = la_col<T, RX>(ay, ks, t0 + t);
                if constexpr (BF) {
#pragma unroll
                    for (int term = la_terms<T, 3>() - 1; term >= 0; --term)
#pragma unroll
                        for (int t = 0; t < 2; ++t) S[t0 + t] = la_mfma(y[t].v, la_term(zt, term), S[t0 + t]);
                } else {
                    // on top of S each of the 32 products would round it
                    f32x4 add[2];
#pragma unroll
                    for (int t = 0; t < 2; ++t) add[t] = la_mfma(y[t].v, la_term(zt, 0), zero);
#pragma unroll
                    for (int t = 0; t < 2; ++t) S[t0 + t] = S[t0 + t] + add[t];
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if (gate_wave && n + 1 < nc) decays(n + 1, next_la);
        if constexpr (!STATE) {
            if (dots) fetch_w(n);
            finish();
        }
    }
    if constexpr (!STATE) {
        lds_barrier();
        Pieces ro;
        if constexpr (BF)
#pragma unroll
            for (int i = 0; i < NZ; ++i) ro[i] = lds_ld<uint4>(la_lds(slot_z[i]));
        store(nc - 1, ro);
        if (dots) {
            dot_rows();
            lds_barrier();
            store_dots(nc - 1);
        }
    }

    float* end = nullptr;
    if constexpr (STATE) {
        end = ps.seg + ((size_t)seq * a.nseg + sg) * elems;
        if (gate_wave && (la_fresh(tid) & 63) == 0)
            ps.segdec[(size_t)seq * a.nseg + sg] = la_exp2(seg_total);
    } else if (ps.end && sg == (rev ? 0 : a.nseg - 1)) {
        end = ps.end + seq * elems;
    }
    const int l_end = la_fresh(tid) & 63, g_end = l_end >> 4, zc_end = zc0 + (l_end & 15);
    if (end && zc_end < Dz) {
        const bool tr = ps.tr != 0;
        float* e = tr ? end + (size_t)zc_end * Dx + 4 * g_end : end + (size_t)(4 * g_end) * Dz + zc_end;
#pragma unroll
        for (int t = 0; t < TX; ++t) {
            if (16 * t + 4 * g_end >= Dx) continue;
            if (tr) {
                *reinterpret_cast<f32x4*>(e + 16 * t) = S[t];
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) e[(16 * t + j) * Dz] = S[t][j];
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
    if (waves == 8) return la_launch<T, DX, 8, NT, STATE>(a, slot, st);
    if (waves == 4) return la_launch<T, DX, 4, NT, STATE>(a, slot, st);
    return la_launch<T, DX, 2, NT, STATE>(a, slot, st);
}

}  // namespace dr
