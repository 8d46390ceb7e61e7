// dr_seqops.h -- argument blocks and launchers of the RMS norm, the short causal
// convolution and the gated linear recurrence (dr_seqops_abi.hip on the host side,
// dr_rmsnorm.hip, dr_conv.hip and dr_scan.hip the kernels).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "dr_layernorm.h"

namespace dr {

struct SeqRows {
    int64_t b, t;   // strides in elements
};

// ------------------------------------------------------------ RMS norm
// Rows, groups and strides as in LnArgs.
struct RnArgs {
    const void* x;
    const void* r;        // the residual, or NULL; backward: the sum's gradient
    const float* w;       // [groups][D] or NULL (ones)
    const float* rstd;    // backward: the forward's, [B][H][L]
    const void* dy;
    void* y;              // y, or dx
    void* total;          // x + r, in r's type
    float* scale;         // [B][H][L][blocks of a row]; set: y is e4m3
    float* rstd_out;      // or NULL
    float* part;          // backward: [groups][blocks][D] partial sums, or NULL
    float* dw;
    LnRows sx, sr, sy, st, sdy;
    int B, H, L, D;
    int per_head;
    unsigned groups, rows, blocks;
    float eps;
    int block;            // columns that share a scale: 128, or 0 for a row
    int x_f32, r_f32, y_f32, dy_f32;
};
// rows: of all groups
LnShape rn_shape(int D, size_t rows);
int rn_pass_rows(int D, size_t rows);
hipError_t launch_rn_fwd(const RnArgs& a, int slot, hipStream_t st);
hipError_t launch_rn_bwd(const RnArgs& a, int slot, hipStream_t st);

// ------------------------------------------------------------ short convolution
struct ScArgs {
    const void* x;
    const float* w;       // [C][W]
    const float* bias;    // [C] or NULL
    const void* state;    // [B][W - 1][C], x's type, or NULL (zeros)
    void* y;              // or dx
    void* state_out;      // or NULL
    const void* dy;
    const float* dstate_in;   // gradient of the final state, [B][W - 1][C], or NULL
    float* dstate;            // gradient of the initial state, or NULL
    float* part;          // backward: [blocks][C][W + 1] partial sums, or NULL
    float* dw;            // [C][W] or NULL
    float* db;            // [C] or NULL
    SeqRows sx, sy, sdy;
    int B, L, C, W;
    int silu;
    int run;              // tokens of a thread
    unsigned tiles;       // 16 runs each, over all sequences
    unsigned blocks;      // backward: workgroups that share a channel tile's tiles
    int x_f32, y_f32, dy_f32;
};
int sc_run(int W);    // a thread's tokens are a multiple of this
hipError_t launch_sc_fwd(const ScArgs& a, int slot, hipStream_t st);
hipError_t launch_sc_bwd(const ScArgs& a, int slot, hipStream_t st);
hipError_t launch_sc_step(const ScArgs& a, int slot, hipStream_t st);
// `bytes` (a multiple of 2) copied, or zeroed where from is NULL
hipError_t launch_seq_copy(void* to, const void* from, size_t bytes, int slot, hipStream_t st);

// ------------------------------------------------------------ gated linear recurrence
// A divisor of numbers below 2^31: n / d = n factor >> shift.
struct GsDivide {
    unsigned factor, shift;
};
inline GsDivide gs_divider(unsigned d) {
    unsigned l = 0;
    while (((uint64_t)1 << l) < d) ++l;
    return {(unsigned)((((uint64_t)1 << (31 + l)) / d) + 1), 31 + l};
}

struct GsArgs {
    const void* x;
    const void* g;
    const float* h0;      // [B][C] or NULL
    const void* h;        // backward: the forward's h
    const void* dh;
    const float* dlast;   // backward: gradient of the last state, or NULL
    void* out;            // h, or dx
    void* dg;
    float* last;          // forward: the last state; backward: dh0; or NULL
    SeqRows sx, sg, sh, sdh, so, sdg;
    int B, L, C;
    int groups;           // runs of tokens side by side in a workgroup
    int nseg;             // tiles of a sequence
    unsigned columns;     // B times the channel tiles
    unsigned padded;      // columns, and some that are left out
    unsigned tiles;       // channel tiles
    GsDivide by_columns, by_tiles;   // padded columns
    uint64_t* maps;       // where a column's tiles have workgroups of their own, else NULL; for each
                          // column [nseg][64] what each tile does to the state, [nseg][64] what it
                          // starts with
    unsigned* counters;   // tiles drawn, of each column; the maps stand behind them
    size_t words;         // 64-bit words of both
    int x_f32, g_f32, h_f32, dh_f32, out_f32;
    int logit;            // decay: 0 e^g, 1 sigmoid(g)
    int inputs;           // 0 plain, 1 blend, 2 unit
};
constexpr int kGsTile = 64;    // channels of a workgroup
constexpr int kGsRun = 4;      // tokens of a thread, forward and backward
hipError_t launch_gs_fwd(const GsArgs& a, int slot, hipStream_t st);
hipError_t launch_gs_bwd(const GsArgs& a, int slot, hipStream_t st);
hipError_t launch_gs_clear(const GsArgs& a, int slot, hipStream_t st);
constexpr int kGsCounter = 32; // a column's counter has 128 bytes to itself
hipError_t launch_gs_step(const GsArgs& a, int slot, hipStream_t st);

}  // namespace dr
