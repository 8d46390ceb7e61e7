// dr_layernorm.h -- argument blocks and launchers of the layer norm
// (dr_linattn_abi.hip on the host side, dr_layernorm.hip the kernels).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dr {

struct LnRows {
    int64_t b, h, t;   // strides in elements
};

// Rows (b, h, l) of D values.  Rows that share a weight form a group: one per
// head (per_head; rows_per_group = B * L), or one in all (B * H * L).
struct LnArgs {
    const void* x;
    const float* w;     // [groups][D] or NULL (ones)
    const float* bias;  // [groups][D] or NULL (zeros)
    const float* mean;  // backward: the forward's statistics, [B][H][L]
    const float* rstd;
    const void* dy;
    void* y;            // y, or dx
    float* mean_out;    // forward: statistics, or NULL
    float* rstd_out;
    float* part;        // backward: [groups][blocks][2][D] partial sums, or NULL
    float* dw;          // [groups][D] or NULL
    float* db;
    LnRows sx, sy, sdy;
    int B, H, L, D;
    int per_head;
    unsigned groups, rows;   // rows per group
    unsigned blocks;         // workgroups per group
    float eps;
    int x_f32, y_f32, dy_f32;
};

// Lanes per row and 8-value vectors per lane for rows of D values.
struct LnShape {
    int lanes, vecs;
};
LnShape ln_shape(int D);
// Rows that a workgroup takes in one pass.
int ln_pass_rows(int D);
// width: values read or written at once, 8, 2 or 1 (D and every stride a
// multiple of it)
hipError_t launch_ln_fwd(const LnArgs& a, int width, int slot, hipStream_t st);
hipError_t launch_ln_bwd(const LnArgs& a, int width, int slot, hipStream_t st);
hipError_t launch_ln_zero(float* p, size_t n, int slot, hipStream_t st);

}  // namespace dr
