// dr_rmsnorm.h -- what the RMS norm's kernels share (dr_rmsnorm.hip forward,
// dr_rmsnorm_bwd.hip the backward).
//
// A row is held by 8 to 256 lanes, 8 values per lane and vector; columns of vector v
// of a lane: 8 (lane + lanes v) and the seven behind it.
#pragma once

#include <hip/hip_runtime.h>

#include "dr_device.h"
#include "dr_internal.h"
#include "dr_norm_rows.h"
#include "dr_octet.h"
#include "dr_seqops.h"

namespace dr {

// Rows in flight per lane group, as for the layer norm.
template <int VPT>
constexpr int rn_rows() { return VPT == 1 ? 2 : 1; }
template <int VPT>
constexpr bool rn_ahead() { return VPT < 8; }

// Of a row as loaded: values that are another lane's, or behind the row, count as 0.
template <bool TAIL, bool SMALL, bool F32>
__device__ __forceinline__ float rn_value(const Oct<F32>& r, const OctPlace& p, int e) {
    const float x = oct_value(r, e);
    return (TAIL || SMALL ? oct_own<SMALL>(p, e) : p.own != 0) ? x : 0.f;
}

template <int LPR>
__device__ __forceinline__ OctPlace rn_place(int lane, int v, int D) {
    return oct_place(lane + LPR * v, D);
}

template <bool TAIL, bool SMALL, int LPR, int VPT>
__device__ __forceinline__ void rn_weights(const RnArgs& a, unsigned g, int lane, float (&w)[VPT][8]) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const OctPlace p = rn_place<LPR>(lane, v, a.D);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = a.w ? a.w[(size_t)g * a.D + (SMALL ? min(e, a.D - 1) : p.at + e)] : 1.f;
            w[v][e] = (TAIL || SMALL ? oct_own<SMALL>(p, e) : p.own != 0) ? x : 0.f;
        }
    }
}

}  // namespace dr
