// dr_linattn32.hip -- the chunked kernel of linear attention with a decay per
// head for fp32 inputs (dr_linattn_kernel.h), on the fp32 matrix ops.

#include "dr_linattn_kernel.h"

namespace dr {

hipError_t launch_la32(const LaArgs& a, int dx, int waves, bool state_only, int slot, hipStream_t st) {
    if (state_only)
        return dx == 64 ? la_launch_w<float, 64, 1, true>(a, waves, slot, st)
                        : la_launch_w<float, 128, 1, true>(a, waves, slot, st);
    return dx == 64 ? la_launch_w<float, 64, 1, false>(a, waves, slot, st)
                    : la_launch_w<float, 128, 1, false>(a, waves, slot, st);
}

}  // namespace dr
