// gmm_mxw_launch.hpp -- host-side launch entry point of the product of a bf16
// lhs with microscaled fp4 weights.
#pragma once

#include "gmm_launch.hpp"

namespace gmmk {

// Its size class: the large-group kernel's 256-row tiles pay from about 128
// rows a group on (32 groups of 128 rows, 1408 x 1408: 29.5 us against 35.0
// with the few-rows kernel; 128 of 64: 80 against 71; 1 of 4096: 34 against 36;
// 8 of 256, 4096 x 4096: 104 against 95).
inline SizeClass mxw_size(long long M, long long Ga) {
  return M >= 4096 && M >= 128 * Ga ? SizeClass::Big : SizeClass::Small;
}

// Queue it (gmm_mxw.hip); p.rhs_scale points to E8M0 bytes [Ga, K/32, 1, N].
hipError_t launch_mxw(const Params& p, SizeClass size, int cu_count, int grid_cap, hipStream_t stream);

}  // namespace gmmk
