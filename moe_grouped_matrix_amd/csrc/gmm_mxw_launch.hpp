// gmm_mxw_launch.hpp -- host-side launch entry point of the product of a bf16
// lhs with microscaled fp4 weights.
#pragma once

#include "gmm_launch.hpp"

namespace gmmk {

// Its size class: the large-group kernel's 256-row tiles pay from about 128
// rows a group on, and once there are enough of them for the compute units.
// Few-rows / large-group kernel in us, equal groups:
//   groups x rows      1408 x 1408    4096 x 4096    N 2048, K 7168
//   128 x 64            71 / 82       433 / 561      407 / 483
//   128 x 128          120 / 91       815 / 628      737 / 550
//   32 x 128            34 / 29       199 / 161      192 / 142
//   8 x 256             23 / 32        93 / 108       86 / 140
//   8 x 512             34 / 34       190 / 110      173 / 162
//   1 x 2048            23 / 31        95 / 81        83 / 123
//   1 x 4096            33 / 32       178 / 107      148 / 124
// (One group of 2048 rows of 4096 x 4096 is on its wrong side.)
inline SizeClass mxw_size(long long M, long long Ga) {
  return M >= 4096 && M >= 128 * Ga ? SizeClass::Big : SizeClass::Small;
}

// Queue it (gmm_mxw.hip); p.rhs_scale points to E8M0 bytes [Ga, K/32, 1, N].
hipError_t launch_mxw(const Params& p, SizeClass size, int cu_count, int grid_cap, hipStream_t stream);

}  // namespace gmmk
