// gmm_mxw.hip -- the grouped matmul of a bf16 lhs with microscaled fp4
// weights: e2m1 codes with one E8M0 scale per 32 elements of K.  A weight is
// widened to bf16 on its way to the matrix cores by the conversion that takes
// the scale with it (2^e times a value of at most two significant bits is a
// bf16), so no scale is folded into sums and the products are plain bf16 ones
// with fp32 sums.
#include "gmm_general.hpp"

namespace gmmk {

hipError_t launch_mxw(const Params& p, const KernelChoice& c, int cu, hipStream_t st) {
  constexpr int FMT = 5 << 3;
  if (c.size == SizeClass::Big)
    return launch_cfg<typename Pick<Op::BF16, false, true, false, SizeClass::Big, FMT, true>::type>(p, cu, c.grid_cap,
                                                                                                   st);
  return launch_cfg<typename Pick<Op::BF16, false, true, false, SizeClass::Small, FMT, true>::type>(p, cu, c.grid_cap,
                                                                                                   st);
}

}  // namespace gmmk
