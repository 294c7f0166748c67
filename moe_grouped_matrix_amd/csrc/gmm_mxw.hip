// gmm_mxw.hip -- the grouped matmul of a bf16 lhs with microscaled fp4
// weights: e2m1 codes with one E8M0 scale per 32 elements of K.  A weight is
// widened to bf16 on its way to the matrix cores by the conversion that takes
// the scale with it (2^e times a value of at most two significant bits is a
// bf16), so no scale is folded into sums and the products are plain bf16 ones
// with fp32 sums.
#include "gmm_general.hpp"
#include "gmm_mxw_big.hpp"
#include "gmm_mxw_rows.hpp"

namespace gmmk {

template <bool OUT_F32>
static hipError_t launch_rows(const Params& p, int cu, int cap, hipStream_t st) {
  static std::atomic<int> occ_cache{0};
  int occ = occ_cache.load();
  if (occ <= 0) {
    const hipError_t e = hipOccupancyMaxActiveBlocksPerMultiprocessor(&occ, gmm_mxw_rows_kernel<OUT_F32>, RowsCfg::T, 0);
    if (e != hipSuccess) return e;
    if (occ < 1) occ = 1;
    occ_cache.store(occ);
  }
  const long long items = ((p.M + RowsCfg::BM - 1LL) / RowsCfg::BM + p.Ga) * ((p.N + RowsCfg::BN - 1) / RowsCfg::BN);
  long long grid = (long long)cu * occ;
  if (grid > items && items >= cu) grid = items;
  if (grid >= 8) grid -= grid % 8;
  if (grid < 1) grid = 1;
  grid = apply_cap(grid, cap);
  hipLaunchKernelGGL(gmm_mxw_rows_kernel<OUT_F32>, dim3((unsigned)grid), dim3(RowsCfg::T), 0, st, p);
  return hipGetLastError();
}

template <bool OUT_F32, bool BIAS>
static hipError_t launch_mxw_big(const Params& p, int cu, int cap, hipStream_t st) {
  using C = MxwBigCfg<OUT_F32, BIAS>;
  const long long tiles = ((p.M + C::BM - 1LL) / C::BM + p.Ga) * ((p.N + C::BN - 1) / C::BN);
  long long grid = cu;  // one workgroup per CU (LDS-bound)
  if (grid > tiles && tiles >= 8) grid = tiles;
  if (grid >= 8) grid -= grid % 8;
  if (grid < 1) grid = 1;
  grid = apply_cap(grid, cap);
  hipLaunchKernelGGL(gmm_mxw_big_kernel<C>, dim3((unsigned)grid), dim3(C::T), 0, st, p);
  return hipGetLastError();
}

hipError_t launch_mxw(const Params& p, const KernelChoice& c, int cu, hipStream_t st) {
  constexpr int FMT = 5 << 3;
  // the big kernel runs a tile in steps of 64, three at least
  if (c.size == SizeClass::Big && p.K >= 192) {
    const bool bias = p.rhs_bias != nullptr;
    if (p.out_f32)
      return bias ? launch_mxw_big<true, true>(p, cu, c.grid_cap, st) : launch_mxw_big<true, false>(p, cu, c.grid_cap, st);
    return bias ? launch_mxw_big<false, true>(p, cu, c.grid_cap, st) : launch_mxw_big<false, false>(p, cu, c.grid_cap, st);
  }
  if (c.size == SizeClass::Big)
    return launch_cfg<typename Pick<Op::BF16, false, true, false, SizeClass::Big, FMT, true>::type>(p, cu, c.grid_cap,
                                                                                                   st);
  return p.out_f32 ? launch_rows<true>(p, cu, c.grid_cap, st) : launch_rows<false>(p, cu, c.grid_cap, st);
  return launch_cfg<typename Pick<Op::BF16, false, true, false, SizeClass::Small, FMT, true>::type>(p, cu, c.grid_cap,
                                                                                                   st);
}

}  // namespace gmmk
