// gmm_mxw.hip -- the grouped matmul of a bf16 lhs with microscaled fp4
// weights (e2m1 codes with one E8M0 scale per 32 elements of K): launchers of
// the kernel for few rows per group (gmm_mxw_rows.hpp) and the one for large
// groups (gmm_mxw_big.hpp).  Both widen a weight to bf16 on its way to the
// matrix cores with the conversion that takes the scale along (a power of two
// times a value of two significant bits is a bf16), so no scale is folded into
// sums: the products are plain bf16 ones with fp32 sums.
#include <atomic>

#include "gmm_mxw_big.hpp"
#include "gmm_mxw_launch.hpp"
#include "gmm_mxw_rows.hpp"

namespace gmmk {

namespace {

// Every kernel walks its tiles with a stride, so any grid is correct; a
// positive cap (a test hook) makes each workgroup run many tiles.
template <class Kernel>
hipError_t launch(Kernel kernel, const Params& p, long long grid, int threads, int cap, hipStream_t st) {
  if (grid >= 8) grid -= grid % 8;
  if (grid < 1) grid = 1;
  if (cap > 0 && grid > cap) grid = cap;
  hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(threads), 0, st, p);
  return hipGetLastError();
}

// Upper bound on the tiles of a problem: group-aligned row tiles are at most
// ceil(M / BM) + Ga.
template <class C>
long long most_tiles(const Params& p) {
  return ((p.M + C::BM - 1LL) / C::BM + p.Ga) * ((p.N + C::BN - 1LL) / C::BN);
}

template <bool OUT_F32>
hipError_t launch_rows(const Params& p, int cu, int cap, hipStream_t st) {
  using C = RowsCfg;
  static std::atomic<int> occ_cache{0};
  int occ = occ_cache.load();
  if (occ <= 0) {
    const hipError_t e = hipOccupancyMaxActiveBlocksPerMultiprocessor(&occ, gmm_mxw_rows_kernel<OUT_F32>, C::T, 0);
    if (e != hipSuccess) return e;
    if (occ < 1) occ = 1;
    occ_cache.store(occ);
  }
  // all workgroups that fit, or as many as there can be tiles, but at least
  // one per compute unit: they share the rows outside the active groups too
  long long grid = (long long)cu * occ;
  const long long tiles = most_tiles<C>(p);
  if (grid > tiles) grid = tiles > cu ? tiles : cu;
  return launch(gmm_mxw_rows_kernel<OUT_F32>, p, grid, C::T, cap, st);
}

template <bool OUT_F32, bool BIAS>
hipError_t launch_big(const Params& p, int cu, int cap, hipStream_t st) {
  using C = MxwBigCfg<OUT_F32, BIAS>;
  long long grid = cu;  // one workgroup per CU (LDS-bound)
  if (grid > most_tiles<C>(p) && most_tiles<C>(p) >= 8) grid = most_tiles<C>(p);
  return launch(gmm_mxw_big_kernel<C>, p, grid, C::T, cap, st);
}

}  // namespace

hipError_t launch_mxw(const Params& p, SizeClass size, int cu, int cap, hipStream_t st) {
  // The large-group kernel runs a tile in steps of 64, three at least; below
  // that a product is its output's stores, and the few-rows kernel is the
  // faster one (131072 rows, K = 128, N = 1408: 181 us, 369 MB written).
  if (size == SizeClass::Big && p.K >= 3 * 64) {
    const bool bias = p.rhs_bias != nullptr;
    if (p.out_f32)
      return bias ? launch_big<true, true>(p, cu, cap, st) : launch_big<true, false>(p, cu, cap, st);
    return bias ? launch_big<false, true>(p, cu, cap, st) : launch_big<false, false>(p, cu, cap, st);
  }
  return p.out_f32 ? launch_rows<true>(p, cu, cap, st) : launch_rows<false>(p, cu, cap, st);
}

}  // namespace gmmk
