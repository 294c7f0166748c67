// gmm_general.hpp -- tile shapes and launcher of the general kernel
// (gmm_device.hpp), for the translation units that instantiate it.
#pragma once

#include <atomic>

#include "gmm_device.hpp"
#include "gmm_launch.hpp"

namespace gmmk {

// Tile shapes.  Big: 256 x 128 output tile, four waves of 128 x 64 (for
// large groups); with scales, eight waves of 64 x 64, since the per-block
// partial and the running total both stay in registers.  Small: 32 x 64,
// four waves of 32 x 16 (decode-sized groups).  F32 uses 64 x 64 tiles of
// four 32 x 32 waves.
template <Op OP, bool NN, bool BF8, bool SC, SizeClass SZ, int FMT, bool MX = false>
struct Pick {
  using type = Cfg<OP, NN, BF8, 256, 128, SC ? 4 : 2, 2, SC, FMT, MX>;
};
template <Op OP, bool NN, bool BF8, bool SC, int FMT, bool MX>
struct Pick<OP, NN, BF8, SC, SizeClass::Small, FMT, MX> {
  using type = Cfg<OP, NN, BF8, 32, 64, 1, 4, SC, FMT, MX>;
};

// Every kernel below walks its work items with a grid stride, so any grid
// size is correct; a positive cap (a test hook) makes each workgroup run
// many tiles, with the operand streams carried from one tile to the next.
inline long long apply_cap(long long grid, int cap) { return cap > 0 && grid > cap ? cap : grid; }

template <class C>
hipError_t launch_cfg(const Params& p, int cu_count, int cap, hipStream_t stream) {
  static std::atomic<int> occ_cache{0};
  int occ = occ_cache.load();
  if (occ <= 0) {
    hipError_t e = hipOccupancyMaxActiveBlocksPerMultiprocessor(&occ, gmm_kernel<C>, C::T, 0);
    if (e != hipSuccess) return e;
    if (occ < 1) occ = 1;
    occ_cache.store(occ);
  }
  // Upper bound on work items: group-aligned m-tiles are at most
  // ceil(M/BM) + Ga, times the n-tiles, plus the zero-fill chunks.
  const long long n_tiles = (p.N + C::BN - 1) / C::BN;
  const long long m_tiles = (p.M + C::BM - 1) / C::BM + p.Ga;
  const long long row_bytes = (long long)p.N * (p.out_f32 ? 4 : 2);
  const long long zero_items = ((long long)p.M * row_bytes + kZeroChunk - 1) / kZeroChunk + 2;
  const long long bound = m_tiles * n_tiles + zero_items;
  long long grid = (long long)cu_count * occ;
  if (grid > bound) grid = bound;
  if (grid >= 8) grid -= grid % 8;
  if (grid < 1) grid = 1;
  grid = apply_cap(grid, cap);
  hipLaunchKernelGGL(gmm_kernel<C>, dim3((unsigned)grid), dim3(C::T), 0, stream, p);
  return hipGetLastError();
}

}  // namespace gmmk
