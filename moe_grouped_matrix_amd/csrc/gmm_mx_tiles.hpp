// gmm_mx_tiles.hpp -- the weight tiles of the microscaled fp4 quantiser and
// widening (plain integer code, also compiled for the host by the tests).
#pragma once

#ifndef GMM_HD
#define GMM_HD __host__ __device__
#endif

namespace gmmk {

constexpr int kMxRows = 64;    // rows of a weight tile
constexpr int kMxPanel = 128;  // most blocks of K in a weight tile

// A weight tile: rows [64 t, 64 t + rows) of group g, blocks [b0, b0 + nb).
struct MxTile {
  long long row0;    // first row of all
  long long scales;  // of (b0, the tile's first row) in [Ga, K/32, 1, N]
  int rows, b0, nb;
};

GMM_HD inline int mx_panels(int K) { return (K / 32 + kMxPanel - 1) / kMxPanel; }
// (N may be 2^31 - 1: no sum past it)
GMM_HD inline int mx_strips(int N) { return (N - 1) / kMxRows + 1; }

// Tiles of `rows` rows in groups of N >= 1, and tile i of them.
GMM_HD inline long long mx_tiles(long long rows, int N, int K) { return rows / N * mx_strips(N) * mx_panels(K); }

GMM_HD inline MxTile mx_tile(int N, int K, long long i) {
  const int all = K / 32, panels = mx_panels(K), strips = mx_strips(N);
  MxTile t;
  const long long s = i / panels;
  t.b0 = (int)(i - s * panels) * kMxPanel;
  t.nb = all - t.b0 < kMxPanel ? all - t.b0 : kMxPanel;
  const long long g = s / strips;
  const int n0 = (int)(s - g * strips) * kMxRows;
  t.rows = N - n0 < kMxRows ? N - n0 : kMxRows;
  t.row0 = g * N + n0;
  t.scales = (g * all + t.b0) * N + n0;
  return t;
}

}  // namespace gmmk
