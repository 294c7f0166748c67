"""The weight tiles of the microscaled fp4 quantiser and widening
(gmm_mx_tiles.hpp) on the CPU: the header is compiled for the host, and over
shapes up to the entry points' limits (Ga * N below 2^31, K below 2^28) every
row and block lies in exactly one tile, at the offsets of [Ga,N,K/32] rows and
[Ga,K/32,1,N] scales."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CXX = shutil.which("g++") or shutil.which("c++")

CHECK = r"""
#include <cstdio>
#include <vector>
#include "gmm_mx_tiles.hpp"
using namespace gmmk;

static bool fits(const MxTile& t, long long Ga, long long N, long long all) {
  const long long g = t.row0 / N, n0 = t.row0 % N;
  return t.rows >= 1 && t.rows <= kMxRows && t.nb >= 1 && t.nb <= kMxPanel && t.b0 >= 0 && t.b0 + t.nb <= all &&
         t.row0 >= 0 && g < Ga && n0 % kMxRows == 0 && n0 + t.rows <= N && t.scales == (g * all + t.b0) * N + n0;
}

// every tile: each (row, block) once
static bool whole(long long Ga, int N, int K) {
  const long long all = K / 32, rows = Ga * N;
  std::vector<unsigned char> seen((size_t)(rows * all));
  for (long long i = 0; i < mx_tiles(rows, N, K); ++i) {
    const MxTile t = mx_tile(N, K, i);
    if (!fits(t, Ga, N, all)) return false;
    for (int r = 0; r < t.rows; ++r)
      for (int b = 0; b < t.nb; ++b)
        if (seen[(size_t)((t.row0 + r) * all + t.b0 + b)]++) return false;
  }
  for (unsigned char c : seen)
    if (c != 1) return false;
  return true;
}

// the largest shapes: the count of tiles, and the first and last ones of a group and of all
static bool edges(long long Ga, int N, int K) {
  const long long all = K / 32, rows = Ga * N;
  const long long strips = ((long long)N + 63) / 64, panels = (all + 127) / 128, tiles = mx_tiles(rows, N, K);
  if (tiles != Ga * strips * panels) return false;
  const long long at[] = {0, 1, panels - 1, panels, strips * panels - 1, strips * panels, tiles / 2, tiles - 2, tiles - 1};
  for (long long i : at) {
    if (i < 0 || i >= tiles) continue;
    const MxTile t = mx_tile(N, K, i);
    if (!fits(t, Ga, N, all)) return false;
    const long long g = i / panels / strips, s = i / panels % strips;
    if (t.row0 != g * N + 64 * s || t.b0 != 128 * (i % panels)) return false;
  }
  return true;
}

#define TRY(F, GA, N, K) \
  if (!F((GA), (N), (K))) { std::printf("%s Ga=%lld N=%d K=%d\n", #F, (long long)(GA), (int)(N), (int)(K)); return 1; }

int main() {
  const int ns[] = {1, 2, 3, 63, 64, 65, 130, 200}, ks[] = {32, 64, 4064, 4096, 4128, 8192, 9600};
  for (int n : ns)
    for (int k : ks) {
      TRY(whole, 1, n, k);
      TRY(whole, 3, n, k);
    }
  const int top = 2147483647, bigk = (1 << 28) - 32;
  for (int d = 0; d < 70; ++d) TRY(edges, 1, top - d, 32);
  TRY(edges, 1, top, 4128);
  TRY(edges, 1, 1 << 30, bigk);
  TRY(edges, 2, (1 << 30) - 1, 96);
  TRY(edges, top, 1, bigk);
  TRY(edges, top / 65, 65, 8224);
  std::printf("ok\n");
  return 0;
}
"""


def test_weight_tiles_cover_every_row_and_block_once(tmp_path):
    if not CXX:
        pytest.skip("no C++ compiler")
    (tmp_path / "c.cpp").write_text(CHECK)
    exe = tmp_path / "c"
    # (a signed overflow ends the program)
    subprocess.run([CXX, "-O1", "-std=c++17", "-Wall", "-Werror", "-ftrapv", "-DGMM_HD=",
                    "-I" + os.path.join(ROOT, "moe_grouped_matrix_amd", "csrc"), str(tmp_path / "c.cpp"), "-o", str(exe)],
                   check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0 and run.stdout == "ok\n", (run.returncode, run.stdout)
