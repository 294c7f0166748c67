// gmm_mxw_rows.hpp -- bf16 lhs x microscaled fp4 weights for few rows per
// group (decode), where the run time is the time to read every active group's
// weight once from HBM.
//
// A workgroup of four waves takes a tile of up to 32 rows x 256 columns of one
// group, each wave 64 of the columns over the whole of K, in steps of 256.
// Weights never pass through LDS: a step's 64 columns x 128 bytes (whole HBM
// lines) go straight into the registers that the matrix instruction reads.
// Lane (q, r) of the 16x16x32 product holds column 4 r + c of block c at K
// elements 32 q + [0, 32) of each half of the step, one 16-byte load.  That is
// one scale block, so a lane needs one scale byte a column, and with columns
// 4 r + c in blocks c = 0..3 its four bytes are one dword.  Which eight K
// elements a lane feeds to product i is free as long as both operands agree:
// 32 q + 8 i + [0, 8).  The lhs rows of a step, which all four waves need, pass
// through a double-buffered LDS stage, loaded a step ahead into registers.  The
// next step's loads (of this tile or the workgroup's next one) are in flight
// while a step is multiplied.  In the result lane (q, r) holds row r and columns
// 16 q + [0, 16).
//
// 2048 rows of 128 experts, 1408 x 1408 (148 MB): 47 us, 3.1 TB/s (39 us with 16
// rows in every group); 16 rows in every one of 128 groups of 4096 x 4096 (1.17
// GB) 4.8 TB/s.  What bounds it: 5 us
// pass before the first weight (launch, group sizes, plan); a bare read of the
// same weights in the same pieces with a barrier a step takes 29 us; the rest is
// the lhs, which every column tile reads again through the same L1, and the
// products, which two waves a SIMD hide in part.  Tried on the way there: waves
// that share out K and read the lhs straight from the L2, 62 us; steps of 128
// (64-byte pieces of a line) 61 us with two to four workgroups a CU; weights two
// or three steps ahead, the lhs two ahead, 512-column tiles of eight waves, no
// gain; 64-row tiles spill (75 us).
#pragma once

#include "gmm_big.hpp"
#include "gmm_mx.hpp"

namespace gmmk {

struct RowsCfg {
  static constexpr int BM = 32, BN = 256, BK = 256, NW = 4, T = 64 * NW;
  static constexpr int A_ROW = BK * 2, STAGE = BM * A_ROW;
};

struct RowsItem {
  int h, row0, rows, n0, ncols;
};

__device__ __forceinline__ RowsItem decode_rows(const Plan& pl, int L, int n_ntiles, int N) {
  RowsItem it;
  const int t = L / n_ntiles, j = L % n_ntiles;
  const int h = find_group(pl, t);
  const int row0 = pl.row_start[h] + (t - pl.tile_start[h]) * RowsCfg::BM;
  const int left = pl.row_start[h + 1] - row0;
  it.h = __builtin_amdgcn_readfirstlane(h);
  it.row0 = __builtin_amdgcn_readfirstlane(row0);
  it.rows = __builtin_amdgcn_readfirstlane(left < RowsCfg::BM ? left : RowsCfg::BM);
  it.n0 = __builtin_amdgcn_readfirstlane(j * RowsCfg::BN);
  it.ncols = N - it.n0 < RowsCfg::BN ? N - it.n0 : RowsCfg::BN;
  return it;
}

struct RowsSrc {
  __amdgpu_buffer_rsrc_t w, s, a;
};

// The wave's 64 columns of the tile (none may be left of a last tile).
__device__ __forceinline__ RowsSrc rows_src(const Params& p, const RowsItem& it, int w) {
  const int K = p.K, N = p.N;
  const int c0 = it.n0 + 64 * w, cols = it.ncols - 64 * w;
  RowsSrc r;
  r.w = uniform_rsrc(reinterpret_cast<const char*>(p.rhs) + ((long long)it.h * N + c0) * (K / 2),
                     cols > 0 ? (cols < 64 ? cols : 64) * (K / 2) : 0);
  r.s = uniform_rsrc(reinterpret_cast<const char*>(p.rhs_scale) + (long long)it.h * p.nb * N + c0,
                     cols > 0 ? p.nb * N - c0 : 0);
  r.a = uniform_rsrc(reinterpret_cast<const char*>(p.lhs) + (long long)it.row0 * K * 2, it.rows * K * 2);
  return r;
}

// One wave's weights of a step: both 128-element halves of the four column
// blocks, and the lane's scale bytes.
struct RowsWeights {
  i32x4 w[2][4];
  int s[2];
};

constexpr int kOutOfRange = (int)0x80000000;

// The range checks look at the lane's own offset only, so everything that can
// leave a row at its end -- K elements past K in a last step, scales of columns
// past the tile's -- gets an offset out of range and reads zeros.
__device__ __forceinline__ void rows_load_w(RowsWeights& f, const RowsSrc& src, int sc, int K, int N, int cols, int q,
                                            int r16) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const bool live = sc * 256 + 128 * h + 32 * q < K && 4 * r16 < cols;
    const int vw = live ? 4 * r16 * (K / 2) + 64 * h + 16 * q : kOutOfRange;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      f.w[h][c] = __builtin_amdgcn_raw_buffer_load_b128(src.w, vw, c * (K / 2) + sc * 128, 0);
    f.s[h] = __builtin_amdgcn_raw_buffer_load_b32(src.s, live ? (4 * h + q) * N + 4 * r16 : kOutOfRange, sc * 8 * N, 0);
  }
}

// Thread t's share of a step's lhs: row t / 8, 16-byte chunks t % 8 + 8 j.
// Chunk c of row r is kept at chunk c ^ (r & 15): sixteen rows read at one
// chunk hit all banks once.
__device__ __forceinline__ void rows_load_a(i32x4 (&a)[4], const RowsSrc& src, int sc, int K, int tid) {
  const int r = tid >> 3, c = tid & 7;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const bool live = sc * 256 + 8 * (c + 8 * j) < K;
    a[j] = __builtin_amdgcn_raw_buffer_load_b128(src.a, live ? r * K * 2 + 16 * (c + 8 * j) : kOutOfRange, sc * 512, 0);
  }
}

__device__ __forceinline__ void rows_store_a(char* st, const i32x4 (&a)[4], int tid) {
  const int r = tid >> 3, c = tid & 7;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<i32x4*>(st + r * RowsCfg::A_ROW + (((c + 8 * j) ^ (r & 15)) << 4)) = a[j];
}

// acc[t][c] += weights (column block c) x lhs rows 16 t + [0, 16).  Where the
// weight reads zeros past K the lhs does too; a column past the tile's has
// weight 0 (and is not stored).
template <int RT>
__device__ __forceinline__ void rows_mma(f32x4 (&acc)[2][4], const RowsWeights& f, const char* st, int q, int r16) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    i32x4 a[RT][4];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        a[t][i] = *reinterpret_cast<const i32x4*>(st + (16 * t + r16) * RowsCfg::A_ROW +
                                                  (((16 * h + 4 * q + i) ^ r16) << 4));
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int byte = (f.s[h] >> (8 * c)) & 255;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bf16x8 w = __builtin_bit_cast(bf16x8, fp4x8_scaled_bf16((unsigned)f.w[h][c][i], byte));
#pragma unroll
        for (int t = 0; t < RT; ++t)
          acc[t][c] =
              __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8, a[t][i]), acc[t][c], 0, 0, 0);
      }
    }
  }
}

template <bool OUT_F32>
__global__ __launch_bounds__(RowsCfg::T, 2) void gmm_mxw_rows_kernel(Params p) {
  using C = RowsCfg;
  __shared__ __attribute__((aligned(16))) char smem[2 * C::STAGE];
  __shared__ Plan pl;
  if (threadIdx.x == 0) pl.flags = 0;
  __syncthreads();
  build_plan<C::T>(p, pl, C::BM);
  report_flags(p, pl);

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int q = lane >> 4, r16 = lane & 15;
  const int M = p.M, N = p.N, K = p.K;
  const int P = gridDim.x, slot = xcd_slot(blockIdx.x, P);  // (of the fill)
  const int n_ntiles = (N + C::BN - 1) / C::BN;
  // Every XCD gets a contiguous eighth of the tiles (they share lhs rows and,
  // in groups of more than one row tile, weights in its L2), which its
  // workgroups take in turn.  Whole rounds over the grid left the last round to
  // some XCDs only: 50 against 39 us for 768 tiles on 512 workgroups.
  const int all_items = __builtin_amdgcn_readfirstlane(pl.n_mtiles) * n_ntiles;
  const int X = P % 8 == 0 ? 8 : 1, x = blockIdx.x % X;
  const int step_items = P / X, n_items = (int)((long long)all_items * (x + 1) / X);
  const int first = (int)((long long)all_items * x / X) + blockIdx.x / X;
  const int NS = (K + C::BK - 1) / C::BK;
  constexpr int es = OUT_F32 ? 4 : 2;

  if (first < n_items) {
    // the current item and the workgroup's next one, found ahead of its turn
    RowsItem it = decode_rows(pl, first, n_ntiles, N), it1 = it;
    RowsSrc src = rows_src(p, it, w), src1 = src;
    int L = first, sc = 0, buf = 0;
    RowsWeights wa{}, wb{};
    i32x4 a[4];
    rows_load_w(wa, src, 0, K, N, it.ncols - 64 * w, q, r16);
    rows_load_a(a, src, 0, K, tid);
    if (first + step_items < n_items) {
      it1 = decode_rows(pl, first + step_items, n_ntiles, N);
      src1 = rows_src(p, it1, w);
    }
    rows_store_a(smem, a, tid);
    f32x4 acc[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[t][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    __syncthreads();

    // One step: returns false after the workgroup's last.
    auto step = [&](const RowsWeights& cur, RowsWeights& nxt) __attribute__((always_inline)) -> bool {
      const bool last = sc + 1 == NS;
      const bool more = !last || L + step_items < n_items;
      const int sc1 = last ? 0 : sc + 1;
      const int row0 = it.row0, rows = it.rows, n0 = it.n0, ncols = it.ncols;
      const long long h = it.h;
      if (last) {
        it = it1;
        src = src1;
      }
      if (more) {
        // the lhs first: it is waited for at this step's end, and loads return
        // in order, so weights asked for before it would be waited for too
        rows_load_a(a, src, sc1, K, tid);
        __builtin_amdgcn_sched_barrier(0);
        rows_load_w(nxt, src, sc1, K, N, it.ncols - 64 * w, q, r16);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (last) {
        L += step_items;
        if (L + step_items < n_items) {
          it1 = decode_rows(pl, L + step_items, n_ntiles, N);
          src1 = rows_src(p, it1, w);
        }
      }
      const char* st = smem + buf * C::STAGE;
      if (rows > 16)
        rows_mma<2>(acc, cur, st, q, r16);
      else
        rows_mma<1>(acc, cur, st, q, r16);
      if (last) {
        // columns 64 w + 16 q + 4 i + c: eight at a time (N is a multiple of 8)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int row = 16 * t + r16;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int col = 64 * w + 16 * q + 8 * u;
            if (row < rows && col < ncols) {
              float v[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = acc[t][e & 3][2 * u + (e >> 2)];
              if (p.rhs_bias) {
                const long long b = h * N + n0 + col;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  v[e] += p.bias_f32 ? reinterpret_cast<const float*>(p.rhs_bias)[b + e]
                                     : bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(p.rhs_bias)[b + e]);
              }
              char* o = reinterpret_cast<char*>(p.out) + ((long long)(row0 + row) * N + n0 + col) * es;
              if constexpr (OUT_F32) {
                reinterpret_cast<f32x4*>(o)[0] = f32x4{v[0], v[1], v[2], v[3]};
                reinterpret_cast<f32x4*>(o)[1] = f32x4{v[4], v[5], v[6], v[7]};
              } else {
                *reinterpret_cast<i32x4*>(o) = i32x4{(int)pk_bf16_rne(v[0], v[1]), (int)pk_bf16_rne(v[2], v[3]),
                                                     (int)pk_bf16_rne(v[4], v[5]), (int)pk_bf16_rne(v[6], v[7])};
              }
            }
          }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[t][c] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
      if (!more) return false;
      buf ^= 1;
      rows_store_a(smem + buf * C::STAGE, a, tid);
      // the stage is written, and nobody reads the other one any more; a bare
      // barrier, so that the weights in flight stay in flight
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      sc = sc1;
      return true;
    };
    while (step(wa, wb) && step(wb, wa)) {
    }
  }

  // rows outside the active groups
  const long long row_bytes = (long long)N * es;
  const int lo_row = pl.row_start[0], hi_row = pl.row_start[pl.ga];
  const long long z1 = fill_rows(p, lo_row) * row_bytes;
  const long long z2b = (long long)hi_row * row_bytes;
  const long long total = z1 + fill_rows(p, M - hi_row) * row_bytes;
  for (long long o = ((long long)slot * C::T + tid) * 16; o < total; o += (long long)P * C::T * 16)
    fill16(p, o < z1 ? o : z2b + (o - z1));
}

}  // namespace gmmk
