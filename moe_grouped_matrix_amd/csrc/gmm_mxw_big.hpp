// gmm_mxw_big.hpp -- bf16 lhs x microscaled fp4 weights for large groups, on
// the tiles, waves and epilogue of the bf16 kernel (gmm_big.hpp): 256 x 256
// output tiles, eight waves of 128 x 64 with 32x32x16 bf16 MFMAs, a persistent
// grid whose operand stream runs on across tiles.
//
// K is consumed 64 at a time.  A stage holds 256 lhs rows of 128 bytes, 256
// weight columns of 32 bytes (the codes as they lie in memory) and the two
// scale rows that cover them; three stages form a ring filled by direct-to-LDS
// loads two steps ahead.  A step is four products of 16 K elements; lane half
// kh takes the elements 32 kh + 8 h + [0, 8) for product h, so its codes of a
// column are one 16-byte chunk with one scale byte, and its lhs elements whole
// 16-byte chunks too.  The codes are widened (with their scale) by each wave
// for its own 64 columns right before their product.
//
// The lhs fragments of two products are held in registers.  Those of products
// 2 and 3 are read while 0 and 1 run, those of the next step's 0 and 1 while 2
// and 3 run, so the wait for the next stage and the barrier stand in the
// middle of a step.
//
// 262144 rows x 1408 x 1408, 128 experts: 0.94-0.96 ms from card to card, 1086 to
// 1106 TFLOP/s (the bf16 kernel on widened weights 0.98-1.03 ms; a library product
// of the dense bf16 shape 1.01-1.06 ms).  The matrix cores are busy 0.62 of the
// cycles at a clock that the power cap holds near 1.8 GHz; no LDS bank conflicts;
// without the widening conversions it would take 0.03 ms less.  What it saves
// against the bf16 kernel is operand stream: 43 KB a 64-element step instead of
// 64.  The few registers that spill are stored once and read at tile boundaries
// only (they would only lengthen a wait: the constant waits count operations that
// must at least be there).
#pragma once

#include "gmm_big.hpp"
#include "gmm_mx.hpp"

namespace gmmk {

template <bool OUT_F32_, bool BIAS_>
struct MxwBigCfg {
  static constexpr bool OUT_F32 = OUT_F32_;
  static constexpr bool BIAS = BIAS_;
  static constexpr int BM = 256, BN = 256;
  static constexpr int WM = 2, WN = 4, NWAVES = WM * WN, T = 64 * NWAVES;
  static constexpr int FM = 4, FN = 2;  // 32 x 32 blocks of a full-tile wave
  static constexpr int BK = 64;
  static constexpr int ROW = BK * 2, W_ROW = BK / 2;  // bytes of an lhs row, of a weight column in a stage
  static constexpr int A_BYTES = BM * ROW, W_BYTES = BN * W_ROW;
  // 256 bytes a wave: the scale rows of waves 0 and 1, the others' stay empty
  static constexpr int S_OFF = A_BYTES + W_BYTES, S_BYTES = 256 * NWAVES;
  static constexpr int STAGE = S_OFF + S_BYTES;
  static constexpr int S = 3;
  static constexpr int RING = S * STAGE;
  static constexpr int BIAS_SLOT = 2048;
  static constexpr int LDS = RING + 2 * BIAS_SLOT;
  // direct-to-LDS operations per wave and step: four of lhs rows, one of codes,
  // one of scales
  static constexpr int OPS = 6;
  static constexpr int es_out = OUT_F32 ? 4 : 2;
  static constexpr int ST_BLOCK = OUT_F32 ? 4 : 2;
  static constexpr int E_FULL = FM * FN * ST_BLOCK, E = E_FULL;
  static_assert(A_BYTES == 4 * 1024 * NWAVES && W_BYTES == 1024 * NWAVES, "load split");
};

// Sources of one tile; zero-size past the end of the stream, so that every
// step issues the same operations.
struct MxwTile {
  __amdgpu_buffer_rsrc_t a, w, s, bias;
  int vs;  // this lane's offset in a scale row, or out of range
};

template <class C>
__device__ __forceinline__ MxwTile mxw_tile(const Params& p, const BigItem& it, bool live, int w, int lane) {
  const int K = p.K, N = p.N;
  MxwTile t;
  t.a = uniform_rsrc(reinterpret_cast<const char*>(p.lhs) + (long long)it.row0 * K * 2, live ? it.rows * K * 2 : 0);
  t.w = uniform_rsrc(reinterpret_cast<const char*>(p.rhs) + ((long long)it.h * N + it.n0) * (K / 2),
                     live ? it.ncols * (K / 2) : 0);
  t.s = uniform_rsrc(reinterpret_cast<const char*>(p.rhs_scale) + (long long)it.h * p.nb * N + it.n0,
                     live ? p.nb * N - it.n0 : 0);
  const int bes = p.bias_f32 ? 4 : 2;
  t.bias = p.rhs_bias ? uniform_rsrc(reinterpret_cast<const char*>(p.rhs_bias) + ((long long)it.h * N + it.n0) * bes,
                                     live ? it.ncols * bes : 0)
                      : uniform_rsrc(reinterpret_cast<const char*>(p.lhs), 0);
  t.vs = w < 2 && 4 * lane < it.ncols ? 4 * lane : (int)0x80000000;
  return t;
}

// This wave's loads of a step: lhs operation i fills rows 32 w + 8 i + lane/8,
// chunk lane%8 (which holds chunk lane%8 ^ swz_w(row) of the row); the code
// operation fills columns 32 w + lane/2, chunk lane%2 (^ bit 3 of the column).
struct MxwOff {
  int a[4], w;
};

__device__ __forceinline__ MxwOff mxw_offsets(int K, int w, int lane) {
  MxwOff o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 32 * w + 8 * i + (lane >> 3);
    o.a[i] = r * K * 2 + (((lane & 7) ^ ((r & 7) ^ ((r >> 3) & 1))) << 4);
  }
  const int n = 32 * w + (lane >> 1);
  o.w = n * (K / 2) + (((lane & 1) ^ ((n >> 3) & 1)) << 4);
  return o;
}

// Operation J of K step k into stage st: 0..3 lhs, 4 codes, 5 scales (waves 0
// and 1: blocks 2 k and 2 k + 1), 6 the wave's piece of the tile's bias row.
template <class C, int J>
__device__ __forceinline__ void mxw_op(const MxwTile& t, const MxwOff& off, int k, int N, char* st, char* bias_slot,
                                       int w, int lane) {
  if constexpr (J < 4) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(t.a, (lds_ptr_t)(st + w * 4096 + J * 1024), 16, off.a[J], k * C::ROW, 0,
                                             0);
  } else if constexpr (J == 4) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(t.w, (lds_ptr_t)(st + C::A_BYTES + w * 1024), 16, off.w, k * C::W_ROW, 0,
                                             0);
  } else if constexpr (J == 5) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(t.s, (lds_ptr_t)(st + C::S_OFF + w * 256), 4, t.vs, (2 * k + (w & 1)) * N,
                                             0, 0);
  } else {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(t.bias, (lds_ptr_t)(bias_slot + w * 256), 4, w * 256 + lane * 4, 0, 0, 0);
  }
}

template <class C>
__global__ __launch_bounds__(C::T) void gmm_mxw_big_kernel(Params p) {
  // one LDS array (a second LDS variable would make the compiler drain the
  // direct-to-LDS loads in flight before every LDS read)
  __shared__ __attribute__((aligned(1024))) char smem[C::LDS + sizeof(Plan)];
  Plan& pl = *reinterpret_cast<Plan*>(smem + C::LDS);
  if (threadIdx.x == 0) pl.flags = 0;
  __syncthreads();
  build_plan<C::T>(p, pl, C::BM);
  report_flags(p, pl);

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kh = lane >> 5, r32 = lane & 31;
  const int M = p.M, N = p.N, K = p.K;
  const int P = gridDim.x;
  const int slot = xcd_slot(blockIdx.x, P);

  // rows outside the active groups: fill them first (grid-stride)
  {
    const long long row_bytes = (long long)N * C::es_out;
    const int lo_row = pl.row_start[0], hi_row = pl.row_start[pl.ga];
    const long long z1 = fill_rows(p, lo_row) * row_bytes;
    const long long z2b = (long long)hi_row * row_bytes;
    const long long total = z1 + fill_rows(p, M - hi_row) * row_bytes;
    for (long long off = ((long long)slot * C::T + tid) * 16; off < total; off += (long long)P * C::T * 16)
      fill16(p, off < z1 ? off : z2b + (off - z1));
  }

  const int n_ntiles = (N + C::BN - 1) / C::BN;
  const int n_items = __builtin_amdgcn_readfirstlane(pl.n_mtiles) * n_ntiles;
  const int KT = K / C::BK;  // steps per tile; the launcher guarantees KT >= 3
  if (slot >= n_items) return;

  BigItem cur = decode_big<C>(pl, slot, n_ntiles, N, w);
  BigItem nxt = cur;
  int L = slot;
  bool last_item = L + P >= n_items;
  if (!last_item) nxt = decode_big<C>(pl, L + P, n_ntiles, N, w);
  MxwTile dcur = mxw_tile<C>(p, cur, true, w, lane), dnxt = mxw_tile<C>(p, nxt, !last_item, w, lane);
  const MxwOff off = mxw_offsets(K, w, lane);
  char* const bias0 = smem + C::RING;

  // the first tile's bias and steps 0 and 1
  mxw_op<C, 6>(dcur, off, 0, N, smem, bias0, w, lane);
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    char* st = smem + s * C::STAGE;
    mxw_op<C, 0>(dcur, off, s, N, st, bias0, w, lane);
    mxw_op<C, 1>(dcur, off, s, N, st, bias0, w, lane);
    mxw_op<C, 2>(dcur, off, s, N, st, bias0, w, lane);
    mxw_op<C, 3>(dcur, off, s, N, st, bias0, w, lane);
    mxw_op<C, 4>(dcur, off, s, N, st, bias0, w, lane);
    mxw_op<C, 5>(dcur, off, s, N, st, bias0, w, lane);
  }
  wait_vmcnt<0>();
  __syncthreads();

  // lane parts of the fragment addresses: fragment rows start at multiples of
  // 32, so the swizzle depends on the lane alone
  const int swz_r = (r32 & 7) ^ ((r32 >> 3) & 1);
  int a_off[4];
#pragma unroll
  for (int h = 0; h < 4; ++h) a_off[h] = r32 * C::ROW + (((4 * kh + h) ^ swz_r) << 4);
  const int w_off = C::A_BYTES + r32 * C::W_ROW + ((kh ^ ((r32 >> 3) & 1)) << 4);
  const int s_off = C::S_OFF + kh * 256 + r32;
  auto a_frag = [&](const char* st, const BigItem& it, int f, int h) __attribute__((always_inline)) {
    return *reinterpret_cast<const i32x4*>(st + (it.rbase + 32 * f) * C::ROW + a_off[h]);
  };
  // the codes of column block f and their scale byte
  i32x4 code[C::FN];
  int byte[C::FN];
  auto read_w = [&](const char* st, const BigItem& it) __attribute__((always_inline)) {
#pragma unroll
    for (int f = 0; f < C::FN; ++f) {
      code[f] = *reinterpret_cast<const i32x4*>(st + (it.cbase + 32 * f) * C::W_ROW + w_off);
      byte[f] = *reinterpret_cast<const uint8_t*>(st + it.cbase + 32 * f + s_off);
    }
  };

  i32x4 a[C::FM][2];  // products 0 and 1, or 2 and 3, of a step
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int f = 0; f < C::FM; ++f) a[f][h] = a_frag(smem, cur, f, h);
  read_w(smem, cur);

  f32x16 acc[C::FM][C::FN];
  int stage = 0, par = 0;

  // One K step.  At its middle the next stage is complete (this wave's loads,
  // then every wave's after the barrier) once at most WAIT newer operations
  // are outstanding: in a tile's first step the previous tile's E stores, else
  // none.  Past the barrier every wave has consumed the previous stage, which
  // takes the loads of the step after the next (this tile's step kd, or the
  // next tile's when NEXT).  In a tile's last step every wave's reads of the
  // current stage are complete at the barrier too: the epilogue stages its
  // output there.
  auto kstep = [&](auto full_tag, auto wait_tag, auto next_tag, auto bias_tag, auto last_tag, int kd)
      __attribute__((always_inline)) {
    constexpr bool FULL = decltype(full_tag)::value;
    constexpr int WAIT = decltype(wait_tag)::value;
    constexpr bool NEXT = decltype(next_tag)::value, BIAS = decltype(bias_tag)::value;
    constexpr bool LAST = decltype(last_tag)::value;
    constexpr int FMA = FULL ? C::FM : C::FM / 2;
    constexpr int NM = 2 * FMA * C::FN;  // products of the half step that issues the loads
    constexpr int NOPS = C::OPS + (BIAS ? 1 : 0);
    const int s1 = stage == C::S - 1 ? 0 : stage + 1, s2 = stage == 0 ? C::S - 1 : stage - 1;
    const char* const st = smem + stage * C::STAGE;
    const char* const st1 = smem + s1 * C::STAGE;
    char* const st2 = smem + s2 * C::STAGE;
    char* const bslot = bias0 + (par ^ 1) * C::BIAS_SLOT;
    const MxwTile& d = NEXT ? dnxt : dcur;
    const BigItem& it1 = LAST ? nxt : cur;
    auto op = [&](int m) __attribute__((always_inline)) {
      // with the bias piece it goes first (older than the operands)
      if constexpr (BIAS) {
        if (m == 0 * NM / NOPS) mxw_op<C, 6>(d, off, kd, N, st2, bslot, w, lane);
      }
      constexpr int B0 = BIAS ? 1 : 0;
      if (m == (B0 + 0) * NM / NOPS) mxw_op<C, 0>(d, off, kd, N, st2, bslot, w, lane);
      if (m == (B0 + 1) * NM / NOPS) mxw_op<C, 1>(d, off, kd, N, st2, bslot, w, lane);
      if (m == (B0 + 2) * NM / NOPS) mxw_op<C, 2>(d, off, kd, N, st2, bslot, w, lane);
      if (m == (B0 + 3) * NM / NOPS) mxw_op<C, 3>(d, off, kd, N, st2, bslot, w, lane);
      if (m == (B0 + 4) * NM / NOPS) mxw_op<C, 4>(d, off, kd, N, st2, bslot, w, lane);
      if (m == (B0 + 5) * NM / NOPS) mxw_op<C, 5>(d, off, kd, N, st2, bslot, w, lane);
    };
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      if (h == 2) {
        wait_vmcnt<WAIT>();
        if constexpr (LAST) __builtin_amdgcn_s_waitcnt(0xF | (0x7 << 4) | (0x0 << 8) | (0x3 << 14));
        ring_barrier();
      }
      i32x4 b[C::FN];
#pragma unroll
      for (int fn = 0; fn < C::FN; ++fn) b[fn] = fp4x8_scaled_bf16((unsigned)code[fn][h], byte[fn]);
      if (h == 3) read_w(st1, it1);
#pragma unroll
      for (int fm = 0; fm < FMA; ++fm) {
#pragma unroll
        for (int fn = 0; fn < C::FN; ++fn) {
          acc[fm][fn] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, b[fn]),
                                                                __builtin_bit_cast(bf16x8, a[fm][h & 1]),
                                                                acc[fm][fn], 0, 0, 0);
          if (h >= 2) op(((h - 2) * FMA + fm) * C::FN + fn);
          __builtin_amdgcn_sched_barrier(0);  // keep this order
        }
        a[fm][h & 1] = h < 2 ? a_frag(st, cur, fm, h + 2) : a_frag(st1, it1, fm, h - 2);
      }
      if (h >= 2) {
#pragma unroll
        for (int fm = FMA; fm < C::FM; ++fm) a[fm][h & 1] = a_frag(st1, it1, fm, h - 2);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    stage = s1;
  };
  using T_ = std::true_type;
  using F_ = std::false_type;
  using WE = std::integral_constant<int, C::E>;
  using W0 = std::integral_constant<int, 0>;
  auto ktile = [&](auto full_tag) __attribute__((always_inline)) {
    constexpr bool FULL = decltype(full_tag)::value;
    constexpr int FMA = FULL ? C::FM : C::FM / 2;
    kstep(full_tag, WE{}, F_{}, F_{}, F_{}, 2);
    for (int kt = 1; kt + 2 < KT; ++kt) kstep(full_tag, W0{}, F_{}, F_{}, F_{}, kt + 2);
    kstep(full_tag, W0{}, T_{}, T_{}, F_{}, 0);  // the next tile's step 0 and bias row
    kstep(full_tag, W0{}, T_{}, F_{}, T_{}, 1);
    // the last step's stage (free, see above) holds the staging slices
    const int last = stage == 0 ? C::S - 1 : stage - 1;
    big_epilogue<C, FMA, C::BIAS>(p, acc, cur, bias0 + par * C::BIAS_SLOT, smem + last * C::STAGE + w * 4096, kh, r32,
                                  lane);
  };

  while (true) {
#pragma unroll
    for (int x = 0; x < C::FM; ++x)
#pragma unroll
      for (int y = 0; y < C::FN; ++y)
#pragma unroll
        for (int z = 0; z < 16; ++z) acc[x][y][z] = 0.f;
    if (!cur.half)
      ktile(std::true_type{});
    else
      ktile(std::false_type{});
    if (last_item) break;
    L += P;
    last_item = L + P >= n_items;
    cur = nxt;
    dcur = dnxt;
    par ^= 1;
    if (!last_item) nxt = decode_big<C>(pl, L + P, n_ntiles, N, w);
    dnxt = mxw_tile<C>(p, nxt, !last_item, w, lane);
  }
}

}  // namespace gmmk
