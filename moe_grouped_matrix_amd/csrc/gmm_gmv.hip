// gmm_gmv.hip -- products of a few tokens with their experts' four-bit
// weights, by expert id (gmm_layer.h, gmm_gmv_run).
//
// What bounds it is reading every touched expert's weight once -- for few rows an
// expert: every sixteen rows are another pass over it, each with its loads and
// conversions.  Sort, dispatch and the grouped product overtake it at some 16 rows
// an expert (128 experts, top-8, 1408 x 1408 int4: 1024 slots 48 against 62 us, 2048
// 74 and 77, 4096 138 and 79), with one expert of 8192 x 4096 at some 80 rows (64: 39.5
// against 51, 128: 75 and 51).  A workgroup
// takes 16 NT columns of one expert and all slots that chose it (up to 16 at a
// time); its four waves share out K in contiguous chunks of 128 and join their
// sums in LDS, so nothing is read by two waves and nothing waits for a barrier on
// the way.  Which slots chose an expert every workgroup finds out by itself from
// the ids.
//
// 8 experts of 1408 x 1408 int4 for one token (8.4 MB): 4.9 us on the GPU; 32
// tokens, top-8 of 128 (75 experts touched, 79 MB): 25-27 us, 3.1 TB/s; 64 experts
// with a row each (67 MB) 17 us, 3.9 TB/s; dense 8192 x 4096 fp4 for four tokens
// 7.3 us.  What is left: ids, weights and join follow one another in a workgroup
// that reads 22 KB a tile, so that five workgroups a CU are needed to keep HBM
// busy, and popular experts take x of 16 rows with every tile.  Tried: x of a
// wave's chunks kept in registers and tiles taken in turn behind a bare barrier
// (34-36 us for the 32 tokens: one tile ahead is too little in flight), two blocks
// an operand for up to eight rows (no gain), three chunks ahead (42 us: registers;
// as it is, 32 columns with zero points spill four),
// eight waves a workgroup (42 us), weights loaded past the caches (47 against 39
// us: a load takes half a line of each row).  Loads that wait for one another cost
// most on the way: ids, scales and zero points are loaded as bits, without
// branches, and converted when they are used (the same work with a conversion or
// a branch behind a load: 32 against 29.5 us, and 30 against 21 for blocks of 32
// with zero points).
//
// The products run on the matrix cores, x rows as the first operand of the
// 16x16x32 product and weights as the second: that leaves the vector units
// nothing but widening the codes, and up to 16 rows cost what one does.  A
// lane (q, n) loads 16 bytes, 32 codes of column n's block q of the chunk; a
// 4 x 4 exchange between the four lanes of a column (two swaps of halves and
// two of quarters, in registers) then makes each register a block of 32, so
// that a product covers one block and its scale and zero point meet the sum:
//   tot += scale * (sum of code * x  -  zero * sum of x),
// sum of x by a product with ones.  Codes of int4 and uint4 are bytes 0..15,
// which the e4m3 format reads as code * 2^-9: its conversion to bf16, scaled by
// 2^9, widens them exactly, two an instruction (int4 with its sign bit turned,
// that is 8 more, and a zero point 8 higher).  fp4 codes have a conversion of
// their own, which takes an E8M0 scale along (exact, no fold).
//
// The sums that are rounded are thus of (code + 8) x and of 8 x for int4: an error
// goes by (|code| + 16) |x|, not by |code| |x|.  int4 as sign and magnitude, worked
// out for a register's eight codes at once, has no such term and needs no sums of x,
// but five instructions more for eight codes: 12.6 against 12.0 us (8 tokens, top-8 of 128,
// 1408 x 1408), 27.8 against 27.3 (32 tokens), 8.5 against 8.0 (one token, weighted),
// and in blocks of 32 with zero points 15.8 against 14.1 and 35.5 against 32.6.
//
// With up to four rows (FEW) one load and one operand bring a chunk's x: row
// 4 r + j of the operand is row r's block j.  The product with block i's
// weights then has the wanted sum in row 4 r + i, which is register i of lane
// group r; the other rows are blocks that do not belong together, and are left
// alone.  One product with ones gives the sums of x of all four blocks.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gmm_layer_launch.hpp"
#include "gmm_mx.hpp"

namespace gmmk {

namespace {

constexpr int kWaves = 4;  // of a workgroup
constexpr int kDepth = 2;  // chunks of a wave in flight
constexpr int kManyX = 1;  // and of x with more than four rows

// The id of a slot, as it was loaded (a 64-bit one in two halves), and the
// expert that it names, -1 for none.
struct SlotId {
  unsigned lo, hi;
};
__device__ __forceinline__ SlotId load_id(const GmvParams& p, int i) {
  const unsigned* const w = static_cast<const unsigned*>(p.ids) + ((long long)i << p.ids64);
  return {w[0], w[p.ids64]};
}
__device__ __forceinline__ int expert_of(const GmvParams& p, SlotId id) {
  return id.lo < (unsigned)p.G && (!p.ids64 || id.hi == 0) ? (int)id.lo : -1;
}
__device__ __forceinline__ int slot_expert(const GmvParams& p, int i) { return p.ids ? expert_of(p, load_id(p, i)) : 0; }
__device__ __forceinline__ float slot_weight(const GmvParams& p, int i) {
  return p.w_f32 ? static_cast<const float*>(p.weights)[i] : bf16_bits_to_f32(static_cast<const uint16_t*>(p.weights)[i]);
}

__device__ __forceinline__ void store_out(const GmvParams& p, long long o, float v) {
  if (p.out_f32)
    static_cast<float*>(p.out)[o] = v;
  else
    static_cast<uint16_t*>(p.out)[o] = f32_to_bf16_rne(v);
}

// How codes become operands, and how scales meet them.
enum Kind : int {
  kInt,    // int4, uint4: a scale per block of a multiple of 32
  kZero,   // the same with zero points
  kFp4,    // fp4 with such scales
  kMicro,  // fp4 with E8M0 scales of blocks of 32
};
constexpr bool integer(Kind k) { return k == kInt || k == kZero; }

// A scale or zero point as it was loaded: f32 bits, bf16 bits, or an E8M0 byte.
// What is loaded is left alone until it is used, and types are the kernel's, not
// the loads', so that no load waits for another.
template <class S>
__device__ __forceinline__ int as_f32(int bits) {
  return sizeof(S) == 2 ? bits << 16 : bits;
}

// Eight codes as bf16, in the order of ordered_x.
template <Kind KIND>
__device__ __forceinline__ bf16x8 widen8(unsigned w, int byte) {
  i32x4 r;
  if constexpr (integer(KIND)) {
    const unsigned even = w & 0x0F0F0F0Fu, odd = (w >> 4) & 0x0F0F0F0Fu;
    r[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(even, 512.f, false));
    r[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(even, 512.f, true));
    r[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(odd, 512.f, false));
    r[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(odd, 512.f, true));
  } else {
    r = fp4x8_scaled_bf16(w, KIND == kMicro ? byte : 127);
  }
  return __builtin_bit_cast(bf16x8, r);
}

// Eight x values in the order in which widen8 gives the codes: elements 0 2 4 6
// 1 3 5 7 for int4 and uint4.
template <Kind KIND>
__device__ __forceinline__ bf16x8 ordered_x(i32x4 x) {
  if constexpr (!integer(KIND)) return __builtin_bit_cast(bf16x8, x);
  const i32x4 r{(int)__builtin_amdgcn_perm(x[1], x[0], 0x05040100), (int)__builtin_amdgcn_perm(x[3], x[2], 0x05040100),
                (int)__builtin_amdgcn_perm(x[1], x[0], 0x07060302), (int)__builtin_amdgcn_perm(x[3], x[2], 0x07060302)};
  return __builtin_bit_cast(bf16x8, r);
}

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void swap_halves(int& a, int& b) {  // lanes 32-63 of a with 0-31 of b
  const u32x2 r = __builtin_amdgcn_permlane32_swap((unsigned)a, (unsigned)b, false, false);
  a = (int)r[0];
  b = (int)r[1];
}
__device__ __forceinline__ void swap_rows(int& a, int& b) {  // rows 1 and 3 of a with rows 0 and 2 of b
  const u32x2 r = __builtin_amdgcn_permlane16_swap((unsigned)a, (unsigned)b, false, false);
  a = (int)r[0];
  b = (int)r[1];
}
// Register i of lane (q, n) and register q of lane (i, n) change places.
__device__ __forceinline__ void transpose4(i32x4& d) {
  int a = d[0], b = d[1], c = d[2], e = d[3];
  swap_halves(a, c);
  swap_halves(b, e);
  swap_rows(a, b);
  swap_rows(c, e);
  d = i32x4{a, b, c, e};
}
// out[i] = lane (i, n)'s v, in every lane of column n.
__device__ __forceinline__ i32x4 spread4(int v) {
  int a = v, c = v;
  swap_halves(a, c);
  int b = a, e = c;
  swap_rows(a, b);
  swap_rows(c, e);
  return i32x4{a, b, c, e};
}

// A lane's share of one chunk of 128 elements of K of its column: the codes of
// its own block of 32, and that block's scale and zero point.
struct Weights {
  i32x4 w;
  int s, z;
};

// Where a wave reads one expert's column: the lane's row of codes, and the index
// of its column's first scale.
struct Column {
  const uint8_t* w;
  long long scale;
};

__device__ __forceinline__ Column column_of(const GmvParams& p, int expert, int col) {
  const int c = col < p.N ? col : p.N - 1;  // (past the last: read, and not stored)
  return {p.rhs + ((long long)expert * p.N + c) * (p.K / 2), (long long)expert * p.nb * p.N + c};
}

template <Kind KIND, class S>
__device__ __forceinline__ void load_weights(Weights& d, const GmvParams& p, const Column& src, int c, int q) {
  const int k0 = 128 * c, mine = k0 + 32 * q < p.K ? k0 + 32 * q : k0;  // (past K: read elsewhere, and not used)
  d.w = *reinterpret_cast<const i32x4*>(src.w + mine / 2);
  const int b = KIND == kMicro ? mine >> 5 : (int)(((unsigned long long)((unsigned)mine >> 5) * p.blk_magic) >> 31);
  const long long i = src.scale + (long long)b * p.N;
  d.s = static_cast<int>(static_cast<const S*>(p.scale)[i]);
  if constexpr (KIND == kZero) d.z = static_cast<int>(static_cast<const S*>(p.zero)[i]);
}

// The x operands of one chunk: of its four blocks, or (FEW) of all at once.
template <bool FEW>
struct Rows {
  i32x4 x[FEW ? 1 : 4];
};

template <bool FEW>
__device__ __forceinline__ void load_rows(Rows<FEW>& d, const GmvParams& p, const uint16_t* x, int c, int q) {
  const int k0 = 128 * c;
  if constexpr (FEW) {
    const int i = threadIdx.x & 3, k = k0 + 32 * i < p.K ? k0 + 32 * i : k0;
    d.x[0] = *reinterpret_cast<const i32x4*>(x + k + 8 * q);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = k0 + 32 * i < p.K ? k0 + 32 * i : k0;
      d.x[i] = *reinterpret_cast<const i32x4*>(x + k + 8 * q);
    }
  }
}

__device__ __forceinline__ bf16x8 ones() {
  const i32x4 one4{0x3F803F80, 0x3F803F80, 0x3F803F80, 0x3F803F80};
  return __builtin_bit_cast(bf16x8, one4);
}

// The wave's sums: tot[r] of lane (q, n) for column n of the tile and row q (FEW)
// or 4 q + r.  fp4 with E8M0 scales needs no folds, and sums in the matrix
// cores' results, run (FEW: one for each block of a chunk).
template <bool FEW>
struct Sums {
  float tot[FEW ? 1 : 4];
  f32x4 run[FEW ? 4 : 1];
};

template <bool FEW>
__device__ __forceinline__ void clear(Sums<FEW>& a) {
#pragma unroll
  for (float& v : a.tot) v = 0.f;
#pragma unroll
  for (f32x4& v : a.run) v = f32x4{0.f, 0.f, 0.f, 0.f};
}

// Adds the products of chunk c, the rows being in order (ordered_x).  WHOLE: its
// four blocks share their scale (scale blocks are multiples of 128).  WEIGHTED:
// times `weight`.
template <Kind KIND, class S, bool WHOLE, bool WEIGHTED, bool FEW>
__device__ __forceinline__ void use_chunk(Sums<FEW>& a, Weights d, const Rows<FEW>& rows, const GmvParams& p, int c,
                                          float weight) {
  const int left = (p.K >> 5) - 4 * c;  // blocks from here on
  const f32x4 none{0.f, 0.f, 0.f, 0.f};
  const bool int4 = integer(KIND) && p.fmt == 3;
  const float base = int4 ? 8.f : 0.f;
  constexpr bool CHAIN = KIND == kMicro && !WEIGHTED, TOGETHER = WHOLE || KIND == kMicro;
  i32x4 s4, z4;
  if constexpr (integer(KIND)) d.w ^= int4 ? (int)0x88888888u : 0;
  transpose4(d.w);
  if constexpr (KIND == kMicro || !WHOLE) {
    s4 = spread4(d.s);
    if constexpr (KIND == kZero) z4 = spread4(d.z);
  }
  // sums of products `got` and of x `sum`, for row r
  auto fold = [&](int r, float got, float sum, int scale, int zero) __attribute__((always_inline)) {
    float s = KIND == kMicro ? 1.f : __int_as_float(as_f32<S>(scale));
    if constexpr (WEIGHTED) s *= weight;
    if constexpr (integer(KIND))
      got = __builtin_fmaf(-(KIND == kZero ? __int_as_float(as_f32<S>(zero)) + base : base), sum, got);
    a.tot[r] = __builtin_fmaf(s, got, a.tot[r]);
  };
  f32x4 acc = none, sum = none;
  float few = 0.f, few_sum = 0.f;
  bf16x8 x = __builtin_bit_cast(bf16x8, rows.x[0]);
  if constexpr (FEW && integer(KIND)) sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, ones(), none, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i >= left) break;
    if constexpr (!FEW) {
      if (i > 0) x = __builtin_bit_cast(bf16x8, rows.x[i]);
      if constexpr (integer(KIND)) sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, ones(), WHOLE ? sum : none, 0, 0, 0);
    }
    const bf16x8 w = widen8<KIND>((unsigned)d.w[i], KIND == kMicro ? s4[i] : 0);
    if constexpr (CHAIN) {
      f32x4& run = a.run[FEW ? i : 0];
      run = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, w, run, 0, 0, 0);
      continue;
    }
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, w, TOGETHER && !FEW ? acc : none, 0, 0, 0);
    if constexpr (!TOGETHER) {
      if constexpr (FEW) {
        fold(0, acc[i], sum[i], s4[i], z4[i]);
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) fold(r, acc[r], sum[r], s4[i], z4[i]);
      }
    } else if constexpr (FEW) {
      few += acc[i];
      few_sum += sum[i];
    }
  }
  if constexpr (!CHAIN && TOGETHER) {
    if constexpr (FEW) {
      fold(0, few, few_sum, d.s, d.z);
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r) fold(r, acc[r], sum[r], d.s, d.z);
    }
  }
}

// What the sums came to.
template <Kind KIND, bool WEIGHTED, bool FEW>
__device__ __forceinline__ float total(const Sums<FEW>& a, int r) {
  if constexpr (KIND != kMicro || WEIGHTED) return a.tot[r];
  if constexpr (FEW) return (a.run[0][0] + a.run[1][1]) + (a.run[2][2] + a.run[3][3]);
  return a.run[0][r];
}

// The slots of the r-th expert that any slot chose: into list, in their order;
// returns how many, and the expert (-1: fewer than r + 1 were chosen).  In which
// order the experts are counted does not matter, but that of the slots does: the
// place in the list decides whether a slot's row is one of up to four (FEW) or of
// sixteen, which add in different orders.  Up to 64 slots each wave looks for
// itself: equal ids find each other by a ballot per bit of the id, and an expert's
// first slot stands for it.
struct Found {
  int expert, count;
};

// (without ids every slot has expert 0)
__device__ __forceinline__ Found find_all(const GmvParams& p, uint16_t* list) {
  for (int i = threadIdx.x & 63; i < p.n; i += 64) list[i] = (uint16_t)i;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  return {0, p.n};
}

__device__ __forceinline__ Found find_few(const GmvParams& p, int r, uint16_t* list) {
  const int lane = threadIdx.x & 63;
  const int id = lane < p.n ? slot_expert(p, lane) : -1;
  const unsigned long long live = __ballot(id >= 0);
  unsigned long long peers = live;
  const int bits = 32 - __builtin_clz(p.G);
  for (int b = 0; b < bits; ++b) {
    const bool bit = (id >> b) & 1;
    const unsigned long long m = __ballot(bit);
    peers &= bit ? m : ~m;
  }
  const unsigned long long below = (1ull << lane) - 1;
  const unsigned long long firsts = __ballot(id >= 0 && (peers & below) == 0);
  if (r >= __builtin_popcountll(firsts)) return {-1, 0};
  // the lane that is the r-th first one
  const unsigned long long at = __ballot(((firsts >> lane) & 1) && __builtin_popcountll(firsts & below) == r);
  const int g = __builtin_amdgcn_readlane(id, __builtin_ctzll(at));
  const unsigned long long mine = __ballot(id == g);
  if (id == g) list[__builtin_popcountll(mine & below)] = (uint16_t)lane;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  return {g, (int)__builtin_popcountll(mine)};
}

// The slots of expert g; every wave looks through all ids for itself (and
// writes the same list), eight of them a lane at a time.
__device__ __forceinline__ Found find_slots(const GmvParams& p, int g, uint16_t* list) {
  const int lane = threadIdx.x & 63;
  const unsigned long long below = (1ull << lane) - 1;
  int count = 0;
  for (int i0 = 0; i0 < p.n; i0 += 512) {
    SlotId id[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = i0 + 64 * u + lane;
      id[u] = load_id(p, i < p.n ? i : p.n - 1);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = i0 + 64 * u + lane;
      const bool hit = i < p.n && expert_of(p, id[u]) == g;
      const unsigned long long mine = __ballot(hit);
      if (hit) list[count + __builtin_popcountll(mine & below)] = (uint16_t)i;
      count += __builtin_popcountll(mine);
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  return {count ? g : -1, count};
}

// (fewer slots than half the experts; their experts are kept, so that the ids are
// asked for once)
__device__ __forceinline__ Found find_many(const GmvParams& p, int r, uint16_t* list) {
  __shared__ uint8_t chosen[kMaxGroups];
  __shared__ int16_t experts[kMaxGroups / 2];
  __shared__ int wave_tot[16];
  __shared__ int expert;
  constexpr int T = 64 * kWaves, per = kMaxGroups / T;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  for (int g = tid; g < kMaxGroups; g += T) chosen[g] = 0;
  if (tid == 0) expert = -1;
  __syncthreads();
  for (int i = tid; i < p.n; i += T) {
    const int g = slot_expert(p, i);
    experts[i] = (int16_t)g;
    if (g >= 0) chosen[g] = 1;
  }
  __syncthreads();
  int mine = 0;
  for (int j = 0; j < per; ++j)
    mine += chosen[tid * per + j];
  int incl = mine;
#pragma unroll
  for (int s = 1; s < 64; s *= 2) {
    const int o = __shfl_up(incl, s, 64);
    if (lane >= s) incl += o;
  }
  if (lane == 63) wave_tot[w] = incl;
  __syncthreads();
  int at = incl - mine;
  for (int i = 0; i < w; ++i) at += wave_tot[i];
  if (at <= r && r < at + mine) {
    int g = tid * per;
    for (int left = r - at;; ++g)
      if (chosen[g] && left-- == 0) break;
    expert = g;
  }
  __syncthreads();
  const int g = expert;
  if (g < 0) return {-1, 0};
  const unsigned long long below = (1ull << lane) - 1;
  int count = 0;
  for (int i0 = 0; i0 < p.n; i0 += 64) {  // (every wave writes the same list)
    const bool hit = i0 + lane < p.n && experts[i0 + lane] == g;
    const unsigned long long here = __ballot(hit);
    if (hit) list[count + __builtin_popcountll(here & below)] = (uint16_t)(i0 + lane);
    count += __builtin_popcountll(here);
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  return {g, count};
}

// The join: every wave's sums go to LDS, join[wave][row][column], and all threads
// add them up, in the waves' order, and store.
template <Kind KIND, bool FEW, int NT>
__device__ __forceinline__ void join_tiles(const GmvParams& p, const Sums<FEW> (&sums)[NT], float* join, const uint16_t* list,
                                           int rows, int n0) {
  constexpr int ROWS = FEW ? 4 : 16, COLS = 16 * NT;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, q = lane >> 4, n = lane & 15;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < ROWS / 4; ++r)
      join[(w * ROWS + (FEW ? q : 4 * q + r)) * COLS + 16 * t + n] = total<KIND, false>(sums[t], r);
  __syncthreads();
  for (int i = threadIdx.x; i < rows * COLS; i += 64 * kWaves) {
    const int col = n0 + i % COLS;
    float v = 0.f;
#pragma unroll
    for (int j = 0; j < kWaves; ++j) v += join[j * ROWS * COLS + i];
    if (col < p.N) {
      const long long o = (long long)list[i / COLS] * p.N + col;
      if (p.weights)
        p.work[o] = v;
      else
        store_out(p, o, v);
    }
  }
}

// One pass over the workgroup's columns, NT tiles of 16, for the rows of list (up
// to four: FEW, or 16).  The waves share out K in contiguous runs of chunks; a wave
// has D chunks of codes, scales and x in flight.
template <Kind KIND, class S, bool WHOLE, bool FEW, int NT>
__device__ __forceinline__ void pass(const GmvParams& p, int expert, const uint16_t* list, int rows, int n0, float* join) {
  constexpr int D = kDepth, DX = FEW ? kDepth : kManyX;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, n = lane & 15;
  const int chunks = (p.K + 127) >> 7, lo = chunks * w / kWaves, hi = chunks * (w + 1) / kWaves;
  Column src[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) src[t] = column_of(p, expert, n0 + 16 * t + n);
  const int row = FEW ? n >> 2 : n;
  const int slot = list[row < rows ? row : 0];
  const uint16_t* const x = p.x + (long long)(p.per_slot ? slot : slot / p.k) * p.K;
  Weights d[D][NT];
  Rows<FEW> xs[DX];
  auto load = [&](int i, int c) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < NT; ++t) load_weights<KIND, S>(d[i][t], p, src[t], c, q);
  };
  Sums<FEW> sums[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) clear(sums[t]);
  const int last = hi - 1;
  if (lo < hi) {
#pragma unroll
    for (int i = 0; i < D; ++i) load(i, lo + i < hi ? lo + i : last);
#pragma unroll
    for (int i = 0; i < DX; ++i) load_rows(xs[i], p, x, lo + i < hi ? lo + i : last, q);
    for (int c = lo; c < hi; c += D) {
#pragma unroll
      for (int i = 0; i < D; ++i)
        if (c + i < hi) {
          Rows<FEW>& xi = xs[i % DX];
          for (i32x4& v : xi.x) v = __builtin_bit_cast(i32x4, ordered_x<KIND>(v));
#pragma unroll
          for (int t = 0; t < NT; ++t) use_chunk<KIND, S, WHOLE, false>(sums[t], d[i][t], xi, p, c + i, 1.f);
          if (c + i + DX < hi) load_rows(xi, p, x, c + i + DX, q);
          if (c + i + D < hi) load(i, c + i + D);
        }
    }
  }
  join_tiles<KIND, FEW, NT>(p, sums, join, list, rows, n0);
}

template <Kind KIND, class S, bool WHOLE, int NT>
__global__ __launch_bounds__(64 * kWaves, 5) void gmv_kernel(GmvParams p) {
  __shared__ float join[kWaves * 16 * 16 * NT];
  extern __shared__ uint16_t list[];  // [n]
  const int n0 = blockIdx.x * 16 * NT;
  if ((int)blockIdx.y == p.experts) {  // slots without an expert: zeros
    const int lane = threadIdx.x & 63;
    for (int i0 = 64 * (threadIdx.x >> 6); p.ids && i0 < p.n; i0 += 64 * kWaves) {
      const SlotId id = load_id(p, i0 + lane < p.n ? i0 + lane : p.n - 1);
      unsigned long long none = __ballot(i0 + lane < p.n && expert_of(p, id) < 0);
      for (; none; none &= none - 1) {
        const long long slot = i0 + __builtin_ctzll(none);
        if (lane < 16 * NT && n0 + lane < p.N) store_out(p, slot * p.N + n0 + lane, 0.f);
      }
    }
    return;
  }
  const Found f = !p.ids ? find_all(p, list)
                  : p.n <= 64 ? find_few(p, blockIdx.y, list)
                  : p.experts == p.G ? find_slots(p, blockIdx.y, list)
                                     : find_many(p, blockIdx.y, list);
  if (f.expert < 0) return;
  for (int first = 0; first < f.count; first += 16) {
    const int rows = f.count - first < 16 ? f.count - first : 16;
    if (first > 0) __syncthreads();  // (the join's buffer is free again)
    if (rows <= 4)
      pass<KIND, S, WHOLE, true, NT>(p, f.expert, list + first, rows, n0, join);
    else
      pass<KIND, S, WHOLE, false, NT>(p, f.expert, list + first, rows, n0, join);
  }
}

// A token's weighted sum over its slots, at once: a workgroup takes 16 columns
// of one token, its 16 waves share out the chunks of all its slots.  For a few
// tokens, whose experts are mostly different ones, this saves the second
// launch (top-8, 1408 x 704 uint4 in blocks of 32: one token 6.1 against 8.7 us, two
// 6.8 and 10, four 12.5 and 12; 1408 x 1408 int4: 8.0 and 9.3, 8.6 and 12, 17 and
// 13.8: hence up to 16 slots).  88 workgroups for 1408 columns is what bounds it;
// with eight or four columns each they take 6.4 and 10.8 us.
template <Kind KIND, class S, bool WHOLE>
__global__ __launch_bounds__(1024) void gmv_token_kernel(GmvParams p) {
  constexpr int W = 16;
  __shared__ int order[64];
  __shared__ float join[W][16];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), q = lane >> 4, n = lane & 15;
  const int n0 = blockIdx.x * 16, t = blockIdx.y;
  // lane j takes slot j, then lane i the i-th slot that has an expert (every wave
  // writes the same list for itself)
  const int own = t * p.k + (lane < p.k ? lane : 0);
  const float own_weight = slot_weight(p, own);
  const int own_id = lane < p.k ? slot_expert(p, own) : -1;
  const unsigned long long live = __ballot(own_id >= 0);
  if (own_id >= 0) order[__builtin_popcountll(live & ((1ull << lane) - 1))] = lane;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  const int count = __builtin_popcountll(live), from = lane < count ? order[lane] : 0;
  const int id = __shfl(own_id, from, 64), slot = t * p.k + from;
  const float scale = __shfl(own_weight, from, 64);
  const int chunks = (p.K + 127) >> 7, all = count * chunks;
  const int lo = (int)((long long)all * w / W), hi = (int)((long long)all * (w + 1) / W);
  Sums<true> sums;
  clear(sums);
  constexpr int D = 3;
  Weights d[D];
  Rows<true> xs[D];
  float weight[D];
  int at[D];  // the chunks
  int slot_at = lo / chunks, chunk_at = lo - slot_at * chunks;  // of the next load
  auto load = [&](int i) __attribute__((always_inline)) {
    const int j = __builtin_amdgcn_readfirstlane(slot_at), c = __builtin_amdgcn_readfirstlane(chunk_at);
    weight[i] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(scale), j));
    at[i] = c;
    load_weights<KIND, S>(d[i], p, column_of(p, __builtin_amdgcn_readlane(id, j), n0 + n), c, q);
    load_rows(xs[i], p, p.x + (long long)(p.per_slot ? __builtin_amdgcn_readlane(slot, j) : t) * p.K, c, q);
    if (++chunk_at == chunks) {
      chunk_at = 0;
      ++slot_at;
    }
  };
#pragma unroll
  for (int i = 0; i < D; ++i)
    if (lo + i < hi) load(i);
  for (int c = lo; c < hi; c += D) {
#pragma unroll
    for (int i = 0; i < D; ++i)
      if (c + i < hi) {
        xs[i].x[0] = __builtin_bit_cast(i32x4, ordered_x<KIND>(xs[i].x[0]));
        use_chunk<KIND, S, WHOLE, true>(sums, d[i], xs[i], p, at[i], weight[i]);
        if (c + i + D < hi) load(i);
      }
  }
  if (q == 0) join[w][n] = total<KIND, true>(sums, 0);
  __syncthreads();
  if (threadIdx.x < 16 && n0 + n < p.N) {
    float v = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) v += join[j][n];
    store_out(p, (long long)t * p.N + n0 + n, v);
  }
}

// out[t] = sum over its routed slots of weight * row.
__global__ __launch_bounds__(256) void gmv_join_kernel(GmvParams p) {
  const int n = blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
  if (n >= p.N) return;
  float sum = 0.f;
  for (int j = 0; j < p.k; ++j) {
    const int i = t * p.k + j;
    if (slot_expert(p, i) < 0) continue;
    sum = __builtin_fmaf(slot_weight(p, i), p.work[(long long)i * p.N + n], sum);
  }
  store_out(p, (long long)t * p.N + n, sum);
}

template <Kind KIND, class S, bool WHOLE>
hipError_t launch(const GmvParams& p, int cu_count, hipStream_t s) {
  const int all = (p.N + 15) / 16;
  if (p.at_once) return queue(gmv_token_kernel<KIND, S, WHOLE>, dim3(all, p.T), dim3(1024), 0, s, p);
  const unsigned experts = p.experts + (p.weights ? 0 : 1);
  // 32 columns a workgroup halve what every one of them spends on ids and x, 16
  // give twice the workgroups: from four of 32 columns a CU on, 32 (top-8 of 128,
  // 1408 x 1408, 16 against 32: 16 slots 6.7 and 7.1 us, 32 slots 9.1 and 8.6, 256
  // slots 34.9 and 29.5; dense 16384 x 4096 10.1 and 10.8, 32768 x 4096 17.8 and 16.4)
  const size_t lds = (size_t)p.n * 2;
  hipError_t e;
  if ((long long)((p.N + 31) / 32) * p.experts >= 4 * cu_count)
    e = queue(gmv_kernel<KIND, S, WHOLE, 2>, dim3((p.N + 31) / 32, experts), dim3(64 * kWaves), lds, s, p);
  else
    e = queue(gmv_kernel<KIND, S, WHOLE, 1>, dim3(all, experts), dim3(64 * kWaves), lds, s, p);
  if (e != hipSuccess || !p.weights) return e;
  return queue(gmv_join_kernel, dim3((p.N + 255) / 256, p.T), dim3(256), 0, s, p);
}

template <Kind KIND>
hipError_t by_scale(const GmvParams& p, int cu_count, hipStream_t s) {
  const bool whole = p.blk % 128 == 0;
  if (p.scale_kind == kGmvF32)
    return whole ? launch<KIND, uint32_t, true>(p, cu_count, s) : launch<KIND, uint32_t, false>(p, cu_count, s);
  return whole ? launch<KIND, uint16_t, true>(p, cu_count, s) : launch<KIND, uint16_t, false>(p, cu_count, s);
}

}  // namespace

hipError_t launch_gmv(const GmvParams& p, int cu_count, hipStream_t s) {
  if (p.scale_kind == kGmvE8m0) return launch<kMicro, uint8_t, false>(p, cu_count, s);
  if (p.fmt == 5) return by_scale<kFp4>(p, cu_count, s);
  return p.zero ? by_scale<kZero>(p, cu_count, s) : by_scale<kInt>(p, cu_count, s);
}

}  // namespace gmmk
