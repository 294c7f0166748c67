// gmm_gmv.hip -- products of a few tokens with their experts' four-bit
// weights, by expert id (gmm_layer.h, gmm_gmv_run).
//
// What bounds it is reading every touched expert's weight once.  A workgroup
// takes 16 NT columns of one expert and all slots that chose it (up to 16 at a
// time); its waves share out K in contiguous chunks of 128 and join their sums
// in LDS, so nothing is read by two waves and nothing waits for a barrier on
// the way.  Which slots chose the r-th of the experts that were chosen at all,
// every workgroup finds out by itself from the ids.
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

constexpr int kMaxSlots = 4096;

__device__ __forceinline__ int slot_expert(const GmvParams& p, int i) {
  if (!p.ids) return 0;
  const long long id = p.ids64 ? static_cast<const int64_t*>(p.ids)[i] : static_cast<const int32_t*>(p.ids)[i];
  return id >= 0 && id < p.G ? (int)id : -1;
}
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
  kInt,    // int4, uint4: scale and zero point per block of a multiple of 32
  kFp4,    // fp4 with f32 or bf16 scales
  kMicro,  // fp4 with E8M0 scales of blocks of 32
};

// Eight codes as bf16, in the order of ordered_x.
template <Kind KIND>
__device__ __forceinline__ bf16x8 widen8(unsigned w, int byte) {
  i32x4 r;
  if constexpr (KIND == kInt) {
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
  if constexpr (KIND != kInt) return __builtin_bit_cast(bf16x8, x);
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

// One chunk of 128 elements of K: the lane's codes of NT column tiles, its
// scales and zero points (of its own block of 32), and its x elements of the
// four blocks (FEW: of one of them).
template <int NT, bool FEW>
struct Chunk {
  i32x4 w[NT];
  int s[NT], z[NT];
  i32x4 x[FEW ? 1 : 4];
};

// What a wave reads for one expert.
template <int NT>
struct Source {
  const uint8_t* w;   // the expert's codes
  long long scale;    // index of its first scale
  long long row[NT];  // the lane's columns: offset of the codes
  int col[NT];        // and the columns
  const uint16_t* x;  // the lane's row of x
};

template <Kind KIND, int NT, bool FEW>
__device__ __forceinline__ void load_chunk(Chunk<NT, FEW>& d, const GmvParams& p, const Source<NT>& src, int c, int q) {
  const int k0 = 128 * c, mine = k0 + 32 * q < p.K ? k0 + 32 * q : k0;  // (past K: read elsewhere, and not used)
#pragma unroll
  for (int t = 0; t < NT; ++t)
    d.w[t] = *reinterpret_cast<const i32x4*>(src.w + src.row[t] + mine / 2);
  const int b = KIND == kMicro ? mine >> 5 : (int)(((unsigned long long)((unsigned)mine >> 5) * p.blk_magic) >> 31);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const long long i = src.scale + (long long)b * p.N + src.col[t];
    if constexpr (KIND == kMicro) {
      d.s[t] = static_cast<const uint8_t*>(p.scale)[i];
    } else if (p.scale_kind == kGmvF32) {
      d.s[t] = static_cast<const int*>(p.scale)[i];
    } else {
      d.s[t] = static_cast<const uint16_t*>(p.scale)[i] << 16;
    }
    if constexpr (KIND == kInt)
      if (p.zero)
        d.z[t] = p.scale_kind == kGmvF32 ? static_cast<const int*>(p.zero)[i] : static_cast<const uint16_t*>(p.zero)[i] << 16;
  }
  if constexpr (FEW) {
    const int i = threadIdx.x & 3, k = k0 + 32 * i < p.K ? k0 + 32 * i : k0;
    d.x[0] = *reinterpret_cast<const i32x4*>(src.x + k + 8 * q);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = k0 + 32 * i < p.K ? k0 + 32 * i : k0;
      d.x[i] = *reinterpret_cast<const i32x4*>(src.x + k + 8 * q);
    }
  }
}

// The wave's sums: tot[t][r] of lane (q, n) for column n of tile t and row q
// (FEW) or 4 q + r.  fp4 with E8M0 scales needs no folds, and sums in the matrix
// cores' results, run (FEW: one for each block of a chunk).
template <int NT, bool FEW>
struct Sums {
  float tot[NT][FEW ? 1 : 4];
  f32x4 run[NT][FEW ? 4 : 1];
};

template <int NT, bool FEW>
__device__ __forceinline__ void clear(Sums<NT, FEW>& a) {
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (float& v : a.tot[t]) v = 0.f;
#pragma unroll
    for (f32x4& v : a.run[t]) v = f32x4{0.f, 0.f, 0.f, 0.f};
  }
}

// Adds the products of chunk c.  WHOLE: its four blocks share their scale (scale
// blocks are multiples of 128).  WEIGHTED: times `weight`.
template <Kind KIND, bool WHOLE, bool WEIGHTED, int NT, bool FEW>
__device__ __forceinline__ void use_chunk(Sums<NT, FEW>& a, Chunk<NT, FEW>& d, const GmvParams& p, int c, float weight) {
  const int left = (p.K >> 5) - 4 * c;  // blocks from here on
  const f32x4 none{0.f, 0.f, 0.f, 0.f};
  const i32x4 one4{0x3F803F80, 0x3F803F80, 0x3F803F80, 0x3F803F80};
  const bf16x8 ones = __builtin_bit_cast(bf16x8, one4);
  const float base = KIND == kInt && p.fmt == 3 ? 8.f : 0.f;
  const int flip = KIND == kInt && p.fmt == 3 ? (int)0x88888888u : 0;
  constexpr bool CHAIN = KIND == kMicro && !WEIGHTED;
  constexpr int ROWS = FEW ? 1 : 4;
  i32x4 s4[NT], z4[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if constexpr (KIND == kInt) d.w[t] ^= flip;
    transpose4(d.w[t]);
    if constexpr (KIND == kMicro || !WHOLE) {
      s4[t] = spread4(d.s[t]);
      if constexpr (KIND == kInt)
        if (p.zero) z4[t] = spread4(d.z[t]);
    }
  }
  // sums of products `got` and of x `sum`, for row r
  auto fold = [&](int t, int r, float got, float sum, int scale, int zero) __attribute__((always_inline)) {
    float s = KIND == kMicro ? 1.f : __int_as_float(scale);
    if constexpr (WEIGHTED) s *= weight;
    if constexpr (KIND == kInt) got = __builtin_fmaf(-(p.zero ? __int_as_float(zero) + base : base), sum, got);
    a.tot[t][r] = __builtin_fmaf(s, got, a.tot[t][r]);
  };
  f32x4 acc[NT], sum = none;
  float few[NT], few_sum = 0.f;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    acc[t] = none;
    few[t] = 0.f;
  }
  bf16x8 x = ordered_x<KIND>(d.x[0]);
  if constexpr (FEW && KIND == kInt) sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, ones, none, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i >= left) break;
    if constexpr (!FEW) {
      if (i > 0) x = ordered_x<KIND>(d.x[i]);
      if constexpr (KIND == kInt) sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, ones, WHOLE ? sum : none, 0, 0, 0);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const bf16x8 w = widen8<KIND>((unsigned)d.w[t][i], KIND == kMicro ? s4[t][i] : 0);
      if constexpr (CHAIN) {
        f32x4& run = a.run[t][FEW ? i : 0];
        run = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, w, run, 0, 0, 0);
        continue;
      }
      constexpr bool TOGETHER = WHOLE || KIND == kMicro;
      acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, w, TOGETHER && !FEW ? acc[t] : none, 0, 0, 0);
      if constexpr (!TOGETHER) {
        if constexpr (FEW) {
          fold(t, 0, acc[t][i], sum[i], s4[t][i], z4[t][i]);
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) fold(t, r, acc[t][r], sum[r], s4[t][i], z4[t][i]);
        }
      } else if constexpr (FEW) {
        few[t] += acc[t][i];
      }
    }
    if constexpr (FEW && WHOLE) few_sum += sum[i];
  }
  if constexpr (!CHAIN && (WHOLE || KIND == kMicro)) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < ROWS; ++r) fold(t, r, FEW ? few[t] : acc[t][r], FEW ? few_sum : sum[r], d.s[t], d.z[t]);
  }
}

// What the sums came to.
template <Kind KIND, bool WEIGHTED, int NT, bool FEW>
__device__ __forceinline__ float total(const Sums<NT, FEW>& a, int t, int r) {
  if constexpr (KIND != kMicro || WEIGHTED) return a.tot[t][r];
  if constexpr (FEW) return (a.run[t][0][0] + a.run[t][1][1]) + (a.run[t][2][2] + a.run[t][3][3]);
  return a.run[t][0][r];
}

// The slots of the r-th expert that any slot chose: into list; returns how
// many, and the expert (-1: fewer than r + 1 were chosen).  In which order the
// experts are counted, and the slots listed, does not matter.  Up to 64 slots
// each wave looks for itself: equal ids find each other by a ballot per bit of
// the id, and an expert's first slot stands for it.
struct Found {
  int expert, count;
};

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
    int id[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = i0 + 64 * u + lane;
      id[u] = i < p.n ? slot_expert(p, i) : -1;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const unsigned long long mine = __ballot(id[u] == g);
      if (id[u] == g) list[count + __builtin_popcountll(mine & below)] = (uint16_t)(i0 + 64 * u + lane);
      count += __builtin_popcountll(mine);
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  return {count ? g : -1, count};
}

template <int T>
__device__ __forceinline__ Found find_many(const GmvParams& p, int r, uint16_t* list) {
  __shared__ int chosen[kMaxGroups];
  __shared__ int wave_tot[T / 64];
  __shared__ int expert, count;
  constexpr int PER = kMaxGroups / T;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  for (int g = tid; g < kMaxGroups; g += T) chosen[g] = 0;
  if (tid == 0) {
    expert = -1;
    count = 0;
  }
  __syncthreads();
  for (int i = tid; i < p.n; i += T) {
    const int g = slot_expert(p, i);
    if (g >= 0) chosen[g] = 1;
  }
  __syncthreads();
  int mine = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) mine += chosen[tid * PER + j];
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
    int g = tid * PER;
    for (int left = r - at;; ++g)
      if (chosen[g] && left-- == 0) break;
    expert = g;
  }
  __syncthreads();
  const int g = expert;
  if (g < 0) return {-1, 0};
  for (int i = tid; i < p.n; i += T)
    if (slot_expert(p, i) == g) list[atomicAdd(&count, 1)] = (uint16_t)i;
  __syncthreads();
  return {g, count};
}

template <int NT>
__device__ __forceinline__ void set_columns(Source<NT>& src, const GmvParams& p, int n0, int n) {
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int col = n0 + 16 * t + n;
    src.col[t] = col < p.N ? col : p.N - 1;  // (past the last: read, and not stored)
    src.row[t] = (long long)src.col[t] * (p.K / 2);
  }
}

// One pass over the expert's columns for rows list[first ..].
template <Kind KIND, bool WHOLE, int NT, bool FEW, int W>
__device__ __forceinline__ void pass(const GmvParams& p, Source<NT>& src, const uint16_t* list, int first, int rows, int n0,
                                     float* join) {
  constexpr int D = NT == 1 ? 3 : 2;  // chunks in flight
  constexpr int ROWS = FEW ? 4 : 16;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), q = lane >> 4, n = lane & 15;
  const int row = FEW ? n >> 2 : n;
  const int slot = list[first + (row < rows ? row : 0)];
  src.x = p.x + (long long)(p.per_slot ? slot : slot / p.k) * p.K;
  const int chunks = (p.K + 127) >> 7, lo = chunks * w / W, hi = chunks * (w + 1) / W;
  Sums<NT, FEW> sums;
  clear(sums);
  Chunk<NT, FEW> d[D];
#pragma unroll
  for (int i = 0; i < D; ++i)
    if (lo + i < hi) load_chunk<KIND>(d[i], p, src, lo + i, q);
  for (int c = lo; c < hi; c += D) {
#pragma unroll
    for (int i = 0; i < D; ++i)
      if (c + i < hi) {
        use_chunk<KIND, WHOLE, false>(sums, d[i], p, c + i, 1.f);
        if (c + i + D < hi) load_chunk<KIND>(d[i], p, src, c + i + D, q);
      }
  }
  // join[wave][row][column]
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < ROWS / 4; ++r)
      join[(w * ROWS + (FEW ? q : 4 * q + r)) * (16 * NT) + 16 * t + n] = total<KIND, false>(sums, t, r);
  __syncthreads();
  for (int i = threadIdx.x; i < rows * 16 * NT; i += 64 * W) {
    const int rr = i / (16 * NT), col = i % (16 * NT);
    if (n0 + col < p.N) {
      float v = 0.f;
#pragma unroll
      for (int j = 0; j < W; ++j) v += join[(j * ROWS + rr) * (16 * NT) + col];
      const long long o = (long long)list[first + rr] * p.N + n0 + col;
      if (p.weights)
        p.work[o] = v;
      else
        store_out(p, o, v);
    }
  }
  __syncthreads();
}

template <Kind KIND, bool WHOLE, int NT>
__global__ __launch_bounds__(256, 4) void gmv_kernel(GmvParams p) {
  constexpr int W = 4;
  __shared__ uint16_t list[kMaxSlots];
  __shared__ float join[W * 16 * 16 * NT];
  const int n0 = blockIdx.x * 16 * NT, n = threadIdx.x & 15;
  if ((int)blockIdx.y == p.experts) {  // slots without an expert: zeros
    for (int i = threadIdx.x / (16 * NT); i < p.n; i += 256 / (16 * NT)) {
      const int col = n0 + threadIdx.x % (16 * NT);
      if (col < p.N && slot_expert(p, i) < 0) store_out(p, (long long)i * p.N + col, 0.f);
    }
    return;
  }
  const Found f = p.n <= 64 ? find_few(p, blockIdx.y, list)
                  : p.experts == p.G ? find_slots(p, blockIdx.y, list)
                                     : find_many<64 * W>(p, blockIdx.y, list);
  if (f.expert < 0) return;
  Source<NT> src;
  set_columns(src, p, n0, n);
  src.w = p.rhs + (long long)f.expert * p.N * (p.K / 2);
  src.scale = (long long)f.expert * p.nb * p.N;
  for (int first = 0; first < f.count; first += 16) {
    const int rows = f.count - first < 16 ? f.count - first : 16;
    if (rows <= 4)
      pass<KIND, WHOLE, NT, true, W>(p, src, list, first, rows, n0, join);
    else
      pass<KIND, WHOLE, NT, false, W>(p, src, list, first, rows, n0, join);
  }
}

// A token's weighted sum over its slots, at once: a workgroup takes 16 columns
// of one token, its 16 waves share out the chunks of all its slots.  For a few
// tokens, whose experts are mostly different ones, this saves the second
// launch.
template <Kind KIND, bool WHOLE>
__global__ __launch_bounds__(1024) void gmv_token_kernel(GmvParams p) {
  constexpr int W = 16;
  __shared__ int expert[64];
  __shared__ int slot[64];
  __shared__ float join[W][16];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), q = lane >> 4, n = lane & 15;
  const int n0 = blockIdx.x * 16, t = blockIdx.y;
  // (every wave writes the same list for itself)
  const int id = lane < p.k ? slot_expert(p, t * p.k + lane) : -1;
  const unsigned long long live = __ballot(id >= 0);
  if (id >= 0) {
    const int at = __builtin_popcountll(live & ((1ull << lane) - 1));
    expert[at] = id;
    slot[at] = t * p.k + lane;
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  Source<1> src;
  set_columns(src, p, n0, n);
  const int chunks = (p.K + 127) >> 7, all = __builtin_popcountll(live) * chunks;
  const int lo = all * w / W, hi = all * (w + 1) / W;
  Sums<1, true> sums;
  clear(sums);
  constexpr int D = 3;
  Chunk<1, true> d[D];
  float weight[D];
  auto load = [&](Chunk<1, true>& into, float& wt, int item) __attribute__((always_inline)) {
    const int j = item / chunks;
    const int g = __builtin_amdgcn_readfirstlane(expert[j]), i = __builtin_amdgcn_readfirstlane(slot[j]);
    src.w = p.rhs + (long long)g * p.N * (p.K / 2);
    src.scale = (long long)g * p.nb * p.N;
    src.x = p.x + (long long)(p.per_slot ? i : t) * p.K;
    wt = slot_weight(p, i);
    load_chunk<KIND>(into, p, src, item - j * chunks, q);
  };
#pragma unroll
  for (int i = 0; i < D; ++i)
    if (lo + i < hi) load(d[i], weight[i], lo + i);
  for (int c = lo; c < hi; c += D) {
#pragma unroll
    for (int i = 0; i < D; ++i)
      if (c + i < hi) {
        use_chunk<KIND, WHOLE, true>(sums, d[i], p, (c + i) % chunks, weight[i]);
        if (c + i + D < hi) load(d[i], weight[i], c + i + D);
      }
  }
  if (q == 0) join[w][n] = total<KIND, true>(sums, 0, 0);
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

template <Kind KIND, bool WHOLE>
hipError_t launch(const GmvParams& p, int cu_count, hipStream_t s) {
  if (p.at_once) {
    hipLaunchKernelGGL((gmv_token_kernel<KIND, WHOLE>), dim3((p.N + 15) / 16, p.T), dim3(1024), 0, s, p);
    return hipGetLastError();
  }
  const unsigned experts = p.experts + (p.weights ? 0 : 1);
  if ((long long)((p.N + 31) / 32) * p.experts >= 2 * cu_count)
    hipLaunchKernelGGL((gmv_kernel<KIND, WHOLE, 2>), dim3((p.N + 31) / 32, experts), dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL((gmv_kernel<KIND, WHOLE, 1>), dim3((p.N + 15) / 16, experts), dim3(256), 0, s, p);
  if (p.weights) hipLaunchKernelGGL(gmv_join_kernel, dim3((p.N + 255) / 256, p.T), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gmv(const GmvParams& p, int cu_count, hipStream_t stream) {
  if (p.scale_kind == kGmvE8m0) return launch<kMicro, false>(p, cu_count, stream);
  const bool whole = p.blk % 128 == 0;
  if (p.fmt == 5) return whole ? launch<kFp4, true>(p, cu_count, stream) : launch<kFp4, false>(p, cu_count, stream);
  return whole ? launch<kInt, true>(p, cu_count, stream) : launch<kInt, false>(p, cu_count, stream);
}

}  // namespace gmmk
