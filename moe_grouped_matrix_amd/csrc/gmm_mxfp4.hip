// gmm_mxfp4.hip -- microscaled fp4 on gfx950: bf16 or f32 tensors to e2m1
// codes with one E8M0 scale per 32 elements of K, and back (the arithmetic and
// layouts are those of gmm_moe.h).
//
// With amax's binary32 exponent field f, floor(log2 amax) - 2 + 127 is f - 2,
// so the scale byte is an integer subtraction (0 below f = 2, subnormals
// among them, 127 for an all-zero block, 255 where f = 255: an infinity or a
// NaN).  The scaled conversions divide (or multiply) by 2^(byte - 127) and
// round once, to nearest, ties to the even code, and keep magnitudes past 6 at
// 6: checked on every scale byte, every code pair and every bf16 value.
//
// Both directions are HBM-bound.  Codes lie as their elements do, so element
// data is a flat run; what does not lie flat is a weight's scales,
// [Ga, K/32, 1, N], whose neighbours along K are N bytes apart.  A workgroup
// takes 64 rows of one group (a contiguous run of codes while K is one panel)
// and turns their scales around in LDS, so that they are written and read in
// runs of 64 bytes.  An activation's scales [M, K/32] lie flat like the rest.
// A lane takes eight elements: one 16-byte load of bf16, one word of codes.
//
// 128 x 1408 x 704 bf16 weights: quantised in 60 us (321 MB, 5.3 TB/s), widened
// in 64 us (5.0 TB/s), a copy's rate (5.14 TB/s); counted HBM traffic is the
// algorithmic one.  With scale bytes written where they belong one at a time,
// and sixteen elements a lane, it was 78 and 94 us.  2048 x 1408 activations
// take 3.4 and 3.3 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gmm_device.hpp"
#include "gmm_mx.hpp"
#include "gmm_mx_tiles.hpp"
#include "gmm_moe_launch.hpp"

namespace gmmk {

namespace {

constexpr int kMxT = 256;
constexpr int kMxUnits = 4;    // units a thread has in flight
constexpr int kMxPitch = kMxRows + 4;
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// Eight consecutive values (one word of codes): the words of 8 bf16 or f32.
template <bool F32>
struct Eight {
  i32x4 w[F32 ? 2 : 1];
};

template <bool F32>
__device__ __forceinline__ Eight<F32> load8(const void* p, long long word) {
  Eight<F32> h;
  const i32x4* s = static_cast<const i32x4*>(p) + word * (F32 ? 2 : 1);
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) {
    // two loads 32 bytes apart share lines in the cache, so f32 goes without
    // the hint (58 against 63 us for 63 M elements; bf16 with it 31, without 33)
    if constexpr (F32)
      h.w[i] = s[i];
    else
      h.w[i] = __builtin_nontemporal_load(s + i);
  }
  return h;
}

// Largest magnitude as binary32 bits (non-negative floats order as integers).
template <bool F32>
__device__ __forceinline__ unsigned amax8(const Eight<F32>& h) {
  if constexpr (F32) {
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, (unsigned)h.w[i / 4][i % 4] & 0x7FFFFFFFu);
    return m;
  } else {
    u16x2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, (unsigned)h.w[0][i] & 0x7FFF7FFFu));
    return (unsigned)max(m[0], m[1]) << 16;
  }
}

__device__ __forceinline__ int scale_byte(unsigned amax_bits) {
  const int f = (int)(amax_bits >> 23);
  if (amax_bits == 0) return 127;
  return f == 255 ? 255 : (f < 2 ? 0 : f - 2);
}

// Four neighbouring lanes hold a block; all get its scale byte.
template <bool F32>
__device__ __forceinline__ int block_byte(const Eight<F32>& h) {
  unsigned m = amax8<F32>(h);
  m = max(m, (unsigned)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, false));  // quad_perm [1,0,3,2]
  m = max(m, (unsigned)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, false));  // quad_perm [2,3,0,1]
  return scale_byte(m);
}

template <bool F32>
__device__ __forceinline__ unsigned codes8(const Eight<F32>& h, int byte) {
  const float s = e8m0_operand(byte);
  unsigned c = 0;
  if constexpr (F32) {
    auto v = [&](int e) { return __int_as_float(h.w[e / 4][e % 4]); };
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v(0), v(1), s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v(2), v(3), s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v(4), v(5), s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v(6), v(7), s, 3);
  } else {
    auto v = [&](int e) {
      const int pair = h.w[0][e];  // (a bit cast of the vector's element itself takes element 0)
      return __builtin_bit_cast(bf16x2, pair);
    };
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, v(0), s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, v(1), s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, v(2), s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, v(3), s, 3);
  }
  return byte == 255 ? 0 : c;
}

__device__ __forceinline__ void store_codes(void* q, long long word, unsigned c) {
  __builtin_nontemporal_store(c, static_cast<unsigned*>(q) + word);
}

// Activations: words of codes in a flat run, scale bytes four to a store.
template <bool F32>
__global__ __launch_bounds__(kMxT) void quant_mxfp4_flat_kernel(Mxfp4Params p) {
  const long long words = p.rows * (p.K / 8);
  const long long stride = (long long)gridDim.x * (kMxT * kMxUnits);
  for (long long i0 = (long long)blockIdx.x * (kMxT * kMxUnits) + threadIdx.x; i0 < words; i0 += stride) {
    Eight<F32> h[kMxUnits];
#pragma unroll
    for (int u = 0; u < kMxUnits; ++u)
      if (i0 + u * kMxT < words) h[u] = load8<F32>(p.src, i0 + u * kMxT);
#pragma unroll
    for (int u = 0; u < kMxUnits; ++u) {
      // the count of words is a multiple of 4: a block's lanes are all in or all out
      const long long i = i0 + u * kMxT;
      if (i >= words) continue;
      const int byte = block_byte<F32>(h[u]);
      store_codes(p.dst, i, codes8<F32>(h[u], byte));
      // lanes 16 m, 16 m + 4, .. + 12 hold the bytes of four blocks
      int b4 = byte | __builtin_amdgcn_update_dpp(0, byte, 0x104, 0xF, 0xF, false) << 8;  // row_shl 4
      b4 |= __builtin_amdgcn_update_dpp(0, b4, 0x108, 0xF, 0xF, false) << 16;             // row_shl 8
      if ((i | 15) < words) {
        if ((i & 15) == 0) *reinterpret_cast<int*>(p.scale + (i >> 2)) = b4;
      } else if ((i & 3) == 0) {
        p.scale[i >> 2] = (uint8_t)byte;
      }
    }
  }
}

// u / d for u < 2^16, 2 <= d <= 2^9: magic = floor(2^32 / d) + 1 is off 2^32/d
// by at most 1, times u below 2^32 / d.
__device__ __forceinline__ unsigned div_small(unsigned u, unsigned magic) { return __umulhi(u, magic); }

template <bool F32>
__global__ __launch_bounds__(kMxT) void quant_mxfp4_weight_kernel(Mxfp4Params p) {
  __shared__ alignas(16) uint8_t sc[kMxPanel * kMxPitch];
  const long long tiles = mx_tiles(p.rows, p.rhs, p.K);
  const int tid = threadIdx.x, N = p.rhs;
  const long long row_words = p.K / 8;
  for (long long i = blockIdx.x; i < tiles; i += gridDim.x) {
    const MxTile t = mx_tile(p.rhs, p.K, i);
    const unsigned per = 4 * t.nb, units = t.rows * per;
    const unsigned magic = (unsigned)(0x100000000ull / per) + 1;
    for (unsigned u0 = tid; u0 < units; u0 += kMxT * kMxUnits) {
      Eight<F32> h[kMxUnits];
      unsigned row[kMxUnits];
#pragma unroll
      for (int k = 0; k < kMxUnits; ++k) {
        const unsigned u = u0 + k * kMxT;
        row[k] = div_small(u, magic);
        if (u < units) h[k] = load8<F32>(p.src, (t.row0 + row[k]) * row_words + 4 * t.b0 + (u - row[k] * per));
      }
#pragma unroll
      for (int k = 0; k < kMxUnits; ++k) {
        const unsigned u = u0 + k * kMxT, x = u - row[k] * per;
        if (u >= units) continue;
        const int byte = block_byte<F32>(h[k]);
        store_codes(p.dst, (t.row0 + row[k]) * row_words + 4 * t.b0 + x, codes8<F32>(h[k], byte));
        if ((x & 3) == 0) sc[(x >> 2) * kMxPitch + row[k]] = (uint8_t)byte;
      }
    }
    __syncthreads();
    for (int w = tid; w < t.nb * (kMxRows / 4); w += kMxT) {
      const int b = w / (kMxRows / 4), r = w % (kMxRows / 4) * 4;
      uint8_t* const d = p.scale + t.scales + (long long)b * N + r;
      if (N % 4 == 0) {  // runs of four are whole and aligned
        if (r < t.rows) *reinterpret_cast<int*>(d) = *reinterpret_cast<const int*>(sc + b * kMxPitch + r);
      } else {
        for (int e = 0; e < 4 && r + e < t.rows; ++e) d[e] = sc[b * kMxPitch + r + e];
      }
    }
    __syncthreads();
  }
}

// Eight codes (a word) under a scale byte to 16 bytes of bf16 or 32 of f32.
template <bool F32>
__device__ __forceinline__ void widen8(void* y, long long word, unsigned w, int byte) {
  if constexpr (F32) {
    const float s = e8m0_operand(byte);
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1);
    const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3);
    f32x4* const o = static_cast<f32x4*>(y) + word * 2;
    __builtin_nontemporal_store(f32x4{a[0], a[1], b[0], b[1]}, o);
    __builtin_nontemporal_store(f32x4{c[0], c[1], d[0], d[1]}, o + 1);
  } else {
    __builtin_nontemporal_store(fp4x8_scaled_bf16(w, byte), static_cast<i32x4*>(y) + word);
  }
}

template <bool F32>
__global__ __launch_bounds__(kMxT) void widen_mxfp4_flat_kernel(Mxfp4Params p) {
  const long long words = p.rows * (p.K / 8);
  const unsigned* const q = static_cast<const unsigned*>(p.src);
  const long long stride = (long long)gridDim.x * (kMxT * kMxUnits);
  for (long long i0 = (long long)blockIdx.x * (kMxT * kMxUnits) + threadIdx.x; i0 < words; i0 += stride) {
    unsigned w[kMxUnits];
    int byte[kMxUnits];
#pragma unroll
    for (int u = 0; u < kMxUnits; ++u) {
      const long long i = i0 + u * kMxT;
      if (i >= words) continue;
      w[u] = __builtin_nontemporal_load(q + i);
      byte[u] = p.scale[i >> 2];
    }
#pragma unroll
    for (int u = 0; u < kMxUnits; ++u)
      if (i0 + u * kMxT < words) widen8<F32>(p.dst, i0 + u * kMxT, w[u], byte[u]);
  }
}

template <bool F32>
__global__ __launch_bounds__(kMxT) void widen_mxfp4_weight_kernel(Mxfp4Params p) {
  __shared__ alignas(16) uint8_t sc[kMxPanel * kMxPitch];
  const long long tiles = mx_tiles(p.rows, p.rhs, p.K);
  const int tid = threadIdx.x, N = p.rhs;
  const long long row_words = p.K / 8;
  const unsigned* const q = static_cast<const unsigned*>(p.src);
  for (long long i = blockIdx.x; i < tiles; i += gridDim.x) {
    const MxTile t = mx_tile(p.rhs, p.K, i);
    for (int w = tid; w < t.nb * (kMxRows / 4); w += kMxT) {
      const int b = w / (kMxRows / 4), r = w % (kMxRows / 4) * 4;
      const uint8_t* const s = p.scale + t.scales + (long long)b * N + r;
      if (N % 4 == 0) {
        if (r < t.rows) *reinterpret_cast<int*>(sc + b * kMxPitch + r) = *reinterpret_cast<const int*>(s);
      } else {
        for (int e = 0; e < 4 && r + e < t.rows; ++e) sc[b * kMxPitch + r + e] = s[e];
      }
    }
    __syncthreads();
    const unsigned per = 4 * t.nb, units = t.rows * per;
    const unsigned magic = (unsigned)(0x100000000ull / per) + 1;
    for (unsigned u0 = tid; u0 < units; u0 += kMxT * kMxUnits) {
      unsigned w[kMxUnits], row[kMxUnits];
#pragma unroll
      for (int k = 0; k < kMxUnits; ++k) {
        const unsigned u = u0 + k * kMxT;
        row[k] = div_small(u, magic);
        if (u < units) w[k] = __builtin_nontemporal_load(q + (t.row0 + row[k]) * row_words + 4 * t.b0 + (u - row[k] * per));
      }
#pragma unroll
      for (int k = 0; k < kMxUnits; ++k) {
        const unsigned u = u0 + k * kMxT, x = u - row[k] * per;
        if (u < units)
          widen8<F32>(p.dst, (t.row0 + row[k]) * row_words + 4 * t.b0 + x, w[k], sc[(x >> 2) * kMxPitch + row[k]]);
      }
    }
    __syncthreads();
  }
}

unsigned flat_grid(long long units, int cu_count) {
  long long grid = (units + kMxT * kMxUnits - 1) / (kMxT * kMxUnits);
  const long long cap = (long long)cu_count * 16;
  if (grid > cap) grid = cap;
  return (unsigned)(grid < 1 ? 1 : grid);
}

unsigned weight_grid(const Mxfp4Params& p, int cu_count) {
  long long grid = mx_tiles(p.rows, p.rhs, p.K);
  const long long cap = (long long)cu_count * 8;
  if (grid > cap) grid = cap;
  return (unsigned)(grid < 1 ? 1 : grid);
}

}  // namespace

hipError_t launch_quant_mxfp4(const Mxfp4Params& p, int cu, hipStream_t st) {
  const auto kernel = p.rhs == 0 ? (p.wide_f32 ? quant_mxfp4_flat_kernel<true> : quant_mxfp4_flat_kernel<false>)
                                 : (p.wide_f32 ? quant_mxfp4_weight_kernel<true> : quant_mxfp4_weight_kernel<false>);
  const unsigned grid = p.rhs == 0 ? flat_grid(p.rows * (p.K / 8), cu) : weight_grid(p, cu);
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(kMxT), 0, st, p);
  return hipGetLastError();
}

hipError_t launch_widen_mxfp4(const Mxfp4Params& p, int cu, hipStream_t st) {
  const auto kernel = p.rhs == 0 ? (p.wide_f32 ? widen_mxfp4_flat_kernel<true> : widen_mxfp4_flat_kernel<false>)
                                 : (p.wide_f32 ? widen_mxfp4_weight_kernel<true> : widen_mxfp4_weight_kernel<false>);
  const unsigned grid = p.rhs == 0 ? flat_grid(p.rows * (p.K / 8), cu) : weight_grid(p, cu);
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(kMxT), 0, st, p);
  return hipGetLastError();
}

}  // namespace gmmk
