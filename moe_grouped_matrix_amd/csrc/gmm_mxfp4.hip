// gmm_mxfp4.hip -- microscaled fp4 on gfx950: bf16 or f32 tensors to e2m1
// codes with one E8M0 scale per 32 elements of K, and back (the arithmetic and
// layouts are those of gmm_moe.h).
//
// With amax's binary32 exponent field f, floor(log2 amax) - 2 + 127 is f - 2,
// so the scale byte is an integer subtraction (0 below f = 2, subnormals
// among them, 127 for an all-zero block, 255 where f = 255: an infinity or a
// NaN).  x * 2^(127 - byte) is exact in binary32 wherever it can decide a code
// (a product that underflows lies far below the first rounding border, 1/4).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gmm_device.hpp"
#include "gmm_moe_launch.hpp"

namespace gmmk {

namespace {

constexpr int kMxT = 256;
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Sixteen consecutive values of a row as binary32.
template <bool F32>
__device__ __forceinline__ void load16(const void* p, long long at, float (&v)[16]) {
  if constexpr (F32) {
    const f32x4* s = reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4 a = s[i];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * i + e] = a[e];
    }
  } else {
    const i32x4* s = reinterpret_cast<const i32x4*>(static_cast<const uint16_t*>(p) + at);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const i32x4 a = s[i];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[8 * i + 2 * e] = __uint_as_float((uint32_t)a[e] << 16);
        v[8 * i + 2 * e + 1] = __uint_as_float((uint32_t)a[e] & 0xFFFF0000u);
      }
    }
  }
}

__device__ __forceinline__ int scale_byte(uint32_t amax_bits) {
  const int f = (int)(amax_bits >> 23);
  if (amax_bits == 0) return 127;
  return f == 255 ? 255 : (f < 2 ? 0 : f - 2);
}

// Eight values times 2^e as e2m1 codes, the first in the low nibble.
__device__ __forceinline__ uint32_t codes8(const float* v, int e) {
  uint32_t w = 0;
  float t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = __builtin_ldexpf(v[i], e);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, t[0], t[1], 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, t[2], t[3], 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, t[4], t[5], 1.0f, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, t[6], t[7], 1.0f, 3);
  return w;
}

// Where block b of row r keeps its scale.
__device__ __forceinline__ long long scale_at(const Mxfp4Params& p, long long r, int b) {
  const int nb = p.K / 32;
  if (p.rhs == 0) return r * nb + b;
  return ((r / p.rhs) * nb + b) * p.rhs + r % p.rhs;
}

// Two neighbouring lanes take a block, sixteen elements each.
template <bool F32>
__global__ __launch_bounds__(kMxT) void quant_mxfp4_kernel(Mxfp4Params p) {
  const int nb = p.K / 32;
  const long long halves = p.rows * nb * 2;
  const long long stride = (long long)gridDim.x * kMxT;
  // neighbours differ in the last bit of i only, so both are in or out
  for (long long i = (long long)blockIdx.x * kMxT + threadIdx.x; i < halves; i += stride) {
    float v[16];
    load16<F32>(p.src, i * 16, v);
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) m = max(m, __float_as_uint(v[e]) & 0x7FFFFFFFu);
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, false));  // quad_perm [1,0,3,2]
    const int byte = scale_byte(m);
    i32x2 w = {0, 0};
    if (byte != 255) {
      w[0] = (int)codes8(v, 127 - byte);
      w[1] = (int)codes8(v + 8, 127 - byte);
    }
    *reinterpret_cast<i32x2*>(static_cast<uint8_t*>(p.dst) + i * 8) = w;
    if ((i & 1) == 0) {
      const long long j = i >> 1;
      p.scale[scale_at(p, j / nb, (int)(j % nb))] = (uint8_t)byte;
    }
  }
}

template <bool F32>
__global__ __launch_bounds__(kMxT) void widen_mxfp4_kernel(Mxfp4Params p) {
  const int nb = p.K / 32;
  const long long halves = p.rows * nb * 2;
  const long long stride = (long long)gridDim.x * kMxT;
  for (long long i = (long long)blockIdx.x * kMxT + threadIdx.x; i < halves; i += stride) {
    const long long j = i >> 1;
    const int byte = p.scale[scale_at(p, j / nb, (int)(j % nb))];
    const i32x2 w = *reinterpret_cast<const i32x2*>(static_cast<const uint8_t*>(p.src) + i * 8);
    float v[16];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[h], 1.0f, 0);
      const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[h], 1.0f, 1);
      const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[h], 1.0f, 2);
      const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[h], 1.0f, 3);
      const float u[8] = {a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[8 * h + e] = byte == 255 ? __builtin_nanf("") : __builtin_ldexpf(u[e], byte - 127);
    }
    if constexpr (F32) {
      f32x4* const d = reinterpret_cast<f32x4*>(static_cast<float*>(p.dst) + i * 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) d[e] = f32x4{v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]};
    } else {
      i32x4* const d = reinterpret_cast<i32x4*>(static_cast<uint16_t*>(p.dst) + i * 16);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        d[h] = i32x4{(int)pk_bf16_rne(v[8 * h], v[8 * h + 1]), (int)pk_bf16_rne(v[8 * h + 2], v[8 * h + 3]),
                     (int)pk_bf16_rne(v[8 * h + 4], v[8 * h + 5]), (int)pk_bf16_rne(v[8 * h + 6], v[8 * h + 7])};
    }
  }
}

unsigned mx_grid(const Mxfp4Params& p, int cu_count) {
  long long grid = (p.rows * (p.K / 32) * 2 + kMxT - 1) / kMxT;
  const long long cap = (long long)cu_count * 16;
  if (grid > cap) grid = cap;
  return (unsigned)(grid < 1 ? 1 : grid);
}

}  // namespace

hipError_t launch_quant_mxfp4(const Mxfp4Params& p, int cu, hipStream_t st) {
  if (p.wide_f32)
    hipLaunchKernelGGL(quant_mxfp4_kernel<true>, dim3(mx_grid(p, cu)), dim3(kMxT), 0, st, p);
  else
    hipLaunchKernelGGL(quant_mxfp4_kernel<false>, dim3(mx_grid(p, cu)), dim3(kMxT), 0, st, p);
  return hipGetLastError();
}

hipError_t launch_widen_mxfp4(const Mxfp4Params& p, int cu, hipStream_t st) {
  if (p.wide_f32)
    hipLaunchKernelGGL(widen_mxfp4_kernel<true>, dim3(mx_grid(p, cu)), dim3(kMxT), 0, st, p);
  else
    hipLaunchKernelGGL(widen_mxfp4_kernel<false>, dim3(mx_grid(p, cu)), dim3(kMxT), 0, st, p);
  return hipGetLastError();
}

}  // namespace gmmk
