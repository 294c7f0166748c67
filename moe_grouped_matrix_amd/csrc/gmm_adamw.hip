// gmm_adamw.hip -- the AdamW step of many tensors (gmm_layer.h,
// gmm_adamw_run), with states in fp32 or in eight bits.
//
// A launch takes up to kAdamItems tensors, whose addresses travel in its
// arguments (nothing is copied to the device first, so a step can be captured
// and its tensors may change from call to call); a workgroup takes chunks of
// kAdamChunk elements, a wave blocks of 256 of them, four consecutive elements
// a lane, so that a block's largest state is one reduction over the wave.
//
// Every operation is rounded on its own and in a fixed order (no contraction),
// so that the eight-bit codes, which turn on single roundings, are those of the
// formula in any other correctly rounded arithmetic.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gmm_device.hpp"
#include "gmm_layer_launch.hpp"

namespace gmmk {

namespace {

constexpr int kAdamT = 256;

typedef short short2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ f32x4 load4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
__device__ __forceinline__ f32x4 load4(const uint16_t* p) {
  const i32x2 w = *reinterpret_cast<const i32x2*>(p);
  return f32x4{__int_as_float(w[0] << 16), __int_as_float(w[0] & (int)0xFFFF0000), __int_as_float(w[1] << 16),
               __int_as_float(w[1] & (int)0xFFFF0000)};
}
__device__ __forceinline__ void store4(float* p, f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; }
__device__ __forceinline__ void store4(uint16_t* p, f32x4 v) {
  *reinterpret_cast<i32x2*>(p) = i32x2{(int)pk_bf16_rne(v[0], v[1]), (int)pk_bf16_rne(v[2], v[3])};
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_bits_to_f32(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = f32_to_bf16_rne(v); }

// Elements [0, n) of the lane's four (the last ones of a tensor may miss).
template <class E>
__device__ __forceinline__ f32x4 load_some(const E* p, int n) {
  if (n >= 4) return load4(p);
  f32x4 v{0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < 3; ++i)
    if (i < n) v[i] = load1(p + i);
  return v;
}
template <class E>
__device__ __forceinline__ void store_some(E* p, f32x4 v, int n) {
  if (n >= 4) return store4(p, v);
  for (int i = 0; i < 3; ++i)
    if (i < n) store1(p + i, v[i]);
}
__device__ __forceinline__ unsigned load_codes(const uint8_t* p, int n) {
  if (n >= 4) return *reinterpret_cast<const unsigned*>(p);
  unsigned w = 0;
  for (int i = 0; i < 3; ++i)
    if (i < n) w |= (unsigned)p[i] << (8 * i);
  return w;
}
__device__ __forceinline__ void store_codes(uint8_t* p, unsigned w, int n) {
  if (n >= 4) {
    *reinterpret_cast<unsigned*>(p) = w;
    return;
  }
  for (int i = 0; i < 3; ++i)
    if (i < n) p[i] = (uint8_t)(w >> (8 * i));
}

__device__ __forceinline__ f32x4 widen_codes(unsigned w, float scale) {
  const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  return f32x4{lo[0] * scale, lo[1] * scale, hi[0] * scale, hi[1] * scale};
}

__device__ __forceinline__ unsigned wave_max(unsigned v) {
#pragma unroll
  for (int s = 1; s < 64; s *= 2) v = max(v, (unsigned)__shfl_xor((int)v, s, 64));
  return v;
}

// The wave's block x as e4m3 codes; returns the scale.
template <bool POSITIVE>
__device__ __forceinline__ float quantise(f32x4 x, unsigned& codes) {
#pragma clang fp contract(off)
  unsigned am = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) am = max(am, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  am = wave_max(am);
  if (am >= 0x7F800000u) {
    codes = 0;
    return __builtin_nanf("");
  }
  const float amax = __uint_as_float(am);
  const float s = am == 0 ? 1.f : fmaxf(amax * (1.f / 448.f), 0x1p-126f);
  float t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t[i] = x[i] / s;
    if (POSITIVE && x[i] > 0.f) t[i] = fmaxf(t[i], 0x1p-9f);
    t[i] = fminf(fmaxf(t[i], -448.f), 448.f);
  }
  short2_t c = {0, 0};
  c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, t[0], t[1], 1.0f, false);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, t[2], t[3], 1.0f, true);
  codes = __builtin_bit_cast(unsigned, c);
  return s;
}

template <class P, class G, bool EIGHT>
__global__ __launch_bounds__(kAdamT) void adamw_kernel(AdamParams a) {
#pragma clang fp contract(off)
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  AdamFactors f{a.decay, a.rate, a.root_scale};
  if (a.step_at || a.lr_at)
    f = adam_factors(a.lr_at ? (double)a.lr_at[0] : a.lr, a.beta1, a.beta2, a.weight_decay,
                     a.step_at ? (long long)a.step_at[0] : a.step);
  const float gscale = a.grad_scale ? a.grad_scale[0] : 1.f;
  const int chunks = a.first[a.count];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    int lo = 0, hi = a.count;  // the last tensor whose first chunk is not behind c
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (a.first[mid] <= c)
        lo = mid;
      else
        hi = mid;
    }
    const AdamItem& t = a.item[lo];
    const long long base = (long long)(c - a.first[lo]) * kAdamChunk;
    for (int b = w; b < kAdamChunk / kAdamBlock; b += kAdamT / 64) {
      const long long at = base + b * kAdamBlock;
      if (at >= t.n) break;
      const long long i = at + lane * 4;
      const int n = (int)(t.n - i < 4 ? t.n - i : 4);  // (may be negative)
      P* const pp = static_cast<P*>(t.p) + i;
      f32x4 p = load_some(pp, n), g = load_some(static_cast<const G*>(t.g) + i, n), m, v;
      if constexpr (EIGHT) {
        const long long blk = at / kAdamBlock;
        m = widen_codes(load_codes(static_cast<const uint8_t*>(t.m) + i, n), t.ms[blk]);
        v = widen_codes(load_codes(static_cast<const uint8_t*>(t.v) + i, n), t.vs[blk]);
      } else {
        m = load_some(static_cast<const float*>(t.m) + i, n);
        v = load_some(static_cast<const float*>(t.v) + i, n);
      }
      f32x4 root;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = a.grad_scale ? g[e] * gscale : g[e];
        const float v0 = EIGHT ? v[e] * v[e] : v[e];
        m[e] = m[e] * a.b1 + x * a.c1;
        v[e] = v0 * a.b2 + (x * x) * a.c2;
        root[e] = __builtin_sqrtf(v[e]);
        p[e] = p[e] * f.decay - f.rate * (m[e] / (root[e] * f.root_scale + a.eps));
      }
      if constexpr (EIGHT) {
        // (elements past the end count for nothing)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e >= n) m[e] = root[e] = 0.f;
        unsigned cm, cv;
        const float sm = quantise<false>(m, cm), sv = quantise<true>(root, cv);
        const long long blk = at / kAdamBlock;
        store_codes(static_cast<uint8_t*>(t.m) + i, cm, n);
        store_codes(static_cast<uint8_t*>(t.v) + i, cv, n);
        if (lane == 0) {
          t.ms[blk] = sm;
          t.vs[blk] = sv;
        }
      } else {
        store_some(static_cast<float*>(t.m) + i, m, n);
        store_some(static_cast<float*>(t.v) + i, v, n);
      }
      store_some(pp, p, n);
      if (t.copy) store_some(t.copy + i, p, n);
    }
  }
}

template <class P, class G>
hipError_t launch(const AdamParams& p, bool eight, int grid, hipStream_t stream) {
  if (eight)
    hipLaunchKernelGGL((adamw_kernel<P, G, true>), dim3(grid), dim3(kAdamT), 0, stream, p);
  else
    hipLaunchKernelGGL((adamw_kernel<P, G, false>), dim3(grid), dim3(kAdamT), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_adamw(const AdamParams& p, bool p_f32, bool g_f32, bool eight, int cu_count, hipStream_t stream) {
  const int chunks = p.first[p.count];
  if (chunks == 0) return hipSuccess;
  const int grid = chunks < cu_count * 8 ? chunks : cu_count * 8;
  if (p_f32) return g_f32 ? launch<float, float>(p, eight, grid, stream) : launch<float, uint16_t>(p, eight, grid, stream);
  return g_f32 ? launch<uint16_t, float>(p, eight, grid, stream) : launch<uint16_t, uint16_t>(p, eight, grid, stream);
}

}  // namespace gmmk
