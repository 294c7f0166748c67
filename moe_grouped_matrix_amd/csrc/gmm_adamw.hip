// gmm_adamw.hip -- the AdamW step of many tensors (gmm_layer.h,
// gmm_adamw_run), with states in fp32 or in eight bits.
//
// A launch takes up to kAdamItems tensors, whose addresses travel in its
// arguments (nothing is copied to the device first, so a step can be captured
// and its tensors may change from call to call).  A workgroup takes 2048
// elements of one, a wave two blocks of 256, four consecutive elements a lane,
// so that a block's largest state is one reduction over the wave, in registers.
//
// It is bound by HBM: 128 x 1408 x (1408 + 704) weights in fp32 with bf16
// gradients and copies and eight-bit states (16 bytes each, 6.1 GB) take 1050 to
// 1110 us (5.8 to 5.5 TB/s, card to card), where a copy reaches 5.1 TB/s; where
// they took 1110, in chunks of 4096 elements 1165, of 8192 1192, in a grid of
// eight workgroups a CU that takes chunk after chunk 1290, with one block of a
// wave in flight there 1300, and with a division for every code and reductions
// through LDS 1500.  Loads past the caches help a large step (1165 against 1258
// us; 12 bytes of state and gradient of 15.9M weights 76 against 88) and hurt one
// that the last-level cache holds (4M weights: 24 against 19, 120 tensors of 4.4M
// weights: 34 against 27; about even from 64 to 128 MB read), hence kAdamCached.
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
static_assert(kAdamMost * kAdamT < (1ll << 32), "a launch has fewer than 2^32 threads");

typedef short short2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef unsigned u32x2_t __attribute__((ext_vector_type(2)));

// Every value is read and written once.  A large step's loads go past the caches
// (STREAM), a small one's may find what ran before it there; stores always do.
template <bool STREAM, class T>
__device__ __forceinline__ T load_as(const void* p) {
  if constexpr (STREAM) return __builtin_nontemporal_load(static_cast<const T*>(p));
  return *static_cast<const T*>(p);
}
template <bool STREAM>
__device__ __forceinline__ f32x4 load4(const float* p) {
  return load_as<STREAM, f32x4>(p);
}
template <bool STREAM>
__device__ __forceinline__ f32x4 load4(const uint16_t* p) {
  const i32x2 w = load_as<STREAM, i32x2>(p);
  return f32x4{__int_as_float(w[0] << 16), __int_as_float(w[0] & (int)0xFFFF0000), __int_as_float(w[1] << 16),
               __int_as_float(w[1] & (int)0xFFFF0000)};
}
__device__ __forceinline__ void store4(float* p, f32x4 v) { __builtin_nontemporal_store(v, reinterpret_cast<f32x4*>(p)); }
__device__ __forceinline__ void store4(uint16_t* p, f32x4 v) {
  const i32x2 w{(int)pk_bf16_rne(v[0], v[1]), (int)pk_bf16_rne(v[2], v[3])};
  __builtin_nontemporal_store(w, reinterpret_cast<i32x2*>(p));
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_bits_to_f32(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = f32_to_bf16_rne(v); }

// Elements [0, n) of the lane's four: all of them, or (FULL false) as many as
// the tensor has left.
template <bool FULL, bool STREAM, class E>
__device__ __forceinline__ f32x4 load_some(const E* p, int n) {
  if (FULL || n >= 4) return load4<STREAM>(p);
  f32x4 v{0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < 3; ++i)
    if (i < n) v[i] = load1(p + i);
  return v;
}
template <bool FULL, class E>
__device__ __forceinline__ void store_some(E* p, f32x4 v, int n) {
  if (FULL || n >= 4) return store4(p, v);
  for (int i = 0; i < 3; ++i)
    if (i < n) store1(p + i, v[i]);
}
template <bool FULL, bool STREAM>
__device__ __forceinline__ unsigned load_codes(const uint8_t* p, int n) {
  if (FULL || n >= 4) return load_as<STREAM, unsigned>(p);
  unsigned w = 0;
  for (int i = 0; i < 3; ++i)
    if (i < n) w |= (unsigned)p[i] << (8 * i);
  return w;
}
template <bool FULL>
__device__ __forceinline__ void store_codes(uint8_t* p, unsigned w, int n) {
  if (FULL || n >= 4) return __builtin_nontemporal_store(w, reinterpret_cast<unsigned*>(p));
  for (int i = 0; i < 3; ++i)
    if (i < n) p[i] = (uint8_t)(w >> (8 * i));
}

__device__ __forceinline__ f32x4 widen_codes(unsigned w, float scale) {
  const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  return f32x4{lo[0] * scale, lo[1] * scale, hi[0] * scale, hi[1] * scale};
}

// The largest of the wave's values (bit patterns of non-negative floats), in
// every lane: within rows of 16 by permutations, then by swaps of rows and halves.
__device__ __forceinline__ unsigned wave_max(unsigned v) {
  v = max(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));   // quad_perm [1,0,3,2]
  v = max(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));   // quad_perm [2,3,0,1]
  v = max(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, true));  // row_half_mirror
  v = max(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, true));  // row_mirror
  const u32x2_t r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(r[0], r[1]);
  const u32x2_t h = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(h[0], h[1]);
}

// x / s correctly rounded, given y = 1/s correctly rounded, for a quotient that
// can decide a code (2^-11 and more; the remainder is exact then from s = 2^-92 on).
__device__ __forceinline__ float quotient(float x, float s, float y) {
#pragma clang fp contract(off)
  const float q0 = x * y;
  const float r = __builtin_fmaf(-q0, s, x);
  return __builtin_copysignf(__builtin_fmaf(r, y, q0), x);
}

// The wave's block x as e4m3 codes; returns the scale.
template <bool POSITIVE>
__device__ __forceinline__ float quantise(f32x4 x, unsigned& codes) {
#pragma clang fp contract(off)
  unsigned am = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) am = max(am, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  // (the same in every lane: a scalar, and the branches on it with it)
  am = (unsigned)__builtin_amdgcn_readfirstlane((int)wave_max(am));
  if (am >= 0x7F800000u) {
    codes = 0;
    return __builtin_nanf("");
  }
  const float amax = __uint_as_float(am);
  const float s = am == 0 ? 1.f : fmaxf(amax * (1.f / 448.f), 0x1p-126f);
  float t[4];
  if (s >= 0x1p-92f) {
    const float y = 1.f / s;
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = quotient(x[i], s, y);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = x[i] / s;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (POSITIVE) t[i] = x[i] > 0.f ? fmaxf(t[i], 0x1p-9f) : t[i];
    t[i] = fminf(fmaxf(t[i], -448.f), 448.f);
  }
  short2_t c = {0, 0};
  c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, t[0], t[1], 1.0f, false);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, t[2], t[3], 1.0f, true);
  codes = __builtin_bit_cast(unsigned, c);
  return s;
}

// A lane's four elements of one block.
struct Lane {
  f32x4 p, g, m, v;
  unsigned cm, cv;
  float ms, vs;
};

template <class P, class G, bool EIGHT, bool FULL, bool STREAM>
__device__ __forceinline__ void load_block(Lane& x, const AdamItem& t, long long at, long long i, int n) {
  x.p = load_some<FULL, STREAM>(static_cast<const P*>(t.p) + i, n);
  x.g = load_some<FULL, STREAM>(static_cast<const G*>(t.g) + i, n);
  if constexpr (EIGHT) {
    x.cm = load_codes<FULL, STREAM>(static_cast<const uint8_t*>(t.m) + i, n);
    x.cv = load_codes<FULL, STREAM>(static_cast<const uint8_t*>(t.v) + i, n);
    x.ms = t.ms[at / kAdamBlock];
    x.vs = t.vs[at / kAdamBlock];
  } else {
    x.m = load_some<FULL, STREAM>(static_cast<const float*>(t.m) + i, n);
    x.v = load_some<FULL, STREAM>(static_cast<const float*>(t.v) + i, n);
  }
}

template <class P, class G, bool EIGHT, bool FULL>
__device__ __forceinline__ void step_block(Lane& x, const AdamParams& a, const AdamFactors& f, float gscale, const AdamItem& t,
                                           long long at, long long i, int n) {
#pragma clang fp contract(off)
  if constexpr (EIGHT) {
    x.m = widen_codes(x.cm, x.ms);
    x.v = widen_codes(x.cv, x.vs);
  }
  f32x4 root;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float g = a.grad_scale ? x.g[e] * gscale : x.g[e];
    const float v0 = EIGHT ? x.v[e] * x.v[e] : x.v[e];
    x.m[e] = x.m[e] * a.b1 + g * a.c1;
    x.v[e] = v0 * a.b2 + (g * g) * a.c2;
    root[e] = __builtin_sqrtf(x.v[e]);
    x.p[e] = x.p[e] * f.decay - f.rate * (x.m[e] / (root[e] * f.root_scale + a.eps));
  }
  store_some<FULL>(static_cast<P*>(t.p) + i, x.p, n);
  if (t.copy) store_some<FULL>(t.copy + i, x.p, n);
  if constexpr (EIGHT) {
    if constexpr (!FULL) {  // (elements past the end count for nothing)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e >= n) x.m[e] = root[e] = 0.f;
    }
    unsigned cm, cv;
    const float sm = quantise<false>(x.m, cm), sv = quantise<true>(root, cv);
    store_codes<FULL>(static_cast<uint8_t*>(t.m) + i, cm, n);
    store_codes<FULL>(static_cast<uint8_t*>(t.v) + i, cv, n);
    if ((threadIdx.x & 63) == 0) {
      t.ms[at / kAdamBlock] = sm;
      t.vs[at / kAdamBlock] = sv;
    }
  } else {
    store_some<FULL>(static_cast<float*>(t.m) + i, x.m, n);
    store_some<FULL>(static_cast<float*>(t.v) + i, x.v, n);
  }
}

template <class P, class G, bool EIGHT, bool STREAM>
__global__ __launch_bounds__(kAdamT) void adamw_kernel(AdamParams a) {
  constexpr int U = kAdamChunk / kAdamT / 4;  // blocks of a wave, all in flight together
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = blockIdx.x;
  int at = 0, hi = a.count;  // the chunk's tensor: the last one whose first chunk is not behind c
  while (hi - at > 1) {
    const int mid = (at + hi) / 2;
    if (a.first[mid] <= c)
      at = mid;
    else
      hi = mid;
  }
  const AdamItem& t = a.item[at];
  const long long base = (long long)(c - a.first[at]) * kAdamChunk + w * U * kAdamBlock;
  if (base >= t.n) return;
  const bool full = base + U * kAdamBlock <= t.n;
  Lane x[U];
  if (full) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long first = base + u * kAdamBlock;
      load_block<P, G, EIGHT, true, STREAM>(x[u], t, first, first + lane * 4, 4);
    }
  }
  AdamFactors f{a.decay, a.rate, a.root_scale};
  if (a.step_at || a.lr_at)  // (worked out while the loads are on their way)
    f = adam_factors(a.lr_at ? (double)a.lr_at[0] : a.lr, a.beta1, a.beta2, a.weight_decay,
                     a.step_at ? (long long)a.step_at[0] : a.step);
  const float gscale = a.grad_scale ? a.grad_scale[0] : 1.f;
  if (full) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long first = base + u * kAdamBlock;
      step_block<P, G, EIGHT, true>(x[u], a, f, gscale, t, first, first + lane * 4, 4);
    }
    return;
  }
  for (int u = 0; u < U; ++u) {
    const long long first = base + u * kAdamBlock, i = first + lane * 4;
    if (first >= t.n) break;
    const int n = (int)(t.n - i < 4 ? t.n - i : 4);  // (may be negative)
    load_block<P, G, EIGHT, false, STREAM>(x[0], t, first, i, n);
    step_block<P, G, EIGHT, false>(x[0], a, f, gscale, t, first, i, n);
  }
}

template <class P, class G>
hipError_t launch(const AdamParams& p, bool eight, bool stream_loads, hipStream_t stream) {
  const dim3 grid(p.first[p.count]), block(kAdamT);
  if (eight && stream_loads) return queue(adamw_kernel<P, G, true, true>, grid, block, 0, stream, p);
  if (eight) return queue(adamw_kernel<P, G, true, false>, grid, block, 0, stream, p);
  if (stream_loads) return queue(adamw_kernel<P, G, false, true>, grid, block, 0, stream, p);
  return queue(adamw_kernel<P, G, false, false>, grid, block, 0, stream, p);
}

}  // namespace

hipError_t launch_adamw(const AdamParams& p, bool p_f32, bool g_f32, bool eight, bool stream_loads, hipStream_t s) {
  if (p_f32) return g_f32 ? launch<float, float>(p, eight, stream_loads, s) : launch<float, uint16_t>(p, eight, stream_loads, s);
  return g_f32 ? launch<uint16_t, float>(p, eight, stream_loads, s) : launch<uint16_t, uint16_t>(p, eight, stream_loads, s);
}

}  // namespace gmmk
