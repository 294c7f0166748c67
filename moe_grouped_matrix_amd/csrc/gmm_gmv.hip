// gmm_gmv.hip -- products of a few tokens with their experts' four-bit
// weights, by expert id (gmm_layer.h, gmm_gmv_run).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gmm_device.hpp"
#include "gmm_layer_launch.hpp"

namespace gmmk {

namespace {

__device__ __forceinline__ int slot_expert(const GmvParams& p, int i) {
  if (!p.ids) return 0;
  const long long id = p.ids64 ? static_cast<const int64_t*>(p.ids)[i] : static_cast<const int32_t*>(p.ids)[i];
  return id >= 0 && id < p.G ? (int)id : -1;
}

__device__ __forceinline__ float block_scale(const GmvParams& p, const void* s, long long i) {
  if (p.scale_kind == kGmvF32) return static_cast<const float*>(s)[i];
  if (p.scale_kind == kGmvBf16) return bf16_bits_to_f32(static_cast<const uint16_t*>(s)[i]);
  const int byte = static_cast<const uint8_t*>(s)[i];
  return byte == 255 ? __builtin_nanf("") : __builtin_ldexpf(1.f, byte - 127);
}

// A wave per slot and column.
template <int F>
__global__ __launch_bounds__(256) void gmv_kernel(GmvParams p) {
  const int lane = threadIdx.x & 63, n = blockIdx.x * 4 + (threadIdx.x >> 6), i = blockIdx.y;
  if (n >= p.N) return;
  const int g = slot_expert(p, i);
  float sum = 0.f;
  if (g >= 0) {
    const unsigned* w = reinterpret_cast<const unsigned*>(p.rhs + ((long long)g * p.N + n) * (p.K / 2));
    const uint16_t* x = p.x + (long long)(p.per_slot ? i : i / p.k) * p.K;
    for (int c = lane; c < p.K / 8; c += 64) {
      const i32x4 v = nib8_to_bf16x8<F>(w[c]);
      const long long b = ((long long)g * p.nb + c * 8 / p.blk) * p.N + n;
      const float zero = p.zero ? block_scale(p, p.zero, b) : 0.f;
      float part = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        part += (bf16_bits_to_f32((uint16_t)((unsigned)v[e >> 1] >> (16 * (e & 1)))) - zero) * bf16_bits_to_f32(x[c * 8 + e]);
      sum += block_scale(p, p.scale, b) * part;
    }
  }
#pragma unroll
  for (int s = 1; s < 64; s *= 2) sum += __shfl_xor(sum, s, 64);
  if (lane == 0) {
    const long long o = (long long)i * p.N + n;
    if (p.weights)
      p.work[o] = sum;
    else if (p.out_f32)
      static_cast<float*>(p.out)[o] = sum;
    else
      static_cast<uint16_t*>(p.out)[o] = f32_to_bf16_rne(sum);
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
    const float w = p.w_f32 ? static_cast<const float*>(p.weights)[i]
                            : bf16_bits_to_f32(static_cast<const uint16_t*>(p.weights)[i]);
    sum += w * p.work[(long long)i * p.N + n];
  }
  const long long o = (long long)t * p.N + n;
  if (p.out_f32)
    static_cast<float*>(p.out)[o] = sum;
  else
    static_cast<uint16_t*>(p.out)[o] = f32_to_bf16_rne(sum);
}

}  // namespace

hipError_t launch_gmv(const GmvParams& p, int, hipStream_t stream) {
  const dim3 grid((p.N + 3) / 4, p.n);
  if (p.fmt == 3)
    hipLaunchKernelGGL(gmv_kernel<3>, grid, dim3(256), 0, stream, p);
  else if (p.fmt == 4)
    hipLaunchKernelGGL(gmv_kernel<4>, grid, dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL(gmv_kernel<5>, grid, dim3(256), 0, stream, p);
  if (p.weights) hipLaunchKernelGGL(gmv_join_kernel, dim3((p.N + 255) / 256, p.T), dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace gmmk
