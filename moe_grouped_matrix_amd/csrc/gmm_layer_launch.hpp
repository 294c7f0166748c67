// gmm_layer_launch.hpp -- arguments and launch entry points of the kernels
// behind gmm_layer.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gmm_params.hpp"

namespace gmmk {

// Queues a kernel; returns this launch's own status (hipGetLastError may hold an
// error that another call of the thread has left, which is not for us to take).
template <class... P>
hipError_t queue(void (*kernel)(P...), dim3 grid, dim3 block, size_t lds, hipStream_t stream, const P&... args) {
  void* at[] = {const_cast<P*>(&args)...};
  const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, block, at, lds, stream);
  if (e != hipSuccess) (void)hipGetLastError();  // (it is returned)
  return e;
}

constexpr int kRouterT = 256;    // threads of the choice and the gradient: four waves
constexpr int kBalanceT = 1024;  // of the balance loss: a thread an expert at its end
constexpr int kBalanceBlocks = 256;  // its most workgroups

// The router's tensors: T tokens, E experts, k choices.
struct RouterParams {
  const void* logits;    // [T,E] f32 or bf16
  const uint8_t* valid;  // [T] or nullptr
  const void* ids;       // [T,k] int32 or int64
  const float* bias;     // [E] or nullptr (choice)
  const void* dweights;  // [T,k] f32 or bf16, or nullptr (gradient)
  const int32_t* counts;  // [E] or nullptr (gradient)
  const int32_t* tokens;  // [1]
  const float* dloss;     // [1] or nullptr (1)
  int32_t* ids_out;       // [T,k]
  float* weights_out;     // [T,k]
  void* dlogits;          // [T,E], logits' type
  float* loss_out;        // [1]
  int32_t* counts_out;    // [E]
  int32_t* tokens_out;    // [1]
  float* work;            // balance loss: blocks * (2 E + 2) words
  long long T;
  int32_t E, k;
  int32_t x_f32, ids64, dw_f32, sigmoid, renorm;
  float scale, coef, z_coef;
};
hipError_t launch_route(const RouterParams& p, int cu_count, hipStream_t stream);
hipError_t launch_balance_loss(const RouterParams& p, int blocks, hipStream_t stream);
hipError_t launch_router_grad(const RouterParams& p, int cu_count, hipStream_t stream);

// Products by expert id: n = T*k slots, weights [G,N,K] in four bits with
// scales (and zero points) [G,nb,1,N].
enum GmvScale : int32_t { kGmvF32 = 0, kGmvBf16 = 1, kGmvE8m0 = 2 };
struct GmvParams {
  const uint16_t* x;    // [T,K] or, per_slot, [T,k,K]
  const uint8_t* rhs;   // [G,N,K/2]
  const void* scale;    // [G,nb,1,N]
  const void* zero;     // the same, or nullptr
  const void* ids;      // [T,k], or nullptr (all 0)
  const void* weights;  // [T,k] f32 or bf16, or nullptr
  void* out;            // [T,k,N], or with weights [T,N]
  float* work;          // [n,N] with weights
  int32_t T, k, n, G, N, K, nb, blk;
  int32_t fmt;  // 3 int4, 4 uint4, 5 fp4 e2m1
  int32_t scale_kind, ids64, w_f32, out_f32, per_slot;
  int32_t experts;     // workgroups' experts: the r-th of those chosen, r < experts, or (experts = G) every one
  uint32_t blk_magic;  // block b of 32 elements lies in scale block b * blk_magic >> 31
  int32_t at_once;     // the weighted sums are taken in one launch, without the workspace
};
// For scale blocks of d * 32 elements: ceil(2^31 / d), exact for b d < 2^31.
inline uint32_t gmv_magic(int blk) {
  const uint64_t d = (uint64_t)blk / 32;
  return (uint32_t)(((1ull << 31) + d - 1) / d);
}
hipError_t launch_gmv(const GmvParams& p, int cu_count, hipStream_t stream);

// AdamW: up to kAdamItems tensors a launch, cut into chunks.
constexpr int kAdamItems = 48;
constexpr int kAdamBlock = 256;   // elements that share a scale
constexpr int kAdamChunk = 2048;  // elements of a workgroup
constexpr long long kAdamMost = 1 << 23;  // chunks of a launch
constexpr long long kAdamCached = 96 << 20;  // a step that reads more streams past the caches
struct AdamItem {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  uint16_t* copy;
  long long n;
};
struct AdamParams {
  AdamItem item[kAdamItems];
  int32_t first[kAdamItems + 1];  // first chunk of each tensor
  int32_t count;
  // the factors of gmm_adamw_run, when step and rate are known to the host
  float decay, rate, root_scale;
  float b1, c1, b2, c2, eps;  // c = 1 - b
  // else: what they are made of
  double lr, beta1, beta2, weight_decay;
  long long step;
  const int32_t* step_at;
  const float* lr_at;
  const float* grad_scale;
};
static_assert(sizeof(AdamParams) <= 4096, "kernel arguments");
hipError_t launch_adamw(const AdamParams& p, bool p_f32, bool g_f32, bool eight, bool stream_loads, hipStream_t stream);

struct AdamFactors {
  float decay, rate, root_scale;
};

// The factors of a step, in double and rounded once (the same on the host and
// on the device: powers by squaring).
__host__ __device__ inline AdamFactors adam_factors(double lr, double beta1, double beta2, double weight_decay,
                                                    long long step) {
  double p1 = 1, p2 = 1;
  for (long long s = step < 1 ? 1 : step; s; s >>= 1) {
    if (s & 1) {
      p1 *= beta1;
      p2 *= beta2;
    }
    beta1 *= beta1;
    beta2 *= beta2;
  }
  return {(float)(1 - lr * weight_decay), (float)(lr / (1 - p1)), (float)(1 / __builtin_sqrt(1 - p2))};
}

}  // namespace gmmk
