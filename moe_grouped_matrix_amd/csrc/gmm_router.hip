// gmm_router.hip -- the router of a mixture-of-experts layer on gfx950: the
// choice of k experts and their weights, the balance loss with per-expert
// counts, and the gradient of both.  Layouts and meanings are those of
// gmm_layer.h.
//
// All three kernels give a token a group of L lanes (a DPP row of 16 or the
// whole wave), lane l of which holds experts l + L v, so that a group's loads
// are coalesced whatever E's alignment is and a token's sums and maxima stay
// in registers.  Everything is fp32.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gmm_device.hpp"
#include "gmm_layer_launch.hpp"

namespace gmmk {

namespace {

constexpr float kInf = __builtin_inff();
constexpr float kNan = __builtin_nanf("");

template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_update_dpp(v, v, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(dpp<CTRL>(__float_as_int(v)));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const long long b = __double_as_longlong(v);
  const unsigned lo = (unsigned)dpp<CTRL>((int)b), hi = (unsigned)dpp<CTRL>((int)(b >> 32));
  return __longlong_as_double((long long)(((unsigned long long)hi << 32) | lo));
}

// op over the L lanes of a group; every lane gets the same bits (each step
// pairs lanes that hold the same two values).
template <int L, class T, class Op>
__device__ __forceinline__ T reduce(T v, Op op) {
  v = op(v, dpp<0xB1>(v));   // quad_perm [1,0,3,2]
  v = op(v, dpp<0x4E>(v));   // quad_perm [2,3,0,1]
  v = op(v, dpp<0x141>(v));  // row_half_mirror
  v = op(v, dpp<0x140>(v));  // row_mirror
  if constexpr (L == 64) {
    v = op(v, __shfl_xor(v, 16, 64));
    v = op(v, __shfl_xor(v, 32, 64));
  }
  return v;
}
template <int L, class T>
__device__ __forceinline__ T group_sum(T v) {
  return reduce<L>(v, [](T a, T b) { return a + b; });
}
template <int L>
__device__ __forceinline__ float group_max(float v) {
  return reduce<L>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int L>
__device__ __forceinline__ double group_max(double v) {
  return reduce<L>(v, [](double a, double b) { return __builtin_fmax(a, b); });
}
template <int L>
__device__ __forceinline__ bool group_any(bool b) {
  const unsigned long long m = __ballot(b);
  if constexpr (L == 64) return m != 0;
  return ((m >> (threadIdx.x & 48)) & 0xFFFF) != 0;
}

__device__ __forceinline__ float load_value(const void* p, long long i, bool f32) {
  return f32 ? static_cast<const float*>(p)[i] : bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
}

__device__ __forceinline__ float sigmoid(float z) { return 1.f / (1.f + expf(-z)); }

// A token's logits over its lanes (-inf where there is no expert).
template <int V>
struct Row {
  float z[V];
  float top;    // the largest
  bool counts;  // valid, and not every expert is switched off
  bool bad;     // counts, and holds a NaN or +inf
};

template <int L, int V>
__device__ __forceinline__ Row<V> load_row(const RouterParams& p, long long t, int l) {
  Row<V> r;
  const bool valid = t < p.T && (!p.valid || p.valid[t] != 0);
  float top = -kInf;
  bool bad = false;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = l + L * v;
    r.z[v] = valid && e < p.E ? load_value(p.logits, t * p.E + e, p.x_f32) : -kInf;
    top = fmaxf(top, r.z[v]);
    bad |= !(r.z[v] < kInf);
  }
  r.top = group_max<L>(top);
  r.bad = group_any<L>(bad);
  r.counts = r.bad || r.top > -kInf;
  return r;
}

// ---------------------------------------------------------------------------
// The choice.  A value and its expert make one double: the fp32 value leaves
// its low 29 bits zero, and ten of them take the id, so that of equal values
// the lower id is the larger key (for negative values larger bits are smaller
// keys), every key is another, and one maximum finds both.

__device__ __forceinline__ double choice_key(float value, int e) {
  const float x = value + 0.f;  // (-0 ranks as +0)
  if (!(x > -kInf)) return -__builtin_inf();
  const unsigned tag = x < 0.f ? (unsigned)e : 1023u - (unsigned)e;
  return __longlong_as_double(__double_as_longlong((double)x) | tag);
}
__device__ __forceinline__ int key_expert(double key) {
  const int tag = (int)(__double_as_longlong(key) & 1023);
  return key < 0 ? tag : 1023 - tag;
}

template <int L, int V>
__global__ __launch_bounds__(kRouterT) void route_kernel(RouterParams p) {
  constexpr int R = 64 / L;
  const int l = threadIdx.x & (L - 1), r = (threadIdx.x & 63) / L, w = threadIdx.x >> 6;
  constexpr int W = kRouterT / 64;
  for (long long t0 = (long long)blockIdx.x * (W * R); t0 < p.T; t0 += (long long)gridDim.x * (W * R)) {
    const long long t = t0 + w * R + r;
    Row<V> x = load_row<L, V>(p, t, l);
    float sum = 0.f;  // of the softmax, relative to the largest logit
    if (!p.sigmoid && (p.bias || !p.renorm)) {
#pragma unroll
      for (int v = 0; v < V; ++v) sum += x.counts ? expf(x.z[v] - x.top) : 0.f;
      sum = group_sum<L>(sum);
    }
    double key[V];
    bool bad = x.bad;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = l + L * v;
      float rank = x.z[v];
      if (p.bias && rank > -kInf && e < p.E) {
        rank = (p.sigmoid ? sigmoid(rank) : expf(rank - x.top) / sum) + p.bias[e];
        bad |= !(rank < kInf);
      }
      key[v] = choice_key(rank, e);
    }
    if (p.bias) bad = group_any<L>(bad);
    // round by round; lane j keeps the j-th choice
    double mine = -__builtin_inf();
    for (int j = 0; j < p.k; ++j) {
      double best = key[0];
#pragma unroll
      for (int v = 1; v < V; ++v) best = __builtin_fmax(best, key[v]);
      best = group_max<L>(best);
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = key[v] == best ? -__builtin_inf() : key[v];
      if (l == j) mine = best;
    }
    const bool there = mine > -__builtin_inf() && !bad;
    const int id = there ? key_expert(mine) : -1;
    float s = 0.f;
    if (there) s = load_value(p.logits, t * p.E + id, p.x_f32);
    if (p.sigmoid) {
      s = there ? sigmoid(s) : 0.f;
    } else {
      const float from = p.renorm ? group_max<L>(there ? s : -kInf) : x.top;
      s = there ? expf(s - from) : 0.f;
      if (!p.renorm) s = s / sum;
    }
    if (p.renorm) {
      const float total = group_sum<L>(s);
      s = total > 0.f ? s / total : 0.f;
    }
    if (t < p.T && l < p.k) {
      p.ids_out[t * p.k + l] = id;
      p.weights_out[t * p.k + l] = bad ? kNan : there ? p.scale * s : 0.f;
    }
  }
}

// ---------------------------------------------------------------------------
// The balance loss: every workgroup's sums of p, counts of choices, sum of
// squared logsumexp and count of tokens, in a row of the workspace; a second
// launch adds the rows up in order.

template <int L, int V>
__global__ __launch_bounds__(kRouterT) void balance_partial_kernel(RouterParams p) {
  constexpr int R = 64 / L, W = kRouterT / 64;
  __shared__ int hist[kMaxGroups];
  __shared__ float part[W * R][L * V];
  __shared__ float zsum[W * R];
  __shared__ int nsum[W * R];
  const int l = threadIdx.x & (L - 1), r = (threadIdx.x & 63) / L, w = threadIdx.x >> 6;
  for (int e = threadIdx.x; e < p.E; e += kRouterT) hist[e] = 0;
  __syncthreads();
  float acc[V], z2 = 0.f;
  int n = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
  for (long long t0 = (long long)blockIdx.x * (W * R); t0 < p.T; t0 += (long long)gridDim.x * (W * R)) {
    const long long t = t0 + w * R + r;
    Row<V> x = load_row<L, V>(p, t, l);
    float e[V], sum = 0.f, ssum = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      e[v] = x.counts ? expf(x.z[v] - x.top) : 0.f;
      sum += e[v];
    }
    sum = group_sum<L>(sum);
    const float lse = x.bad ? kNan : x.top + logf(sum);
    if (p.sigmoid) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        e[v] = x.counts && x.z[v] > -kInf ? sigmoid(x.z[v]) : 0.f;
        ssum += e[v];
      }
      sum = group_sum<L>(ssum);
    }
    if (x.counts) {
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] += x.bad ? kNan : sum > 0.f ? e[v] / sum : 0.f;
      z2 += lse * lse;
      ++n;
    }
    if (t < p.T)
      for (int j = l; j < p.k; j += L) {
        const long long i = t * p.k + j;
        const long long id = p.ids64 ? static_cast<const int64_t*>(p.ids)[i] : static_cast<const int32_t*>(p.ids)[i];
        if (id >= 0 && id < p.E) atomicAdd(&hist[id], 1);
      }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) part[w * R + r][l + L * v] = acc[v];
  if (l == 0) {
    zsum[w * R + r] = z2;
    nsum[w * R + r] = n;
  }
  __syncthreads();
  float* const out = p.work + (long long)blockIdx.x * (2 * p.E + 2);
  for (int e = threadIdx.x; e < p.E; e += kRouterT) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < W * R; ++i) s += part[i][e];
    out[e] = s;
    reinterpret_cast<int*>(out)[p.E + e] = hist[e];
  }
  if (threadIdx.x == 0) {
    float s = 0.f;
    int c = 0;
    for (int i = 0; i < W * R; ++i) {
      s += zsum[i];
      c += nsum[i];
    }
    out[2 * p.E] = s;
    reinterpret_cast<int*>(out)[2 * p.E + 1] = c;
  }
}

__global__ __launch_bounds__(1024) void balance_final_kernel(RouterParams p, int blocks) {
  __shared__ double dot[1024], num[1024];
  __shared__ double z2;
  __shared__ int tokens;
  const int e = threadIdx.x, S = 2 * p.E + 2;
  double P = 0, c = 0;
  if (e < p.E) {
    long long count = 0;
    for (int b = 0; b < blocks; ++b) {
      P += p.work[(long long)b * S + e];
      count += reinterpret_cast<const int*>(p.work)[(long long)b * S + p.E + e];
    }
    c = (double)count;
    p.counts_out[e] = (int)count;
  }
  dot[e] = c * P;
  num[e] = c;
  if (e == 0) {
    double z = 0;
    int n = 0;
    for (int b = 0; b < blocks; ++b) {
      z += p.work[(long long)b * S + 2 * p.E];
      n += reinterpret_cast<const int*>(p.work)[(long long)b * S + 2 * p.E + 1];
    }
    z2 = z;
    tokens = n;
    p.tokens_out[0] = n;
  }
  __syncthreads();
  for (int s = 512; s > 0; s >>= 1) {
    if (e < s) {
      dot[e] += dot[e + s];
      num[e] += num[e + s];
    }
    __syncthreads();
  }
  if (e == 0) {
    const double n = tokens > 0 ? tokens : 1, all = num[0] > 0 ? num[0] : 1;
    p.loss_out[0] = (float)((double)p.coef * p.E * dot[0] / (all * n) + (double)p.z_coef * z2 / n);
  }
}

// ---------------------------------------------------------------------------
// The gradient.  With s the scores, p = s / sum s, a[e] = dloss coef E f[e] / n:
//   balance part   softmax: p (a - sum a p);  sigmoid: p (1 - s) (a - sum a p)
//   logit term     2 dloss z_coef / n * lse * softmax
//   weights part   of the chosen experts, with u_j = s_j ds_j:
//                  renormalised: u_j = scale q_j (g_j - sum_i q_i g_i), q_j = s_j / S
//                  else u_j = scale s_j g_j
//                  softmax: + u_j, and - s sum_j u_j for every expert where
//                  not renormalised (the sum is 0 there); sigmoid: + u_j (1 - s_j)

template <int L, int V>
__global__ __launch_bounds__(kRouterT) void router_grad_kernel(RouterParams p) {
  constexpr int R = 64 / L, W = kRouterT / 64;
  __shared__ float picked[W * R][L * V];
  const int l = threadIdx.x & (L - 1), r = (threadIdx.x & 63) / L, w = threadIdx.x >> 6;
  const int lane0 = (threadIdx.x & 63) & ~(L - 1);
  float* const mine = picked[w * R + r];
  float a[V], zfac = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    a[v] = 0.f;
    mine[l + L * v] = 0.f;
  }
  if (p.counts) {
    double c[V], all = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      c[v] = l + L * v < p.E ? (double)p.counts[l + L * v] : 0.0;
      all += c[v];
    }
    all = group_sum<L>(all);
    const int tokens = p.tokens[0];
    const double up = (p.dloss ? (double)p.dloss[0] : 1.0) / (tokens > 0 ? tokens : 1);
#pragma unroll
    for (int v = 0; v < V; ++v) a[v] = (float)(up * p.coef * p.E * c[v] / (all > 0 ? all : 1));
    zfac = (float)(2 * up * p.z_coef);
  }
  for (long long t0 = (long long)blockIdx.x * (W * R); t0 < p.T; t0 += (long long)gridDim.x * (W * R)) {
    const long long t = t0 + w * R + r;
    Row<V> x = load_row<L, V>(p, t, l);
    float soft[V], sum = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      soft[v] = x.counts ? expf(x.z[v] - x.top) : 0.f;
      sum += soft[v];
    }
    sum = group_sum<L>(sum);
    const float lse = x.top + logf(sum);
    float s[V], ssum = 0.f, about = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      soft[v] = x.counts ? soft[v] / sum : 0.f;
      s[v] = !p.sigmoid ? soft[v] : x.counts && x.z[v] > -kInf ? sigmoid(x.z[v]) : 0.f;
      ssum += s[v];
    }
    if (p.sigmoid) ssum = group_sum<L>(ssum);
    float pr[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      pr[v] = !p.sigmoid ? s[v] : ssum > 0.f ? s[v] / ssum : 0.f;
      about += a[v] * pr[v];
    }
    about = group_sum<L>(about);

    float off = 0.f;
    if (p.dweights) {
      // lane j takes slot j
      int id = -1;
      float g = 0.f, q = 0.f, z = -kInf;
      if (x.counts && l < p.k) {
        const long long i = t * p.k + l;
        const long long e = p.ids64 ? static_cast<const int64_t*>(p.ids)[i] : static_cast<const int32_t*>(p.ids)[i];
        if (e >= 0 && e < p.E) {
          id = (int)e;
          g = load_value(p.dweights, i, p.dw_f32);
          z = load_value(p.logits, t * p.E + id, p.x_f32);
        }
      }
      const bool there = z > -kInf;  // (an expert that is switched off has score 0)
      if (!there) g = 0.f;
      float not_q = 1.f;
      if (p.sigmoid) {
        q = there ? sigmoid(z) : 0.f;
        not_q = there ? sigmoid(-z) : 0.f;
      } else {
        const float from = p.renorm ? group_max<L>(z) : x.top;
        q = there ? expf(z - from) : 0.f;
        if (!p.renorm) q = there ? q / sum : 0.f;
      }
      if (p.renorm) {
        const float total = group_sum<L>(q);
        q = total > 0.f ? q / total : 0.f;
        g -= group_sum<L>(q * g);
      }
      float u = p.scale * q * g;
      if (!p.sigmoid && !p.renorm) off = group_sum<L>(u);
      u *= not_q;
      // slots of one expert are added up in their order, by the first of them
      float total = 0.f;
      bool first = there;
      for (int j = 0; j < p.k; ++j) {
        const int other = __shfl(id, lane0 + j, 64);
        const float uj = __shfl(u, lane0 + j, 64);
        if (other == id) {
          total += uj;
          first = first && j >= l;
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if (first) mine[id] = total;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = l + L * v;
      float d = pr[v] * (a[v] - about);
      if (p.sigmoid) d *= 1.f - s[v];
      if (p.counts) d += zfac * lse * soft[v];
      d -= off * soft[v];
      if (p.dweights) {
        d += mine[e];
        mine[e] = 0.f;
      }
      if (x.bad) d = kNan;
      if (!x.counts || x.z[v] == -kInf) d = 0.f;
      if (t < p.T && e < p.E) {
        if (p.x_f32)
          static_cast<float*>(p.dlogits)[t * p.E + e] = d;
        else
          static_cast<uint16_t*>(p.dlogits)[t * p.E + e] = f32_to_bf16_rne(d);
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// Lanes and values a lane for E experts and k choices (a choice needs a lane).
template <template <int, int> class F, class... A>
hipError_t by_size(int E, int k, A... a) {
  if (E <= 128 && k <= 16) {
    if (E <= 16) return F<16, 1>::run(a...);
    if (E <= 32) return F<16, 2>::run(a...);
    if (E <= 64) return F<16, 4>::run(a...);
    return F<16, 8>::run(a...);
  }
  if (E <= 128) return F<64, 2>::run(a...);
  if (E <= 256) return F<64, 4>::run(a...);
  if (E <= 512) return F<64, 8>::run(a...);
  return F<64, 16>::run(a...);
}

int row_grid(const RouterParams& p, int L, int cu_count) {
  const long long rows = (kRouterT / 64) * (64 / L);
  long long b = (p.T + rows - 1) / rows;
  const long long most = (long long)cu_count * 8;
  return (int)(b < 1 ? 1 : b > most ? most : b);
}

template <int L, int V>
struct Route {
  static hipError_t run(const RouterParams* p, int cus, hipStream_t s) {
    hipLaunchKernelGGL((route_kernel<L, V>), dim3(row_grid(*p, L, cus)), dim3(kRouterT), 0, s, *p);
    return hipGetLastError();
  }
};
template <int L, int V>
struct Balance {
  static hipError_t run(const RouterParams* p, int blocks, hipStream_t s) {
    hipLaunchKernelGGL((balance_partial_kernel<L, V>), dim3(blocks), dim3(kRouterT), 0, s, *p);
    return hipGetLastError();
  }
};
template <int L, int V>
struct Grad {
  static hipError_t run(const RouterParams* p, int cus, hipStream_t s) {
    hipLaunchKernelGGL((router_grad_kernel<L, V>), dim3(row_grid(*p, L, cus)), dim3(kRouterT), 0, s, *p);
    return hipGetLastError();
  }
};

}  // namespace

hipError_t launch_route(const RouterParams& p, int cu_count, hipStream_t stream) {
  return by_size<Route>(p.E, p.k, &p, cu_count, stream);
}

hipError_t launch_balance_loss(const RouterParams& p, int blocks, hipStream_t stream) {
  const hipError_t e = by_size<Balance>(p.E, p.k, &p, blocks, stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(balance_final_kernel, dim3(1), dim3(1024), 0, stream, p, blocks);
  return hipGetLastError();
}

hipError_t launch_router_grad(const RouterParams& p, int cu_count, hipStream_t stream) {
  return by_size<Grad>(p.E, p.k, &p, cu_count, stream);
}

}  // namespace gmmk
