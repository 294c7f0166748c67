// gmm_router.hip -- the router of a mixture-of-experts layer on gfx950: the
// choice of k experts and their weights, the balance loss with per-expert
// counts, and the gradient of both.  Layouts and meanings are those of
// gmm_layer.h.
//
// All three kernels give a token a group of L lanes (half a DPP row, a row, or
// the whole wave), lane l of which holds experts l + L v, so that a group's
// loads are coalesced whatever E's alignment is and a token's sums and maxima
// stay in registers.  Everything is fp32.
//
// 32768 tokens of 128 experts, k = 8 (16.8 MB of f32 logits; a copy of them, which
// moves twice that, takes 6.2 us): choice 7.1 us, loss 13.1, gradient 11.1.  The
// largest part of the choice and the gradient is the vector units' work, 84 and 98
// instructions a token (each issued in four cycles on one of 1024 SIMDs: 4.5 and
// 5.2 us at 2.4 GHz), and the loss is two dependent launches of 8 and 4 to 6 us.
// With a wave a token and fp32 functions of the library the three took 12, 109 and
// 17 us.
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
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);  // (every lane reads another)
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
  if constexpr (L >= 16) v = op(v, dpp<0x140>(v));  // row_mirror
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
  return ((m >> (threadIdx.x & 63 & ~(L - 1))) & ((1ull << (L & 63)) - 1)) != 0;
}

__device__ __forceinline__ float load_value(const void* p, long long i, bool f32) {
  return f32 ? static_cast<const float*>(p)[i] : bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
}

// e^x of an x that is at most 0 (or -inf), within 2 u of itself: 2^t by the
// exponential instruction (1 ulp), t = x log2 e rounded, times 1 + (what the
// rounding left) ln 2.  Below 2^-126 it gives 0.
__device__ __forceinline__ float exp_of(float x) {
  x = fmaxf(x, -160.f);  // (2^-230: 0; no infinity meets the fma)
  const float t = x * 0x1.715476p+0f;
  const float left = __builtin_fmaf(x, 0x1.4ae0cp-26f, __builtin_fmaf(x, 0x1.715476p+0f, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e, left * 0x1.62e43p-1f, e);
}

// The logarithm of a sum of exponentials of which one is 1, and reciprocals: the
// instructions' (1 ulp); no reciprocal of a sum of scores below 2^-126, which
// counts as 0.
__device__ __forceinline__ float log_of(float x) { return __builtin_amdgcn_logf(x) * 0x1.62e43p-1f; }
__device__ __forceinline__ float over_of(float x) { return __builtin_amdgcn_rcpf(x); }
__device__ __forceinline__ float over_scores(float sum) { return sum >= 0x1p-126f ? over_of(sum) : 0.f; }

// The sigmoids of z and of -z, each within a few u of itself.
__device__ __forceinline__ void sigmoids(float z, float& s, float& not_s) {
  const float e = exp_of(-fabsf(z)), r = over_of(1.f + e), er = e * r;
  s = z >= 0.f ? r : er;
  not_s = z >= 0.f ? er : r;
}
__device__ __forceinline__ float sigmoid(float z) {
  float s, n;
  sigmoids(z, s, n);
  return s;
}

// Choice j of token t, -1 where there is none.
__device__ __forceinline__ long long load_id(const RouterParams& p, long long t, int j) {
  if (t >= p.T || j >= p.k) return -1;
  const long long i = t * p.k + j;
  return p.ids64 ? static_cast<const int64_t*>(p.ids)[i] : static_cast<const int32_t*>(p.ids)[i];
}

// A token's logits over its lanes (-inf where there is no expert).
template <int V>
struct Row {
  float z[V];
  float top;    // the largest
  bool counts;  // valid, and not every expert is switched off
  bool bad;     // counts, and holds a NaN or +inf
};

// Asks for the logits; what is out of range is read elsewhere in the tensor
// (which must have a token) and put right by row_state, so that the loads need
// no branches.  FULL: E is L V, and a lane's experts are a constant apart; with
// other numbers the bounds cost instructions and registers (32768 tokens, choice
// and gradient: 96 experts 9.9 and 11.0 us, 128 7.4 and 11.6; 200 17.4 and 18.9,
// 256 11.9 and 16.9; the ordered lists of 16 values a lane spill 14 to 16 there).
template <int L, int V, bool FULL>
__device__ __forceinline__ bool load_row(Row<V>& r, const RouterParams& p, long long t, int l) {
  const long long row = (t < p.T ? t : p.T - 1) * p.E;
  const int last = p.E - 1;
  auto at = [&](int v) __attribute__((always_inline)) { return FULL || l + L * v < last ? l + L * v : last; };
  if (p.x_f32) {
    const float* const z = static_cast<const float*>(p.logits) + row;
#pragma unroll
    for (int v = 0; v < V; ++v) r.z[v] = z[at(v)];
  } else {
    const uint16_t* const z = static_cast<const uint16_t*>(p.logits) + row;
#pragma unroll
    for (int v = 0; v < V; ++v) r.z[v] = bf16_bits_to_f32(z[at(v)]);
  }
  return t < p.T && (!p.valid || p.valid[t] != 0);
}

// What the row is.  (The logits of padding stay what they are: nothing that
// comes of a token that does not count is kept.)
template <int L, int V, bool FULL>
__device__ __forceinline__ void row_state(Row<V>& r, const RouterParams& p, bool valid, int l) {
  float top = -kInf;
  // a NaN or +inf is the largest of the bit patterns as signed numbers, or, with
  // its sign set, as unsigned ones
  int high = 0;
  unsigned low = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if constexpr (!FULL) r.z[v] = l + L * v < p.E ? r.z[v] : -kInf;
    top = fmaxf(top, r.z[v]);
    high = max(high, __float_as_int(r.z[v]));
    low = max(low, __float_as_uint(r.z[v]));
  }
  r.top = group_max<L>(top);
  r.bad = group_any<L>(valid && (high >= 0x7F800000 || low > 0xFF800000u));
  r.counts = valid && (r.bad || r.top > -kInf);
}

// ---------------------------------------------------------------------------
// The choice.  A value and its expert make one double: the fp32 value leaves
// its low 29 bits zero, and ten of them take the id, so that of equal values
// the lower id is the larger key (for negative values larger bits are smaller
// keys), every key is another, and one maximum finds both.
//
// Up to eight choices (K8; 32768 x 128: 7.1 against 11.3 us), a lane first brings its values into order, eight at
// a time by a network of 19 exchanges (a maximum and a minimum each), lists of
// eight being merged to their eight largest; a round then looks at the heads of
// the lanes' lists alone, and the lane that held the best one moves its list
// up.  More choices, and few values a lane, look at every value in every round.

constexpr double kDead = -0x1p1000;  // of an expert that is switched off (its key has the id, too)

__device__ __forceinline__ double choice_key(float value, int e) {
  const float x = value + 0.f;  // (-0 ranks as +0)
  const unsigned tag = ~((unsigned)(__float_as_int(x) >> 31) ^ (unsigned)e) & 1023u;
  return __longlong_as_double(__double_as_longlong(__builtin_fmax((double)x, kDead)) | tag);
}
__device__ __forceinline__ bool alive(double key) { return key > 0.5 * kDead; }
__device__ __forceinline__ int key_expert(double key) {
  const int tag = (int)(__double_as_longlong(key) & 1023);
  return key < 0 ? tag : 1023 - tag;
}

__device__ __forceinline__ void exchange(double& a, double& b) {  // the larger first
  const double hi = __builtin_fmax(a, b);
  b = __builtin_fmin(a, b);
  a = hi;
}
// A bitonic list of eight into falling order.
__device__ __forceinline__ void order_bitonic(double* k) {
#pragma unroll
  for (int d = 4; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((i & d) == 0) exchange(k[i], k[i + d]);
}
// Eight keys into falling order (Batcher's odd-even merge sort).
__device__ __forceinline__ void order8(double* k) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) exchange(k[i], k[i + 1]);
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    exchange(k[i], k[i + 2]);
    exchange(k[i + 1], k[i + 3]);
    exchange(k[i + 1], k[i + 2]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) exchange(k[i], k[i + 4]);
  exchange(k[2], k[4]);
  exchange(k[3], k[5]);
  exchange(k[1], k[2]);
  exchange(k[3], k[4]);
  exchange(k[5], k[6]);
}

template <int L, int V, bool K8, bool FULL>
__global__ __launch_bounds__(kRouterT, 4) void route_kernel(RouterParams p) {
  constexpr int R = 64 / L;
  const int l = threadIdx.x & (L - 1), r = (threadIdx.x & 63) / L, w = threadIdx.x >> 6;
  constexpr int W = kRouterT / 64;
  for (long long t0 = (long long)blockIdx.x * (W * R); t0 < p.T; t0 += (long long)gridDim.x * (W * R)) {
    const long long t = t0 + w * R + r;
    Row<V> x;
    const bool valid = load_row<L, V, FULL>(x, p, t, l);
    row_state<L, V, FULL>(x, p, valid, l);
    float over_sum = 0.f;  // of the softmax, relative to the largest logit
    if (!p.sigmoid && (p.bias || !p.renorm)) {
      float sum = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) sum += exp_of(x.z[v] - x.top);
      over_sum = over_of(group_sum<L>(sum));
    }
    double key[V];
    bool bad = x.bad;
    if (p.bias) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = l + L * v;
        float rank = x.z[v];
        if (rank > -kInf && e < p.E) {
          rank = (p.sigmoid ? sigmoid(rank) : exp_of(rank - x.top) * over_sum) + p.bias[e];
          bad |= x.counts && !(rank < kInf);
        }
        key[v] = choice_key(rank, e);
      }
      bad = group_any<L>(bad);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = choice_key(x.z[v], l + L * v);
    }
    // lane j keeps the j-th choice
    double mine = kDead;
    if constexpr (K8) {
#pragma unroll
      for (int i = 0; i < V; i += 8) order8(key + i);
#pragma unroll
      for (int n = V / 8; n > 1; n /= 2)
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
#pragma unroll
          for (int j = 0; j < 8; ++j) key[8 * i + j] = __builtin_fmax(key[8 * i + j], key[8 * (i + n / 2) + 7 - j]);
          order_bitonic(key + 8 * i);
        }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j == p.k) break;
        const double best = group_max<L>(key[0]);
        mine = l == j ? best : mine;
        const bool won = key[0] == best;
#pragma unroll
        for (int i = 0; i < 7 - j; ++i) key[i] = won ? key[i + 1] : key[i];
      }
    } else {
      for (int j = 0; j < p.k; ++j) {
        double best = key[0];
#pragma unroll
        for (int v = 1; v < V; ++v) best = __builtin_fmax(best, key[v]);
        best = group_max<L>(best);
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = key[v] == best ? kDead : key[v];
        mine = l == j ? best : mine;
      }
    }
    const bool there = alive(mine) && x.counts && !bad;
    const int id = there ? key_expert(mine) : -1;
    float z = -kInf;
    if (!p.bias)
      z = there ? (float)__longlong_as_double(__double_as_longlong(mine) & ~1023ll) : -kInf;
    else if (there)
      z = load_value(p.logits, t * p.E + id, p.x_f32);
    float s;
    if (p.sigmoid) {
      s = there ? sigmoid(z) : 0.f;
    } else {
      const float from = p.renorm ? group_max<L>(z) : x.top;
      s = there ? exp_of(z - from) : 0.f;
      if (!p.renorm) s *= over_sum;
    }
    if (p.renorm) {
      const float total = group_sum<L>(s);
      s *= over_scores(total);
    }
    if (t < p.T && l < p.k) {
      p.ids_out[t * p.k + l] = id;
      p.weights_out[t * p.k + l] = bad ? kNan : there ? p.scale * s : 0.f;
    }
  }
}

// ---------------------------------------------------------------------------
// The balance loss: every workgroup's sums of p, counts of choices, sum of
// squared logsumexp and count of tokens, in the workspace (planes [blocks][E]
// of sums and of counts, then [blocks] of each of the others); a second launch
// adds them up in order.  One workgroup alone finishes by itself.  (Joining in
// one launch by the last workgroup to arrive would need a counter that is zero
// before the call.)

// loss, given thread e's sum of p and count of expert e (0 past the last).
__device__ __forceinline__ void finish_loss(const RouterParams& p, double P, long long count, double z2, int tokens) {
  __shared__ double dots[kBalanceT / 64], alls[kBalanceT / 64];
  double dot = (double)count * P, all = (double)count;
  dot = group_sum<64>(dot);
  all = group_sum<64>(all);
  if ((threadIdx.x & 63) == 0) {
    dots[threadIdx.x >> 6] = dot;
    alls[threadIdx.x >> 6] = all;
  }
  if ((int)threadIdx.x < p.E) p.counts_out[threadIdx.x] = (int)count;
  __syncthreads();
  if (threadIdx.x == 0) {
    dot = all = 0;
    for (int i = 0; i < kBalanceT / 64; ++i) {
      dot += dots[i];
      all += alls[i];
    }
    const double n = tokens > 0 ? tokens : 1;
    // (without the term its sum is not looked at: squares of far logits overflow)
    const double squares = p.z_coef != 0.f ? (double)p.z_coef * z2 / n : 0.0;
    p.loss_out[0] = (float)((double)p.coef * p.E * dot / ((all > 0 ? all : 1) * n) + squares);
    p.tokens_out[0] = tokens;
  }
}

template <int L, int V, bool FULL>
__global__ __launch_bounds__(kBalanceT) void balance_partial_kernel(RouterParams p) {
  constexpr int R = 64 / L, W = kBalanceT / 64;
  __shared__ int hist[kMaxGroups];
  __shared__ float part[W][L * V];
  __shared__ float zsum[W];
  __shared__ int nsum[W];
  const int l = threadIdx.x & (L - 1), r = (threadIdx.x & 63) / L, w = threadIdx.x >> 6;
  float acc[V], z2 = 0.f;
  int n = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
  // the next token is asked for before the present one is worked on
  const long long step = (long long)gridDim.x * (W * R);
  long long t = (long long)blockIdx.x * (W * R) + w * R + r;
  const long long end = p.T + w * R + r;
  Row<V> next;
  bool next_valid = false;
  if (p.T > 0) next_valid = load_row<L, V, FULL>(next, p, t, l);  // (there may be no token at all)
  long long id = load_id(p, t, l);
  if ((int)threadIdx.x < p.E) hist[threadIdx.x] = 0;
  __syncthreads();
  for (; t < end; t += step) {
    Row<V> x = next;
    const bool valid = next_valid;
    if (t + step < end) next_valid = load_row<L, V, FULL>(next, p, t + step, l);
    row_state<L, V, FULL>(x, p, valid, l);
    float e[V], sum = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      e[v] = exp_of(x.z[v] - x.top);
      sum += e[v];
    }
    sum = group_sum<L>(sum);
    const float lse = x.bad ? kNan : x.top + log_of(sum);
    if (p.sigmoid) {
      sum = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        e[v] = x.z[v] > -kInf ? sigmoid(x.z[v]) : 0.f;
        sum += e[v];
      }
      sum = group_sum<L>(sum);
    }
    if (x.counts) {
      const float over = x.bad ? kNan : over_scores(sum);
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = __builtin_fmaf(e[v], over, acc[v]);
      z2 = __builtin_fmaf(lse, lse, z2);
      ++n;
    }
    if (id >= 0 && id < p.E) atomicAdd(&hist[id], 1);
    for (int j = l + L; j < p.k; j += L) {
      id = load_id(p, t, j);
      if (id >= 0 && id < p.E) atomicAdd(&hist[id], 1);
    }
    id = load_id(p, t + step, l);
  }
  // the wave's groups (they hold the same experts), then the workgroup's waves
#pragma unroll
  for (int s = L; s < 64; s *= 2) {
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] += __shfl_xor(acc[v], s, 64);
    z2 += __shfl_xor(z2, s, 64);
    n += __shfl_xor(n, s, 64);
  }
  if (r == 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) part[w][l + L * v] = acc[v];
  }
  if ((threadIdx.x & 63) == 0) {
    zsum[w] = z2;
    nsum[w] = n;
  }
  __syncthreads();
  const int e = threadIdx.x, B = gridDim.x, b = blockIdx.x;
  float P = 0.f, z = 0.f;
  int c = 0;
  if (e < p.E)
#pragma unroll
    for (int i = 0; i < W; ++i) P += part[i][e];
  for (int i = 0; i < W; ++i) {
    z += zsum[i];
    c += nsum[i];
  }
  const int count = e < p.E ? hist[e] : 0;
  if (B == 1) return finish_loss(p, P, count, z, c);
  int* const counts = reinterpret_cast<int*>(p.work + (long long)B * p.E);
  float* const zs = p.work + 2ll * B * p.E;
  if (e < p.E) {
    p.work[(long long)b * p.E + e] = P;
    counts[(long long)b * p.E + e] = count;
  }
  if (e == 0) {
    zs[b] = z;
    reinterpret_cast<int*>(zs)[B + b] = c;
  }
}

// Thread (slice, e) adds up every n-th workgroup's row from `slice` on; U rows
// of both planes are in flight together.
template <int U>
__global__ __launch_bounds__(kBalanceT) void balance_final_kernel(RouterParams p, int B, int slices) {
  __shared__ double sums[kBalanceT];
  __shared__ int counts[kBalanceT];
  __shared__ double zs[kBalanceBlocks / 64];
  __shared__ int ns[kBalanceBlocks / 64];
  const int width = kBalanceT / slices, e = threadIdx.x % width, s = threadIdx.x / width;
  const int* const cplane = reinterpret_cast<const int*>(p.work + (long long)B * p.E);
  const float* const zplane = p.work + 2ll * B * p.E;
  float z = 0.f;
  int n = 0;
  if ((int)threadIdx.x < B) {
    z = zplane[threadIdx.x];
    n = reinterpret_cast<const int*>(zplane)[B + threadIdx.x];
  }
  double P = 0;
  int count = 0;
  if (e < p.E)
    for (int b0 = s; b0 < B; b0 += U * slices) {
      float f[U];
      int c[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int b = b0 + u * slices < B ? b0 + u * slices : B - 1;
        f[u] = p.work[(long long)b * p.E + e];
        c[u] = cplane[(long long)b * p.E + e];
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (b0 + u * slices < B) {
          P += f[u];
          count += c[u];
        }
    }
  sums[threadIdx.x] = P;
  counts[threadIdx.x] = count;
  if (threadIdx.x < kBalanceBlocks) {  // (whole waves)
    const double z64 = group_sum<64>((double)z);
    n = group_sum<64>(n);
    if ((threadIdx.x & 63) == 0) {
      zs[threadIdx.x >> 6] = z64;
      ns[threadIdx.x >> 6] = n;
    }
  }
  __syncthreads();
  double total = 0, z2 = 0;
  int all = 0;
  n = 0;
  if ((int)threadIdx.x < p.E)
    for (int i = 0; i < slices; ++i) {
      total += sums[i * width + threadIdx.x];
      all += counts[i * width + threadIdx.x];
    }
#pragma unroll
  for (int i = 0; i < kBalanceBlocks / 64; ++i) {
    z2 += zs[i];
    n += ns[i];
  }
  finish_loss(p, total, all, z2, n);
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
// The u_j go to their experts' lanes through a row of LDS a group.

template <int L, int V, bool SIGMOID, bool FULL>
__global__ __launch_bounds__(kRouterT) void router_grad_kernel(RouterParams p) {
  constexpr int R = 64 / L, W = kRouterT / 64;
  __shared__ float picked[W * R][L * V];
  const int l = threadIdx.x & (L - 1), r = (threadIdx.x & 63) / L, w = threadIdx.x >> 6;
  const int lane0 = (threadIdx.x & 63) & ~(L - 1);
  float* const mine = picked[w * R + r];
  const long long step = (long long)gridDim.x * (W * R);
  long long t = (long long)blockIdx.x * (W * R) + w * R + r;
  const long long end = p.T + w * R + r;
  // A token's logits, and lane j's slot j; the next token's are asked for
  // before the present one is worked on.
  Row<V> next;
  bool next_valid = load_row<L, V, FULL>(next, p, t, l);
  long long next_id = -1;
  float next_g = 0.f;
  auto load_slot = [&](long long t1) __attribute__((always_inline)) {
    next_id = load_id(p, t1, l);
    if (next_id >= 0 && next_id < p.E)
      next_g = load_value(p.dweights, t1 * p.k + l, p.dw_f32);
    else
      next_id = -1;
  };
  if (p.dweights) load_slot(t);
  float a[V], zfac = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) a[v] = 0.f;
  if (p.counts) {
    int c[V];
    double all = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] = p.counts[l + L * v < p.E ? l + L * v : p.E - 1];
    const int tokens = p.tokens[0];
    const float up = p.dloss ? p.dloss[0] : 1.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (l + L * v >= p.E) c[v] = 0;
      all += c[v];
    }
    all = group_sum<L>(all);
    const double n = tokens > 0 ? tokens : 1, per = (double)up * p.coef * p.E / ((all > 0 ? all : 1) * n);
#pragma unroll
    for (int v = 0; v < V; ++v) a[v] = (float)(per * c[v]);
    zfac = 2.f * up * p.z_coef / (float)n;
  }
  for (; t < end; t += step) {
    Row<V> x = next;
    const bool valid = next_valid;
    const int id = (int)next_id;
    float g = next_g;
    if (t + step < end) {
      next_valid = load_row<L, V, FULL>(next, p, t + step, l);
      if (p.dweights) load_slot(t + step);
    }
    row_state<L, V, FULL>(x, p, valid, l);
    float z = -kInf;
    if (p.dweights) {  // the chosen logits, from their lanes
#pragma unroll
      for (int v = 0; v < V; ++v) mine[l + L * v] = x.z[v];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if (id >= 0) z = mine[id];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int v = 0; v < V; ++v) mine[l + L * v] = 0.f;
    }
    float slope[V], soft[V], sum = 0.f, about = 0.f;  // slope: s (1 - s), 1 - s being the sigmoid of -z in full precision
#pragma unroll
    for (int v = 0; v < V; ++v) {
      soft[v] = exp_of(x.z[v] - x.top);
      sum += soft[v];
    }
    sum = group_sum<L>(sum);
    const float over_sum = over_of(sum), lse = x.top + log_of(sum);
    float over = over_sum;  // of the sum of the scores
    if constexpr (SIGMOID) {
      float ssum = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float e = exp_of(-fabsf(x.z[v])), r = over_of(1.f + e);  // sigmoids are r and e r (1 and 0 of -inf)
        const float score = x.z[v] >= 0.f ? r : e * r;
        slope[v] = e * r * r;
        asm("" : "+v"(slope[v]));  // (worked out here: two values for each, r and e r, would be kept for later)
        ssum += score;
        about = __builtin_fmaf(a[v], score, about);
      }
      ssum = group_sum<L>(ssum);
      over = over_scores(ssum);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) about = __builtin_fmaf(a[v], soft[v], about);
    }
    about = group_sum<L>(about) * over;

    float off = 0.f;
    if (p.dweights) {
      const bool there = x.counts && z > -kInf;  // (an expert that is switched off has score 0)
      if (!there) g = 0.f;
      float q, not_q = 1.f;
      if constexpr (SIGMOID) {
        sigmoids(z, q, not_q);
        if (!there) q = 0.f;
      } else {
        const float from = p.renorm ? group_max<L>(z) : x.top;
        q = there ? exp_of(z - from) : 0.f;
        if (!p.renorm) q *= over_sum;
      }
      if (p.renorm) {
        const float total = group_sum<L>(q);
        q *= over_scores(total);
        g -= group_sum<L>(q * g);
      }
      float u = p.scale * q * g;
      if (!SIGMOID && !p.renorm) off = group_sum<L>(u);
      u *= not_q;
      // Every slot leaves its lane at its expert; where another lane's stands
      // afterwards, slots of one expert meet, and are added up in their order
      // by the first of them.
      int* const owner = reinterpret_cast<int*>(mine);
      bool first = there;
      if (there) owner[id] = l;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      const bool lost = there && owner[id] != l;
      if (__ballot(lost) != 0) {
        float total = 0.f;
        for (int j = 0; j < p.k; ++j) {
          const int other = __shfl(id, lane0 + j, 64);
          const float uj = __shfl(u, lane0 + j, 64);
          if (other == id) {
            total += uj;
            first = first && j >= l;
          }
        }
        u = total;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if (first) mine[id] = u;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    float d[V];
    const float c = p.counts ? zfac * lse : 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if constexpr (SIGMOID)
        d[v] = slope[v] * over * (a[v] - about) + soft[v] * over_sum * c;
      else
        d[v] = soft[v] * over_sum * (a[v] - about - off + c);
      if (p.dweights) d[v] += mine[l + L * v];
      if (x.z[v] == -kInf) d[v] = 0.f;
    }
    if (__ballot(x.bad || !x.counts) != 0) {
#pragma unroll
      for (int v = 0; v < V; ++v) d[v] = x.bad ? kNan : x.counts ? d[v] : 0.f;
    }
    if (t < p.T) {
      if (p.x_f32) {
        float* const out = static_cast<float*>(p.dlogits) + t * p.E;
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (FULL || l + L * v < p.E) out[l + L * v] = d[v];
      } else {
        uint16_t* const out = static_cast<uint16_t*>(p.dlogits) + t * p.E;
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (FULL || l + L * v < p.E) out[l + L * v] = f32_to_bf16_rne(d[v]);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

int row_grid(const RouterParams& p, int L, int cu_count, int per_cu) {
  const long long rows = (kRouterT / 64) * (64 / L);
  long long b = (p.T + rows - 1) / rows;
  const long long most = (long long)cu_count * per_cu;
  return (int)(b < 1 ? 1 : b > most ? most : b);
}

template <int L, int V, bool K8>
hipError_t route(const RouterParams& p, int cus, hipStream_t s) {
  const dim3 grid(row_grid(p, L, cus, 8)), block(kRouterT);
  return queue(p.E == L * V ? route_kernel<L, V, K8, true> : route_kernel<L, V, K8, false>, grid, block, 0, s, p);
}
template <int L, int V>
hipError_t balance(const RouterParams& p, int blocks, hipStream_t s) {
  return queue(p.E == L * V ? balance_partial_kernel<L, V, true> : balance_partial_kernel<L, V, false>, dim3(blocks),
               dim3(kBalanceT), 0, s, p);
}
template <int L, int V, bool SIGMOID>
hipError_t grad_of(const RouterParams& p, int cus, hipStream_t s) {
  const dim3 grid(row_grid(p, L, cus, 4)), block(kRouterT);
  return queue(p.E == L * V ? router_grad_kernel<L, V, SIGMOID, true> : router_grad_kernel<L, V, SIGMOID, false>, grid,
               block, 0, s, p);
}
template <int L, int V>
hipError_t grad(const RouterParams& p, int cus, hipStream_t s) {
  return p.sigmoid ? grad_of<L, V, true>(p, cus, s) : grad_of<L, V, false>(p, cus, s);
}

}  // namespace

// Lanes a token: as few as keep a token's values in registers, since the rounds
// and reductions cost the same for 8 tokens a wave as for one.  32768 tokens, k =
// 8, in us, with 8, 16 and 64 lanes: 64 experts 5.5, 9.1, 32; 128: 7.7, 9.4, 32;
// 256: 20.5, 12.4, 32; 512 with 16 and 64: 57, 31.  A few tokens of 128 take 3.0 us
// with 16 lanes and 3.3 with 8 (4096: 3.5 and 3.85, 8192: 4.0 and 3.9).  k = 10 and
// 16: 12.6 and 17.2 us for 128 experts, 33.5 and 47.2 for 256; k = 8 with a bias:
// 11.3 and 18.9.
hipError_t launch_route(const RouterParams& p, int cus, hipStream_t s) {
  const int E = p.E;
  if (p.k <= 8) {
    if (E <= 64) return route<8, 8, true>(p, cus, s);
    if (E <= 128) return p.T > 4096 ? route<8, 16, true>(p, cus, s) : route<16, 8, true>(p, cus, s);
    if (E <= 256) return route<16, 16, true>(p, cus, s);
    if (E <= 512) return route<64, 8, true>(p, cus, s);
    return route<64, 16, true>(p, cus, s);
  }
  // (a choice needs a lane)
  if (E <= 128 && p.k <= 16) return route<16, 8, false>(p, cus, s);
  if (E <= 128) return route<64, 2, false>(p, cus, s);
  if (E <= 256) return route<64, 4, false>(p, cus, s);
  if (E <= 512) return route<64, 8, false>(p, cus, s);
  return route<64, 16, false>(p, cus, s);
}

// (16 against 64 lanes a token, 32768 tokens: 32 experts 9.7 and 15 us, 64: 9.8
// and 15, 128: 14.9 and 18, 256: 20.4 and 22.  Of the second launch's sixteen rows
// in flight a few workgroups' sums need four: 1024 tokens of 128 experts 7.4
// against 8.5 us.)
hipError_t launch_balance_loss(const RouterParams& p, int blocks, hipStream_t s) {
  const int E = p.E;
  const hipError_t e = E <= 32 ? balance<16, 2>(p, blocks, s)
                       : E <= 64 ? balance<16, 4>(p, blocks, s)
                       : E <= 128 ? balance<16, 8>(p, blocks, s)
                       : E <= 256 ? balance<16, 16>(p, blocks, s)
                       : E <= 512 ? balance<64, 8>(p, blocks, s)
                                  : balance<64, 16>(p, blocks, s);
  if (e != hipSuccess || blocks == 1) return e;
  int slices = 1;
  while (slices < 32 && E * slices * 2 <= kBalanceT) slices *= 2;
  return queue(blocks <= 4 * slices ? balance_final_kernel<4> : balance_final_kernel<16>, dim3(1), dim3(kBalanceT), 0, s, p,
               blocks, slices);
}

// (16 against 64 lanes a token, 32768 tokens: 32 experts 6.0 and 17.4 us, 64: 8.2
// and 19.7, 128: 11.9 and 20.4, 256: 17.4 and 23.8; 1024 tokens of 256: 4.8 and 3.95.
// Eight lanes for 128 experts: 12.4.)
hipError_t launch_router_grad(const RouterParams& p, int cus, hipStream_t s) {
  const int E = p.E;
  if (E <= 128 && p.k <= 16) {
    if (E <= 32) return grad<16, 2>(p, cus, s);
    if (E <= 64) return grad<16, 4>(p, cus, s);
    return grad<16, 8>(p, cus, s);
  }
  if (E <= 128) return grad<64, 2>(p, cus, s);
  if (E <= 256) return p.T > 4096 && p.k <= 16 ? grad<16, 16>(p, cus, s) : grad<64, 4>(p, cus, s);
  if (E <= 512) return grad<64, 8>(p, cus, s);
  return grad<64, 16>(p, cus, s);
}

}  // namespace gmmk
