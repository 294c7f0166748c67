// gmm_moe.hip -- the steps around the grouped matmul on gfx950: the stable
// sort of token slots by expert, the dispatch of tokens to expert rows, the
// weighted combine back and its gradient.  Layouts and meanings are those of
// gmm_moe.h: slot_row[t,j] is the row of slot (t,j), or the complement of its
// row when the slot is unrouted.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gmm_device.hpp"
#include "gmm_moe_launch.hpp"

namespace gmmk {

namespace {

// ---------------------------------------------------------------------------
// Stable sort by expert.  A counting sort: row(s) = (slots of smaller keys) +
// (earlier slots of the same key), the key of an unrouted slot being G.  The
// slots are cut into contiguous runs, one per workgroup; the first launch
// counts every run's keys, and in the second each workgroup adds up the counts
// of all runs (what stands before its own, and the totals) and ranks its
// slots.  Within a wave equal keys find each other by one ballot per key bit;
// a wave takes 64 consecutive slots at a time, in order, so the rank of a slot
// is its wave's running count plus the equal lanes below it.

__device__ __forceinline__ int sort_key(const SortParams& p, long long i) {
  const long long id = p.ids64 ? reinterpret_cast<const int64_t*>(p.ids)[i]
                               : (long long)reinterpret_cast<const int32_t*>(p.ids)[i];
  return id >= 0 && id < p.G ? (int)id : p.G;
}

__global__ __launch_bounds__(kSortCountT) void sort_count_kernel(SortParams p) {
  __shared__ int hist[kMaxGroups + 1];
  for (int g = threadIdx.x; g <= p.G; g += kSortCountT) hist[g] = 0;
  __syncthreads();
  const long long lo = blockIdx.x * p.per, hi = lo + p.per < p.n ? lo + p.per : p.n;
  for (long long i = lo + threadIdx.x; i < hi; i += kSortCountT) atomicAdd(&hist[sort_key(p, i)], 1);
  __syncthreads();
  int32_t* const ws = p.counts + (long long)blockIdx.x * (p.G + 1);
  for (int g = threadIdx.x; g <= p.G; g += kSortCountT) ws[g] = hist[g];
}

template <int T>
__global__ __launch_bounds__(T) void sort_place_kernel(SortParams p) {
  constexpr int W = T / 64, ITEMS = 4;
  constexpr int E = (kMaxGroups + T - 1) / T;
  // per wave and key: the wave's count of the round, then the row of its next slot
  __shared__ int cnt[W * (kMaxGroups + 1)];
  __shared__ int base[kMaxGroups + 1];   // per key: the row of the workgroup's next slot
  __shared__ int total[kMaxGroups + 1];  // per key: all slots
  __shared__ long long wave_tot[W];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int S = p.G + 1;
  const bool alone = gridDim.x == 1;
  const int bits = 32 - __builtin_clz(p.G);  // keys 0 .. G
  const long long lo = blockIdx.x * p.per, hi = lo + p.per < p.n ? lo + p.per : p.n;

  for (int g = tid; g < S; g += T) base[g] = total[g] = 0;
  __syncthreads();
  if (!alone) {
    for (int b = w; b < (int)gridDim.x; b += W) {
      const int32_t* const ws = p.counts + (long long)b * S;
      for (int g = lane; g < S; g += 64) {
        const int c = ws[g];
        atomicAdd(&total[g], c);
        if (b < (int)blockIdx.x) atomicAdd(&base[g], c);
      }
    }
  }

  bool first = true;
  for (long long r0 = lo; first || r0 < hi; r0 += T * ITEMS) {
    for (int i = tid; i < W * S; i += T) cnt[i] = 0;
    __syncthreads();
    int key[ITEMS], rank[ITEMS];
    const long long w0 = r0 + w * (64 * ITEMS);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const long long s = w0 + i * 64 + lane;
      key[i] = s < hi ? sort_key(p, s) : -1;
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      rank[i] = 0;
      if (w0 + i * 64 < hi) {
        const bool live = key[i] >= 0;
        unsigned long long peers = __ballot(live);
        for (int b = 0; b < bits; ++b) {
          const bool bit = (key[i] >> b) & 1;
          const unsigned long long m = __ballot(bit);
          peers &= bit ? m : ~m;
        }
        // (a lane past the end has key -1; its peers are nobody's business)
        const int leader = live ? __builtin_ctzll(peers) : 0;
        int before = 0;
        if (live && lane == leader) before = atomicAdd(&cnt[w * S + key[i]], __builtin_popcountll(peers));
        before = __shfl(before, leader, 64);
        rank[i] = before + __builtin_popcountll(peers & ((1ull << lane) - 1));
      }
    }
    __syncthreads();
    if (first) {
      if (alone) {
        for (int g = tid; g < S; g += T) {
          int c = 0;
#pragma unroll
          for (int i = 0; i < W; ++i) c += cnt[i * S + g];
          total[g] = c;
        }
        __syncthreads();
      }
      // keys tid*E .. of this thread: rows of smaller keys
      long long sum = 0, all;
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (tid * E + e < p.G) sum += total[tid * E + e];
      long long at = block_excl_scan<T>(sum, wave_tot, &all);
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (tid * E + e < p.G) {
          base[tid * E + e] += (int)at;
          at += total[tid * E + e];
        }
      if (tid == 0) base[p.G] += (int)all;
      if (blockIdx.x == 0)
        for (int g = tid; g < p.G; g += T) p.group_sizes[g] = total[g];
      __syncthreads();
    }
    for (int g = tid; g < S; g += T) {
      int c[W], run = base[g];
#pragma unroll
      for (int i = 0; i < W; ++i) c[i] = cnt[i * S + g];
#pragma unroll
      for (int i = 0; i < W; ++i) {
        cnt[i * S + g] = run;
        run += c[i];
      }
      base[g] = run;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const long long s = w0 + i * 64 + lane;
      if (key[i] >= 0) {
        const int row = cnt[w * S + key[i]] + rank[i];
        p.slot_row[s] = key[i] < p.G ? row : ~row;
      }
    }
    __syncthreads();
    first = false;
  }
}

// ---------------------------------------------------------------------------
// Rows.  A wave takes one token's columns in chunks of V elements per lane.  A
// row whose width is not a multiple of V ends in a chunk that starts V before
// the end and overlaps the chunk before it (both write the same values); rows
// narrower than V go one element at a time.

template <typename E, int V>
struct Vec {
  E v[V];
};

template <int V>
__device__ __forceinline__ int chunk_start(int c, int D) {
  return c * V + V <= D ? c * V : D - V;
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(uint16_t v) { return bf16_bits_to_f32(v); }
__device__ __forceinline__ void from_f32(float f, float& v) { v = f; }
__device__ __forceinline__ void from_f32(float f, uint16_t& v) { v = f32_to_bf16_rne(f); }

// rows start at any multiple of the element size: the copies say so
template <typename E, int V>
__device__ __forceinline__ Vec<E, V> load_vec(const E* p) {
  Vec<E, V> r;
  __builtin_memcpy(&r, p, sizeof r);
  return r;
}
template <typename E, int V>
__device__ __forceinline__ void store_vec(E* p, const Vec<E, V>& r) {
  __builtin_memcpy(p, &r, sizeof r);
}

__device__ __forceinline__ void bad_row(const RowParams& p) { atomicOr(p.flags, kFlagBadRow); }

// The row that slot entry r names (as itself or as a complement), or -1 and
// the flag for one outside [0, n).
__device__ __forceinline__ int named_row(const RowParams& p, int r, int lane) {
  const int row = r < 0 ? ~r : r;
  if (row < p.n) return row;
  if (lane == 0) bad_row(p);
  return -1;
}

template <int V>
__global__ __launch_bounds__(kRowT) void dispatch_kernel(RowParams p) {
  const int lane = threadIdx.x & 63;
  const int D = p.D;  // bytes of a row
  const int chunks = (D + V - 1) / V;
  const long long waves = (long long)gridDim.x * (kRowT / 64);
  for (long long t = (long long)blockIdx.x * (kRowT / 64) + (threadIdx.x >> 6); t < p.T; t += waves) {
    const uint8_t* const src = static_cast<const uint8_t*>(p.a) + t * D;
    for (int c = lane; c < chunks; c += 64) {
      const int at = chunk_start<V>(c, D);
      const Vec<uint8_t, V> x = load_vec<uint8_t, V>(src + at);
      for (int j = 0; j < p.k; ++j) {
        const int r = p.slot_row[t * p.k + j];
        const int row = named_row(p, r, lane);
        if (row < 0) continue;
        Vec<uint8_t, V> v = x;
        if (r < 0) v = Vec<uint8_t, V>{};
        store_vec(static_cast<uint8_t*>(p.out) + (long long)row * D + at, v);
      }
    }
  }
}

// out[t] = sum over j of w[t,j] * rows[slot_row[t,j]]
template <typename R, typename O, int V>
__global__ __launch_bounds__(kRowT) void combine_kernel(RowParams p) {
  const int lane = threadIdx.x & 63;
  const int D = p.D;
  const int chunks = (D + V - 1) / V;
  const long long waves = (long long)gridDim.x * (kRowT / 64);
  for (long long t = (long long)blockIdx.x * (kRowT / 64) + (threadIdx.x >> 6); t < p.T; t += waves) {
    for (int c = lane; c < chunks; c += 64) {
      const int at = chunk_start<V>(c, D);
      float acc[V];
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = 0.f;
      for (int j = 0; j < p.k; ++j) {
        const int r = p.slot_row[t * p.k + j];
        const int row = named_row(p, r, lane);
        if (r < 0 || row < 0) continue;
        float w = 1.f;
        if (p.weights) w = p.w_f32 ? static_cast<const float*>(p.weights)[t * p.k + j]
                                   : bf16_bits_to_f32(static_cast<const uint16_t*>(p.weights)[t * p.k + j]);
        const Vec<R, V> x = load_vec<R, V>(static_cast<const R*>(p.a) + (long long)row * D + at);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = __builtin_fmaf(w, to_f32(x.v[i]), acc[i]);
      }
      Vec<O, V> o;
#pragma unroll
      for (int i = 0; i < V; ++i) from_f32(acc[i], o.v[i]);
      store_vec(static_cast<O*>(p.out) + t * D + at, o);
    }
  }
}

// drows[slot_row[t,j]] = w[t,j] * dout[t], dweights[t,j] = <dout[t], rows[slot_row[t,j]]>
template <typename G, typename R, int V>
__global__ __launch_bounds__(kRowT) void combine_grad_kernel(RowParams p) {
  const int lane = threadIdx.x & 63;
  const int D = p.D;
  const int chunks = (D + V - 1) / V;
  const long long waves = (long long)gridDim.x * (kRowT / 64);
  const long long slots = p.T * p.k;
  for (long long s = (long long)blockIdx.x * (kRowT / 64) + (threadIdx.x >> 6); s < slots; s += waves) {
    const long long t = s / p.k;
    const int r = p.slot_row[s];
    const int row = named_row(p, r, lane);
    float dot = 0.f;
    if (row >= 0) {
      const float w = r < 0 ? 0.f
                            : (p.w_f32 ? static_cast<const float*>(p.weights)[s]
                                       : bf16_bits_to_f32(static_cast<const uint16_t*>(p.weights)[s]));
      const G* const g = static_cast<const G*>(p.b) + t * D;
      const R* const x = static_cast<const R*>(p.a) + (long long)row * D;
      R* const o = static_cast<R*>(p.out) + (long long)row * D;
      for (int c = lane; c < chunks; c += 64) {
        const int at = chunk_start<V>(c, D);
        Vec<R, V> d{};
        if (r >= 0) {
          const Vec<G, V> gv = load_vec<G, V>(g + at);
          const Vec<R, V> xv = load_vec<R, V>(x + at);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float gi = to_f32(gv.v[i]);
            // elements of an overlapping last chunk count once
            if (at + i >= c * V) dot = __builtin_fmaf(gi, to_f32(xv.v[i]), dot);
            from_f32(w * gi, d.v[i]);
          }
        }
        store_vec(o + at, d);
      }
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) dot += __shfl_xor(dot, d, 64);
    if (lane == 0) {
      if (p.w_f32)
        static_cast<float*>(p.dweights)[s] = dot;
      else
        static_cast<uint16_t*>(p.dweights)[s] = f32_to_bf16_rne(dot);
    }
  }
}

unsigned row_grid(long long items, int cu_count) {
  long long grid = (items + kRowT / 64 - 1) / (kRowT / 64);
  const long long cap = (long long)cu_count * 32;
  if (grid > cap) grid = cap;
  return (unsigned)(grid < 1 ? 1 : grid);
}

}  // namespace

hipError_t launch_sort(const SortParams& p, int blocks, hipStream_t stream) {
  if (blocks > 1) {
    hipLaunchKernelGGL(sort_count_kernel, dim3((unsigned)blocks), dim3(kSortCountT), 0, stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (p.per <= 1024)
    hipLaunchKernelGGL(sort_place_kernel<256>, dim3((unsigned)blocks), dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL(sort_place_kernel<1024>, dim3((unsigned)blocks), dim3(1024), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_dispatch(const RowParams& p, int cu, hipStream_t st) {
  const unsigned grid = row_grid(p.T, cu);
  if (p.D >= 16)
    hipLaunchKernelGGL(dispatch_kernel<16>, dim3(grid), dim3(kRowT), 0, st, p);
  else
    hipLaunchKernelGGL(dispatch_kernel<1>, dim3(grid), dim3(kRowT), 0, st, p);
  return hipGetLastError();
}

template <typename R, typename O>
static void combine_by_width(const RowParams& p, unsigned grid, hipStream_t st) {
  if (p.D >= 8)
    hipLaunchKernelGGL((combine_kernel<R, O, 8>), dim3(grid), dim3(kRowT), 0, st, p);
  else
    hipLaunchKernelGGL((combine_kernel<R, O, 1>), dim3(grid), dim3(kRowT), 0, st, p);
}

hipError_t launch_combine(const RowParams& p, bool rows_f32, bool out_f32, int cu, hipStream_t st) {
  const unsigned grid = row_grid(p.T, cu);
  if (rows_f32)
    out_f32 ? combine_by_width<float, float>(p, grid, st) : combine_by_width<float, uint16_t>(p, grid, st);
  else
    out_f32 ? combine_by_width<uint16_t, float>(p, grid, st) : combine_by_width<uint16_t, uint16_t>(p, grid, st);
  return hipGetLastError();
}

template <typename G, typename R>
static void grad_by_width(const RowParams& p, unsigned grid, hipStream_t st) {
  if (p.D >= 8)
    hipLaunchKernelGGL((combine_grad_kernel<G, R, 8>), dim3(grid), dim3(kRowT), 0, st, p);
  else
    hipLaunchKernelGGL((combine_grad_kernel<G, R, 1>), dim3(grid), dim3(kRowT), 0, st, p);
}

hipError_t launch_combine_grad(const RowParams& p, bool dout_f32, bool rows_f32, int cu, hipStream_t st) {
  const unsigned grid = row_grid(p.T * p.k, cu);
  if (dout_f32)
    rows_f32 ? grad_by_width<float, float>(p, grid, st) : grad_by_width<float, uint16_t>(p, grid, st);
  else
    rows_f32 ? grad_by_width<uint16_t, float>(p, grid, st) : grad_by_width<uint16_t, uint16_t>(p, grid, st);
  return hipGetLastError();
}

}  // namespace gmmk
