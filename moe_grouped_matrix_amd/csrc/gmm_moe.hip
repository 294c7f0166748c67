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
// counts every run's keys (kept key by key, so that a wave reads a key's counts
// with one load a lane), and in the second each workgroup adds up the counts of
// all runs (what stands before its own, and the totals) and ranks its slots.
// Within a wave equal keys find each other by one ballot per key bit; a wave
// takes 64 consecutive slots at a time, in order, so the rank of a slot is its
// wave's running count plus the equal lanes below it.  Up to 4096 slots one
// workgroup does it all in one launch.
//
// Latency is what it costs: 2.9 us for one token's 8 slots, 5.9 us for 4096,
// 3.4 + 7.9 us for 262144 slots of 128 experts (3 MB read and written, which a
// copy moves in 1 us).  With the counts kept run by run and added with LDS
// atomics the second launch took 13 us, and so it did read key by key, one key a
// wave at a time; eight keys a wave at a time 8.9 us; the ids asked for before
// the counts are waited for, and the scan of the keys in lane shifts, 7.9 us.
// Reading every workgroup's counts grows with the experts: a call takes 10.6 us
// at 127 of them, 11.1 at 128, 15.8 at 256 and 41.7 at 1024.

// Inclusive prefix sum and sum over the wave's lanes, by row shifts and row
// broadcasts (the order of the additions is fixed).
__device__ __forceinline__ int wave_incl_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
  return v;
}
__device__ __forceinline__ int wave_sum(int v) { return __builtin_amdgcn_readlane(wave_incl_scan(v), 63); }
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_f32(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xF, false));
}
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp_f32<0x111, 0xF>(v);
  v += dpp_f32<0x112, 0xF>(v);
  v += dpp_f32<0x114, 0xF>(v);
  v += dpp_f32<0x118, 0xF>(v);
  v += dpp_f32<0x142, 0xA>(v);
  v += dpp_f32<0x143, 0xC>(v);
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

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
  for (int g = threadIdx.x; g <= p.G; g += kSortCountT) p.counts[(long long)g * gridDim.x + blockIdx.x] = hist[g];
}

// T threads, ITEMS slots a thread in a round.
template <int T, int ITEMS>
__global__ __launch_bounds__(T) void sort_place_kernel(SortParams p) {
  constexpr int W = T / 64;
  constexpr int E = (kMaxGroups + T - 1) / T;
  // per wave and key: the wave's count of the round, then the row of its next slot
  __shared__ int cnt[W * (kMaxGroups + 1)];
  __shared__ int base[kMaxGroups + 1];   // per key: the row of the workgroup's next slot
  __shared__ int total[kMaxGroups + 1];  // per key: all slots
  __shared__ int wave_tot[W];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int S = p.G + 1;
  const bool alone = gridDim.x == 1;
  const int bits = 32 - __builtin_clz(p.G);  // keys 0 .. G
  const long long lo = blockIdx.x * p.per, hi = lo + p.per < p.n ? lo + p.per : p.n;

  // the first round's keys are asked for before the counts are waited for
  int key[ITEMS];
  auto load_keys = [&](long long r0) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const long long s = r0 + w * (64 * ITEMS) + i * 64 + lane;
      key[i] = s < hi ? sort_key(p, s) : -1;
    }
  };
  load_keys(lo);
  for (int i = tid; i < W * S; i += T) cnt[i] = 0;
  if (alone) {
    for (int g = tid; g < S; g += T) base[g] = 0;
  } else {
    // eight keys a wave at a time: their loads are in flight together
    const int B = gridDim.x;  // at most kSortBlocks
    constexpr int KB = 8, NI = kSortBlocks / 64;
    for (int g0 = w; g0 < S; g0 += W * KB) {
      int c[KB][NI];
#pragma unroll
      for (int k = 0; k < KB; ++k)
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int g = g0 + k * W, b = lane + 64 * i;
          c[k][i] = g < S && b < B ? p.counts[(long long)g * B + b] : 0;
        }
#pragma unroll
      for (int k = 0; k < KB; ++k) {
        int all = 0, before = 0;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          all += c[k][i];
          before += lane + 64 * i < (int)blockIdx.x ? c[k][i] : 0;
        }
        all = wave_sum(all);
        before = wave_sum(before);
        if (lane == 0 && g0 + k * W < S) {
          total[g0 + k * W] = all;
          base[g0 + k * W] = before;
        }
      }
    }
  }

  bool first = true;
  for (long long r0 = lo; first || r0 < hi; r0 += T * ITEMS) {
    __syncthreads();
    int rank[ITEMS];
    const long long w0 = r0 + w * (64 * ITEMS);
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
      int sum = 0;
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (tid * E + e < p.G) sum += total[tid * E + e];
      const int incl = wave_incl_scan(sum);
      if (lane == 63) wave_tot[w] = incl;
      __syncthreads();
      int at = incl - sum, all = 0;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const int t = wave_tot[i];
        at += i < w ? t : 0;
        all += t;
      }
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (tid * E + e < p.G) {
          base[tid * E + e] += at;
          at += total[tid * E + e];
        }
      if (tid == 0) base[p.G] += all;
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
    first = false;
    if (r0 + T * ITEMS < hi) {
      load_keys(r0 + T * ITEMS);
      __syncthreads();
      for (int i = tid; i < W * S; i += T) cnt[i] = 0;
    }
  }
}

// ---------------------------------------------------------------------------
// Rows.  All three kernels stream rows once and are HBM-bound; what they need
// is many independent 16-byte loads in flight.  A wave takes one token and up
// to U chunks of V elements a lane (a segment of its columns), and loads the
// token's slot entries (k <= 64) with one load, a slot a lane; the slots' rows
// then come from lanes into scalar registers, so that a row's address is a
// scalar and its rows' loads do not wait for one another.  A row whose width
// is not a multiple of V ends in a chunk that starts V before its end and
// overlaps the one before (both write the same values); rows narrower than V
// go one element at a time.  Rows start at any multiple of the element size.
//
// 32768 tokens x top-8 of 128, 1408 bf16 columns, against a copy of as many
// bytes (5.14 TB/s): dispatch 157 us (832 MB, 5.3 TB/s), combine 158 us (831 MB),
// its gradient 307 us (1572 MB, 5.1 TB/s); counted HBM traffic 1.00 times those
// bytes.  One row at a time and loads through the caches took 173, 180 and 374
// us.  For a decode step of 256 tokens a lane takes one chunk, so that three
// times the waves share the rows: dispatch 3.7 us (8.7 with a wave a token),
// combine of f32 rows 4.4 us (13.9).
//
// Narrow rows leave lanes idle: 32768 x 8 bf16 rows of 128 columns run at 5.5
// TB/s (dispatch), 2.6 (combine) and 2.7 (its gradient), of 64 at 3.6, 1.4 and
// 1.6; from 512 on dispatch and
// combine run at the copy's rate, the gradient at 0.8 to 1.05 of it.

typedef int i32x4_any __attribute__((ext_vector_type(4), aligned(1)));

template <typename E, int V>
struct Vec {
  E v[V];
};

template <typename E, int V>
__device__ __forceinline__ Vec<E, V> load_vec(const E* p) {
  Vec<E, V> r;
  constexpr int B = sizeof(E) * V;
  if constexpr (B % 16 == 0) {
    i32x4 w[B / 16];
#pragma unroll
    for (int i = 0; i < B / 16; ++i) {
      // eight f32 are two loads that share lines, and go without the hint
      // (combine of 16384 x 8 f32 rows of 1408: 152 against 157 us; of bf16 rows
      // with it 156, without 162)
      if constexpr (B == 32)
        w[i] = reinterpret_cast<const i32x4_any*>(p)[i];
      else
        w[i] = __builtin_nontemporal_load(reinterpret_cast<const i32x4_any*>(p) + i);
    }
    __builtin_memcpy(&r, w, B);
  } else {
    __builtin_memcpy(&r, p, B);
  }
  return r;
}
template <typename E, int V>
__device__ __forceinline__ void store_vec(E* p, const Vec<E, V>& r) {
  constexpr int B = sizeof(E) * V;
  if constexpr (B % 16 == 0) {
    i32x4 w[B / 16];
    __builtin_memcpy(w, &r, B);
#pragma unroll
    for (int i = 0; i < B / 16; ++i)
      __builtin_nontemporal_store((i32x4_any)w[i], reinterpret_cast<i32x4_any*>(p) + i);
  } else {
    __builtin_memcpy(p, &r, B);
  }
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(uint16_t v) { return bf16_bits_to_f32(v); }
__device__ __forceinline__ void from_f32(float f, float& v) { v = f; }
__device__ __forceinline__ void from_f32(float f, uint16_t& v) { v = f32_to_bf16_rne(f); }

// The slot entries of token t, slot j in lane j: the row it names (as itself
// or as a complement), -1 for none or for one outside [0, n) (flagged), and
// whether the slot is routed.
struct Slots {
  int row, routed;
  float w;
};

__device__ __forceinline__ Slots load_slots(const RowParams& p, long long t, int lane) {
  Slots s{-1, 0, 0.f};
  if (lane < p.k) {
    const long long i = t * p.k + lane;
    const int r = p.slot_row[i];
    s.row = r < 0 ? ~r : r;
    s.routed = r >= 0;
    if (s.row >= p.n) {
      s.row = -1;
      atomicOr(p.flags, kFlagBadRow);
    }
    s.w = 1.f;
    if (p.weights)
      s.w = p.w_f32 ? static_cast<const float*>(p.weights)[i]
                    : bf16_bits_to_f32(static_cast<const uint16_t*>(p.weights)[i]);
  }
  return s;
}

__device__ __forceinline__ int of_lane(int v, int j) { return __builtin_amdgcn_readlane(v, j); }
__device__ __forceinline__ float of_lane(float v, int j) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), j));
}

// First element of the chunk that chunk number c of a row covers.
template <int V>
__device__ __forceinline__ int chunk_start(int c, int D) {
  return c * V + V <= D ? c * V : D - V;
}

// Work item i of a row kernel: a token and a segment of 64 U chunks.
struct RowItem {
  long long t;
  int c0, chunks;
};

template <int V, int U>
__device__ __forceinline__ RowItem row_item(const RowParams& p, long long i) {
  const int chunks = (p.D + V - 1) / V, segs = (chunks + 64 * U - 1) / (64 * U);
  if (segs == 1) return {p.t0 + i, 0, chunks};
  const long long t = i / segs;
  return {p.t0 + t, (int)(i - t * segs) * 64 * U, chunks};
}

template <int V, int U>
__global__ __launch_bounds__(kRowT) void dispatch_kernel(RowParams p) {
  const int lane = threadIdx.x & 63;
  const long long item = (long long)blockIdx.x * (kRowT / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const RowItem it = row_item<V, U>(p, item);
  if (it.t >= p.t1) return;
  const int D = p.D;  // bytes of a row
  const uint8_t* const src = static_cast<const uint8_t*>(p.a) + it.t * D;
  int at[U];
  Vec<uint8_t, V> x[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = it.c0 + 64 * u + lane;
    at[u] = c < it.chunks ? chunk_start<V>(c, D) : -1;
    if (at[u] >= 0) x[u] = load_vec<uint8_t, V>(src + at[u]);
  }
  const Slots s = load_slots(p, it.t, lane);
  for (int j = 0; j < p.k; ++j) {
    const int row = of_lane(s.row, j);
    if (row < 0) continue;
    uint8_t* const dst = static_cast<uint8_t*>(p.out) + (long long)row * D;
    if (of_lane(s.routed, j)) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (at[u] >= 0) store_vec(dst + at[u], x[u]);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (at[u] >= 0) store_vec(dst + at[u], Vec<uint8_t, V>{});
    }
  }
}

// out[t] = sum over j of w[t,j] * rows[slot_row[t,j]], four rows in flight
template <typename R, typename O, int V, int U>
__global__ __launch_bounds__(kRowT) void combine_kernel(RowParams p) {
  constexpr int JB = 4;
  const int lane = threadIdx.x & 63;
  const long long item = (long long)blockIdx.x * (kRowT / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const RowItem it = row_item<V, U>(p, item);
  if (it.t >= p.t1) return;
  const int D = p.D;
  const Slots s = load_slots(p, it.t, lane);
  int at[U];
  float acc[U][V];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = it.c0 + 64 * u + lane;
    at[u] = c < it.chunks ? chunk_start<V>(c, D) : -1;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[u][e] = 0.f;
  }
  for (int j = 0; j < p.k; j += JB) {
    Vec<R, V> x[JB][U];
    bool live[JB];
#pragma unroll
    for (int b = 0; b < JB; ++b) {
      // (lanes past k hold no row)
      const int row = j + b < p.k ? of_lane(s.row, j + b) : -1;
      live[b] = row >= 0 && of_lane(s.routed, j + b < p.k ? j + b : 0);
      if (!live[b]) continue;
      const R* const src = static_cast<const R*>(p.a) + (long long)row * D;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (at[u] >= 0) x[b][u] = load_vec<R, V>(src + at[u]);
    }
#pragma unroll
    for (int b = 0; b < JB; ++b) {
      if (!live[b]) continue;
      const float w = of_lane(s.w, j + b);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < V; ++e) acc[u][e] = __builtin_fmaf(w, to_f32(x[b][u].v[e]), acc[u][e]);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (at[u] < 0) continue;
    Vec<O, V> o;
#pragma unroll
    for (int e = 0; e < V; ++e) from_f32(acc[u][e], o.v[e]);
    store_vec(static_cast<O*>(p.out) + it.t * D + at[u], o);
  }
}

// drows[slot_row[t,j]] = w[t,j] * dout[t], dweights[t,j] = <dout[t], rows[slot_row[t,j]]>.
// A wave takes p.part of a token's slots over all its columns, so a product's
// sum never leaves the wave: per segment it is added up over the lanes, and
// lane j keeps slot j's.
template <typename G, typename R, int V, int U>
__global__ __launch_bounds__(kRowT) void combine_grad_kernel(RowParams p) {
  constexpr int JB = 2;
  const int lane = threadIdx.x & 63;
  const long long item = (long long)blockIdx.x * (kRowT / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int parts = (p.k + p.part - 1) / p.part;
  const long long rel = parts == 1 ? item : item / parts, t = p.t0 + rel;
  if (t >= p.t1) return;
  const int j0 = parts == 1 ? 0 : (int)(item - rel * parts) * p.part;
  const int j1 = j0 + p.part < p.k ? j0 + p.part : p.k;
  const int D = p.D, chunks = (D + V - 1) / V;
  const Slots s = load_slots(p, t, lane);
  const G* const g = static_cast<const G*>(p.b) + t * D;
  float mine = 0.f;
  for (int c0 = 0; c0 < chunks; c0 += 64 * U) {
    int at[U];
    Vec<G, V> gv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + 64 * u + lane;
      at[u] = c < chunks ? chunk_start<V>(c, D) : -1;
      gv[u] = Vec<G, V>{};
      if (at[u] >= 0) gv[u] = load_vec<G, V>(g + at[u]);
    }
    // elements of the last chunk that the one before has: they count once
    const bool tail = c0 + 64 * U >= chunks && D % V != 0;
    for (int j = j0; j < j1; j += JB) {
      Vec<R, V> x[JB][U];
      int row[JB];
      bool routed[JB];
#pragma unroll
      for (int b = 0; b < JB; ++b) {
        const int jb = j + b < j1 ? j + b : j;
        row[b] = j + b < j1 ? of_lane(s.row, jb) : -1;
        routed[b] = row[b] >= 0 && of_lane(s.routed, jb);
        if (!routed[b]) continue;
        const R* const src = static_cast<const R*>(p.a) + (long long)row[b] * D;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          x[b][u] = Vec<R, V>{};
          if (at[u] >= 0) x[b][u] = load_vec<R, V>(src + at[u]);
        }
      }
#pragma unroll
      for (int b = 0; b < JB; ++b) {
        if (row[b] < 0) continue;
        R* const dst = static_cast<R*>(p.out) + (long long)row[b] * D;
        if (!routed[b]) {
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (at[u] >= 0) store_vec(dst + at[u], Vec<R, V>{});
          continue;
        }
        const float w = of_lane(s.w, j + b);
        float dot = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          Vec<R, V> d;
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float ge = to_f32(gv[u].v[e]);
            from_f32(w * ge, d.v[e]);
            // (a select of the sum, not of a factor: 0 times an infinity would count)
            const bool count = !tail || at[u] + e >= (c0 + 64 * u + lane) * V;
            const float sum = __builtin_fmaf(ge, to_f32(x[b][u].v[e]), dot);
            dot = count ? sum : dot;
          }
          if (at[u] >= 0) store_vec(dst + at[u], d);
        }
        dot = wave_sum(dot);
        if (lane == j + b) mine += dot;
      }
    }
  }
  if (lane >= j0 && lane < j1) {
    const long long i = t * p.k + lane;
    if (p.w_f32)
      static_cast<float*>(p.dweights)[i] = mine;
    else
      static_cast<uint16_t*>(p.dweights)[i] = f32_to_bf16_rne(mine);
  }
}

}  // namespace

hipError_t launch_sort(const SortParams& p, int blocks, hipStream_t stream) {
  if (blocks > 1) {
    hipLaunchKernelGGL(sort_count_kernel, dim3((unsigned)blocks), dim3(kSortCountT), 0, stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (blocks > 1)
    hipLaunchKernelGGL((sort_place_kernel<1024, 2>), dim3((unsigned)blocks), dim3(1024), 0, stream, p);
  else if (p.per <= 1024)
    hipLaunchKernelGGL((sort_place_kernel<256, 4>), dim3((unsigned)blocks), dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL((sort_place_kernel<1024, 4>), dim3((unsigned)blocks), dim3(1024), 0, stream, p);
  return hipGetLastError();
}

// Chunks a lane takes: a whole row in one segment up to four a lane, but with
// too few tokens to fill the card one, so that more waves share the rows.  One /
// several, us, 8 rows a token, bf16: combine of 1024 tokens x 1408 9.0 / 14.7, of
// 2048 10.9 / 16.7, of 8192 36.5 / 40.7, of 32768 137 / 156 (several chunks do not
// pay there either); dispatch within 5% at every size (1024: 5.3 / 5.3, 8192:
// 36.4 / 38.4, 32768: 152 / 156).
static int row_unroll(long long tokens, int D, int V, int cu) {
  const int chunks = (D + V - 1) / V;
  const int u = (chunks + 63) / 64;
  if (tokens < 8LL * cu) return 1;
  return u > 4 ? 4 : u;
}

// Runs launch(p, blocks) over all tokens with `per_token` waves each, in
// slices of tokens that keep a launch to 2^31 threads at most.
template <class LaunchFn>
static hipError_t by_slices(RowParams p, long long per_token, LaunchFn launch) {
  const long long most = (1LL << 25) / per_token > 0 ? (1LL << 25) / per_token : 1;
  for (p.t0 = 0; p.t0 < p.T; p.t0 = p.t1) {
    p.t1 = p.t0 + most < p.T ? p.t0 + most : p.T;
    launch(p, (unsigned)(((p.t1 - p.t0) * per_token + kRowT / 64 - 1) / (kRowT / 64)));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

static long long row_segs(const RowParams& p, int V, int U) { return ((p.D + V - 1LL) / V + 64 * U - 1) / (64 * U); }

#define GMM_LAUNCH(KERNEL) hipLaunchKernelGGL(KERNEL, dim3(blocks), dim3(kRowT), 0, st, q)

template <int V, int U>
static hipError_t dispatch_u(const RowParams& p, hipStream_t st) {
  return by_slices(p, row_segs(p, V, U),
                   [=](const RowParams& q, unsigned blocks) { GMM_LAUNCH((dispatch_kernel<V, U>)); });
}

hipError_t launch_dispatch(const RowParams& p, int cu, hipStream_t st) {
  if (p.D < 16) return dispatch_u<1, 1>(p, st);
  switch (row_unroll(p.T, p.D, 16, cu)) {
    case 1: return dispatch_u<16, 1>(p, st);
    case 2: return dispatch_u<16, 2>(p, st);
    case 3: return dispatch_u<16, 3>(p, st);
    default: return dispatch_u<16, 4>(p, st);
  }
}

template <typename R, typename O, int V, int U>
static hipError_t combine_u(const RowParams& p, hipStream_t st) {
  return by_slices(p, row_segs(p, V, U),
                   [=](const RowParams& q, unsigned blocks) { GMM_LAUNCH((combine_kernel<R, O, V, U>)); });
}

template <typename R, typename O>
static hipError_t combine_by_width(const RowParams& p, int cu, hipStream_t st) {
  if (p.D < 8) return combine_u<R, O, 1, 1>(p, st);
  switch (row_unroll(p.T, p.D, 8, cu)) {
    case 1: return combine_u<R, O, 8, 1>(p, st);
    case 2: return combine_u<R, O, 8, 2>(p, st);
    case 3: return combine_u<R, O, 8, 3>(p, st);
    default: return combine_u<R, O, 8, 4>(p, st);
  }
}

hipError_t launch_combine(const RowParams& p, bool rows_f32, bool out_f32, int cu, hipStream_t st) {
  if (rows_f32) return out_f32 ? combine_by_width<float, float>(p, cu, st) : combine_by_width<float, uint16_t>(p, cu, st);
  return out_f32 ? combine_by_width<uint16_t, float>(p, cu, st) : combine_by_width<uint16_t, uint16_t>(p, cu, st);
}

template <typename G, typename R, int V, int U>
static hipError_t grad_u(const RowParams& p, hipStream_t st) {
  return by_slices(p, (p.k + p.part - 1) / p.part,
                   [=](const RowParams& q, unsigned blocks) { GMM_LAUNCH((combine_grad_kernel<G, R, V, U>)); });
}

template <typename G, typename R>
static hipError_t grad_by_width(RowParams p, int cu, hipStream_t st) {
  // a wave takes all of a token's slots, or with too few tokens one (a slot / all,
  // us, 8 rows of 1408 bf16 a token: 1024 tokens 16.3 / 22.6, 2048 26.6 / 27.8, 2944
  // 36.8 / 32.7, 8192 92 / 84; rows of 256, 8192 tokens: 32 / 17.5)
  p.part = p.T < 8LL * cu ? 1 : p.k;
  if (p.D < 8) return grad_u<G, R, 1, 1>(p, st);
  switch (((p.D + 7) / 8 + 63) / 64) {
    case 1: return grad_u<G, R, 8, 1>(p, st);
    case 2: return grad_u<G, R, 8, 2>(p, st);
    case 3: return grad_u<G, R, 8, 3>(p, st);
    default: return grad_u<G, R, 8, 4>(p, st);
  }
}
#undef GMM_LAUNCH

hipError_t launch_combine_grad(const RowParams& p, bool dout_f32, bool rows_f32, int cu, hipStream_t st) {
  if (dout_f32) return rows_f32 ? grad_by_width<float, float>(p, cu, st) : grad_by_width<float, uint16_t>(p, cu, st);
  return rows_f32 ? grad_by_width<uint16_t, float>(p, cu, st) : grad_by_width<uint16_t, uint16_t>(p, cu, st);
}

}  // namespace gmmk
