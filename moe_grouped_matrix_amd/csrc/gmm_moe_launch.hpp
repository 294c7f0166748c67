// gmm_moe_launch.hpp -- arguments and launch entry points of the kernels
// behind gmm_moe.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gmm_params.hpp"

namespace gmmk {

constexpr uint32_t kFlagBadRow = 0x10u;

constexpr int kSortCountT = 256;  // threads of the sort's counting launch
constexpr int kSortBlocks = 256;  // most workgroups of the split sort
constexpr int kRowT = 256;        // threads of the row kernels: four waves

// Stable sort of n slots by expert: each of `blocks` workgroups takes `per`
// consecutive slots.
struct SortParams {
  const void* ids;  // [n] int32 or int64
  int32_t* group_sizes;
  int32_t* slot_row;
  int32_t* counts;  // [G + 1][blocks], with more than one workgroup
  long long n, per;
  int32_t G, ids64;
};
hipError_t launch_sort(const SortParams& p, int blocks, hipStream_t stream);

// Row kernels: T tokens, k slots each, n = T*k rows of D elements (dispatch:
// D bytes).
struct RowParams {
  const void* a;        // dispatch: x; combine and its gradient: rows
  const void* b;        // gradient: dout
  const int32_t* slot_row;
  const void* weights;  // [T,k] f32 or bf16, or nullptr (all 1)
  void* out;            // dispatch: rows; combine: out; gradient: drows
  void* dweights;       // gradient, of weights' type
  uint32_t* flags;
  long long T, n;
  long long t0, t1;  // the launch's tokens
  int32_t k, D, w_f32;
  int32_t part;  // gradient: slots of a token that one wave takes
};
hipError_t launch_dispatch(const RowParams& p, int cu_count, hipStream_t stream);
hipError_t launch_combine(const RowParams& p, bool rows_f32, bool out_f32, int cu_count, hipStream_t stream);
hipError_t launch_combine_grad(const RowParams& p, bool dout_f32, bool rows_f32, int cu_count, hipStream_t stream);

// Microscaled fp4: `rows` rows of K elements (K % 32 == 0), codes packed two a
// byte.  Scales [rows,K/32], or with rhs > 0 [rows/rhs, K/32, rhs] (rhs = N
// rows per group).
struct Mxfp4Params {
  const void* src;  // quantise: the wide tensor; widen: the codes
  void* dst;        // quantise: the codes; widen: the wide tensor
  uint8_t* scale;
  long long rows;
  int32_t K, rhs, wide_f32;
};
hipError_t launch_quant_mxfp4(const Mxfp4Params& p, int cu_count, hipStream_t stream);
hipError_t launch_widen_mxfp4(const Mxfp4Params& p, int cu_count, hipStream_t stream);

}  // namespace gmmk
