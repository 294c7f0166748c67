// gmm_moe_checks.hpp -- argument checks of the entry points of gmm_moe.h
// (plain host C++: no HIP, no device access).  Each returns GMM_OK or the
// refusal and its text; nothing is queued before its check has passed.
#pragma once

#include <initializer_list>
#include <string>

#include "gmm_moe.h"
#include "gmm_params.hpp"
#include "gmm_tensor.hpp"

namespace gmmh {

constexpr long long kMaxTopK = 64;
constexpr long long kMaxExtent = 1LL << 31;
constexpr long long kMaxCols = 1LL << 28;

struct Check {
  gmm_status status = GMM_OK;
  std::string text;
  explicit operator bool() const { return status == GMM_OK; }
};

inline Check invalid(const std::string& t) { return {GMM_E_INVALID, t}; }
inline Check unsupported(const std::string& t) { return {GMM_E_UNSUPPORTED, t}; }

inline bool is_any(int dtype, std::initializer_list<int> of) {
  for (int d : of)
    if (dtype == d) return true;
  return false;
}

inline bool has_shape(const gmm_tensor* t, std::initializer_list<long long> shape) {
  if (t->ndim != (int)shape.size()) return false;
  int i = 0;
  for (long long s : shape)
    if (t->shape[i++] != s) return false;
  return true;
}

// Data pointers (needed where a tensor holds elements), their alignment, and
// that no output overlaps an input or another output.  The extents are
// checked before (numel does not overflow).
inline Check check_memory(std::initializer_list<const gmm_tensor*> ins, std::initializer_list<const gmm_tensor*> outs) {
  for (auto list : {ins, outs})
    for (const gmm_tensor* t : list) {
      if (!t) continue;
      if (numel(t) > 0 && !t->data) return invalid("null data pointer");
      if (!aligned16(t->data)) return invalid("tensor data must be 16-byte aligned");
    }
  for (const gmm_tensor* o : outs) {
    for (const gmm_tensor* t : ins)
      if (overlaps(t, o)) return invalid("an output overlaps an input");
    for (const gmm_tensor* t : outs)
      if (t != o && overlaps(t, o)) return invalid("two outputs overlap");
  }
  return {};
}

// The sort's split of the slots into contiguous runs, one per workgroup.  One
// workgroup alone (no workspace) sorts up to kSortSmall slots.  In the split
// sort every workgroup reads the counts of all of them, [G + 1][blocks], so
// their number falls with G.
constexpr long long kSortSmall = 4096;

struct SortSplit {
  int blocks;     // 1: one launch, no workspace
  long long per;  // slots per workgroup, a multiple of 1024 unless blocks == 1
};

inline SortSplit sort_split(long long slots, long long groups) {
  if (slots <= kSortSmall) return {1, slots};
  long long most = 32768 / (groups + 1);
  most = most > 256 ? 256 : (most < 32 ? 32 : most);
  long long per = (slots + most - 1) / most;
  per = per < 2048 ? 2048 : (per + 1023) / 1024 * 1024;
  return {(int)((slots + per - 1) / per), per};
}

inline Check check_sort_limits(long long slots, long long groups) {
  if (slots < 0) return invalid("negative number of slots");
  if (groups < 1) return invalid("at least one group is required");
  if (groups > gmmk::kMaxGroups) return unsupported("more than 1024 groups");
  if (slots >= kMaxExtent) return unsupported("2^31 slots or more");
  return {};
}

// Counts of every workgroup for every group and for the unrouted slots.
inline size_t sort_workspace_bytes(long long slots, long long groups) {
  const SortSplit s = sort_split(slots, groups);
  return s.blocks == 1 ? 0 : (size_t)s.blocks * (size_t)(groups + 1) * sizeof(int32_t);
}

// [T,k] I32 slots (or expert ids): T >= 0, 1 <= k <= 64, T*k < 2^31.
inline Check check_slots(const gmm_tensor* t, const char* name) {
  if (t->ndim != 2 || t->shape[0] < 0 || t->shape[1] < 1)
    return invalid(std::string("expected ") + name + " of shape (T, k) with k >= 1");
  if (t->shape[1] > kMaxTopK) return unsupported("more than 64 choices per token");
  if (t->shape[0] >= kMaxExtent || t->shape[0] * t->shape[1] >= kMaxExtent) return unsupported("T*k beyond 2^31");
  return {};
}

inline Check check_sort_tokens(const gmm_tensor* ids, const gmm_tensor* sizes, const gmm_tensor* slot_row,
                               const void* workspace, size_t workspace_bytes) {
  if (!ids || !sizes || !slot_row) return invalid("expert_ids, group_sizes and slot_row are required");
  if (!is_any(ids->dtype, {GMM_I32, GMM_I64})) return invalid("expert_ids must be int32 or int64");
  Check c = check_slots(ids, "expert_ids");
  if (!c) return c;
  if (sizes->ndim != 1 || sizes->dtype != GMM_I32) return invalid("expected a 1-d int32 group_sizes");
  const long long T = ids->shape[0], k = ids->shape[1], G = sizes->shape[0];
  if (!(c = check_sort_limits(T * k, G))) return c;
  if (slot_row->dtype != GMM_I32 || !has_shape(slot_row, {T, k}))
    return invalid("slot_row must be int32 of expert_ids' shape, got " + shape_str(slot_row));
  if (!(c = check_memory({ids}, {sizes, slot_row}))) return c;
  const size_t need = sort_workspace_bytes(T * k, G);
  if (need > 0) {
    if (!workspace || workspace_bytes < need)
      return invalid("the workspace needs " + std::to_string(need) + " bytes");
    if (!aligned16(workspace)) return invalid("the workspace must be 16-byte aligned");
    const gmm_tensor w{workspace, GMM_I8, 1, {(int64_t)need, 0, 0, 0}};
    if (overlaps(&w, ids) || overlaps(&w, sizes) || overlaps(&w, slot_row))
      return invalid("the workspace overlaps a tensor");
  }
  return {};
}

// A [T*k,D] or [T,D] tensor beside slot_row [T,k].
inline Check check_rows(const gmm_tensor* t, const char* name, long long rows, long long D) {
  if (!has_shape(t, {rows, D}))
    return invalid(std::string("expected ") + name + " of shape (" + std::to_string(rows) + "," + std::to_string(D) +
                   "), got " + shape_str(t));
  return {};
}

inline Check check_cols(long long D) {
  if (D < 1) return invalid("negative or zero extent");
  if (D >= kMaxCols) return unsupported("2^28 columns or more");
  return {};
}

inline Check check_slot_row(const gmm_tensor* slot_row) {
  if (slot_row->dtype != GMM_I32) return invalid("slot_row must be int32");
  return check_slots(slot_row, "slot_row");
}

inline Check check_dispatch(const gmm_tensor* x, const gmm_tensor* slot_row, const gmm_tensor* out) {
  if (!x || !slot_row || !out) return invalid("x, slot_row and out are required");
  Check c = check_slot_row(slot_row);
  if (!c) return c;
  const long long T = slot_row->shape[0], k = slot_row->shape[1];
  if (!is_any(x->dtype, {GMM_F32, GMM_BF16, GMM_F8E4M3FN, GMM_F8E5M2, GMM_E8M0, GMM_I8, GMM_I32}))
    return invalid("x: unsupported dtype");
  if (x->ndim != 2) return invalid("expected a 2-tensor for x");
  const long long D = x->shape[1];
  if (!(c = check_cols(D))) return c;
  if (!(c = check_rows(x, "x", T, D))) return c;
  if (!(c = check_rows(out, "out", T * k, D))) return c;
  if (out->dtype != x->dtype) return invalid("out must have x's dtype");
  return check_memory({x, slot_row}, {out});
}

inline Check check_weights(const gmm_tensor* w, long long T, long long k) {
  if (!is_any(w->dtype, {GMM_F32, GMM_BF16})) return invalid("weights must be f32 or bf16");
  if (!has_shape(w, {T, k})) return invalid("weights must have slot_row's shape, got " + shape_str(w));
  return {};
}

inline Check check_combine(const gmm_tensor* rows, const gmm_tensor* slot_row, const gmm_tensor* weights,
                           const gmm_tensor* out) {
  if (!rows || !slot_row || !out) return invalid("rows, slot_row and out are required");
  Check c = check_slot_row(slot_row);
  if (!c) return c;
  const long long T = slot_row->shape[0], k = slot_row->shape[1];
  if (!is_any(rows->dtype, {GMM_F32, GMM_BF16}) || !is_any(out->dtype, {GMM_F32, GMM_BF16}))
    return invalid("rows and out must be f32 or bf16");
  if (rows->ndim != 2) return invalid("expected a 2-tensor for rows");
  const long long D = rows->shape[1];
  if (!(c = check_cols(D))) return c;
  if (!(c = check_rows(rows, "rows", T * k, D))) return c;
  if (!(c = check_rows(out, "out", T, D))) return c;
  if (weights && !(c = check_weights(weights, T, k))) return c;
  return check_memory({rows, slot_row, weights}, {out});
}

inline Check check_combine_grad(const gmm_tensor* dout, const gmm_tensor* rows, const gmm_tensor* slot_row,
                                const gmm_tensor* weights, const gmm_tensor* drows, const gmm_tensor* dweights) {
  if (!dout || !rows || !slot_row || !weights || !drows || !dweights)
    return invalid("dout, rows, slot_row, weights, drows and dweights are required");
  Check c = check_slot_row(slot_row);
  if (!c) return c;
  const long long T = slot_row->shape[0], k = slot_row->shape[1];
  if (!is_any(dout->dtype, {GMM_F32, GMM_BF16}) || !is_any(rows->dtype, {GMM_F32, GMM_BF16}))
    return invalid("dout and rows must be f32 or bf16");
  if (rows->ndim != 2) return invalid("expected a 2-tensor for rows");
  const long long D = rows->shape[1];
  if (!(c = check_cols(D))) return c;
  if (!(c = check_rows(dout, "dout", T, D))) return c;
  if (!(c = check_rows(rows, "rows", T * k, D))) return c;
  if (!(c = check_weights(weights, T, k))) return c;
  if (!(c = check_rows(drows, "drows", T * k, D))) return c;
  if (drows->dtype != rows->dtype) return invalid("drows must have rows' dtype");
  if (dweights->dtype != weights->dtype || !has_shape(dweights, {T, k}))
    return invalid("dweights must have weights' dtype and shape, got " + shape_str(dweights));
  return check_memory({dout, rows, slot_row, weights}, {drows, dweights});
}

// The pair (q, scale) of a microscaled tensor and the wide tensor beside it:
// [M,K] with scale [M,K/32], or [Ga,N,K] with scale [Ga,K/32,1,N].
inline Check check_mxfp4(const gmm_tensor* wide, const gmm_tensor* q, const gmm_tensor* scale, bool quantise) {
  const char* const name = quantise ? "x" : "y";
  if (!wide || !q || !scale) return invalid(std::string(name) + ", q and scale are required");
  if (!is_any(wide->dtype, {GMM_F32, GMM_BF16})) return invalid(std::string(name) + " must be f32 or bf16");
  if (wide->ndim != 2 && wide->ndim != 3) return invalid(std::string("expected a 2- or 3-tensor for ") + name);
  const bool rhs = wide->ndim == 3;
  const long long Ga = rhs ? wide->shape[0] : 1, N = wide->shape[rhs ? 1 : 0], K = wide->shape[rhs ? 2 : 1];
  if (Ga < 0 || N < 0 || K < 1) return invalid("negative or zero extent");
  if (K % 32) return invalid("K must be a multiple of the 32-element block");
  if (K >= kMaxCols) return unsupported("2^28 columns or more");
  if (Ga >= kMaxExtent || N >= kMaxExtent || Ga * N >= kMaxExtent) return unsupported("2^31 rows or more");
  if (q->dtype != GMM_F4E2M1 || !(rhs ? has_shape(q, {Ga, N, K}) : has_shape(q, {N, K})))
    return invalid(std::string("q must be fp4 e2m1 of ") + name + "'s shape, got " + shape_str(q));
  if (scale->dtype != GMM_E8M0 || !(rhs ? has_shape(scale, {Ga, K / 32, 1, N}) : has_shape(scale, {N, K / 32})))
    return invalid(std::string("scale must be E8M0 of shape ") + (rhs ? "(Ga, K/32, 1, N)" : "(M, K/32)") + ", got " +
                   shape_str(scale));
  return quantise ? check_memory({wide}, {q, scale}) : check_memory({q, scale}, {wide});
}

}  // namespace gmmh
