// gmm_layer_checks.hpp -- argument checks of the entry points of gmm_layer.h
// (plain host C++: no HIP, no device access).  Each returns GMM_OK or the
// refusal and its text; nothing is queued before its check has passed.
#pragma once

#include <algorithm>
#include <cmath>
#include <utility>
#include <vector>

#include "gmm_layer.h"
#include "gmm_moe_checks.hpp"

namespace gmmh {

constexpr long long kMaxGmvSlots = 4096;
constexpr long long kMaxGmvCols = 1LL << 24;
constexpr long long kMaxGmvK = 1LL << 20;
constexpr long long kMaxAdamElems = 1LL << 34;

// logits [T,E], ids [T,k] of the given types, valid [T].
inline Check check_router(const gmm_tensor* logits, const gmm_tensor* ids, bool ids_written, const gmm_tensor* valid,
                          int scores) {
  if (!is_any(logits->dtype, {GMM_F32, GMM_BF16})) return invalid("logits must be f32 or bf16");
  if (logits->ndim != 2 || logits->shape[0] < 0 || logits->shape[1] < 1)
    return invalid("expected logits of shape (T, E) with E >= 1, got " + shape_str(logits));
  const long long T = logits->shape[0], E = logits->shape[1];
  if (E > gmmk::kMaxGroups) return unsupported("more than 1024 experts");
  if (T >= kMaxExtent || T * E >= kMaxExtent) return unsupported("T*E beyond 2^31");
  if (ids_written ? ids->dtype != GMM_I32 : !is_any(ids->dtype, {GMM_I32, GMM_I64}))
    return invalid(ids_written ? "expert_ids must be int32" : "expert_ids must be int32 or int64");
  Check c = check_slots(ids, "expert_ids");
  if (!c) return c;
  if (ids->shape[0] != T) return invalid("expert_ids and logits differ in their tokens");
  if (ids->shape[1] > E) return invalid("more choices than experts");
  if (valid && (valid->dtype != GMM_I8 || !has_shape(valid, {T})))
    return invalid("valid must be one byte or bool per token, got " + shape_str(valid));
  if (scores != GMM_SCORES_SOFTMAX && scores != GMM_SCORES_SIGMOID) return invalid("unknown kind of scores");
  return {};
}

inline Check check_route(const gmm_tensor* logits, const gmm_tensor* bias, const gmm_tensor* valid, int scores,
                         const gmm_tensor* ids, const gmm_tensor* weights) {
  if (!logits || !ids || !weights) return invalid("logits, expert_ids and weights are required");
  Check c = check_router(logits, ids, true, valid, scores);
  if (!c) return c;
  if (bias && (bias->dtype != GMM_F32 || !has_shape(bias, {logits->shape[1]})))
    return invalid("bias must be f32 of shape (E,), got " + shape_str(bias));
  if (weights->dtype != GMM_F32 || !has_shape(weights, {ids->shape[0], ids->shape[1]}))
    return invalid("weights must be f32 of expert_ids' shape, got " + shape_str(weights));
  return check_memory({logits, bias, valid}, {ids, weights});
}

// Workgroups of the balance loss's first launch, 64 tokens (16 of more than
// 256 experts) at a time.  One workgroup alone needs no second launch and no
// workspace.
inline int balance_blocks(long long T, long long E) {
  const long long rows = E <= 256 ? 64 : 16;
  const long long b = (T + rows - 1) / rows;
  return (int)(b < 1 ? 1 : b > 256 ? 256 : b);
}
inline size_t balance_workspace_bytes(long long T, long long E) {
  const int blocks = balance_blocks(T, E);
  return blocks == 1 ? 0 : (size_t)blocks * (size_t)(2 * E + 2) * sizeof(float);
}

inline Check check_workspace(const void* workspace, size_t bytes, size_t need,
                             std::initializer_list<const gmm_tensor*> tensors) {
  if (need == 0) return {};
  if (!workspace || bytes < need) return invalid("the workspace needs " + std::to_string(need) + " bytes");
  if (!aligned16(workspace)) return invalid("the workspace must be 16-byte aligned");
  const gmm_tensor w{workspace, GMM_I8, 1, {(int64_t)need, 0, 0, 0}};
  for (const gmm_tensor* t : tensors)
    if (overlaps(&w, t)) return invalid("the workspace overlaps a tensor");
  return {};
}

inline Check check_balance_loss(const gmm_tensor* logits, const gmm_tensor* ids, const gmm_tensor* valid, int scores,
                                const gmm_tensor* loss, const gmm_tensor* counts, const gmm_tensor* tokens,
                                const void* workspace, size_t workspace_bytes) {
  if (!logits || !ids || !loss || !counts || !tokens)
    return invalid("logits, expert_ids, loss, counts and tokens are required");
  Check c = check_router(logits, ids, false, valid, scores);
  if (!c) return c;
  if (loss->dtype != GMM_F32 || !has_shape(loss, {1})) return invalid("loss must be one f32");
  if (counts->dtype != GMM_I32 || !has_shape(counts, {logits->shape[1]}))
    return invalid("counts must be int32 of shape (E,), got " + shape_str(counts));
  if (tokens->dtype != GMM_I32 || !has_shape(tokens, {1})) return invalid("tokens must be one int32");
  if (!(c = check_memory({logits, ids, valid}, {loss, counts, tokens}))) return c;
  return check_workspace(workspace, workspace_bytes, balance_workspace_bytes(logits->shape[0], logits->shape[1]),
                         {logits, ids, valid, loss, counts, tokens});
}

inline Check check_router_grad(const gmm_tensor* logits, const gmm_tensor* ids, const gmm_tensor* valid, int scores,
                               const gmm_tensor* dweights, const gmm_tensor* counts, const gmm_tensor* tokens,
                               const gmm_tensor* dloss, const gmm_tensor* dlogits) {
  if (!logits || !ids || !dlogits) return invalid("logits, expert_ids and dlogits are required");
  if (!dweights && !counts) return invalid("dweights or counts are required (without both there is no gradient)");
  if (!counts != !tokens) return invalid("counts and tokens come together");
  if (dloss && !counts) return invalid("dloss without counts and tokens");
  Check c = check_router(logits, ids, false, valid, scores);
  if (!c) return c;
  if (dweights && (!is_any(dweights->dtype, {GMM_F32, GMM_BF16}) || !has_shape(dweights, {ids->shape[0], ids->shape[1]})))
    return invalid("dweights must be f32 or bf16 of expert_ids' shape, got " + shape_str(dweights));
  if (counts && (counts->dtype != GMM_I32 || !has_shape(counts, {logits->shape[1]})))
    return invalid("counts must be int32 of shape (E,), got " + shape_str(counts));
  if (tokens && (tokens->dtype != GMM_I32 || !has_shape(tokens, {1}))) return invalid("tokens must be one int32");
  if (dloss && (dloss->dtype != GMM_F32 || !has_shape(dloss, {1}))) return invalid("dloss must be one f32");
  if (dlogits->dtype != logits->dtype || !has_shape(dlogits, {logits->shape[0], logits->shape[1]}))
    return invalid("dlogits must have logits' dtype and shape, got " + shape_str(dlogits));
  return check_memory({logits, ids, valid, dweights, counts, tokens, dloss}, {dlogits});
}

// Up to so many slots the weighted sums are taken in one launch, without a
// workspace.
constexpr long long kGmvAtOnce = 16;

inline size_t gmv_workspace_bytes(long long slots, long long N, bool weighted) {
  return weighted && slots > kGmvAtOnce ? (size_t)slots * (size_t)N * sizeof(float) : 0;
}

inline Check check_gmv_limits(long long slots, long long N) {
  if (slots < 0 || N < 1) return invalid("negative or zero extent");
  if (slots > kMaxGmvSlots) return unsupported("more than 4096 slots (T*k): gmm_run takes sorted rows");
  if (N >= kMaxGmvCols) return unsupported("2^24 columns or more");
  return {};
}

inline Check check_gmv(const gmm_tensor* x, const gmm_tensor* rhs, const gmm_tensor* scale, const gmm_tensor* zero,
                       const gmm_tensor* ids, const gmm_tensor* weights, const gmm_tensor* out, const void* workspace,
                       size_t workspace_bytes) {
  if (!x || !rhs || !scale || !out) return invalid("x, rhs, rhs_scale and out are required");
  if (x->dtype != GMM_BF16) return invalid("x must be bf16");
  if (!is_any(rhs->dtype, {GMM_I4, GMM_U4, GMM_F4E2M1})) return invalid("rhs must be int4, uint4 or fp4 e2m1");
  if (rhs->ndim != 3 || rhs->shape[0] < 1 || rhs->shape[1] < 1 || rhs->shape[2] < 1)
    return invalid("expected rhs of shape (G, N, K), got " + shape_str(rhs));
  const long long G = rhs->shape[0], N = rhs->shape[1], K = rhs->shape[2];
  if (G > gmmk::kMaxGroups) return unsupported("more than 1024 groups");
  if (K >= kMaxGmvK) return unsupported("K of 2^20 or more");
  if (K % 32) return invalid("K must be a multiple of 32");
  long long T, k;
  Check c;
  if (ids) {
    if (!is_any(ids->dtype, {GMM_I32, GMM_I64})) return invalid("expert_ids must be int32 or int64");
    if (!(c = check_slots(ids, "expert_ids"))) return c;
    T = ids->shape[0], k = ids->shape[1];
  } else {
    if (G != 1) return invalid("expert_ids are required with more than one group");
    if (x->ndim < 2 || x->shape[0] < 0) return invalid("expected x of shape (T, K) or (T, k, K)");
    T = x->shape[0], k = 1;
    if (T >= kMaxExtent) return unsupported("2^31 tokens or more");
  }
  if (!(c = check_gmv_limits(T * k, N))) return c;
  if (!(x->ndim == 3 ? has_shape(x, {T, k, K}) : has_shape(x, {T, K})))
    return invalid("expected x of shape (T, K) or (T, k, K), got " + shape_str(x));
  if (scale->ndim != 4 || scale->shape[0] != G || scale->shape[1] < 1 || scale->shape[2] != 1 || scale->shape[3] != N)
    return invalid("expected rhs_scale of shape (G, nb, 1, N), got " + shape_str(scale));
  const long long nb = scale->shape[1];
  if (nb > K || K % nb || K / nb % 32) return invalid("K/nb must be a multiple of 32");
  if (scale->dtype == GMM_E8M0) {
    if (rhs->dtype != GMM_F4E2M1 || K / nb != 32) return invalid("E8M0 scales belong to fp4 e2m1 in blocks of 32");
  } else if (!is_any(scale->dtype, {GMM_F32, GMM_BF16})) {
    return invalid("rhs_scale must be f32, bf16 or E8M0");
  }
  if (zero) {
    if (rhs->dtype == GMM_F4E2M1) return invalid("fp4 e2m1 has no zero points");
    if (zero->dtype != scale->dtype || !has_shape(zero, {G, nb, 1, N}))
      return invalid("rhs_zero must have rhs_scale's dtype and shape, got " + shape_str(zero));
  }
  if (weights && !(c = check_weights(weights, T, k))) return c;
  if (!is_any(out->dtype, {GMM_F32, GMM_BF16})) return invalid("out must be f32 or bf16");
  if (!(weights ? has_shape(out, {T, N}) : has_shape(out, {T, k, N})))
    return invalid(std::string("expected out of shape ") + (weights ? "(T, N)" : "(T, k, N)") + ", got " + shape_str(out));
  if (!(c = check_memory({x, rhs, scale, zero, ids, weights}, {out}))) return c;
  return check_workspace(workspace, workspace_bytes, gmv_workspace_bytes(T * k, N, weights),
                         {x, rhs, scale, zero, ids, weights, out});
}

// Byte ranges that a step writes must not meet one another or a gradient.
inline bool ranges_overlap(std::vector<std::pair<const char*, const char*>>& r) {
  const auto before = [](const auto& a, const auto& b) { return a.first < b.first; };
  if (!std::is_sorted(r.begin(), r.end(), before)) std::sort(r.begin(), r.end(), before);
  for (size_t i = 1; i < r.size(); ++i)
    if (r[i].first < r[i - 1].second) return true;
  return false;
}

inline Check check_adamw(const gmm_adamw_item* items, int64_t count, const gmm_adamw_args* a) {
  if (!a) return invalid("args are required");
  if (count < 0 || (count > 0 && !items)) return invalid("items are required");
  if (!is_any(a->param_dtype, {GMM_F32, GMM_BF16}) || !is_any(a->grad_dtype, {GMM_F32, GMM_BF16}))
    return invalid("parameters and gradients must be f32 or bf16");
  if (!is_any(a->state_dtype, {GMM_F32, GMM_F8E4M3FN})) return invalid("states must be f32 or e4m3fn");
  if (!(a->lr >= 0) || std::isinf(a->lr)) return invalid("lr must be finite and not negative");
  if (!(a->beta1 >= 0 && a->beta1 < 1 && a->beta2 >= 0 && a->beta2 < 1)) return invalid("betas must be in [0, 1)");
  if (!(a->eps >= 0) || std::isinf(a->eps)) return invalid("eps must be finite and not negative");
  if (!(a->weight_decay >= 0) || std::isinf(a->weight_decay)) return invalid("weight_decay must be finite and not negative");
  if (!a->step_at && a->step < 1) return invalid("steps are counted from 1");
  if ((reinterpret_cast<uintptr_t>(a->step_at) | reinterpret_cast<uintptr_t>(a->lr_at) |
       reinterpret_cast<uintptr_t>(a->grad_scale)) & 3)
    return invalid("step_at, lr_at and grad_scale must be 4-byte aligned");
  const bool eight = a->state_dtype == GMM_F8E4M3FN;
  const int ps = elem_size(a->param_dtype), gs = elem_size(a->grad_dtype), ss = eight ? 1 : 4;
  std::vector<std::pair<const char*, const char*>> out;
  out.reserve(6 * (size_t)count);
  for (int64_t i = 0; i < count; ++i) {
    const gmm_adamw_item& t = items[i];
    const std::string who = "tensor " + std::to_string(i) + ": ";
    if (t.n < 0) return invalid(who + "negative number of elements");
    if (t.n >= kMaxAdamElems) return unsupported(who + "2^34 elements or more");
    if (t.n == 0) continue;
    if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq) return invalid(who + "null data pointer");
    if (eight != (t.exp_avg_scale != nullptr) || eight != (t.exp_avg_sq_scale != nullptr))
      return invalid(who + (eight ? "eight-bit states need scales" : "f32 states have no scales"));
    for (const void* p : {(const void*)t.param, t.grad, (const void*)t.exp_avg, (const void*)t.exp_avg_sq,
                          (const void*)t.exp_avg_scale, (const void*)t.exp_avg_sq_scale, (const void*)t.copy})
      if (!aligned16(p)) return invalid(who + "tensor data must be 16-byte aligned");
    const long long blocks = (t.n + GMM_ADAMW_BLOCK - 1) / GMM_ADAMW_BLOCK;
    const auto add = [&out](const void* p, long long bytes) {
      if (p) out.emplace_back(static_cast<const char*>(p), static_cast<const char*>(p) + bytes);
    };
    add(t.param, t.n * ps);
    add(t.exp_avg, t.n * ss);
    add(t.exp_avg_sq, t.n * ss);
    add(t.exp_avg_scale, blocks * 4);
    add(t.exp_avg_sq_scale, blocks * 4);
    add(t.copy, t.n * 2);
  }
  if (ranges_overlap(out)) return invalid("tensors of the step overlap");
  // (gradients may share memory with one another, not with what is written)
  const auto written = [&out](const void* p, long long bytes) {
    const char* const a = static_cast<const char*>(p);
    if (!a || out.empty()) return false;
    const auto it = std::lower_bound(out.begin(), out.end(), a + bytes,
                                     [](const auto& r, const char* end) { return r.first < end; });
    return it != out.begin() && std::prev(it)->second > a;
  };
  for (int64_t i = 0; i < count; ++i)
    if (items[i].n > 0 && written(items[i].grad, items[i].n * gs)) return invalid("a gradient overlaps a tensor that is written");
  if (written(a->step_at, 4) || written(a->lr_at, 4) || written(a->grad_scale, 4))
    return invalid("step_at, lr_at or grad_scale overlaps a tensor that is written");
  return {};
}

}  // namespace gmmh
