// gmm_layer_api.cpp -- the C entry points of include/gmm_layer.h: the checks
// of gmm_layer_checks.hpp, then the launch.
#include <hip/hip_runtime.h>

#include <string>

#include "gmm_handle.hpp"
#include "gmm_layer.h"
#include "gmm_layer_checks.hpp"
#include "gmm_layer_launch.hpp"

using namespace gmmh;

static_assert(gmmk::kBalanceBlocks == 256, "balance_blocks' most");
static_assert(gmmk::kAdamBlock == GMM_ADAMW_BLOCK, "the kernels' block is the header's");
static_assert(kMaxAdamElems <= gmmk::kAdamMost * gmmk::kAdamChunk, "a tensor fits a launch");

namespace {

// Runs a check and, when it passes, the launch on the handle's device.  No
// exception leaves (an allocation of an error text can throw).
template <class CheckFn, class LaunchFn>
gmm_status checked(gmm_handle* h, CheckFn check, LaunchFn launch) {
  if (!h) return GMM_E_INVALID;
  try {
    h->err.clear();
    const Check c = check();
    if (!c) return fail(h, c.status, c.text);
    DeviceGuard g(h->device);
    const hipError_t e = launch();
    if (e != hipSuccess) return fail(h, GMM_E_HIP, std::string("kernel launch failed: ") + hipGetErrorString(e));
    return GMM_OK;
  } catch (...) {
    return GMM_E_HIP;
  }
}

template <class T>
T* written(const gmm_tensor* t) {
  return static_cast<T*>(const_cast<void*>(t->data));
}

gmmk::RouterParams router_params(const gmm_tensor* logits, const gmm_tensor* ids, const gmm_tensor* valid, int scores) {
  gmmk::RouterParams p{};
  p.logits = logits->data;
  p.x_f32 = logits->dtype == GMM_F32;
  p.T = logits->shape[0];
  p.E = (int32_t)logits->shape[1];
  p.ids = ids->data;
  p.ids64 = ids->dtype == GMM_I64;
  p.k = (int32_t)ids->shape[1];
  p.valid = valid ? static_cast<const uint8_t*>(valid->data) : nullptr;
  p.sigmoid = scores == GMM_SCORES_SIGMOID;
  return p;
}

}  // namespace

extern "C" {

gmm_status gmm_route_run(gmm_handle* h, const gmm_tensor* logits, const gmm_tensor* bias, const gmm_tensor* valid,
                         int scores, int renormalize, float scale, const gmm_tensor* expert_ids,
                         const gmm_tensor* weights, void* stream) {
  return checked(
      h, [&] { return check_route(logits, bias, valid, scores, expert_ids, weights); },
      [&] {
        gmmk::RouterParams p = router_params(logits, expert_ids, valid, scores);
        if (p.T == 0) return hipSuccess;
        p.bias = bias ? static_cast<const float*>(bias->data) : nullptr;
        p.renorm = renormalize != 0;
        p.scale = scale;
        p.ids_out = written<int32_t>(expert_ids);
        p.weights_out = written<float>(weights);
        return gmmk::launch_route(p, h->cu_count, static_cast<hipStream_t>(stream));
      });
}

gmm_status gmm_balance_loss_workspace(int64_t tokens, int64_t experts, size_t* bytes) {
  if (!bytes) return GMM_E_INVALID;
  *bytes = 0;
  try {
    if (tokens < 0 || experts < 1) return GMM_E_INVALID;
    if (experts > gmmk::kMaxGroups || tokens >= kMaxExtent || tokens * experts >= kMaxExtent) return GMM_E_UNSUPPORTED;
  } catch (...) {
    return GMM_E_HIP;
  }
  *bytes = balance_workspace_bytes(tokens, experts);
  return GMM_OK;
}

gmm_status gmm_balance_loss_run(gmm_handle* h, const gmm_tensor* logits, const gmm_tensor* expert_ids,
                                const gmm_tensor* valid, int scores, float coef, float z_coef, const gmm_tensor* loss,
                                const gmm_tensor* counts, const gmm_tensor* tokens, void* workspace,
                                size_t workspace_bytes, void* stream) {
  return checked(
      h,
      [&] {
        return check_balance_loss(logits, expert_ids, valid, scores, loss, counts, tokens, workspace, workspace_bytes);
      },
      [&] {
        gmmk::RouterParams p = router_params(logits, expert_ids, valid, scores);
        p.coef = coef;
        p.z_coef = z_coef;
        p.loss_out = written<float>(loss);
        p.counts_out = written<int32_t>(counts);
        p.tokens_out = written<int32_t>(tokens);
        p.work = static_cast<float*>(workspace);
        return gmmk::launch_balance_loss(p, balance_blocks(p.T, p.E), static_cast<hipStream_t>(stream));
      });
}

gmm_status gmm_router_grad_run(gmm_handle* h, const gmm_tensor* logits, const gmm_tensor* expert_ids,
                               const gmm_tensor* valid, int scores, const gmm_tensor* dweights, int renormalize,
                               float scale, const gmm_tensor* counts, const gmm_tensor* tokens, const gmm_tensor* dloss,
                               float coef, float z_coef, const gmm_tensor* dlogits, void* stream) {
  return checked(
      h,
      [&] { return check_router_grad(logits, expert_ids, valid, scores, dweights, counts, tokens, dloss, dlogits); },
      [&] {
        gmmk::RouterParams p = router_params(logits, expert_ids, valid, scores);
        if (p.T == 0) return hipSuccess;
        p.renorm = renormalize != 0;
        p.scale = scale;
        p.dweights = dweights ? dweights->data : nullptr;
        p.dw_f32 = dweights && dweights->dtype == GMM_F32;
        p.counts = counts ? static_cast<const int32_t*>(counts->data) : nullptr;
        p.tokens = tokens ? static_cast<const int32_t*>(tokens->data) : nullptr;
        p.dloss = dloss ? static_cast<const float*>(dloss->data) : nullptr;
        p.coef = coef;
        p.z_coef = z_coef;
        p.dlogits = written<void>(dlogits);
        return gmmk::launch_router_grad(p, h->cu_count, static_cast<hipStream_t>(stream));
      });
}

gmm_status gmm_gmv_workspace(int64_t slots, int64_t N, int weighted, size_t* bytes) {
  if (!bytes) return GMM_E_INVALID;
  *bytes = 0;
  try {
    const Check c = check_gmv_limits(slots, N);
    if (!c) return c.status;
  } catch (...) {
    return GMM_E_HIP;
  }
  *bytes = gmv_workspace_bytes(slots, N, weighted != 0);
  return GMM_OK;
}

gmm_status gmm_gmv_run(gmm_handle* h, const gmm_tensor* x, const gmm_tensor* rhs, const gmm_tensor* rhs_scale,
                       const gmm_tensor* rhs_zero, const gmm_tensor* expert_ids, const gmm_tensor* weights,
                       const gmm_tensor* out, void* workspace, size_t workspace_bytes, void* stream) {
  return checked(
      h,
      [&] { return check_gmv(x, rhs, rhs_scale, rhs_zero, expert_ids, weights, out, workspace, workspace_bytes); },
      [&] {
        gmmk::GmvParams p{};
        p.T = (int32_t)x->shape[0];
        if (p.T == 0) return hipSuccess;
        p.k = expert_ids ? (int32_t)expert_ids->shape[1] : 1;
        p.n = p.T * p.k;
        p.G = (int32_t)rhs->shape[0];
        p.N = (int32_t)rhs->shape[1];
        p.K = (int32_t)rhs->shape[2];
        p.nb = (int32_t)rhs_scale->shape[1];
        p.blk = p.K / p.nb;
        p.x = static_cast<const uint16_t*>(x->data);
        p.per_slot = x->ndim == 3;
        p.rhs = static_cast<const uint8_t*>(rhs->data);
        p.fmt = rhs->dtype == GMM_I4 ? 3 : rhs->dtype == GMM_U4 ? 4 : 5;
        p.scale = rhs_scale->data;
        p.scale_kind = rhs_scale->dtype == GMM_F32 ? gmmk::kGmvF32 : rhs_scale->dtype == GMM_BF16 ? gmmk::kGmvBf16 : gmmk::kGmvE8m0;
        p.zero = rhs_zero ? rhs_zero->data : nullptr;
        p.ids = expert_ids ? expert_ids->data : nullptr;
        p.ids64 = expert_ids && expert_ids->dtype == GMM_I64;
        p.weights = weights ? weights->data : nullptr;
        p.w_f32 = weights && weights->dtype == GMM_F32;
        p.out = written<void>(out);
        p.out_f32 = out->dtype == GMM_F32;
        p.work = static_cast<float*>(workspace);
        p.experts = 2 * p.n < p.G || p.n <= 64 ? (p.n < p.G ? p.n : p.G) : p.G;
        p.blk_magic = gmmk::gmv_magic(p.blk);
        p.at_once = p.weights && p.n <= kGmvAtOnce;
        return gmmk::launch_gmv(p, h->cu_count, static_cast<hipStream_t>(stream));
      });
}

gmm_status gmm_adamw_run(gmm_handle* h, const gmm_adamw_item* items, int64_t count, const gmm_adamw_args* a,
                         void* stream) {
  return checked(
      h, [&] { return check_adamw(items, count, a); },
      [&] {
        gmmk::AdamParams p{};
        p.lr = a->lr;
        p.beta1 = a->beta1;
        p.beta2 = a->beta2;
        p.weight_decay = a->weight_decay;
        p.step = a->step;
        p.step_at = a->step_at;
        p.lr_at = a->lr_at;
        p.grad_scale = a->grad_scale;
        if (!a->step_at && !a->lr_at) {
          const gmmk::AdamFactors f = gmmk::adam_factors(a->lr, a->beta1, a->beta2, a->weight_decay, a->step);
          p.decay = f.decay;
          p.rate = f.rate;
          p.root_scale = f.root_scale;
        }
        p.b1 = (float)a->beta1;
        p.c1 = (float)(1 - a->beta1);
        p.b2 = (float)a->beta2;
        p.c2 = (float)(1 - a->beta2);
        p.eps = (float)a->eps;
        const bool eight = a->state_dtype == GMM_F8E4M3FN;
        const int per = elem_size(a->param_dtype) + elem_size(a->grad_dtype) + 2 * (eight ? 1 : 4);
        long long bytes = 0;  // that the step reads
        for (int64_t i = 0; i < count; ++i) bytes += items[i].n * per;
        const auto run = [&] {
          return gmmk::launch_adamw(p, a->param_dtype == GMM_F32, a->grad_dtype == GMM_F32, eight,
                                    bytes > gmmk::kAdamCached, static_cast<hipStream_t>(stream));
        };
        hipError_t e = hipSuccess;
        for (int64_t i = 0; i < count; ++i) {
          const gmm_adamw_item& t = items[i];
          if (t.n == 0) continue;
          const long long chunks = (t.n + gmmk::kAdamChunk - 1) / gmmk::kAdamChunk;
          if (p.count && p.first[p.count] + chunks > gmmk::kAdamMost) {
            if ((e = run()) != hipSuccess) return e;
            p.count = 0;
          }
          p.item[p.count] = {t.param, t.grad, t.exp_avg, t.exp_avg_sq, t.exp_avg_scale, t.exp_avg_sq_scale,
                             static_cast<uint16_t*>(t.copy), t.n};
          p.first[p.count + 1] = p.first[p.count] + (int32_t)chunks;
          if (++p.count == gmmk::kAdamItems) {
            if ((e = run()) != hipSuccess) return e;
            p.count = 0;
          }
        }
        return p.count ? run() : e;
      });
}

}  // extern "C"
