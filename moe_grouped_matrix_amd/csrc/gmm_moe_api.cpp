// gmm_moe_api.cpp -- the C entry points of include/gmm_moe.h: the checks of
// gmm_moe_checks.hpp, then the launch.
#include <hip/hip_runtime.h>

#include <string>

#include "gmm_handle.hpp"
#include "gmm_moe.h"
#include "gmm_moe_checks.hpp"
#include "gmm_moe_launch.hpp"

using namespace gmmh;

static_assert(gmmk::kFlagBadRow == GMM_FLAG_BAD_ROW, "the kernels' flag bit is the header's");

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

void* mutable_data(const gmm_tensor* t) { return const_cast<void*>(t->data); }

gmmk::RowParams row_params(const gmm_handle* h, const gmm_tensor* slot_row, const gmm_tensor* weights, long long D) {
  gmmk::RowParams p{};
  p.slot_row = static_cast<const int32_t*>(slot_row->data);
  p.weights = weights ? weights->data : nullptr;
  p.w_f32 = weights && weights->dtype == GMM_F32;
  p.flags = h->flags;
  p.T = slot_row->shape[0];
  p.k = (int32_t)slot_row->shape[1];
  p.n = p.T * p.k;
  p.D = (int32_t)D;
  return p;
}

}  // namespace

extern "C" {

gmm_status gmm_sort_tokens_workspace(int64_t slots, int64_t groups, size_t* bytes) {
  if (!bytes) return GMM_E_INVALID;
  *bytes = 0;
  try {
    const Check c = check_sort_limits(slots, groups);
    if (!c) return c.status;
  } catch (...) {
    return GMM_E_HIP;
  }
  *bytes = sort_workspace_bytes(slots, groups);
  return GMM_OK;
}

gmm_status gmm_sort_tokens_run(gmm_handle* h, const gmm_tensor* expert_ids, const gmm_tensor* group_sizes,
                               const gmm_tensor* slot_row, void* workspace, size_t workspace_bytes, void* stream) {
  return checked(
      h, [&] { return check_sort_tokens(expert_ids, group_sizes, slot_row, workspace, workspace_bytes); },
      [&] {
        gmmk::SortParams p{};
        p.ids = expert_ids->data;
        p.ids64 = expert_ids->dtype == GMM_I64;
        p.group_sizes = static_cast<int32_t*>(mutable_data(group_sizes));
        p.slot_row = static_cast<int32_t*>(mutable_data(slot_row));
        p.counts = static_cast<int32_t*>(workspace);
        p.n = expert_ids->shape[0] * expert_ids->shape[1];
        p.G = (int32_t)group_sizes->shape[0];
        const SortSplit s = sort_split(p.n, p.G);
        p.per = s.per;
        return gmmk::launch_sort(p, s.blocks, static_cast<hipStream_t>(stream));
      });
}

gmm_status gmm_dispatch_run(gmm_handle* h, const gmm_tensor* x, const gmm_tensor* slot_row, const gmm_tensor* out,
                            void* stream) {
  return checked(
      h, [&] { return check_dispatch(x, slot_row, out); },
      [&] {
        gmmk::RowParams p = row_params(h, slot_row, nullptr, x->shape[1] * elem_size(x->dtype));
        if (p.T == 0) return hipSuccess;
        p.a = x->data;
        p.out = mutable_data(out);
        return gmmk::launch_dispatch(p, h->cu_count, static_cast<hipStream_t>(stream));
      });
}

gmm_status gmm_combine_run(gmm_handle* h, const gmm_tensor* rows, const gmm_tensor* slot_row,
                           const gmm_tensor* weights, const gmm_tensor* out, void* stream) {
  return checked(
      h, [&] { return check_combine(rows, slot_row, weights, out); },
      [&] {
        gmmk::RowParams p = row_params(h, slot_row, weights, rows->shape[1]);
        if (p.T == 0) return hipSuccess;
        p.a = rows->data;
        p.out = mutable_data(out);
        return gmmk::launch_combine(p, rows->dtype == GMM_F32, out->dtype == GMM_F32, h->cu_count,
                                    static_cast<hipStream_t>(stream));
      });
}

gmm_status gmm_combine_grad_run(gmm_handle* h, const gmm_tensor* dout, const gmm_tensor* rows,
                                const gmm_tensor* slot_row, const gmm_tensor* weights, const gmm_tensor* drows,
                                const gmm_tensor* dweights, void* stream) {
  return checked(
      h, [&] { return check_combine_grad(dout, rows, slot_row, weights, drows, dweights); },
      [&] {
        gmmk::RowParams p = row_params(h, slot_row, weights, rows->shape[1]);
        if (p.T == 0) return hipSuccess;
        p.a = rows->data;
        p.b = dout->data;
        p.out = mutable_data(drows);
        p.dweights = mutable_data(dweights);
        return gmmk::launch_combine_grad(p, dout->dtype == GMM_F32, rows->dtype == GMM_F32, h->cu_count,
                                         static_cast<hipStream_t>(stream));
      });
}

static gmmk::Mxfp4Params mx_params(const gmm_tensor* wide, const gmm_tensor* scale) {
  gmmk::Mxfp4Params p{};
  const bool rhs = wide->ndim == 3;
  p.rows = rhs ? wide->shape[0] * wide->shape[1] : wide->shape[0];
  p.K = (int32_t)wide->shape[rhs ? 2 : 1];
  p.rhs = rhs ? (int32_t)wide->shape[1] : 0;
  p.wide_f32 = wide->dtype == GMM_F32;
  p.scale = static_cast<uint8_t*>(mutable_data(scale));
  return p;
}

gmm_status gmm_quant_mxfp4_run(gmm_handle* h, const gmm_tensor* x, const gmm_tensor* q, const gmm_tensor* scale,
                               void* stream) {
  return checked(
      h, [&] { return check_mxfp4(x, q, scale, true); },
      [&] {
        gmmk::Mxfp4Params p = mx_params(x, scale);
        if (p.rows == 0) return hipSuccess;
        p.src = x->data;
        p.dst = mutable_data(q);
        return gmmk::launch_quant_mxfp4(p, h->cu_count, static_cast<hipStream_t>(stream));
      });
}

gmm_status gmm_widen_mxfp4_run(gmm_handle* h, const gmm_tensor* q, const gmm_tensor* scale, const gmm_tensor* y,
                               void* stream) {
  return checked(
      h, [&] { return check_mxfp4(y, q, scale, false); },
      [&] {
        gmmk::Mxfp4Params p = mx_params(y, scale);
        if (p.rows == 0) return hipSuccess;
        p.src = q->data;
        p.dst = mutable_data(y);
        return gmmk::launch_widen_mxfp4(p, h->cu_count, static_cast<hipStream_t>(stream));
      });
}

}  // extern "C"
