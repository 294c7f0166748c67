"""ctypes binding of the entry points of include/gmm_moe.h: tokens sorted by
expert, dispatched into expert rows and combined back, with gradients, and
microscaled fp4 tensors.

Argument marshalling only, as in _binding.py: the checks and the computation
are the library's."""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from ._binding import (_DTYPE, _raise, _ref, _view, _view_packed, GMM_E_INVALID, GMM_I64, GmmInvalid, handle, load)

EXPORTED_MOE = ("gmm_sort_tokens_workspace", "gmm_sort_tokens_run", "gmm_dispatch_run", "gmm_combine_run",
                "gmm_combine_grad_run", "gmm_quant_mxfp4_run", "gmm_widen_mxfp4_run")
FLAG_BAD_ROW = 0x10

_ID_DTYPE = {torch.int32: _DTYPE[torch.int32], torch.int64: GMM_I64}


class _Call:
    """The views, stream and handle of one call.  Every tensor lives on the
    first one's device; outputs that the call makes are allocated on the stream
    that writes them, and kept from reuse while the current stream may still
    read them."""

    def __init__(self, stream: Optional[torch.cuda.Stream], first: torch.Tensor, name: str):
        if not isinstance(first, torch.Tensor) or not first.is_cuda:
            raise GmmInvalid(GMM_E_INVALID, f"{name} must be a device tensor")
        self.dev = first.device
        self.stream = stream if stream is not None else torch.cuda.current_stream(self.dev)
        if self.stream.device != self.dev:
            raise GmmInvalid(GMM_E_INVALID, f"the stream is on {self.stream.device}, {name} on {self.dev}")

    def view(self, t: Optional[torch.Tensor], name: str, packed: bool = False, dtypes=_DTYPE):
        if t is not None and t.is_cuda and t.device != self.dev:
            raise GmmInvalid(GMM_E_INVALID, f"{name} is on {t.device}, not on {self.dev}")
        return _view_packed(t, "fp4_e2m1", name) if packed else _view(t, name, dtypes)

    def empty(self, shape, dtype: torch.dtype) -> torch.Tensor:
        current = torch.cuda.current_stream(self.dev)
        with torch.cuda.stream(self.stream):
            t = torch.empty(shape, dtype=dtype, device=self.dev)
        if current != self.stream:
            t.record_stream(current)
        return t

    def run(self, name: str, *args) -> None:
        h = handle(self.dev)
        _raise(getattr(load(), name)(h, *[_ref(a) if hasattr(a, "_fields_") else a for a in args],
                                     ctypes.c_void_p(self.stream.cuda_stream)), h)


def sort_tokens(expert_ids: torch.Tensor, num_groups: int, *,
                group_sizes: Optional[torch.Tensor] = None,
                slot_row: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None):
    """Stable sort of the slots of expert_ids [T,k] (int32 or int64) by expert
    through libgmm.so (gmm_sort_tokens_run).

    Returns (group_sizes int32 [num_groups], as gmm() takes it; slot_row int32
    [T,k], each slot's row in the sorted order).  An id outside [0, num_groups)
    leaves its slot unrouted: its row comes after all others, and slot_row
    holds the row's bitwise complement (a negative number)."""
    load()
    c = _Call(stream, expert_ids, "expert_ids")
    ids = c.view(expert_ids, "expert_ids", dtypes=_ID_DTYPE)
    need = ctypes.c_size_t(0)
    # a refused size is the run's to report, with its text
    load().gmm_sort_tokens_workspace(expert_ids.numel(), int(num_groups), ctypes.byref(need))
    if group_sizes is None:
        group_sizes = c.empty((max(int(num_groups), 0),), torch.int32)
    elif group_sizes.dim() != 1 or group_sizes.numel() != int(num_groups):
        raise GmmInvalid(GMM_E_INVALID, "group_sizes must hold num_groups elements")
    if slot_row is None:
        slot_row = c.empty(tuple(expert_ids.shape), torch.int32)
    work = c.empty((need.value,), torch.uint8) if need.value else None
    c.run("gmm_sort_tokens_run", ids, c.view(group_sizes, "group_sizes"), c.view(slot_row, "slot_row"),
          ctypes.c_void_p(work.data_ptr() if work is not None else None), need)
    return group_sizes, slot_row


def dispatch(x: torch.Tensor, slot_row: torch.Tensor, *, out: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Tokens into expert rows through libgmm.so (gmm_dispatch_run):
    rows[slot_row[t,j]] = x[t], the rows of unrouted slots zeros.  x [T,D] of
    any one-, two- or four-byte dtype, slot_row from sort_tokens(); returns
    rows [T*k,D], the lhs of gmm().  The gradient is combine(drows, slot_row)."""
    load()
    c = _Call(stream, x, "x")
    views = [c.view(x, "x"), c.view(slot_row, "slot_row")]
    if out is None:
        out = c.empty((slot_row.numel(), x.shape[1] if x.dim() == 2 else 0), x.dtype)
    c.run("gmm_dispatch_run", *views, c.view(out, "out"))
    return out


def combine(rows: torch.Tensor, slot_row: torch.Tensor, weights: Optional[torch.Tensor] = None, *,
            out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
            stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Expert rows back to tokens through libgmm.so (gmm_combine_run):
    out[t] = sum over routed slots j of weights[t,j] * rows[slot_row[t,j]], in
    float32, rounded once.  rows [T*k,D] and weights [T,k] float32 or bfloat16
    (weights None: all 1, the gradient of dispatch()); returns out [T,D] of
    out_dtype (rows' dtype by default)."""
    load()
    c = _Call(stream, rows, "rows")
    views = [c.view(rows, "rows"), c.view(slot_row, "slot_row"), c.view(weights, "weights")]
    if out is None:
        out = c.empty((slot_row.shape[0] if slot_row.dim() else 0, rows.shape[1] if rows.dim() == 2 else 0),
                      out_dtype if out_dtype is not None else rows.dtype)
    c.run("gmm_combine_run", *views, c.view(out, "out"))
    return out


def combine_grad(dout: torch.Tensor, rows: torch.Tensor, slot_row: torch.Tensor, weights: torch.Tensor, *,
                 drows: Optional[torch.Tensor] = None, dweights: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None):
    """The gradients of combine() with weights, through libgmm.so
    (gmm_combine_grad_run).  Returns (drows [T*k,D] of rows' dtype, zeros in
    the rows of unrouted slots; dweights [T,k] of weights' dtype, 0 there)."""
    load()
    c = _Call(stream, dout, "dout")
    views = [c.view(dout, "dout"), c.view(rows, "rows"), c.view(slot_row, "slot_row"), c.view(weights, "weights")]
    if weights is None:
        raise GmmInvalid(GMM_E_INVALID, "weights are required (without them the gradient is dispatch())")
    if drows is None:
        drows = c.empty(tuple(rows.shape), rows.dtype)
    if dweights is None:
        dweights = c.empty(tuple(weights.shape), weights.dtype)
    c.run("gmm_combine_grad_run", *views, c.view(drows, "drows"), c.view(dweights, "dweights"))
    return drows, dweights


def _operand(operand: str, dims: int, name: str) -> None:
    if operand not in ("lhs", "rhs"):
        raise GmmInvalid(GMM_E_INVALID, f"operand must be 'lhs' or 'rhs', got {operand!r}")
    if dims != (2 if operand == "lhs" else 3):
        raise GmmInvalid(GMM_E_INVALID, f"{name}: a {operand} is a {2 if operand == 'lhs' else 3}-tensor")


def quant_mxfp4(x: torch.Tensor, *, operand: str = "lhs", q: Optional[torch.Tensor] = None,
                scale: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """Microscaled fp4 quantisation through libgmm.so (gmm_quant_mxfp4_run):
    x bfloat16 or float32, blocks of 32 along the last dimension K.  Returns
    (q uint8 [...,K/2], two fp4 e2m1 codes a byte; scale float8_e8m0fnu) in the
    layouts that gmm() takes: operand "lhs" x [M,K] -> scale [M,K/32] (with
    lhs_format="fp4_e2m1"), "rhs" x [Ga,N,K] -> scale [Ga,K/32,1,N] (with
    rhs_format="fp4_e2m1")."""
    load()
    c = _Call(stream, x, "x")
    _operand(operand, x.dim(), "x")
    xv = c.view(x, "x")
    K = x.shape[-1]
    if q is None:
        q = c.empty(tuple(x.shape[:-1]) + (K // 2,), torch.uint8)
    if scale is None:
        scale = c.empty((x.shape[0], K // 32) if operand == "lhs" else (x.shape[0], K // 32, 1, x.shape[1]),
                        torch.float8_e8m0fnu)
    c.run("gmm_quant_mxfp4_run", xv, c.view(q, "q", packed=True), c.view(scale, "scale"))
    return q, scale


def widen_mxfp4(q: torch.Tensor, scale: torch.Tensor, *, operand: str = "lhs",
                out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The values of a microscaled fp4 tensor through libgmm.so
    (gmm_widen_mxfp4_run), exact in bfloat16 and float32: q and scale as
    quant_mxfp4() returns them for the same operand; returns [...,K]."""
    load()
    c = _Call(stream, q, "q")
    _operand(operand, q.dim(), "q")
    views = [c.view(q, "q", packed=True), c.view(scale, "scale")]
    if out is None:
        out = c.empty(tuple(q.shape[:-1]) + (2 * q.shape[-1],), out_dtype)
    c.run("gmm_widen_mxfp4_run", *views, c.view(out, "out"))
    return out
