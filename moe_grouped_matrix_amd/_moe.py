"""ctypes binding of the entry points of include/gmm_moe.h: tokens sorted by
expert, dispatched into expert rows and combined back, with gradients, and
microscaled fp4 tensors.

Argument marshalling only, as in _binding.py: the checks and the computation
are the library's.  The common call (outputs to be made, the current stream)
is marshalled by compiled host code, _moe_ext.so; every other one here."""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import os
import threading
import warnings
from typing import Optional

import torch

from ._binding import (_DTYPE, _PAD, _TENSOR, _empty, _handles, _raise, _raw_stream, _record, GMM_E_INVALID,
                       GMM_F4E2M1, GMM_I64, GmmInvalid, LIB_PATH, handle, load)

# in the order of _moe_ext's bind() and bind_layer()
EXPORTED_MOE = ("gmm_sort_tokens_workspace", "gmm_sort_tokens_run", "gmm_dispatch_run", "gmm_combine_run",
                "gmm_combine_grad_run", "gmm_quant_mxfp4_run", "gmm_widen_mxfp4_run")
EXPORTED_LAYER = ("gmm_route_run", "gmm_balance_loss_workspace", "gmm_balance_loss_run", "gmm_router_grad_run",
                  "gmm_gmv_workspace", "gmm_gmv_run", "gmm_adamw_run")
FLAG_BAD_ROW = 0x10

_ID_DTYPE = {torch.int32: _DTYPE[torch.int32], torch.int64: GMM_I64}
_BYTE_DTYPE = {**_DTYPE, torch.uint8: _DTYPE[torch.int8]}  # rows that are only copied
_PACKED_DTYPE = {torch.uint8: GMM_F4E2M1, torch.float4_e2m1fn_x2: GMM_F4E2M1}

# These calls take a few microseconds on the GPU for a decode step, so the
# host's share counts.  _moe_ext does the common call without a Python step in
# between; it returns None for every other one, and for a refused one, which
# then goes the long way below and is told why.
EXT_PATH = os.path.join(os.path.dirname(LIB_PATH), "_moe_ext.so")
_ext = None
_ext_lock = threading.Lock()


class _NoExt:
    """Stands in where _moe_ext.so is not built: every call goes the long way."""

    def set_handle(self, *_):
        return None

    sort_tokens = dispatch = combine = combine_grad = quant_mxfp4 = widen_mxfp4 = set_handle
    route = balance_loss = router_grad = gmv = adamw = set_handle


def _load_ext():
    global _ext
    lib = load()
    with _ext_lock:
        if _ext is not None:
            return _ext
        try:
            spec = importlib.util.spec_from_file_location("_moe_ext", EXT_PATH)
            ext = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(ext)
        except ImportError as e:
            warnings.warn(f"{EXT_PATH} is not built or does not load ({e}); the token and fp4 operators are marshalled "
                          "in Python, some microseconds a call slower", RuntimeWarning, stacklevel=3)
            ext = _NoExt()
        else:
            for bind, names in ((ext.bind, EXPORTED_MOE), (ext.bind_layer, EXPORTED_LAYER)):
                bind(*[ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in names])
            for dev, h in list(_handles.items()):
                ext.set_handle(dev, h)
        _ext = ext
        return ext


def _current(t) -> int:
    """The raw current stream of a device tensor's device (0 otherwise)."""
    dev = t.get_device() if isinstance(t, torch.Tensor) else -1
    return torch._C._cuda_getCurrentRawStream(dev) if dev >= 0 else 0


def _refuse(text: str):
    raise GmmInvalid(GMM_E_INVALID, text)


def _unfit(t: torch.Tensor, name: str, dev: torch.device) -> None:
    """Says why _pack does not take a tensor."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _refuse(f"{name} must be a device tensor")
    if t.device != dev:
        _refuse(f"{name} is on {t.device}, not on {dev}")
    if not t.is_contiguous():
        _refuse(f"{name} must be contiguous")
    if t.dim() > 4 or t.dim() == 0:
        _refuse(f"{name}: rank {t.dim()} is not supported")
    _refuse(f"{name}: unsupported dtype {t.dtype}")


def _pack(t: torch.Tensor, name: str, dev: torch.device, dtypes=_DTYPE) -> bytes:
    """The C struct of a dense tensor on `dev`.  Packed four-bit bytes
    (dtypes _PACKED_DTYPE) count elements, two to a byte of the last
    dimension."""
    try:
        code, n = dtypes.get(t.dtype), t.dim()
        if code is None or t.device != dev or not t.is_contiguous() or n > 4 or n == 0:
            _unfit(t, name, dev)
    except AttributeError:
        _unfit(t, name, dev)
    at = t.data_ptr()
    if at & 15 and t.numel() == 0:
        at = 0
    return _struct(at, code, t.shape)


def _struct(at: int, code: int, shape) -> bytes:
    n = len(shape)
    if code == GMM_F4E2M1:
        shape = (*shape[:-1], 2 * shape[-1])
    if n == 2:
        return _TENSOR.pack(at, code, 2, shape[0], shape[1], 0, 0)
    return _TENSOR.pack(at, code, n, *shape, *_PAD[n])


def _device(t: torch.Tensor, name: str) -> torch.device:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        load()
        _refuse(f"{name} must be a device tensor")
    return t.device


def _out(t: Optional[torch.Tensor], name: str, shape, dtype: torch.dtype, dev: torch.device,
         stream: Optional[torch.cuda.Stream], dtypes=_DTYPE):
    """The caller's output or a new one of this shape, and its C struct."""
    if t is not None:
        return t, _pack(t, name, dev, dtypes)
    code = dtypes.get(dtype)
    if code is None:
        _refuse(f"{name}: unsupported dtype {dtype}")
    t = _empty(shape, dtype, dev, stream)
    return t, _struct(t.data_ptr(), code, shape)


def _run(fn, dev: torch.device, stream: Optional[torch.cuda.Stream], tensors, *args) -> None:
    """The call itself.  On a stream of the caller's choice its tensors, the
    caller's own outputs among them, are kept from reuse until that stream is
    done with them."""
    raw = _raw_stream(stream, dev)
    h = handle(dev)
    status = fn(h, *args, raw)
    if status:
        _raise(status, h)
    (_ext or _load_ext()).set_handle(dev.index, h)
    _record(stream, tensors)


@functools.lru_cache(maxsize=4096)
def _sort_workspace(slots: int, groups: int) -> int:
    need = ctypes.c_size_t(0)
    # a refused size is the run's to report, with its text
    load().gmm_sort_tokens_workspace(slots, groups, ctypes.byref(need))
    return need.value


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
    if group_sizes is None and slot_row is None and stream is None:
        made = (_ext or _load_ext()).sort_tokens(expert_ids, int(num_groups), _current(expert_ids))
        if made is not None:
            return made
    dev = _device(expert_ids, "expert_ids")
    ids = _pack(expert_ids, "expert_ids", dev, _ID_DTYPE)
    groups = int(num_groups)
    if group_sizes is not None and (group_sizes.dim() != 1 or group_sizes.numel() != groups):
        _refuse("group_sizes must hold num_groups elements")
    # (a number past the limit of 1024 is refused by the run, whatever the output holds)
    group_sizes, gv = _out(group_sizes, "group_sizes", (min(max(groups, 0), 1025),), torch.int32, dev, stream)
    slot_row, sv = _out(slot_row, "slot_row", expert_ids.shape, torch.int32, dev, stream)
    need = _sort_workspace(expert_ids.numel(), group_sizes.numel())
    work = _empty((need,), torch.uint8, dev, stream) if need else None
    _run(load().gmm_sort_tokens_run, dev, stream, (expert_ids, group_sizes, slot_row), ids, gv, sv, work.data_ptr() if need else None, need)
    return group_sizes, slot_row


def dispatch(x: torch.Tensor, slot_row: torch.Tensor, *, out: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Tokens into expert rows through libgmm.so (gmm_dispatch_run):
    rows[slot_row[t,j]] = x[t], the rows of unrouted slots zeros.  x [T,D] of
    any dtype that gmm() takes, or uint8 (packed fp4 codes; their scales
    [T,K/32] and quant()'s [T,K/128] go the same way), slot_row from
    sort_tokens(); returns rows [T*k,D], the lhs of gmm().  The gradient is
    combine(drows, slot_row)."""
    if out is None and stream is None:
        made = (_ext or _load_ext()).dispatch(x, slot_row, _current(x))
        if made is not None:
            return made
    dev = _device(x, "x")
    xv, sv = _pack(x, "x", dev, _BYTE_DTYPE), _pack(slot_row, "slot_row", dev)
    out, ov = _out(out, "out", (slot_row.numel(), x.shape[1] if x.dim() == 2 else 0), x.dtype, dev, stream, _BYTE_DTYPE)
    _run(load().gmm_dispatch_run, dev, stream, (x, slot_row, out), xv, sv, ov)
    return out


def combine(rows: torch.Tensor, slot_row: torch.Tensor, weights: Optional[torch.Tensor] = None, *,
            out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
            stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Expert rows back to tokens through libgmm.so (gmm_combine_run):
    out[t] = sum over routed slots j of weights[t,j] * rows[slot_row[t,j]], in
    float32, rounded once.  rows [T*k,D] and weights [T,k] float32 or bfloat16
    (weights None: all 1, the gradient of dispatch()); returns out [T,D] of
    out_dtype (rows' dtype by default)."""
    if out is None and stream is None:
        made = (_ext or _load_ext()).combine(rows, slot_row, weights,
                                             -1 if out_dtype is None else _DTYPE.get(out_dtype, -2), _current(rows))
        if made is not None:
            return made
    dev = _device(rows, "rows")
    rv, sv = _pack(rows, "rows", dev), _pack(slot_row, "slot_row", dev)
    wv = _pack(weights, "weights", dev) if weights is not None else None
    out, ov = _out(out, "out", (slot_row.shape[0], rows.shape[1] if rows.dim() == 2 else 0),
                   out_dtype if out_dtype is not None else rows.dtype, dev, stream)
    _run(load().gmm_combine_run, dev, stream, (rows, slot_row, weights, out), rv, sv, wv, ov)
    return out


def combine_grad(dout: torch.Tensor, rows: torch.Tensor, slot_row: torch.Tensor, weights: torch.Tensor, *,
                 drows: Optional[torch.Tensor] = None, dweights: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None):
    """The gradients of combine() with weights, through libgmm.so
    (gmm_combine_grad_run).  Returns (drows [T*k,D] of rows' dtype, zeros in
    the rows of unrouted slots; dweights [T,k] of weights' dtype, 0 there)."""
    if drows is None and dweights is None and stream is None:
        made = (_ext or _load_ext()).combine_grad(dout, rows, slot_row, weights, _current(dout))
        if made is not None:
            return made
    dev = _device(dout, "dout")
    if weights is None:
        _refuse("weights are required (without them the gradient is dispatch())")
    views = [_pack(t, n, dev) for t, n in ((dout, "dout"), (rows, "rows"), (slot_row, "slot_row"),
                                           (weights, "weights"))]
    drows, rv = _out(drows, "drows", rows.shape, rows.dtype, dev, stream)
    dweights, wv = _out(dweights, "dweights", weights.shape, weights.dtype, dev, stream)
    _run(load().gmm_combine_grad_run, dev, stream, (dout, rows, slot_row, weights, drows, dweights), *views, rv,
         wv)
    return drows, dweights


_RANK = {"lhs": 2, "rhs": 3}


def _operand(operand: str, dims: int, name: str) -> None:
    if operand not in _RANK:
        _refuse(f"operand must be 'lhs' or 'rhs', got {operand!r}")
    if dims != _RANK[operand]:
        _refuse(f"{name}: a {operand} is a {_RANK[operand]}-tensor")


def quant_mxfp4(x: torch.Tensor, *, operand: str = "lhs", q: Optional[torch.Tensor] = None,
                scale: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """Microscaled fp4 quantisation through libgmm.so (gmm_quant_mxfp4_run):
    x bfloat16 or float32, blocks of 32 along the last dimension K.  Returns
    (q uint8 [...,K/2], two fp4 e2m1 codes a byte; scale float8_e8m0fnu) in the
    layouts that gmm() takes: operand "lhs" x [M,K] -> scale [M,K/32] (with
    lhs_format="fp4_e2m1"), "rhs" x [Ga,N,K] -> scale [Ga,K/32,1,N] (with
    rhs_format="fp4_e2m1")."""
    if q is None and scale is None and stream is None and operand in _RANK:
        made = (_ext or _load_ext()).quant_mxfp4(x, _RANK[operand], _current(x))
        if made is not None:
            return made
    dev = _device(x, "x")
    _operand(operand, x.dim(), "x")
    xv = _pack(x, "x", dev)
    shape = x.shape
    K = shape[-1]
    q, qv = _out(q, "q", (*shape[:-1], K // 2), torch.uint8, dev, stream, _PACKED_DTYPE)
    scale, sv = _out(scale, "scale", (shape[0], K // 32) if operand == "lhs" else (shape[0], K // 32, 1, shape[1]),
                     torch.float8_e8m0fnu, dev, stream)
    _run(load().gmm_quant_mxfp4_run, dev, stream, (x, q, scale), xv, qv, sv)
    return q, scale


def widen_mxfp4(q: torch.Tensor, scale: torch.Tensor, *, operand: str = "lhs",
                out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The values of a microscaled fp4 tensor through libgmm.so
    (gmm_widen_mxfp4_run), exact in bfloat16 and float32: q and scale as
    quant_mxfp4() returns them for the same operand; returns [...,K]."""
    if out is None and stream is None and operand in _RANK:
        made = (_ext or _load_ext()).widen_mxfp4(q, scale, _RANK[operand], _DTYPE.get(out_dtype, -2), _current(q))
        if made is not None:
            return made
    dev = _device(q, "q")
    _operand(operand, q.dim(), "q")
    qv, sv = _pack(q, "q", dev, _PACKED_DTYPE), _pack(scale, "scale", dev)
    out, ov = _out(out, "out", (*q.shape[:-1], 2 * q.shape[-1]), out_dtype, dev, stream)
    _run(load().gmm_widen_mxfp4_run, dev, stream, (q, scale, out), qv, sv, ov)
    return out
