"""ctypes binding of the entry points of include/gmm_layer.h: the router of a
mixture-of-experts layer with its balance loss and their gradient, the experts'
products of a few tokens by expert id, and the AdamW step.

Argument marshalling only, as in _binding.py and _moe.py: the checks of values
and the computation are the library's, and the common call is marshalled by
_moe_ext.so."""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import Optional, Sequence, Tuple, Union

import torch

from ._binding import (_DTYPE, _empty, _raise, GMM_BF16, GMM_F32, GMM_F8E4M3FN, GmmError, GmmInvalid, GmmTensor,
                       GmmUnsupported, handle, load, PACKED_FORMATS)
from . import _moe
from ._moe import _current, _device, _ID_DTYPE, _load_ext, _out, _pack, _PACKED_DTYPE, _refuse, _run

ADAMW_BLOCK = 256
GMV_SLOTS = 4096

_SCORES = {"softmax": 0, "sigmoid": 1}
_VALID_DTYPE = {t: _DTYPE[torch.int8] for t in (torch.bool, torch.uint8, torch.int8)}


def _kind(scores: str) -> int:
    if scores not in _SCORES:
        _refuse(f"scores must be 'softmax' or 'sigmoid', got {scores!r}")
    return _SCORES[scores]


def _maybe(t: Optional[torch.Tensor], name: str, dev: torch.device, dtypes=_DTYPE) -> Optional[bytes]:
    return None if t is None else _pack(t, name, dev, dtypes)


def route(logits: torch.Tensor, top_k: int, *, scores: str = "softmax", bias: Optional[torch.Tensor] = None,
          renormalize: bool = True, scale: float = 1.0, valid: Optional[torch.Tensor] = None,
          expert_ids: Optional[torch.Tensor] = None, weights: Optional[torch.Tensor] = None,
          stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The router's choice of top_k experts for every token through libgmm.so
    (gmm_route_run): logits [T,E] float32 or bfloat16.  Returns (expert_ids
    int32 [T,k], the best first, equal logits in the order of their experts;
    weights float32 [T,k]: scale * score, divided by the sum of the token's
    chosen scores with renormalize), as sort_tokens(), combine() and gmv() take
    them.

    scores "softmax" (over the experts) or "sigmoid"; with bias float32 [E] the
    choice, not the weight, goes by score + bias.  An expert whose logit is -inf
    is never chosen; choices that are missing, and all of a token whose valid
    [T] (bool) is False, are id -1 with weight 0.  The gradient is
    router_grad()."""
    kind, k = _kind(scores), int(top_k)
    if expert_ids is None and weights is None and stream is None:
        made = (_moe._ext or _load_ext()).route(logits, k, bias, valid, kind, bool(renormalize), scale, _current(logits))
        if made is not None:
            return made
    dev = _device(logits, "logits")
    T = logits.shape[0] if logits.dim() == 2 else 0
    args = [_pack(logits, "logits", dev), _maybe(bias, "bias", dev), _maybe(valid, "valid", dev, _VALID_DTYPE)]
    # (a number of choices that is out of range is refused by the run, whatever the output holds)
    expert_ids, iv = _out(expert_ids, "expert_ids", (T, min(max(k, 0), 1025)), torch.int32, dev, stream)
    if expert_ids.dim() != 2 or expert_ids.shape[1] != k:
        _refuse("expert_ids must hold top_k choices a token")
    weights, wv = _out(weights, "weights", (T, min(max(k, 0), 1025)), torch.float32, dev, stream)
    _run(load().gmm_route_run, dev, stream, (logits, bias, valid, expert_ids, weights), *args, kind,
         int(bool(renormalize)), float(scale), iv, wv)
    return expert_ids, weights


@functools.lru_cache(maxsize=4096)
def _balance_workspace(tokens: int, experts: int) -> int:
    need = ctypes.c_size_t(0)
    load().gmm_balance_loss_workspace(tokens, experts, ctypes.byref(need))
    return need.value


def balance_loss(logits: torch.Tensor, expert_ids: torch.Tensor, *, scores: str = "softmax", coef: float = 1.0,
                 z_coef: float = 0.0, valid: Optional[torch.Tensor] = None, loss: Optional[torch.Tensor] = None,
                 counts: Optional[torch.Tensor] = None, tokens: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The load-balancing loss of a router and its experts' counts through
    libgmm.so (gmm_balance_loss_run): with f[e] the share of the choices
    expert_ids [T,k] (int32 or int64) that went to expert e and P[e] the mean
    over the tokens of its probability (scores divided by their sum),

        loss = coef * E * sum_e f[e] * P[e] + z_coef * mean_t logsumexp(logits[t])^2.

    Returns (loss float32 [1], counts int32 [E], tokens int32 [1]).  Tokens
    whose valid [T] (bool) is False, or whose logits are all -inf, count for
    nothing; tokens is the number of the others.  The gradient is
    router_grad(), which takes the counts and tokens."""
    kind = _kind(scores)
    if loss is None and counts is None and tokens is None and stream is None:
        made = (_moe._ext or _load_ext()).balance_loss(logits, expert_ids, valid, kind, coef, z_coef, _current(logits))
        if made is not None:
            return made
    dev = _device(logits, "logits")
    T, E = logits.shape if logits.dim() == 2 else (0, 1)
    args = [_pack(logits, "logits", dev), _pack(expert_ids, "expert_ids", dev, _ID_DTYPE),
            _maybe(valid, "valid", dev, _VALID_DTYPE)]
    loss, lv = _out(loss, "loss", (1,), torch.float32, dev, stream)
    counts, cv = _out(counts, "counts", (E,), torch.int32, dev, stream)
    tokens, tv = _out(tokens, "tokens", (1,), torch.int32, dev, stream)
    need = _balance_workspace(T, E)
    work = _empty((need,), torch.uint8, dev, stream) if need else None
    _run(load().gmm_balance_loss_run, dev, stream, (logits, expert_ids, valid, loss, counts, tokens), *args, kind,
         float(coef), float(z_coef), lv, cv, tv, work.data_ptr() if need else None, need)
    return loss, counts, tokens


def router_grad(logits: torch.Tensor, expert_ids: torch.Tensor, *, dweights: Optional[torch.Tensor] = None,
                scores: str = "softmax", renormalize: bool = True, scale: float = 1.0,
                counts: Optional[torch.Tensor] = None, tokens: Optional[torch.Tensor] = None,
                dloss: Optional[torch.Tensor] = None, coef: float = 1.0, z_coef: float = 0.0,
                valid: Optional[torch.Tensor] = None, dlogits: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The gradient of a router's logits through libgmm.so
    (gmm_router_grad_run): of route()'s weights, given dweights [T,k] (as
    combine_grad() returns them), and of balance_loss(), given its counts and
    tokens and dloss (float32 [1], 1 without it) -- either or both, added in one
    pass.  scores, renormalize, scale, coef, z_coef and valid are those of the
    forward calls; the counts are constants, and may be sums over ranks.
    Returns dlogits [T,E] of logits' dtype, zeros for tokens that count for
    nothing and for experts that are switched off."""
    kind = _kind(scores)
    if dlogits is None and stream is None:
        made = (_moe._ext or _load_ext()).router_grad(logits, expert_ids, valid, kind, dweights, bool(renormalize), scale, counts,
                                                      tokens, dloss, coef, z_coef, _current(logits))
        if made is not None:
            return made
    dev = _device(logits, "logits")
    args = [_pack(logits, "logits", dev), _pack(expert_ids, "expert_ids", dev, _ID_DTYPE),
            _maybe(valid, "valid", dev, _VALID_DTYPE)]
    more = [_maybe(t, n, dev) for t, n in ((counts, "counts"), (tokens, "tokens"), (dloss, "dloss"))]
    wv = _maybe(dweights, "dweights", dev)
    dlogits, dv = _out(dlogits, "dlogits", logits.shape, logits.dtype, dev, stream)
    _run(load().gmm_router_grad_run, dev, stream, (logits, expert_ids, valid, dweights, counts, tokens, dloss, dlogits), *args,
         kind, wv, int(bool(renormalize)), float(scale), *more, float(coef), float(z_coef), dv)
    return dlogits


def _view_rhs(t: torch.Tensor, fmt: str, dev: torch.device) -> bytes:
    if fmt not in PACKED_FORMATS:
        _refuse(f"rhs: unknown four-bit format {fmt!r}")
    # packed as fp4 codes (two elements to a byte), then named by its format
    view = bytearray(_pack(t, "rhs", dev, _PACKED_DTYPE))
    GmmTensor.from_buffer(view).dtype = PACKED_FORMATS[fmt]
    return bytes(view)


@functools.lru_cache(maxsize=4096)
def _gmv_workspace(slots: int, N: int, weighted: bool) -> int:
    need = ctypes.c_size_t(0)
    load().gmm_gmv_workspace(slots, N, int(weighted), ctypes.byref(need))
    return need.value


def gmv(x: torch.Tensor, rhs: torch.Tensor, expert_ids: Optional[torch.Tensor] = None, *, rhs_scale: torch.Tensor,
        rhs_format: str, rhs_zero: Optional[torch.Tensor] = None, weights: Optional[torch.Tensor] = None,
        out_dtype: torch.dtype = torch.float32, out: Optional[torch.Tensor] = None,
        stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Products of a few tokens with their experts' four-bit weights, by expert
    id, through libgmm.so (gmm_gmv_run): the form of gmm() for a decode step,
    with no sort and no expert rows.

    x bfloat16 [T,K] (a token's vector goes to all its experts) or [T,k,K] (a
    vector a slot); rhs bytes [G,N,K/2] of rhs_format "int4", "uint4" or
    "fp4_e2m1" and rhs_scale [G,nb,1,N], as gmm() takes them (bfloat16 scales
    too); rhs_zero of rhs_scale's shape and dtype, subtracted from the codes
    before they are scaled; expert_ids [T,k] int32 or int64, an id outside
    [0,G) giving zeros (None with one group: a dense product).  Returns
    [T,k,N] of out_dtype, or with weights [T,k] the weighted sum over a token's
    slots, [T,N].  Up to 4096 slots; from some 16 rows an expert on (80 of a
    single expert) sort_tokens(), dispatch() and gmm() are faster."""
    if out is None and stream is None:
        made = (_moe._ext or _load_ext()).gmv(x, rhs, PACKED_FORMATS.get(rhs_format, -1), rhs_scale, rhs_zero, expert_ids, weights,
                                              _DTYPE.get(out_dtype, -2), _current(x))
        if made is not None:
            return made
    dev = _device(x, "x")
    N = rhs.shape[1] if rhs.dim() == 3 else 1
    T = x.shape[0] if x.dim() else 0
    k = expert_ids.shape[1] if expert_ids is not None and expert_ids.dim() == 2 else 1
    args = [_pack(x, "x", dev), _view_rhs(rhs, rhs_format, dev), _pack(rhs_scale, "rhs_scale", dev),
            _maybe(rhs_zero, "rhs_zero", dev), _maybe(expert_ids, "expert_ids", dev, _ID_DTYPE), _maybe(weights, "weights", dev)]
    # (too many slots are refused by the run, whatever the output holds)
    rows = T if T * k <= GMV_SLOTS else 0
    out, ov = _out(out, "out", (rows, k, N) if weights is None else (rows, N), out_dtype, dev, stream)
    need = _gmv_workspace(T * k, N, weights is not None)
    work = _empty((need,), torch.uint8, dev, stream) if need else None
    _run(load().gmm_gmv_run, dev, stream, (x, rhs, rhs_scale, rhs_zero, expert_ids, weights, out), *args, ov,
         work.data_ptr() if need else None, need)
    return out


# gmm_adamw_item and gmm_adamw_args
_ITEM = struct.Struct("@qPPPPPPP")
_ARGS = struct.Struct("@iiidddddqPPP")
_STATE_DTYPE = {torch.float32: GMM_F32, torch.float8_e4m3fn: GMM_F8E4M3FN}
_WIDE_DTYPE = {torch.float32: GMM_F32, torch.bfloat16: GMM_BF16}


def _column(tensors, name: str, like, dev: torch.device, dtypes, sizes) -> Tuple[int, list]:
    """One role's tensors: their common dtype code and their addresses."""
    if len(tensors) != len(like):
        _refuse(f"{len(tensors)} tensors in {name}, {len(like)} in params")
    code, at = None, []
    for t, n in zip(tensors, sizes):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.device != dev:
            _refuse(f"{name} must be device tensors on {dev}")
        if not t.is_contiguous():
            _refuse(f"{name} must be contiguous")
        if t.numel() != n:
            _refuse(f"{name}: a tensor of {t.numel()} elements, expected {n}")
        c = dtypes.get(t.dtype)
        if c is None:
            _refuse(f"{name}: unsupported dtype {t.dtype}")
        if code is None:
            code = c
        elif code != c:
            _refuse(f"{name}: tensors of different dtypes (a call takes one of each role)")
        at.append(t.data_ptr())
    return code, at


def _one(v, name: str, dtype: torch.dtype, dev: torch.device) -> Optional[int]:
    if not isinstance(v, torch.Tensor):
        return None
    if not v.is_cuda or v.device != dev or v.dtype != dtype or v.numel() != 1:
        _refuse(f"{name} must be a number or a one-element {dtype} tensor on {dev}")
    return v.data_ptr()


def _written(tensors) -> None:
    """What has been (or may have been) written is another version to autograd."""
    torch.autograd.graph.increment_version([t for t in tensors if not t.is_inference()])


def adamw(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], exp_avg: Sequence[torch.Tensor],
          exp_avg_sq: Sequence[torch.Tensor], step: Union[int, torch.Tensor], *, lr: Union[float, torch.Tensor],
          betas: Tuple[float, float] = (0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.0,
          exp_avg_scale: Optional[Sequence[torch.Tensor]] = None,
          exp_avg_sq_scale: Optional[Sequence[torch.Tensor]] = None,
          copies: Optional[Sequence[torch.Tensor]] = None, grad_scale: Optional[torch.Tensor] = None,
          stream: Optional[torch.cuda.Stream] = None) -> None:
    """One AdamW step of many tensors, in place, through libgmm.so
    (gmm_adamw_run).  params and grads float32 or bfloat16; the states exp_avg
    and exp_avg_sq float32, or float8_e4m3fn with exp_avg_scale and
    exp_avg_sq_scale, float32 [ceil(n/256)] for a tensor of n elements
    (exp_avg_sq then holds the codes of its square root; zero codes with scales
    of 1 begin).  copies: bfloat16 tensors that take the rounded parameters (the
    weights that gmm() reads, beside float32 params).  step counts from 1; step
    (int32), lr and grad_scale (float32, a factor of the gradients) may be
    one-element device tensors, read when the step runs, as a captured graph
    needs it.  The tensors of a role share a dtype, and none may overlap.  A refused
    call (GmmInvalid, GmmUnsupported) changes nothing; after any other GmmError
    some of the tensors may have taken the step.  To autograd a step is an
    in-place operation: a backward through a graph that keeps what the step
    wrote is refused.

    The products' weights are parameters like any other: params [G,K,N], grads
    as tgmm() returns them."""
    if stream is None and len(params):
        done = (_moe._ext or _load_ext()).adamw(params, grads, exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale, copies, step,
                                                lr, *betas, eps, weight_decay, grad_scale, _current(params[0]))
        if done is not None:
            if done is not True:  # (queued in part: not to be asked for again)
                _raise(done, handle(params[0].device))
            return
    if len(params) == 0:
        load()
        if any(len(t) for t in (grads, exp_avg, exp_avg_sq, exp_avg_scale or (), exp_avg_sq_scale or (), copies or ())):
            _refuse("tensors without params")
        return
    dev = _device(params[0], "params")
    sizes = [t.numel() if isinstance(t, torch.Tensor) else -1 for t in params]
    pc, p = _column(params, "params", params, dev, _WIDE_DTYPE, sizes)
    gc, g = _column(grads, "grads", params, dev, _WIDE_DTYPE, sizes)
    mc, m = _column(exp_avg, "exp_avg", params, dev, _STATE_DTYPE, sizes)
    vc, v = _column(exp_avg_sq, "exp_avg_sq", params, dev, _STATE_DTYPE, sizes)
    if mc != vc:
        _refuse("exp_avg and exp_avg_sq must have one dtype")
    none = [0] * len(params)
    ms = vs = c = none
    blocks = [(n + ADAMW_BLOCK - 1) // ADAMW_BLOCK for n in sizes]
    f32 = {torch.float32: GMM_F32}
    if (exp_avg_scale is None) != (exp_avg_sq_scale is None) or (mc == GMM_F32) != (exp_avg_scale is None):
        _refuse("exp_avg_scale and exp_avg_sq_scale belong to float8_e4m3fn states")
    if exp_avg_scale is not None:
        ms = _column(exp_avg_scale, "exp_avg_scale", params, dev, f32, blocks)[1]
        vs = _column(exp_avg_sq_scale, "exp_avg_sq_scale", params, dev, f32, blocks)[1]
    if copies is not None:
        c = _column(copies, "copies", params, dev, {torch.bfloat16: GMM_BF16}, sizes)[1]
    items = b"".join([_ITEM.pack(*row) for row in zip(sizes, p, g, m, v, ms, vs, c)])
    at = _one(step, "step", torch.int32, dev), _one(lr, "lr", torch.float32, dev), _one(grad_scale, "grad_scale", torch.float32, dev)
    if grad_scale is not None and at[2] is None:
        _refuse("grad_scale must be a one-element float32 device tensor")
    args = _ARGS.pack(pc, gc, mc, 0.0 if at[1] else float(lr), float(betas[0]), float(betas[1]), float(eps),
                      float(weight_decay), 0 if at[0] else int(step), at[0] or 0, at[1] or 0, at[2] or 0)
    written = [*params, *exp_avg, *exp_avg_sq, *(exp_avg_scale or ()), *(exp_avg_sq_scale or ()), *(copies or ())]
    tensors = [*written, *grads]
    tensors += [t for t in (step, lr, grad_scale) if isinstance(t, torch.Tensor)]
    try:
        _run(load().gmm_adamw_run, dev, stream, tensors, items, len(params), args)
    except (GmmInvalid, GmmUnsupported):
        raise
    except GmmError:
        _written(written)
        raise
    _written(written)
