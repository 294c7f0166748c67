"""The Python binding of include/gmm_layer.h on the CPU: memory of calls on a
stream of the caller's choice, what is handed to the library, and refusals
that name the argument (the library and the device allocator are stood in for
by Python objects that keep account)."""
import pytest
import torch

from moe_grouped_matrix_amd import _binding, _layer, _moe
from test_stream_argument import _empty, Stream, check, device, kept, streams  # noqa: F401  (a fixture)

F32, BF16, I32, I64, U8, E4 = (torch.float32, torch.bfloat16, torch.int32, torch.int64, torch.uint8, torch.float8_e4m3fn)


class Ext:
    """Takes no call: every one is marshalled in Python."""

    def __getattr__(self, name):
        return lambda *_: None


@pytest.fixture(autouse=True)
def clear(monkeypatch, request):
    if "streams" in request.fixturenames:
        request.getfixturevalue("streams")
        monkeypatch.setattr(_moe, "_ext", Ext())
        monkeypatch.setattr(_moe, "_current", lambda t: 0)
        monkeypatch.setattr(_layer, "_current", lambda t: 0)
    for cached in (_layer._balance_workspace, _layer._gmv_workspace):
        cached.cache_clear()
    yield
    for cached in (_layer._balance_workspace, _layer._gmv_workspace):
        cached.cache_clear()


def calls():
    """(name, call(**given), inputs, {output: the caller's})"""
    z, ids, valid, bias = device(6, 16, dtype=F32), device(6, 2, dtype=I32), device(6, dtype=torch.bool), device(16, dtype=F32)
    dw, counts, tokens, dloss = device(6, 2, dtype=F32), device(16, dtype=I32), device(1, dtype=I32), device(1, dtype=F32)
    x, q, s = device(6, 64), device(4, 24, 32, dtype=U8), device(4, 2, 1, 24, dtype=F32)
    zero, w = device(4, 2, 1, 24, dtype=F32), device(6, 2, dtype=F32)
    return [
        ("route", lambda **kw: _layer.route(z, 2, bias=bias, valid=valid, **kw), (z, bias, valid),
         dict(expert_ids=device(6, 2, dtype=I32), weights=device(6, 2, dtype=F32))),
        ("balance_loss", lambda **kw: _layer.balance_loss(z, ids, valid=valid, **kw), (z, ids, valid),
         dict(loss=device(1, dtype=F32), counts=device(16, dtype=I32), tokens=device(1, dtype=I32))),
        ("router_grad", lambda **kw: _layer.router_grad(z, ids, dweights=dw, counts=counts, tokens=tokens, dloss=dloss, valid=valid, **kw),
         (z, ids, dw, counts, tokens, dloss, valid), dict(dlogits=device(6, 16, dtype=F32))),
        ("gmv", lambda **kw: _layer.gmv(x, q, ids, rhs_format="int4", rhs_scale=s, rhs_zero=zero, **kw), (x, q, ids, s, zero),
         dict(out=device(6, 2, 24, dtype=F32))),
        ("gmv weighted", lambda **kw: _layer.gmv(x, q, ids, rhs_format="int4", rhs_scale=s, weights=w, **kw), (x, q, ids, s, w),
         dict(out=device(6, 24, dtype=F32))),
    ]


@pytest.mark.parametrize("i", range(5))
def test_a_stream_of_the_callers_choice(streams, i):  # noqa: F811
    for given in (0, 1, 9):
        name, call, ins, outs = calls()[i]
        own = dict(list(outs.items())[:given])
        check(streams, lambda st: call(stream=st, **own), ins, tuple(own.values()))
    far = Stream(0x30)
    far.device = torch.device("cuda", 1)
    before = len(streams[2].raw)
    with pytest.raises(_binding.GmmInvalid, match="stream is on"):
        calls()[i][1](stream=far)
    assert not [r for r in streams[2].raw[before:] if r == 0x30]


def columns(n=3, eight=False, p=F32, g=BF16):
    state = E4 if eight else F32
    made = dict(params=[device(5, 100, dtype=p) for _ in range(n)], grads=[device(5, 100, dtype=g) for _ in range(n)],
                exp_avg=[device(500, dtype=state) for _ in range(n)], exp_avg_sq=[device(500, dtype=state) for _ in range(n)])
    if eight:
        made.update(exp_avg_scale=[device(2, dtype=F32) for _ in range(n)], exp_avg_sq_scale=[device(2, dtype=F32) for _ in range(n)])
    return made


def test_adamw_keeps_its_tensors(streams):  # noqa: F811
    _, other, lib = streams
    cols, one = columns(eight=True), dict(step=device(1, dtype=I32), lr=device(1, dtype=F32), grad_scale=device(1, dtype=F32))
    copies = [device(500, dtype=BF16) for _ in range(3)]
    _layer.adamw(**cols, copies=copies, stream=other, **one)
    assert lib.raw[-1] == other.cuda_stream
    for t in [t for c in cols.values() for t in c] + copies + list(one.values()):
        assert other in kept(t)


def test_adamw_hands_over_its_tensors(streams, monkeypatch):  # noqa: F811
    seen = []
    monkeypatch.setattr(streams[2].__class__, "gmm_adamw_run", lambda self, *a: seen.append(a) or 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0x77, raising=False)
    cols, copies = columns(eight=True), [device(500, dtype=BF16) for _ in range(3)]
    _layer.adamw(**cols, step=7, lr=0.5, betas=(0.25, 0.125), eps=2.0, weight_decay=4.0, copies=copies)
    h, items, count, args, stream = seen[0]
    assert count == 3 and stream == 0x77
    at = [_layer._ITEM.unpack_from(items, i * _layer._ITEM.size) for i in range(3)]
    names = ("params", "grads", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale")
    assert at == [(500, *[cols[n][i].data_ptr() for n in names], copies[i].data_ptr()) for i in range(3)]
    assert _layer._ARGS.unpack(args) == (_binding.GMM_F32, _binding.GMM_BF16, _binding.GMM_F8E4M3FN, 0.5, 0.25, 0.125, 2.0, 4.0, 7, 0, 0, 0)


def test_adamw_refuses(streams):  # noqa: F811
    def refused(word, drop=(), **kw):
        cols = columns(eight="exp_avg_scale" in kw.pop("like", ()))
        for n in drop:
            del cols[n]
        with pytest.raises(_binding.GmmInvalid, match=word):
            _layer.adamw(**dict(dict(cols, step=1, lr=1e-3), **kw))
    eight = columns(eight=True)
    refused("3 in params", grads=[device(500)] * 2)
    refused("500 elements|elements, expected 500", grads=[device(499)] * 3)
    refused("unsupported dtype", grads=[device(500, dtype=I32)] * 3)
    refused("different dtypes", grads=[device(500), device(500, dtype=F32), device(500)])
    refused("contiguous", grads=[device(500, 2)[:, 0]] * 3)
    refused("device tensors", grads=[_empty(500)] * 3)
    refused("device tensor", params=[_empty(500)] * 3)
    refused("one dtype", exp_avg=eight["exp_avg"])
    refused("float8_e4m3fn states", exp_avg=eight["exp_avg"], exp_avg_sq=eight["exp_avg_sq"])
    refused("float8_e4m3fn states", exp_avg_scale=eight["exp_avg_scale"], exp_avg_sq_scale=eight["exp_avg_sq_scale"])
    refused("float8_e4m3fn states", exp_avg_scale=eight["exp_avg_scale"])
    refused("copies: unsupported", copies=[device(500, dtype=F32)] * 3)
    refused("step must be", step=device(1, dtype=I64))
    refused("lr must be", lr=device(2, dtype=F32))
    refused("grad_scale must be", grad_scale=0.5)
    refused("without params", params=[])
    assert streams[2].raw == []
    _layer.adamw([], [], [], [], 1, lr=0.1)
    assert streams[2].raw == []


def test_router_and_gmv_refuse(streams):  # noqa: F811
    z, ids = device(6, 16, dtype=F32), device(6, 2, dtype=I32)
    x, q, s = device(6, 64), device(4, 24, 32, dtype=U8), device(4, 2, 1, 24, dtype=F32)
    for word, call in (
            ("logits must be a device tensor", lambda: _layer.route(_empty(3, 4), 2)),
            ("contiguous", lambda: _layer.route(device(16, 6, dtype=F32).t(), 2)),
            ("scores must be", lambda: _layer.route(z, 2, scores="tanh")),
            ("top_k", lambda: _layer.route(z, 2, expert_ids=device(6, 3, dtype=I32))),
            ("unsupported dtype", lambda: _layer.route(z.half(), 2)),
            ("valid: unsupported", lambda: _layer.route(z, 2, valid=device(6, dtype=I32))),
            ("scores must be", lambda: _layer.balance_loss(z, ids, scores=1)),
            ("expert_ids: unsupported", lambda: _layer.balance_loss(z, device(6, 2))),
            ("scores must be", lambda: _layer.router_grad(z, ids, scores=None)),
            ("dweights: unsupported", lambda: _layer.router_grad(z, ids, dweights=device(6, 2, dtype=torch.float16))),
            ("unknown four-bit format", lambda: _layer.gmv(x, q, ids, rhs_format="int8", rhs_scale=s)),
            ("rhs: unsupported", lambda: _layer.gmv(x, device(4, 24, 32), ids, rhs_format="int4", rhs_scale=s)),
            ("out: unsupported", lambda: _layer.gmv(x, q, ids, rhs_format="int4", rhs_scale=s, out_dtype=torch.float16)),
            ("rhs_scale must be a device tensor", lambda: _layer.gmv(x, q, ids, rhs_format="int4", rhs_scale=torch.ones(4, 2, 1, 24)))):
        with pytest.raises(_binding.GmmInvalid, match=word):
            call()
    assert not [r for r in streams[2].raw if isinstance(r, int) and r > 1]
