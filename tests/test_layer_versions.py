"""adamw() is an in-place operation to autograd: whatever a step writes moves
its version counter, so that a backward through weights which have since been
stepped is refused, as with torch's own optimizers, and not computed with the
new ones.  Gradients and scalars are only read.  (Both ways on the CPU: the
compiled binding with host tensors for device tensors, and the Python one.)"""
import pytest
import torch

from moe_grouped_matrix_amd import _binding, _layer, _moe
from test_layer_step_once import host  # noqa: F401  (a fixture)
from test_moe_ext_host import dev

F32, BF16, I32, E4 = torch.float32, torch.bfloat16, torch.int32, torch.float8_e4m3fn
ROLES = ("params", "grads", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale", "copies")


def columns(eight, copies, n=600, count=3):
    col = lambda d, m=n: [dev(m, dtype=d) for _ in range(count)]  # noqa: E731
    return dict(params=col(F32), grads=col(BF16), exp_avg=col(E4 if eight else F32), exp_avg_sq=col(E4 if eight else F32),
                exp_avg_scale=col(F32, 3) if eight else None, exp_avg_sq_scale=col(F32, 3) if eight else None,
                copies=col(BF16) if copies else None)


def versions(roles):
    return {name: [t._version for t in ts] for name, ts in roles.items() if ts is not None}


@pytest.fixture(params=["compiled", "python"])
def way(request, host, monkeypatch):  # noqa: F811
    ext, c = host

    class Library:
        def gmm_adamw_run(self, *args):
            return way.status

        def gmm_last_error(self, h):
            return b""

    class Way:
        def __init__(self):
            self.expect(0)

        def expect(self, status):
            self.status = status
            c.rec_expect(status)

    class Nothing:
        def set_handle(self, *_):
            pass

        def adamw(self, *_):
            return None

    way = Way()
    monkeypatch.setattr(_binding, "_lib", Library())
    monkeypatch.setattr(_binding, "_handles", {0: 1, None: 1})
    monkeypatch.setattr(_layer, "_current", lambda t: 0x77)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0x77, raising=False)
    monkeypatch.setattr(_moe, "_ext", ext if request.param == "compiled" else Nothing())
    return way


@pytest.mark.parametrize("eight,copies", [(False, False), (False, True), (True, True)])
def test_what_is_written_moves(way, eight, copies):
    roles = columns(eight, copies)
    step, lr, gs = dev(1, dtype=I32), dev(1, dtype=F32), dev(1, dtype=F32)
    before = versions(roles)
    _layer.adamw(*[roles[r] for r in ROLES[:4]], step, lr=lr, grad_scale=gs, **{r: roles[r] for r in ROLES[4:]})
    after = versions(roles)
    for name in after:
        moved = [b < a for b, a in zip(before[name], after[name])]
        assert all(moved) if name != "grads" else not any(moved), name
    assert step._version == lr._version == gs._version == 0


def test_a_refused_step_moves_nothing_and_a_failed_one_does(way):
    for status, cls in ((_binding.GMM_E_INVALID, _binding.GmmInvalid), (_binding.GMM_E_HIP, _binding.GmmError)):
        roles = columns(False, False)
        before = versions(roles)
        way.expect(status)
        with pytest.raises(cls):
            _layer.adamw(*[roles[r] for r in ROLES[:4]], 1, lr=0.1)
        assert (versions(roles)["params"] == before["params"]) == (status == _binding.GMM_E_INVALID)


def test_backward_through_stepped_weights_is_refused(way):
    roles = columns(False, False, count=1)
    w = roles["params"][0].as_subclass(torch.Tensor).requires_grad_()
    x = torch.ones(600, requires_grad=True)
    y = (w * x).sum()  # (keeps w for the gradient of x)
    with torch.no_grad():
        _layer.adamw(*[roles[r] for r in ROLES[:4]], 1, lr=0.1)
    assert w._version == roles["params"][0]._version
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_tensors_of_inference_mode_have_no_counter(way):
    with torch.inference_mode():
        roles = columns(True, True)
        assert all(t.is_inference() for ts in roles.values() for t in ts)
    _layer.adamw(*[roles[r] for r in ROLES[:4]], 1, lr=0.1, **{r: roles[r] for r in ROLES[4:]})
