"""A HIP error that an earlier call of the thread left behind is not taken for
a launch's own: the call succeeds, a step is taken once, and the error is still
there for whoever looks for it."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture
def hip():
    """The HIP runtime that the process has loaded."""
    with open("/proc/self/maps") as f:
        paths = {line.split()[-1] for line in f if "libamdhip64" in line}
    assert len(paths) == 1, paths
    lib = ctypes.CDLL(paths.pop())
    yield lib
    lib.hipGetLastError()


def _operators():
    import moe_grouped_matrix_amd as m
    g = torch.Generator().manual_seed(3)
    T, E, k = 2048, 128, 8
    z = torch.randn(T, E, generator=g).cuda()
    ids, w = m.route(z, k)
    _, counts, tokens = m.balance_loss(z, ids)
    x = torch.randn(40, 256, generator=g).to(BF16).cuda()
    q = torch.randint(0, 256, (E, 48, 128), generator=g, dtype=torch.uint8).cuda()
    s = torch.rand(E, 2, 1, 48, generator=g).cuda()
    some, sw = ids[:40].contiguous(), w[:40].contiguous()
    few, fw = ids[:2].contiguous(), w[:2].contiguous()
    return {
        "route": lambda: m.route(z, k),
        "balance_loss": lambda: m.balance_loss(z, ids),
        "balance_loss, one workgroup": lambda: m.balance_loss(z[:16], ids[:16]),
        "router_grad": lambda: m.router_grad(z, ids, dweights=w, counts=counts, tokens=tokens),
        "gmv": lambda: m.gmv(x, q, some, rhs_format="int4", rhs_scale=s),
        "gmv, weighted": lambda: m.gmv(x, q, some, rhs_format="int4", rhs_scale=s, weights=sw),
        "gmv, weighted, few slots": lambda: m.gmv(x[:2], q, few, rhs_format="int4", rhs_scale=s, weights=fw),
    }


def _leave_error(hip):
    hip.hipGetLastError()
    left = hip.hipSetDevice(10 ** 6)  # (refused on the host)
    assert left != 0 and hip.hipPeekAtLastError() == left
    return left


def test_outputs(hip):
    for name, call in _operators().items():
        call()  # (memory for the outputs is in the allocator afterwards)
        want = call()
        torch.cuda.synchronize()
        left = _leave_error(hip)
        got = call()
        still = hip.hipGetLastError()
        assert still == left, name
        want, got = (r if isinstance(r, tuple) else (r,) for r in (want, got))
        for a, b in zip(want, got):
            assert torch.equal(a, b), name


@pytest.mark.parametrize("count", [1, 100])
def test_a_step_is_taken_once(hip, count):
    import moe_grouped_matrix_amd as m
    g = torch.Generator().manual_seed(count)
    first = [[torch.rand(300, generator=g).cuda() for _ in range(count)] for _ in range(4)]
    want, got = ([[t.clone() for t in role] for role in first] for _ in range(2))
    m.adamw(*want, 1, lr=0.1)
    m.adamw(*[[t.clone() for t in role] for role in first], 1, lr=0.1)
    torch.cuda.synchronize()
    left = _leave_error(hip)
    m.adamw(*got, 1, lr=0.1)
    assert hip.hipGetLastError() == left
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
