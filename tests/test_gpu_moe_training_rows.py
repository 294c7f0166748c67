"""Dispatch, combine and its gradient at the token counts of a training batch,
against the 64-bit forms (taken on the GPU, in elementary operations).

From 2048 tokens on (eight a compute unit) a lane takes up to four chunks of a
row and a wave all of a token's slots; the widths below give one to four chunks
a lane and rows of several segments, ending in whole and in overlapping chunks,
for 16-byte chunks of a copied row and 8-element chunks of a summed one.

Tolerances as for fewer tokens (u = 2^-24): combine k u sum|w x|, drows u |w g|,
dweights D u sum|g x|, each with half a step of the output type."""
import pytest
import torch

import moe_reference as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BITS = {1: torch.uint8, 2: torch.int16, 4: torch.int32}
CASES = [(2048, 2, 40), (2049, 3, 500), (2051, 1, 700), (2051, 7, 1024), (2051, 3, 1027), (2051, 8, 1408),
         (2060, 4, 1800), (2048, 5, 2053), (2050, 2, 5003), (2048, 17, 530), (2300, 2, 5)]


def _slots(T, k, seed, unrouted):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, 11, (T, k), generator=g)
    if unrouted:
        ids[torch.rand(T, k, generator=g) < unrouted] = -1
    return ref.sort_tokens(ids, 11)[1].cuda()


def _big_enough(T):
    assert T >= 8 * torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("unrouted", [0.0, 0.3])
@pytest.mark.parametrize("T,k,D", CASES)
def test_dispatch(T, k, D, unrouted):
    import moe_grouped_matrix_amd as m
    _big_enough(T)
    g = torch.Generator().manual_seed(T + k + D)
    slot_row = _slots(T, k, D, unrouted)
    row, routed = ref._split(slot_row)
    for dtype in (torch.bfloat16, torch.float32, torch.uint8):
        iv = BITS[torch.empty(0, dtype=dtype).element_size()]
        x = torch.randint(-128, 128, (T, D * torch.empty(0, dtype=dtype).element_size()), dtype=torch.int8,
                          generator=g).cuda().view(dtype)
        print(f"dispatch T={T} k={k} D={D} {dtype} unrouted={unrouted}", flush=True)
        out = torch.full((T * k, x.shape[1]), 3.0).to(dtype).cuda()
        m.dispatch(x, slot_row, out=out)
        want = torch.empty((T * k, x.shape[1]), dtype=iv, device="cuda")
        want[row.flatten()] = torch.where(routed[..., None], x.view(iv)[:, None, :],
                                          torch.zeros((), dtype=iv, device="cuda")).reshape(T * k, -1)
        assert torch.equal(out.view(iv), want)


@pytest.mark.parametrize("unrouted", [0.0, 0.3])
@pytest.mark.parametrize("T,k,D", CASES)
def test_combine(T, k, D, unrouted):
    import moe_grouped_matrix_amd as m
    _big_enough(T)
    g = torch.Generator().manual_seed(T + k + D + 1)
    slot_row = _slots(T, k, D, unrouted)
    off = slot_row < 0
    for rd, wd, od in ((torch.bfloat16, torch.float32, torch.bfloat16), (torch.float32, torch.bfloat16, torch.float32),
                       (torch.float32, torch.float32, torch.bfloat16), (torch.bfloat16, None, torch.float32)):
        rows = torch.randn(T * k, D, generator=g).to(rd).cuda()
        weights = None
        if wd is not None:
            weights = torch.randn(T, k, generator=g).to(wd).cuda()
            weights[off] = float("nan")
        rows[(~slot_row[off]).long()] = float("inf")
        print(f"combine T={T} k={k} D={D} {rd} {wd} {od} unrouted={unrouted}", flush=True)
        out = m.combine(rows, slot_row, weights, out_dtype=od)
        row, routed = ref._split(slot_row)
        want, terms = torch.zeros(2, T, D, dtype=torch.float64, device="cuda")
        for j in range(k):
            w = 1.0 if weights is None else weights[:, j, None].double()
            term = torch.where(routed[:, j, None], rows[row[:, j]].double() * w, 0.0)
            want += term
            terms += term.abs()
        ref.within(out, want, k * U * terms + ref.half_step(od, want.abs() + k * U * terms), "combine")


@pytest.mark.parametrize("unrouted", [0.0, 0.3])
@pytest.mark.parametrize("T,k,D", CASES)
def test_combine_grad(T, k, D, unrouted):
    import moe_grouped_matrix_amd as m
    _big_enough(T)
    g = torch.Generator().manual_seed(T + k + D + 2)
    slot_row = _slots(T, k, D, unrouted)
    off = slot_row < 0
    for gd, rd, wd in ((torch.bfloat16, torch.bfloat16, torch.float32), (torch.float32, torch.float32, torch.bfloat16),
                       (torch.bfloat16, torch.float32, torch.float32), (torch.float32, torch.bfloat16, torch.float32)):
        dout = torch.randn(T, D, generator=g).to(gd).cuda()
        rows = torch.randn(T * k, D, generator=g).to(rd).cuda()
        weights = torch.randn(T, k, generator=g).to(wd).cuda()
        weights[off] = float("nan")
        rows[(~slot_row[off]).long()] = float("nan")
        print(f"combine_grad T={T} k={k} D={D} {gd} {rd} {wd} unrouted={unrouted}", flush=True)
        drows, dweights = m.combine_grad(dout, rows, slot_row, weights)
        row, routed = ref._split(slot_row)
        d = dout.double()
        for j in range(k):
            on = routed[:, j]
            wr = torch.where(on[:, None], d * weights[:, j, None].double(), 0.0)
            ref.within(drows[row[:, j]], wr, U * wr.abs() + ref.half_step(rd, wr.abs() * (1 + U)), f"drows, slot {j}")
            term = torch.where(on[:, None], d * rows[row[:, j]].double(), 0.0)
            ww, terms = term.sum(1), term.abs().sum(1)
            ref.within(dweights[:, j], ww, D * U * terms + ref.half_step(wd, ww.abs() + D * U * terms), f"dweights, slot {j}")
        assert bool((dweights[off] == 0).all())


@pytest.mark.parametrize("D", [1027, 1408, 2053])
def test_gradient_of_infinities(D):
    """One infinity a token, in every column in turn: the product is that
    infinity, in overlapping chunks too."""
    import moe_grouped_matrix_amd as m
    T, k = 2 * D if D < 1100 else D + 700, 3
    _big_enough(T)
    slot_row = torch.arange(T * k, dtype=torch.int32, device="cuda").reshape(T, k)
    for dtype in (torch.float32, torch.bfloat16):
        rows = torch.ones(T * k, D, dtype=dtype, device="cuda")
        at = torch.arange(T, device="cuda") % D
        rows[3 * torch.arange(T, device="cuda") + 1, at] = float("inf")
        print(f"infinite rows T={T} D={D} {dtype}", flush=True)
        drows, dw = m.combine_grad(torch.ones(T, D, dtype=dtype, device="cuda"), rows, slot_row,
                                   torch.ones(T, k, device="cuda"))
        want = torch.full((T, k), float(D), device="cuda")
        want[:, 1] = float("inf")
        assert torch.equal(dw, want) and bool((drows == 1).all())
