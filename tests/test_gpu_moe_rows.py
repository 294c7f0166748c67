"""GPU parity of the token operators of include/gmm_moe.h (sort, dispatch,
combine and its gradient) against their plain 64-bit forms.

Tolerances (u = 2^-24, the half step of binary32; h = half a step of the
output type): combine adds k products with one fma each, in order: an error of
at most k u sum|w x| before the output rounding.  A drows element is one
binary32 product: u |w g|.  dweights sums D products in some fixed order: at
most D u sum|g x|."""
import pytest
import torch

import moe_reference as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
IV = {torch.float32: torch.int32, torch.bfloat16: torch.int16}


def _ids(T, k, G, seed, unrouted=0.0, dtype=torch.int64, skew=False):
    g = torch.Generator().manual_seed(seed)
    if skew:  # most slots on one expert
        ids = torch.where(torch.rand(T, k, generator=g) < 0.8, 3 % G, torch.randint(0, G, (T, k), generator=g))
    else:
        ids = torch.randint(0, G, (T, k), generator=g)
    if unrouted:
        off = torch.rand(T, k, generator=g) < unrouted
        wild = torch.tensor([-1, G, G + 5, -2 ** 31, 2 ** 31 - 1])[torch.randint(0, 5, (T, k), generator=g)]
        ids = torch.where(off, wild, ids)
    return ids.to(dtype)


SORTS = [(1, 1, 1), (1, 8, 128), (3, 2, 5), (63, 1, 64), (65, 3, 7), (256, 8, 128), (512, 2, 1024), (341, 3, 200),
         (1024, 4, 128), (4096, 1, 33), (4097, 1, 33), (3001, 5, 128), (20000, 8, 128), (9001, 8, 1024),
         (70001, 4, 256), (40000, 64, 3)]


@pytest.mark.parametrize("unrouted", [0.0, 0.3, 1.0])
@pytest.mark.parametrize("T,k,G", SORTS)
def test_sort_tokens(T, k, G, unrouted):
    import moe_grouped_matrix_amd as m
    for dtype, skew in ((torch.int64, False), (torch.int32, True)):
        ids = _ids(T, k, G, 7 * T + k, unrouted, dtype, skew)
        print(f"sort T={T} k={k} G={G} unrouted={unrouted} {dtype}", flush=True)
        sizes, slot_row = m.sort_tokens(ids.cuda(), G)
        ws, wr = ref.sort_tokens(ids, G)
        assert torch.equal(sizes.cpu(), ws)
        assert torch.equal(slot_row.cpu(), wr)


def test_sort_tokens_wide_ids():
    """int64 ids whose low 32 bits look like an expert are unrouted."""
    import moe_grouped_matrix_amd as m
    ids = torch.tensor([[2 ** 32 + 1, 1], [-2 ** 63, 0], [2 ** 63 - 1, 2]])
    sizes, slot_row = m.sort_tokens(ids.cuda(), 3)
    assert sizes.tolist() == [1, 1, 1]
    assert slot_row.tolist() == [[~3, 1], [~4, 0], [~5, 2]]


def test_sort_tokens_empty():
    import moe_grouped_matrix_amd as m
    sizes, slot_row = m.sort_tokens(torch.zeros(0, 4, dtype=torch.int32, device="cuda"), 9,
                                    group_sizes=torch.full((9,), 5, dtype=torch.int32, device="cuda"))
    assert sizes.tolist() == [0] * 9 and tuple(slot_row.shape) == (0, 4)


def test_sort_tokens_several_rounds_per_workgroup():
    """2^21 slots over 1024 experts: 32 workgroups of 16 rounds each."""
    import moe_grouped_matrix_amd as m
    T, k, G = 1 << 19, 4, 1024
    ids = _ids(T, k, G, 5, 0.1)
    sizes, slot_row = m.sort_tokens(ids.cuda(), G)
    key = torch.where((ids >= 0) & (ids < G), ids, G).flatten()
    order = torch.sort(key, stable=True).indices
    row = torch.empty_like(order)
    row[order] = torch.arange(T * k)
    want = torch.where(key < G, row, ~row).reshape(T, k).int()
    assert torch.equal(slot_row.cpu(), want)
    assert torch.equal(sizes.cpu(), torch.bincount(key, minlength=G + 1)[:G].int())


ROWS = [(1, 1, 1), (1, 8, 1408), (5, 3, 7), (4, 2, 8), (33, 8, 9), (17, 1, 64), (64, 4, 130), (9, 5, 1027),
        (130, 6, 2880), (3, 64, 40), (2, 2, 5003), (700, 8, 1408), (5, 9, 16384)]


def _slots(T, k, seed, unrouted):
    _, slot_row = ref.sort_tokens(_ids(T, k, 6, seed, unrouted), 6)
    return slot_row


@pytest.mark.parametrize("unrouted", [0.0, 0.4])
@pytest.mark.parametrize("T,k,D", ROWS)
def test_dispatch(T, k, D, unrouted):
    import moe_grouped_matrix_amd as m
    g = torch.Generator().manual_seed(T + k + D)
    slot_row = _slots(T, k, D, unrouted)
    for dtype in (torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int8):
        x = torch.randint(-100, 100, (T, D), generator=g).to(dtype)
        print(f"dispatch T={T} k={k} D={D} {dtype} unrouted={unrouted}", flush=True)
        out = torch.full((T * k, D), 3.0).to(dtype).cuda()
        m.dispatch(x.cuda(), slot_row.cuda(), out=out)
        want = ref.dispatch(x.float(), slot_row).to(dtype)
        iv = torch.int32 if dtype == torch.float32 else torch.int16 if dtype == torch.bfloat16 else torch.int8
        assert torch.equal(out.cpu().view(iv), want.view(iv))


def test_dispatch_of_packed_codes():
    """Codes and scales of quantised tokens go the way of the tokens."""
    import moe_grouped_matrix_amd as m
    x = torch.randn(37, 96, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    slot_row = _slots(37, 3, 5, 0.0).cuda()
    q, s = m.quant_mxfp4(x)
    wq, ws = m.quant_mxfp4(m.dispatch(x, slot_row))
    rows, scales = m.dispatch(q, slot_row), m.dispatch(s, slot_row)
    assert rows.dtype == torch.uint8 and torch.equal(rows, wq)
    assert torch.equal(scales.view(torch.uint8), ws.view(torch.uint8))
    assert torch.equal(m.dispatch(q, slot_row, out=torch.empty_like(wq)), wq)


def test_more_groups_than_there_may_be_allocates_nothing_for_them():
    import moe_grouped_matrix_amd as m
    ids = torch.zeros(4, 2, dtype=torch.int64, device="cuda")
    for groups in (1 << 45, 1 << 70):
        with pytest.raises(m.GmmUnsupported):
            m.sort_tokens(ids, groups)


@pytest.mark.parametrize("unrouted", [0.0, 0.4])
@pytest.mark.parametrize("T,k,D", ROWS)
def test_combine(T, k, D, unrouted):
    import moe_grouped_matrix_amd as m
    g = torch.Generator().manual_seed(T + k + D + 1)
    slot_row = _slots(T, k, D, unrouted)
    off = slot_row < 0
    for rd, wd, od in ((torch.bfloat16, torch.float32, torch.bfloat16), (torch.float32, torch.bfloat16, torch.float32),
                       (torch.float32, None, torch.bfloat16), (torch.bfloat16, None, torch.float32)):
        rows = torch.randn(T * k, D, generator=g).to(rd)
        weights = None
        if wd is not None:
            weights = torch.randn(T, k, generator=g).to(wd)
            weights[off] = float("nan")  # an unrouted slot's weight counts for nothing
        rows[(~slot_row[off]).long()] = float("inf")  # nor does its row
        print(f"combine T={T} k={k} D={D} {rd} {wd} {od} unrouted={unrouted}", flush=True)
        out = m.combine(rows.cuda(), slot_row.cuda(), None if weights is None else weights.cuda(), out_dtype=od).cpu()
        want, terms = ref.combine(rows, slot_row, weights)
        assert out.dtype == od
        ref.within(out, want, k * U * terms + ref.half_step(od, want.abs() + k * U * terms), "combine")


@pytest.mark.parametrize("unrouted", [0.0, 0.4])
@pytest.mark.parametrize("T,k,D", ROWS)
def test_combine_grad(T, k, D, unrouted):
    import moe_grouped_matrix_amd as m
    g = torch.Generator().manual_seed(T + k + D + 2)
    slot_row = _slots(T, k, D, unrouted)
    off = slot_row < 0
    for gd, rd, wd in ((torch.bfloat16, torch.bfloat16, torch.float32), (torch.float32, torch.float32, torch.float32),
                       (torch.bfloat16, torch.float32, torch.bfloat16), (torch.float32, torch.bfloat16, torch.bfloat16)):
        dout = torch.randn(T, D, generator=g).to(gd)
        rows = torch.randn(T * k, D, generator=g).to(rd)
        weights = torch.randn(T, k, generator=g).to(wd)
        weights[off] = float("nan")
        rows[(~slot_row[off]).long()] = float("nan")
        print(f"combine_grad T={T} k={k} D={D} {gd} {rd} {wd} unrouted={unrouted}", flush=True)
        drows, dweights = m.combine_grad(dout.cuda(), rows.cuda(), slot_row.cuda(), weights.cuda())
        wr, ww, terms = ref.combine_grad(dout, rows, slot_row, weights)
        assert drows.dtype == rd and dweights.dtype == wd
        ref.within(drows.cpu(), wr, U * wr.abs() + ref.half_step(rd, wr.abs() * (1 + U)), "drows")
        ref.within(dweights.cpu(), ww, D * U * terms + ref.half_step(wd, ww.abs() + D * U * terms), "dweights")
        assert bool((dweights.cpu()[off] == 0).all())


def test_combine_grad_is_the_difference_quotient():
    """<combine(rows + e a, w + e b) - combine(rows - e a, w - e b), dout> / 2e
    against <a, drows> + <b, dweights>, in f32 with inputs on a coarse grid:
    the quotient is exact in 64 bits up to the second-order term of w * rows,
    e^2 a b, which the central difference cancels."""
    import moe_grouped_matrix_amd as m
    g = torch.Generator().manual_seed(3)
    T, k, D, e = 40, 4, 72, 0.25
    slot_row = _slots(T, k, 1, 0.2)
    pick = lambda *s: torch.randint(-8, 9, s, generator=g).float() / 4  # noqa: E731
    rows, w, dout, a, b = pick(T * k, D), pick(T, k), pick(T, D), pick(T * k, D), pick(T, k)
    s = slot_row.cuda()
    up = m.combine((rows + e * a).cuda(), s, (w + e * b).cuda()).cpu().double()
    dn = m.combine((rows - e * a).cuda(), s, (w - e * b).cuda()).cpu().double()
    drows, dweights = m.combine_grad(dout.cuda(), rows.cuda(), s, w.cuda())
    # multiples of 2^-8 below 2^16: every binary32 step above is exact
    want = ((up - dn) * dout.double()).sum() / (2 * e)
    got = (a.double() * drows.cpu().double()).sum() + (b.double() * dweights.cpu().double()).sum()
    assert float(want) == float(got)


def test_combine_grad_repeats_bit_for_bit():
    import moe_grouped_matrix_amd as m
    g = torch.Generator().manual_seed(4)
    slot_row = _slots(500, 8, 2, 0.1).cuda()
    dout, rows = torch.randn(500, 1027, generator=g).cuda(), torch.randn(4000, 1027, generator=g).cuda()
    w = torch.randn(500, 8, generator=g).cuda()
    first = m.combine_grad(dout, rows, slot_row, w)
    for _ in range(3):
        again = m.combine_grad(dout, rows, slot_row, w)
        assert all(torch.equal(x.view(torch.int32), y.view(torch.int32)) for x, y in zip(first, again))


def test_infinities_in_routed_rows_reach_the_sum():
    import moe_grouped_matrix_amd as m
    rows = torch.ones(4, 16)
    rows[1, 3], rows[2, 5] = float("inf"), float("nan")
    slot_row = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32)
    out = m.combine(rows.cuda(), slot_row.cuda(), torch.ones(2, 2).cuda()).cpu()
    want = torch.full((2, 16), 2.0)
    want[0, 3], want[1, 5] = float("inf"), float("nan")
    assert torch.equal(out.nan_to_num(nan=-1.0), want.nan_to_num(nan=-1.0))


@pytest.mark.parametrize("D", [3, 8, 13, 517, 1027])
def test_infinities_in_any_column_reach_the_gradient(D):
    """One infinity a row, each column in turn: the product is that infinity
    (not the NaN of an infinity times a zero), whatever the width."""
    import moe_grouped_matrix_amd as m
    slot_row = torch.arange(D, dtype=torch.int32).reshape(D, 1)
    for dtype in (torch.float32, torch.bfloat16):
        rows = torch.ones(D, D)
        rows[torch.arange(D), torch.arange(D)] = float("inf") * (1 - 2 * (torch.arange(D) % 2)).float()
        want = torch.diagonal(rows)[:, None]
        print(f"infinite rows D={D} {dtype}", flush=True)
        drows, dw = m.combine_grad(torch.ones(D, D).to(dtype).cuda(), rows.to(dtype).cuda(), slot_row.cuda(),
                                   torch.ones(D, 1).cuda())
        assert torch.equal(dw.cpu(), want)
        assert bool((drows == 1).all())


def test_bad_rows_are_flagged_and_write_nothing():
    import moe_grouped_matrix_amd as m
    T, k, D = 6, 2, 40
    slot_row = torch.arange(T * k, dtype=torch.int32).reshape(T, k)
    slot_row[1, 0], slot_row[2, 1], slot_row[3, 0] = 12, 2 ** 31 - 1, -2 ** 31
    m.device_flags()
    x = torch.arange(T * D).reshape(T, D).float()
    out = m.dispatch(x.cuda(), slot_row.cuda(), out=torch.full((T * k, D), -1.0).cuda()).cpu()
    assert m.device_flags() == m.FLAG_BAD_ROW
    want = x.repeat_interleave(k, 0)
    want[[2, 5, 6]] = -1.0
    assert torch.equal(out, want)
    rows = torch.randn(T * k, D)
    w = torch.rand(T, k)
    got = m.combine(rows.cuda(), slot_row.cuda(), w.cuda()).cpu()
    assert m.device_flags() == m.FLAG_BAD_ROW
    good = slot_row.clone()
    good[1, 0], good[2, 1], good[3, 0] = -3, -6, -7
    want = m.combine(rows.cuda(), good.cuda(), w.cuda()).cpu()
    assert torch.equal(got, want)
    drows, dw = m.combine_grad(x.cuda(), rows.cuda(), slot_row.cuda(), w.cuda(),
                               drows=torch.full((T * k, D), -1.0).cuda())
    assert m.device_flags() == m.FLAG_BAD_ROW
    wr, ww = m.combine_grad(x.cuda(), rows.cuda(), good.cuda(), w.cuda())
    assert bool((drows.cpu()[[2, 5, 6]] == -1).all()) and torch.equal(dw, ww)
    keep = [r for r in range(T * k) if r not in (2, 5, 6)]
    assert torch.equal(drows[keep], wr[keep])
    assert m.device_flags() == 0


def test_no_tokens():
    import moe_grouped_matrix_amd as m
    slots = torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    x = torch.zeros(0, 32, dtype=torch.bfloat16, device="cuda")
    assert tuple(m.dispatch(x, slots).shape) == (0, 32)
    assert tuple(m.combine(x, slots).shape) == (0, 32)
    drows, dw = m.combine_grad(x, x, slots, torch.zeros(0, 4, device="cuda"))
    assert tuple(drows.shape) == (0, 32) and tuple(dw.shape) == (0, 4)


def test_rows_past_32_bit_offsets():
    """Rows whose byte offsets pass 2^32: 9 x 64 rows of 2^22 f32 columns
    (9.6 GB), checked where the offsets are largest."""
    import moe_grouped_matrix_amd as m
    T, k, D = 9, 64, 1 << 22
    slot_row = torch.arange(T * k, dtype=torch.int32).flip(0).reshape(T, k).cuda()
    x = torch.arange(T, device="cuda", dtype=torch.float32)[:, None] * torch.ones(D, device="cuda") + 1
    rows = m.dispatch(x, slot_row)
    assert torch.equal(rows.view(T, k, D).amax(2), (T - torch.arange(T, device="cuda")).float()[:, None].expand(T, k))
    assert torch.equal(rows.view(T, k, D).amin(2), (T - torch.arange(T, device="cuda")).float()[:, None].expand(T, k))
    assert torch.equal(m.combine(rows, slot_row), 64 * x)


def test_python_level_refusals():
    import moe_grouped_matrix_amd as m
    ids = torch.zeros(4, 2, dtype=torch.int64, device="cuda")
    with pytest.raises(m.GmmInvalid):
        m.sort_tokens(ids, 0)
    with pytest.raises(m.GmmUnsupported):
        m.sort_tokens(ids, 1025)
    with pytest.raises(m.GmmInvalid):
        m.sort_tokens(ids.float(), 4)
    with pytest.raises(m.GmmInvalid):
        m.sort_tokens(ids.t(), 4)
    with pytest.raises(m.GmmInvalid):
        m.sort_tokens(ids, 4, group_sizes=torch.zeros(5, dtype=torch.int32, device="cuda"))
    x = torch.zeros(4, 64, device="cuda")
    slots = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(m.GmmInvalid):
        m.dispatch(x, slots.long())
    with pytest.raises(m.GmmInvalid):
        m.dispatch(x[:, ::2], slots)
    with pytest.raises(m.GmmInvalid):
        m.dispatch(x.half(), slots)
    with pytest.raises(m.GmmInvalid):
        m.combine(x, slots)
    with pytest.raises(m.GmmInvalid):
        m.combine_grad(x, torch.zeros(8, 64, device="cuda"), slots, None)


def test_more_tokens_than_one_launch_takes():
    """2^26 + 77 one-byte tokens: more waves than a launch holds."""
    import moe_grouped_matrix_amd as m
    T = (1 << 26) + 77
    x = torch.randint(-100, 100, (T, 1), dtype=torch.int8, device="cuda")
    slot_row = torch.arange(T, dtype=torch.int32, device="cuda").flip(0).view(T, 1)
    assert torch.equal(m.dispatch(x, slot_row), x.flip(0))
    assert m.device_flags() == 0
