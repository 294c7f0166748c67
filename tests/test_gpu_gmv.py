"""GPU parity of gmv (include/gmm_layer.h, gmm_gmv_run) against its plain
64-bit form.

Tolerance (u = 2^-24): the products of bf16 values with four-bit codes are
exact in binary32, and their sums over K, in whatever order, are off by at most
one u of the absolute terms an addition: fewer than K/8 + 64 additions lie on
any path from a term to the result (a chain over K in pieces of eight or more,
and the joins of lanes and waves), and scale, zero point and weights add a few
roundings each; `mag` adds up the absolute terms, the zero point's apart from
the code's.  Then half a step of the output's type."""
import math

import pytest
import torch

import layer_reference as ref
from moe_reference import half_step, within

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16, E8 = torch.float32, torch.bfloat16, torch.float8_e8m0fnu


def _case(T, k, G, N, K, fmt, block, scale, zero=False, per_slot=False, weighted=False, seed=0, ids_dtype=torch.int32, wild=0.2):
    g = torch.Generator().manual_seed(seed + 1000 * T + K)
    x = torch.randn((T, k, K) if per_slot else (T, K), generator=g).to(BF16)
    q = torch.randint(0, 256, (G, N, K // 2), generator=g, dtype=torch.uint8)
    nb = K // block
    if scale == E8:
        s = torch.randint(117, 128, (G, nb, 1, N), generator=g, dtype=torch.uint8).view(E8)
    else:
        s = (torch.randn(G, nb, 1, N, generator=g) * 0.1).to(scale)
    z = (torch.rand(G, nb, 1, N, generator=g) * 15).to(scale) if zero else None
    ids = torch.randint(0, G, (T, k), generator=g)
    off = torch.rand(T, k, generator=g) < wild
    ids = torch.where(off, torch.tensor([-1, G, G + 7, 2 ** 31 - 1])[torch.randint(0, 4, (T, k), generator=g)], ids).to(ids_dtype)
    w = torch.rand(T, k, generator=g) if weighted else None
    if weighted:
        w[off] = math.nan  # not read
    return x, q, ids, s, z, w


def _dev(*ts):
    return [t.cuda() if t is not None else None for t in ts]


def _check(case, fmt, out_dtype, what=""):
    import moe_grouped_matrix_amd as m
    x, q, ids, s, z, w = case
    dx, dq, di, ds, dz, dw = _dev(*case)
    got = m.gmv(dx, dq, di, rhs_format=fmt, rhs_scale=ds, rhs_zero=dz, weights=dw, out_dtype=out_dtype)
    want, mag = ref.gmv(x, q, ids, fmt, s, z, w)
    assert got.dtype == out_dtype and got.shape == want.shape
    K = 2 * q.shape[2]
    slack = mag * (K / 8 + 64 + 8) * U + 1e-37
    if out_dtype == BF16:
        slack = slack + half_step(BF16, want) * (1 + 2 ** -7)
    within(got.cpu(), want, slack, what)
    return got


SHAPES = [(1, 1, 1, 1, 32), (1, 8, 16, 64, 128), (1, 8, 128, 33, 704), (2, 3, 5, 17, 160), (3, 1, 1, 130, 1408), (5, 2, 3, 65, 96),
          (16, 2, 4, 48, 256), (17, 1, 1, 31, 512), (33, 2, 2, 20, 192), (64, 8, 32, 40, 64), (1, 64, 70, 24, 96), (200, 1, 3, 9, 224)]


@pytest.mark.parametrize("fmt,scale,zero", [("int4", F32, False), ("int4", BF16, True), ("uint4", F32, True), ("uint4", BF16, False),
                                            ("fp4_e2m1", E8, False), ("fp4_e2m1", F32, False), ("fp4_e2m1", BF16, False)])
@pytest.mark.parametrize("T,k,G,N,K", SHAPES)
def test_shapes_and_formats(T, k, G, N, K, fmt, scale, zero):
    for i, (per_slot, weighted) in enumerate([(False, False), (True, True), (False, True), (True, False)]):
        blocks = [32] if scale == E8 else sorted({b for b in (32, 64, 96, 128, K) if K % b == 0})
        block = blocks[i % len(blocks)]
        case = _case(T, k, G, N, K, fmt, block, scale, zero, per_slot, weighted, i, torch.int64 if i & 1 else torch.int32)
        _check(case, fmt, BF16 if i & 2 else F32, (per_slot, weighted, block))


@pytest.mark.parametrize("fmt,scale,zero,block", [("int4", F32, False, 128), ("uint4", BF16, True, 32), ("fp4_e2m1", E8, False, 32),
                                                  ("int4", BF16, True, 64), ("uint4", F32, False, 1408)])
def test_a_layers_size(fmt, scale, zero, block):
    """8 of 12 experts of 1408 x 1408, one token and several that share experts."""
    for T, weighted in ((1, False), (1, True), (4, False), (30, True)):
        _check(_case(T, 8, 12, 1408, 1408, fmt, block, scale, zero, weighted, weighted, T), fmt, BF16, T)


def test_every_code_and_every_scale_byte():
    """One-hot vectors read every code back exactly under a scale of 1; E8M0
    bytes 1 to 252 and 255 as they stand."""
    import moe_grouped_matrix_amd as m
    K = 32
    q = (torch.arange(256) % 256).to(torch.uint8).reshape(1, 16, 16)
    x = torch.eye(K).to(BF16)
    for fmt in ("int4", "uint4", "fp4_e2m1"):
        got = m.gmv(x.cuda(), q.cuda(), rhs_format=fmt, rhs_scale=torch.ones(1, 1, 1, 16).cuda())
        want = ref.code_values(fmt)[ref.unpack(q).long()][0].t()
        assert torch.equal(got.cpu().double()[:, 0], want), fmt
    scale = torch.arange(256, dtype=torch.uint8).reshape(1, 1, 1, 256).view(E8)
    q = torch.full((1, 256, 16), 0x22, dtype=torch.uint8)  # 1.0
    x = torch.zeros(1, K)
    x[0, 5] = 1
    got = m.gmv(x.to(BF16).cuda(), q.cuda(), rhs_format="fp4_e2m1", rhs_scale=scale.cuda()).cpu()[0, 0].double()
    assert torch.equal(got[1:253], torch.exp2(torch.arange(1, 253).double() - 127))
    assert math.isnan(float(got[255]))


def test_dense_without_ids_and_empty():
    import moe_grouped_matrix_amd as m
    x, q, ids, s, z, w = _case(5, 1, 1, 70, 128, "int4", 64, F32, wild=0.0)
    dx, dq, ds = _dev(x, q, s)
    a = m.gmv(dx, dq, rhs_format="int4", rhs_scale=ds)
    assert torch.equal(a, m.gmv(dx, dq, torch.zeros(5, 1, dtype=torch.int32).cuda(), rhs_format="int4", rhs_scale=ds))
    assert m.gmv(dx[:0], dq, rhs_format="int4", rhs_scale=ds).shape == (0, 1, 70)
    none = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    assert m.gmv(dx[:0], dq, none, rhs_format="int4", rhs_scale=ds, weights=torch.empty(0, 3).cuda()).shape == (0, 70)


def test_all_slots_unrouted_and_infinities():
    """Slots without an expert give zeros whatever their x holds; an infinity in
    one token's x stays in that token's rows."""
    import moe_grouped_matrix_amd as m
    x, q, ids, s, z, w = _case(6, 2, 3, 40, 96, "int4", 32, F32, True, True, True, wild=0.0)
    ids[2], ids[4, 1] = -1, 3
    x[2], x[4, 1] = math.nan, math.inf
    w[2], w[4, 1] = math.nan, math.nan
    dx, dq, di, ds, dz, dw = _dev(x, q, ids, s, z, w)
    got = m.gmv(dx, dq, di, rhs_format="int4", rhs_scale=ds, rhs_zero=dz).cpu()
    assert not bool(got[2].any()) and not bool(got[4, 1].any()) and bool(torch.isfinite(got).all())
    got = m.gmv(dx, dq, di, rhs_format="int4", rhs_scale=ds, rhs_zero=dz, weights=dw).cpu()
    assert not bool(got[2].any()) and bool(torch.isfinite(got).all())
    x[3, 0, 7] = math.inf
    got = m.gmv(x.cuda(), dq, di, rhs_format="int4", rhs_scale=ds).cpu()
    assert not bool(torch.isfinite(got[3, 0]).any())
    others = torch.ones(6, 2, dtype=torch.bool)
    others[3, 0] = False
    assert bool(torch.isfinite(got[others]).all())


def test_most_slots():
    """4096 slots: one expert for all of them, and many experts."""
    _check(_case(64, 64, 1, 33, 64, "int4", 32, F32, wild=0.0), "int4", F32, "one")
    _check(_case(4096, 1, 300, 19, 64, "uint4", 64, BF16, True), "uint4", F32, "many")
    _check(_case(512, 8, 1024, 8, 32, "fp4_e2m1", 32, E8, False, False, True), "fp4_e2m1", BF16, "weighted")


@pytest.mark.parametrize("T,k,G", [(8, 8, 9), (13, 5, 9), (1, 64, 1024), (10, 10, 300), (5, 13, 131), (5, 13, 130), (60, 4, 1000), (2, 8, 40),
                                   (17, 1, 40), (1, 17, 40), (64, 8, 2)])
def test_every_way_to_find_the_slots(T, k, G):
    """Up to 64 slots, more slots than half the experts, fewer; ids that are
    experts only in their low 32 bits are none."""
    for weighted in (False, True):
        x, q, ids, s, z, w = _case(T, k, G, 40, 96, "int4", 32, F32, True, weighted, weighted, G, torch.int64, 0.1)
        ids[0, 0] = 2 ** 32 + 1
        ids[T // 2, k - 1] = -2 ** 63
        if weighted:
            w[0, 0] = w[T // 2, k - 1] = math.nan
        _check((x, q, ids, s, z, w), "int4", F32, weighted)
    one = torch.full((T, k), G - 1)  # every slot on one expert, and none anywhere
    x, q, _, s, z, w = _case(T, k, G, 40, 96, "uint4", 96, BF16, True, True, True, wild=0.0)
    _check((x, q, one, s, z, w), "uint4", F32, "one")
    _check((x, q, torch.full_like(one, -1), s, z, torch.full_like(w, math.nan)), "uint4", F32, "none")


@pytest.mark.parametrize("K,N", [(32, 5000), (64, 1), (16384, 24), (99968, 17), (2 ** 20 - 32, 3)])
def test_long_and_short_k(K, N):
    for fmt, block, scale, zero in (("int4", 32, F32, False), ("uint4", K, BF16, True), ("fp4_e2m1", 32, E8, False)):
        _check(_case(2, 2, 3, N, K, fmt, block, scale, zero, K < 1000, True, 5, wild=0.0), fmt, F32, (fmt, "weighted"))
        _check(_case(7, 1, 1, N, K, fmt, block, scale, zero, False, False, 6, wild=0.0), fmt, BF16, fmt)


def test_two_streams_at_once():
    """Two weighted products that overlap in time, each with a workspace of its own."""
    import moe_grouped_matrix_amd as m
    cases = [_case(40, 4, 10, 1000, 512, "int4", 64, F32, False, True, True, i, wild=0.0) for i in range(2)]
    dev = [_dev(*c) for c in cases]
    call = lambda d, **kw: m.gmv(d[0], d[1], d[2], rhs_format="int4", rhs_scale=d[3], weights=d[5], **kw)  # noqa: E731
    want = [call(d) for d in dev]
    streams = [torch.cuda.Stream() for _ in dev]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    got = [[call(d, stream=st) for d, st in zip(dev, streams)] for _ in range(5)]
    torch.cuda.synchronize()
    for pair in got:
        for a, b in zip(pair, want):
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """1024 groups of 2112 x 2048 (2.2e9 bytes of codes): the last group's product."""
    import moe_grouped_matrix_amd as m
    G, N, K = 1024, 2112, 2048
    q = torch.empty(G, N, K // 2, dtype=torch.uint8, device="cuda")
    q.zero_()
    g = torch.Generator().manual_seed(1)
    last = torch.randint(0, 256, (1, N, K // 2), generator=g, dtype=torch.uint8)
    q[G - 1] = last[0].cuda()
    scale = torch.ones(G, 1, 1, N, device="cuda")
    x = torch.randn(2, K, generator=g).to(BF16)
    got = m.gmv(x.cuda(), q, torch.tensor([[G - 1, 0], [1, G - 1]], dtype=torch.int32).cuda(), rhs_format="int4", rhs_scale=scale).cpu()
    want, mag = ref.gmv(x, last, torch.zeros(2, 1, dtype=torch.int32), "int4", torch.ones(1, 1, 1, N))
    within(got[0, 0], want[0, 0], mag[0, 0] * (K / 8 + 72) * U, "last group")
    within(got[1, 1], want[1, 0], mag[1, 0] * (K / 8 + 72) * U, "last group")
    assert not bool(got[0, 1].any()) and not bool(got[1, 0].any())


def test_matches_the_grouped_product():
    """The same tensors through sort, dispatch and gmm give the same rows, to
    the tolerance of both."""
    import moe_grouped_matrix_amd as m
    T, k, G, N, K = 24, 3, 7, 128, 256
    x, q, ids, s, _, _ = _case(T, k, G, N, K, "int4", 128, F32, wild=0.0)
    dx, dq, di, ds = _dev(x, q, ids, s)
    sizes, slot_row = m.sort_tokens(di, G)
    rows = m.gmm(m.dispatch(dx, slot_row), dq, sizes, rhs_scale=ds, rhs_format="int4")
    _, mag = ref.gmv(x, q, ids, "int4", s)
    got = m.gmv(dx, dq, di, rhs_format="int4", rhs_scale=ds)
    within(got.cpu(), rows[slot_row.long()].cpu().double(), 2 * mag * (K / 8 + 72) * U, "gmm")


@pytest.mark.parametrize("weighted", [False, True])
def test_captured_and_replayed(weighted):
    import moe_grouped_matrix_amd as m
    case = _case(4, 8, 20, 200, 704, "uint4", 32, BF16, True, True, weighted)
    x, q, ids, s, z, w = _dev(*case)
    w2 = torch.nan_to_num(w) if weighted else None

    def step():
        return m.gmv(x, q, ids, rhs_format="uint4", rhs_scale=s, rhs_zero=z, weights=w2, out_dtype=BF16)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = step(), step()  # (two calls of one graph: a workspace each)
    for i in range(4):
        g = torch.Generator().manual_seed(i)
        x.copy_(torch.randn(x.shape, generator=g))
        ids.copy_(torch.randint(-1, 20, ids.shape, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        assert torch.equal(a, want) and torch.equal(b, want)
