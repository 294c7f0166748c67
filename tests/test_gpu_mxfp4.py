"""GPU parity of microscaled fp4: quantisation and widening bit for bit
against the definition, and the grouped product of a bf16 lhs with fp4 weights
and E8M0 block scales against the oracle.

The product's sums run in binary32 over K exact products (a bf16 times a
widened fp4 value has at most 10 significant bits): with u = 2^-24 an error of
at most K u sum|a b| whatever their order, then one rounding to the output
type; inputs on a coarse grid make every sum exact, and those cases have to
agree bit for bit."""
import pytest
import torch

import moe_reference as ref
import oracle

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _e8(t):
    return t.to(torch.uint8).view(torch.float8_e8m0fnu)


def _hard(shape, seed, dtype):
    """Normals over a wide range of block sizes, with every border case of the
    rounding, zeros of both signs, blocks of zeros, the smallest and largest
    values, infinities and NaN sprinkled in."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    nb = shape[-1] // 32
    big = torch.exp2(torch.randint(-140, 120, shape[:-1] + (nb, 1), generator=g).double())
    b = x.reshape(shape[:-1] + (nb, 32)).double() * big
    kind = torch.randint(0, 10, shape[:-1] + (nb, 1), generator=g)
    grid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 6.0, 0.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5,
                         -5.0, -7.0, 0.2490234375, 0.251953125, 4.96875, 5.03125, 7.96875, -0.0, 1e-3, -1e-3, 0.5, 1.0,
                         1.5, 2.0, 3.0, 4.0], dtype=torch.float64)
    b = torch.where(kind == 0, grid * torch.exp2(torch.log2(big).round()), b)
    b = torch.where(kind == 1, torch.zeros_like(b), b)
    b = torch.where(kind == 2, -torch.zeros_like(b), b)
    b = torch.where(kind == 3, b * 2.0 ** -126, b)  # subnormals and underflow
    top = torch.finfo(dtype).max
    b = b.clamp(-top, top).reshape(shape).to(dtype)
    flat = b.reshape(-1)
    n = flat.numel()
    if n >= 3200:
        at = torch.randint(0, n, (6,), generator=g)
        flat[at[0]], flat[at[1]], flat[at[2]] = float("inf"), float("-inf"), float("nan")
        flat[at[3]], flat[at[4]] = top, -top
    return b


LHS = [(1, 32), (1, 64), (3, 96), (7, 1408), (64, 32), (65, 160), (257, 704), (33, 4096), (2048, 1408)]
RHS = [(1, 1, 32), (2, 3, 64), (3, 8, 96), (1, 65, 160), (5, 33, 704), (4, 200, 256), (2, 130, 1408), (7, 64, 32)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", LHS + RHS)
def test_quant_and_widen(shape, dtype):
    import moe_grouped_matrix_amd as m
    x = _hard(shape, sum(shape), dtype)
    side = "lhs" if len(shape) == 2 else "rhs"
    print(f"quant {shape} {dtype}", flush=True)
    q, scale = m.quant_mxfp4(x.cuda(), operand=side)
    codes, byte = ref.quant_mxfp4(x)
    want = byte if side == "lhs" else ref.rhs_layout(byte)
    assert torch.equal(scale.cpu().view(torch.uint8), want)
    assert torch.equal(q.cpu(), ref.pack(codes))
    value = ref.values(codes, byte)
    for od in (torch.float32, torch.bfloat16):
        y = m.widen_mxfp4(q, scale, operand=side, out_dtype=od).cpu()
        iv = torch.int32 if od == torch.float32 else torch.int16
        nan = value.isnan()
        assert torch.equal(y.isnan(), nan)
        assert torch.equal(y[~nan].view(iv), value[~nan].to(od).view(iv))


def test_widen_takes_every_code_and_scale_byte():
    """256 rows, one per scale byte; the widened values are the conversions of
    the 64-bit ones (exact but for the infinities of bytes 253 and 254)."""
    import moe_grouped_matrix_amd as m
    codes = torch.arange(64).remainder(16).to(torch.uint8).repeat(256, 1)
    byte = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 2)
    value = ref.values(codes, byte)
    for od in (torch.float32, torch.bfloat16):
        y = m.widen_mxfp4(ref.pack(codes).cuda(), _e8(byte).cuda(), out_dtype=od).cpu()
        want = value.to(od)
        assert torch.equal(y.isnan(), want.isnan())
        live = ~want.isnan()
        iv = torch.int32 if od == torch.float32 else torch.int16
        assert torch.equal(y[live].view(iv), want[live].view(iv))


def test_quantised_values_survive_quantisation():
    import moe_grouped_matrix_amd as m
    x = torch.randn(64, 256, generator=torch.Generator().manual_seed(1)).cuda()
    q, s = m.quant_mxfp4(x)
    y = m.widen_mxfp4(q, s)
    assert torch.equal(y.float(), m.widen_mxfp4(*m.quant_mxfp4(y), out_dtype=torch.float32))
    # an element is off by at most half a step of its block's grid, or by what lies past 6 (a quarter)
    assert bool(((y - x).abs() <= 0.25 * x.abs().reshape(64, 8, 32).amax(-1).repeat_interleave(32, 1)).all())


# (rows per group, rows past the groups, K, N, lhs rows before an offset shard)
PRODUCTS = [
    ([1], 0, 64, 8), ([3, 0, 2], 2, 128, 72), ([33, 0, 70, 257, 5], 7, 256, 200), ([0, 0, 0], 4, 192, 40),
    ([8] * 40, 0, 384, 264), ([1, 0, 64, 65, 2, 31], 0, 512, 256), ([130, 5], 1, 1408, 136), ([20] * 9, 3, 448, 1408),
    ([5000, 0, 4200, 129], 9, 320, 264), ([9000], 0, 704, 520), ([4096, 4096], 5, 256, 128), ([8200], 0, 64, 48),
    ([300, 9001, 1, 255, 256, 257], 3, 192, 776),
]


def _grid_case(sizes, extra, K, N, seed):
    """lhs in {-3..3}, any code, scales 2^-2 .. 2^2: products are multiples of
    2^-3 below 2^6.2, sums exact in binary32 while K < 2^14."""
    g = torch.Generator().manual_seed(seed)
    M, G = sum(sizes) + extra, len(sizes)
    lhs = torch.randint(-3, 4, (M, K), generator=g).to(torch.bfloat16)
    q = torch.randint(0, 256, (G, N, K // 2), generator=g, dtype=torch.uint8)
    scale = torch.randint(125, 130, (G, K // 32, 1, N), generator=g)
    return lhs, q, _e8(scale), torch.tensor(sizes, dtype=torch.int32)


@pytest.mark.parametrize("policy", [0, 1, 2])
@pytest.mark.parametrize("sizes,extra,K,N", PRODUCTS)
def test_product_is_exact_on_a_grid(sizes, extra, K, N, policy):
    import moe_grouped_matrix_amd as m
    lhs, q, scale, gs = _grid_case(sizes, extra, K, N, K + N)
    bias = torch.randint(-8, 9, (len(sizes), 1, N), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    m.set_tile_policy(policy)
    try:
        for kw, od in ((dict(), torch.float32), (dict(rhs_bias=bias), torch.bfloat16),
                       (dict(rhs_bias=bias.float()), torch.float32), (dict(), torch.bfloat16)):
            print(f"mxfp4 product {sizes[:6]} K={K} N={N} policy={policy} {od} bias={bool(kw)}", flush=True)
            out = m.gmm(lhs.cuda(), q.cuda(), gs.cuda(), rhs_scale=scale.cuda(), rhs_format="fp4_e2m1", out_dtype=od,
                        **{k: v.cuda() for k, v in kw.items()}).cpu()
            want = oracle.round_to(oracle.gmm_reference(lhs, q, gs, rhs_format="fp4_e2m1", rhs_scale=scale, **kw), od)
            iv = torch.int32 if od == torch.float32 else torch.int16
            assert torch.equal(out.view(iv), want.view(iv)), (out.float() - want.float()).abs().max()
    finally:
        m.set_tile_policy(0)
    assert m.device_flags() == 0


@pytest.mark.parametrize("limit", [1, 5, 24])
def test_product_with_few_workgroups(limit):
    """Each workgroup runs many tiles back to back."""
    import moe_grouped_matrix_amd as m
    m.set_grid_limit(limit)
    try:
        for sizes, extra, K, N in (([40, 0, 3, 64, 65, 100], 3, 512, 600), ([4100, 300, 4200, 1], 5, 256, 520)):
            lhs, q, scale, gs = _grid_case(sizes, extra, K, N, 9)
            out = m.gmm(lhs.cuda(), q.cuda(), gs.cuda(), rhs_scale=scale.cuda(), rhs_format="fp4_e2m1").cpu()
            want = oracle.round_to(oracle.gmm_reference(lhs, q, gs, rhs_format="fp4_e2m1", rhs_scale=scale),
                                   torch.float32)
            assert torch.equal(out.view(torch.int32), want.view(torch.int32)), (limit, sizes)
    finally:
        m.set_grid_limit(0)


@pytest.mark.parametrize("sizes,extra,K,N", PRODUCTS)
def test_product_on_random_values(sizes, extra, K, N):
    import moe_grouped_matrix_amd as m
    g = torch.Generator().manual_seed(K)
    M, G = sum(sizes) + extra, len(sizes)
    lhs = torch.randn(M, K, generator=g).to(torch.bfloat16)
    w = torch.randn(G, N, K, generator=g) * 0.02
    codes, byte = ref.quant_mxfp4(w)
    q, scale = m.quant_mxfp4(w.cuda(), operand="rhs")
    gs = torch.tensor(sizes, dtype=torch.int32)
    value = ref.values(codes, byte)
    want, terms = torch.zeros(M, N, dtype=torch.float64), torch.zeros(M, N, dtype=torch.float64)
    lo = 0
    for h, s in enumerate(sizes):
        a = lhs[lo:lo + s].double()
        want[lo:lo + s], terms[lo:lo + s] = a @ value[h].t(), a.abs() @ value[h].t().abs()
        lo += s
    for od in (torch.float32, torch.bfloat16):
        out = m.gmm(lhs.cuda(), q, gs.cuda(), rhs_scale=scale, rhs_format="fp4_e2m1", out_dtype=od).cpu()
        ref.within(out, want, K * U * terms + ref.half_step(od, want.abs() + K * U * terms), f"product {od}")


def test_product_of_a_shard_and_an_existing_output():
    import moe_grouped_matrix_amd as m
    for scale_rows in (1, 60):
        sizes = [s * scale_rows for s in (30, 0, 70, 41, 5, 90)]
        lhs, q, scale, gs = _grid_case(sizes, 6, 384, 136, 4)
        keep = torch.randn(lhs.shape[0], 136, generator=torch.Generator().manual_seed(1))
        for s, Ga in ((2, 3), (0, 2), (5, 1)):
            kw = dict(rhs_format="fp4_e2m1", group_offset=s)
            qs, ss = q[s:s + Ga].contiguous(), scale.view(torch.uint8)[s:s + Ga].contiguous().view(torch.float8_e8m0fnu)
            ref_out = oracle.gmm_reference(lhs, qs, gs, rhs_scale=ss, **kw)
            out = m.gmm(lhs.cuda(), qs.cuda(), gs.cuda(), rhs_scale=ss.cuda(), **kw).cpu()
            assert torch.equal(out, oracle.round_to(ref_out, torch.float32))
            lo, hi = sum(sizes[:s]), sum(sizes[:s + Ga])
            got = m.gmm(lhs.cuda(), qs.cuda(), gs.cuda(), rhs_scale=ss.cuda(), existing_out=keep.cuda(), **kw).cpu()
            assert torch.equal(got[lo:hi], out[lo:hi]) and torch.equal(got[:lo], keep[:lo]) and torch.equal(got[hi:], keep[hi:])


def test_product_scale_bytes_over_their_range():
    """Every scale byte from 0 to 252 on weights of one column each, against
    the exact value: lhs a power of two that brings the product back near 1."""
    import moe_grouped_matrix_amd as m
    K, N = 64, 256
    byte = torch.arange(N).clamp(max=252)
    scale = byte.to(torch.uint8).reshape(1, 1, 1, N).repeat(1, 2, 1, 1)
    q = torch.full((1, N, K // 2), 0x35, dtype=torch.uint8)  # codes 5 (3.0) and 3 (1.5)
    for e in (-100, 0, 100):
        lhs = torch.zeros(1, K)
        lhs[0, 0], lhs[0, 33] = 2.0 ** e, 2.0 ** e
        out = m.gmm(lhs.to(torch.bfloat16).cuda(), q.cuda(), torch.tensor([1], dtype=torch.int32).cuda(),
                    rhs_scale=_e8(scale).cuda(), rhs_format="fp4_e2m1").cpu()[0].double()
        want = 4.5 * torch.exp2(byte.double() - 127 + e)
        live = (want < 2.0 ** 127) & (want > 2.0 ** -120)
        assert int(live.sum()) > 100
        assert torch.equal(out[live], want[live])


def test_product_refusals():
    import moe_grouped_matrix_amd as m
    lhs, q, scale, gs = _grid_case([4], 0, 128, 16, 1)
    a, b, s, n = lhs.cuda(), q.cuda(), scale.cuda(), gs.cuda()
    s8 = scale.view(torch.uint8)
    with pytest.raises(m.GmmUnsupported):  # blocks of 64
        m.gmm(a, b, n, rhs_format="fp4_e2m1", rhs_scale=_e8(s8[:, :2].contiguous()).cuda())
    with pytest.raises(m.GmmUnsupported):  # an E8M0 lhs scale on a bf16 lhs
        m.gmm(a, b, n, rhs_format="fp4_e2m1", rhs_scale=s, lhs_scale=_e8(torch.full((4, 4), 127)).cuda())
    with pytest.raises(m.GmmUnsupported):  # E8M0 scales on int4 weights
        m.gmm(a, b, n, rhs_format="int4", rhs_scale=s)
    with pytest.raises(m.GmmError):  # read in place as [G,K,N]
        m.gmm(a, torch.zeros(1, 128, 8, dtype=torch.uint8, device="cuda"), n, rhs_format="fp4_e2m1", rhs_scale=s,
              transpose_rhs=True)
    with pytest.raises(m.GmmInvalid):
        m.gmm(a, b, n, rhs_format="fp4_e2m1", rhs_scale=_e8(s8.reshape(1, 16, 1, 4)).cuda())
    with pytest.raises(m.GmmInvalid):
        m.quant_mxfp4(a, operand="rhs")
    with pytest.raises(m.GmmInvalid):
        m.quant_mxfp4(a, operand="weights")
    with pytest.raises(m.GmmInvalid):
        m.quant_mxfp4(a[:, :48].contiguous())
