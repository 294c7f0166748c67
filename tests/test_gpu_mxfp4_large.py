"""Microscaled fp4 past the sizes of one panel of K (128 blocks), of one pass
of the quantiser's and widening's grids, and of one product tile in K and N."""
import pytest
import torch

import moe_reference as ref
import oracle

pytestmark = pytest.mark.gpu

BITS = {torch.float32: torch.int32, torch.bfloat16: torch.int16}


def _check(m, x, side, codes, byte):
    """Codes, scales and widened values of x, on the GPU, bit for bit."""
    q, scale = m.quant_mxfp4(x, operand=side)
    assert torch.equal(scale.view(torch.uint8), byte if side == "lhs" else ref.rhs_layout(byte))
    assert torch.equal(q, ref.pack(codes))
    table = torch.from_numpy(ref.E2M1).float().cuda()
    value = table[codes.int()].reshape(byte.shape + (32,)) * torch.exp2(byte.float() - 127)[..., None]  # exact
    for od in (torch.float32, torch.bfloat16):
        y = m.widen_mxfp4(q, scale, operand=side, out_dtype=od)
        assert torch.equal(y.view(BITS[od]), value.reshape(x.shape).to(od).view(BITS[od]))


def _values(shape, seed):
    """Rows of sizes 2^-20 .. 2^20, with zeros and ties."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp2(torch.randint(-20, 21, shape[:-1] + (1,), generator=g).float())
    return torch.where(torch.rand(shape, generator=g) < 0.02, 0.0, x)


# several panels of K; more tiles than workgroups (2048 on 256 compute units); both
RHS = [(2, 70, 4128), (1, 66, 8224), (3, 5, 9600), (1, 64, 4096), (2100, 3, 64), (700, 200, 32), (1100, 66, 32),
       (700, 1, 12320)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", RHS)
def test_weights(shape, dtype):
    import moe_grouped_matrix_amd as m
    print(f"mxfp4 weights {shape} {dtype}", flush=True)
    x = _values(shape, sum(shape)).to(dtype)
    codes, byte = ref.quant_mxfp4(x)
    _check(m, x.cuda(), "rhs", codes.cuda(), byte.cuda())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_activations_past_one_pass_of_the_grid(dtype):
    """25483 x 1408 elements, 36 million: 4096 workgroups take 33.5 million a
    pass.  The rows are a block times a power of two for every repetition."""
    import moe_grouped_matrix_amd as m
    assert torch.cuda.get_device_properties(0).multi_processor_count * 16 * 1024 * 8 < 25483 * 1408
    base = _values((1499, 1408), 5).to(dtype)
    codes, byte = ref.quant_mxfp4(base)
    print(f"mxfp4 activations {dtype}", flush=True)
    x = torch.cat([base.cuda() * 2.0 ** (r - 8) for r in range(17)])
    zero = (base.reshape(1499, 44, 32) == 0).all(-1)  # a block of zeros keeps its byte
    bytes_ = torch.cat([torch.where(zero, byte.int(), byte.int() + r - 8) for r in range(17)]).to(torch.uint8)
    _check(m, x, "lhs", codes.cuda().repeat(17, 1), bytes_.cuda())


@pytest.mark.parametrize("sizes,K,N", [([5, 0, 40, 17], 4160, 2056), ([4200, 130], 4160, 1032), ([64] * 64, 2048, 264)])
def test_product(sizes, K, N):
    """lhs in {-3..3}, any code, scales 2^-2 .. 2^2: sums exact in binary32."""
    import moe_grouped_matrix_amd as m
    g = torch.Generator().manual_seed(K + N)
    G = len(sizes)
    lhs = torch.randint(-3, 4, (sum(sizes) + 2, K), generator=g).to(torch.bfloat16)
    q = torch.randint(0, 256, (G, N, K // 2), generator=g, dtype=torch.uint8)
    scale = torch.randint(125, 130, (G, K // 32, 1, N), generator=g).to(torch.uint8).view(torch.float8_e8m0fnu)
    gs = torch.tensor(sizes, dtype=torch.int32)
    want = oracle.gmm_reference(lhs, q, gs, rhs_format="fp4_e2m1", rhs_scale=scale)
    for od in (torch.float32, torch.bfloat16):
        print(f"mxfp4 product {sizes[:4]} K={K} N={N} {od}", flush=True)
        out = m.gmm(lhs.cuda(), q.cuda(), gs.cuda(), rhs_scale=scale.cuda(), rhs_format="fp4_e2m1", out_dtype=od).cpu()
        assert torch.equal(out.view(BITS[od]), oracle.round_to(want, od).view(BITS[od]))
