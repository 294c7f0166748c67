"""gmv gives equal bits for equal inputs however it finds an expert's slots
(include/gmm_layer.h).  An expert of 17 to 20 slots is done as sixteen rows and a
rest of one to four, which add in another order with scale blocks of 128 or E8M0
scales: which slots are the rest must not depend on which wave comes first.

384 experts with fewer than 192 slots take one way to find them, the first
experts of the same weights, less than twice as many as there are slots,
another that lists them in their order.  Rows and bits have to be the same."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16, E8 = torch.float32, torch.bfloat16, torch.float8_e8m0fnu


def _case(T, k, G, few, N, K, fmt, seed):
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 256, (G, N, K // 2), generator=g, dtype=torch.uint8)
    if fmt == "fp4_e2m1":
        s = torch.randint(117, 128, (G, K // 32, 1, N), generator=g, dtype=torch.uint8).view(E8)
    else:
        s = torch.randn(G, K // 128, 1, N, generator=g) * 0.1
    ids = torch.randint(0, few, (T, k), generator=g, dtype=torch.int32)
    ids[ids == few // 2] = 0
    ids[torch.arange(T), torch.randint(0, k, (T,), generator=g)] = few // 2  # one expert that every token chose
    x = torch.randn(T, K, generator=g).to(BF16)
    return x.cuda(), q.cuda(), ids.cuda(), s.cuda(), torch.rand(T, k, generator=g).cuda()


@pytest.mark.parametrize("fmt", ["int4", "uint4", "fp4_e2m1"])
@pytest.mark.parametrize("T", [17, 18, 20])
def test_equal_bits(T, fmt):
    import moe_grouped_matrix_amd as m
    k, G, few = 8, 384, 200
    x, q, ids, s, w = _case(T, k, G, few, 1408, 1408, fmt, T)
    assert 64 < T * k and 2 * T * k < G and few < 2 * T * k
    for weights in (None, w):
        for out_dtype in (F32, BF16):
            kw = dict(rhs_format=fmt, weights=weights, out_dtype=out_dtype)
            want = m.gmv(x, q[:few], ids, rhs_scale=s[:few], **kw)
            for _ in range(8):
                assert torch.equal(m.gmv(x, q, ids, rhs_scale=s, **kw), want)


@pytest.mark.parametrize("fmt", ["int4", "fp4_e2m1"])
def test_every_slot_on_one_expert(fmt):
    """100 slots (six times sixteen and four) of one of 1024 experts, and of one expert alone."""
    import moe_grouped_matrix_amd as m
    x, q, ids, s, _ = _case(100, 1, 1024, 200, 96, 640, fmt, 1)
    ids.fill_(777)
    one = torch.zeros_like(ids)
    want = m.gmv(x, q[777:778], one, rhs_format=fmt, rhs_scale=s[777:778])
    assert torch.equal(m.gmv(x, q[777:778], rhs_format=fmt, rhs_scale=s[777:778]), want)
    for _ in range(8):
        assert torch.equal(m.gmv(x, q, ids, rhs_format=fmt, rhs_scale=s), want)
