"""What gmv's sums of int4 are off by (include/gmm_layer.h): codes are added as
code + 8 and 8 times the sum of x is taken off again, so that the roundings go by
|scale| (|code| + |zero| + 16) |x|, whatever the codes are.  Codes of -1, 0 and 1,
most of them 0, under x of one sign, against the 64-bit form: nearly all of the
bound is the 16.

Tolerance: the K/8 + 72 roundings of 2^-24 on any path of tests/test_gpu_gmv.py,
of those terms: |code + 8| <= |code| + 8 in the one sum and |zero + 8| <= |zero| + 8
in the other."""
import pytest
import torch

import layer_reference as ref
from moe_reference import within

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16 = torch.bfloat16


def _packed(codes):
    """[G,N,K] four-bit codes, two to a byte, the first in the low half."""
    b = (codes & 15).to(torch.uint8)
    return b[..., 0::2] | b[..., 1::2] << 4


def _run(x, q, ids, fmt="int4", **kw):
    import moe_grouped_matrix_amd as m
    return m.gmv(x.cuda(), q.cuda(), None if ids is None else ids.cuda(), rhs_format=fmt,
                 **{n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in kw.items()}).cpu()


@pytest.mark.parametrize("block", [32, 128])
@pytest.mark.parametrize("T", [1, 4, 7, 20])
@pytest.mark.parametrize("K", [256, 16384])
def test_sparse_codes_of_one(K, T, block):
    g = torch.Generator().manual_seed(K + T)
    G, N, k = 3, 40, 2
    codes = torch.randint(-1, 2, (G, N, K), generator=g) * (torch.rand(G, N, K, generator=g) < 1 / 256)
    q = _packed(codes)
    assert torch.equal(ref.code_values("int4")[ref.unpack(q).long()].reshape(codes.shape), codes.double())
    x = torch.randn(T, K, generator=g).abs().to(BF16)
    s = torch.rand(G, K // block, 1, N, generator=g) + 0.5
    ids = torch.randint(0, G, (T, k), generator=g, dtype=torch.int32)
    sixteen = torch.full_like(q, 0x88)  # code -8 everywhere: 8 |scale| |x|
    for w in (None, torch.rand(T, k, generator=g)):
        want, mag = ref.gmv(x, q, ids, "int4", s, None, w)
        slack = (mag + 2 * ref.gmv(x, sixteen, ids, "int4", s, None, w)[1]) * (K / 8 + 72) * U
        for zero in (None, torch.zeros_like(s)):
            within(_run(x, q, ids, rhs_scale=s, weights=w, rhs_zero=zero), want, slack, (w is not None, zero is not None))


@pytest.mark.parametrize("T", [1, 6])
def test_far_values(T):
    """As long as the sums of (|code| + 8) |x| stay in range, codes of zero give zeros (x 2^100)."""
    N, K = 33, 256
    x = torch.full((T, K), 2.0 ** 100).to(BF16)
    got = _run(x, torch.zeros(1, N, K // 2, dtype=torch.uint8), None, rhs_scale=torch.ones(1, 2, 1, N))
    assert torch.equal(got, torch.zeros(T, 1, N))


@pytest.mark.parametrize("fmt", ["int4", "uint4", "fp4_e2m1"])
def test_every_code_in_every_place(fmt):
    """One-hot vectors read each of the sixteen codes back from every place of a chunk."""
    N, K = 16, 160
    codes = (torch.arange(N)[:, None] + torch.arange(K)[None, :]) % 16
    got = _run(torch.eye(K).to(BF16), _packed(codes[None]), None, fmt, rhs_scale=torch.ones(1, 1, 1, N))[:, 0]
    assert torch.equal(got.double(), ref.code_values(fmt)[codes].t())
