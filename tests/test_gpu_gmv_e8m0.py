"""Every E8M0 byte under every fp4 code in gmv (include/gmm_layer.h): weights
are widened to bf16 with their scale, exactly for bytes 0 to 252; those past the
largest bf16 (bytes 253 and 254) become infinities, and byte 255 makes its block
NaN.  x of one value that keeps the products among binary32's normal numbers, one
code a column, zeros elsewhere: the result is one exact product."""
import pytest
import torch

import layer_reference as ref

pytestmark = pytest.mark.gpu

E8 = torch.float8_e8m0fnu


def _columns(K, at):
    """Column 16 b + c: code c at element `at`, scale byte b in its block, 127 in the others."""
    N = 256 * 16
    byte, code = torch.arange(256).repeat_interleave(16), torch.arange(16).repeat(256)
    q = torch.zeros(1, N, K // 2, dtype=torch.uint8)
    q[0, :, at // 2] = (code << (4 * (at & 1))).to(torch.uint8)
    s = torch.full((1, K // 32, 1, N), 127, dtype=torch.uint8)
    s[0, at // 32, 0] = byte.to(torch.uint8)
    want = ref.code_values("fp4_e2m1")[code] * torch.exp2(byte.double() - 127)
    return q, s.view(E8), byte, want


@pytest.mark.parametrize("T,weighted", [(1, False), (6, False), (1, True), (20, True)])
@pytest.mark.parametrize("K,at", [(32, 5), (160, 138)])
def test_every_byte_and_code(K, at, T, weighted):
    import moe_grouped_matrix_amd as m
    q, s, byte, want = _columns(K, at)
    w = torch.ones(T, 1).cuda() if weighted else None
    for power, these in ((64, byte < 127), (-64, (byte >= 127) & (byte < 255))):
        x = torch.zeros(T, K)
        x[:, at] = 2.0 ** power
        got = m.gmv(x.to(torch.bfloat16).cuda(), q.cuda(), torch.zeros(T, 1, dtype=torch.int32).cuda(), rhs_format="fp4_e2m1",
                    rhs_scale=s.cuda(), weights=w).cpu().reshape(T, -1).double()
        exact = torch.where(want.abs() > torch.finfo(torch.bfloat16).max, torch.sign(want) * torch.inf, want) * 2.0 ** power
        assert bool(exact[these].isinf().any()) == (power < 0)
        for t in range(T):
            assert torch.equal(got[t, these], exact[these]), (power, t)
        assert bool(got[:, byte == 255].isnan().all())
