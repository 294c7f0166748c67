"""The balance loss's gradient of sigmoid scores near 1: the formula's factor
1 - s is the sigmoid of -z, which is a small number of full precision and not what
is left of 1 after s was rounded.

Tolerance (u = 2^-24): every element is p (1 - s) (a - sum a p), with a = coef E f
/ n.  The scores, 1 - s and the sum of the scores come within 8 u each and 8 u for
the sum's additions, and the factors are multiplied with a rounding each: 32 u of
p (1 - s) |a - sum a p|; what is in the brackets is off by (16 + E / 8) u of
|a| + sum |a| p.  There is no absolute term: elements of 10^-12 are held to the
same bound.  The 64-bit form works out 1 - s to 2^-52 / (1 - s), 2^-31 here."""
import pytest
import torch

import layer_reference as ref
from moe_reference import within

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("T,E", [(3, 5), (40, 16), (70, 37), (9, 64), (33, 128), (12, 200), (5, 300), (3, 1024)])
def test_balance_gradient(T, E):
    import moe_grouped_matrix_amd as m
    g = torch.Generator().manual_seed(T + E)
    z = torch.rand(T, E, generator=g) * 10 + 4  # sigmoids from 1 - 0.018 to 1 - 8e-7
    k = min(4, E)
    ids, _ = m.route(z.cuda(), k, scores="sigmoid")
    _, counts, tokens = m.balance_loss(z.cuda(), ids, scores="sigmoid", coef=0.5)
    got = m.router_grad(z.cuda(), ids, scores="sigmoid", counts=counts, tokens=tokens, coef=0.5).cpu()
    want = ref.router_grad(z, ids.cpu(), scores="sigmoid", counts_in=counts.cpu(), tokens_in=int(tokens), coef=0.5)
    s, rest = torch.sigmoid(z.double()), torch.sigmoid(-z.double())
    p = s / s.sum(1, keepdim=True)
    a = 0.5 * E * counts.cpu().double() / int(counts.sum()) / T
    brackets = (a - (a * p).sum(1, keepdim=True)).abs()
    slack = p * rest * (32 * U * brackets + (16 + E / 8) * U * (a + (a * p).sum(1, keepdim=True)))
    within(got, want, slack + 2.0 ** -30 * want.abs(), (T, E))
