"""GPU parity of the router (include/gmm_layer.h: route, balance_loss,
router_grad) against its plain 64-bit forms.

Tolerances (u = 2^-24, the half step of binary32).  A score is an exponential
of a difference of logits: the difference is rounded once (an error of u |z -
top|, which the exponential turns into a relative one), the exponential is
within a few u, and so are the sum over the experts (at most 1024 positive
terms, added in a tree of 16 + 6 levels), the quotient and the scale: a weight
or probability is within (32 + 2 range) u of itself, with `range` the largest
distance of a finite logit from its token's largest (or from 0, which a sigmoid
or a logsumexp starts from).  The loss adds at most T/4 positive terms a chain:
T/4 u more.  A gradient is a sum of products of such factors, whose absolute
values add up to at most `mag` below."""
import math

import pytest
import torch

import layer_reference as ref
from moe_reference import half_step, within

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def _logits(T, E, seed, dtype=F32, off=0.0, pad=0.0, spread=2.0, ties=False):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(T, E, generator=g) * spread
    if ties:
        z = (z * 2).round() / 2
    if off:
        z[torch.rand(T, E, generator=g) < off] = -math.inf
        z[torch.rand(T, generator=g) < 0.1] = -math.inf  # nothing left
    valid = None
    if pad:
        valid = torch.rand(T, generator=g) >= pad
        z[~valid] = math.nan
    return z.to(dtype), valid


def _range(z):
    f = z.double()
    f = torch.where(torch.isfinite(f), f, torch.zeros_like(f))
    return float((f.amax() - f.amin()).abs() + f.abs().amax()) if f.numel() else 0.0


def _dev(*ts):
    return [t.cuda() if t is not None else None for t in ts]


SIZES = [(0, 4, 2), (1, 1, 1), (1, 128, 8), (5, 2, 2), (7, 16, 16), (33, 17, 3), (64, 64, 1), (70, 65, 5), (9, 127, 16),
         (11, 128, 17), (13, 129, 9), (6, 100, 64), (17, 256, 8), (10, 257, 4), (8, 512, 8), (5, 1000, 6), (3, 1024, 64),
         (1025, 37, 3), (260, 128, 8)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scores,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_route(T, E, k, scores, renorm, dtype):
    import moe_grouped_matrix_amd as m
    for n, (off, pad, ties) in enumerate([(0.0, 0.0, False), (0.3, 0.2, True)]):
        z, valid = _logits(T, E, 10 * T + n, dtype, off, pad, ties=ties)
        ids, w = m.route(z.cuda(), k, scores=scores, renormalize=renorm, scale=1.5, valid=None if valid is None else valid.cuda())
        want, ww, _ = ref.route(z, k, scores, None, renorm, 1.5, valid)
        assert ids.dtype == torch.int32 and w.dtype == F32
        assert torch.equal(ids.cpu(), want)
        within(w.cpu(), ww, ww.abs() * (32 + 2 * _range(z)) * U + 1e-37, "weights")


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (50, 16, 4), (33, 128, 8), (9, 300, 20), (5, 1024, 64)])
def test_route_with_a_bias(T, E, k, scores):
    """The keys s + bias are within (32 + 2 range) u of s and u of the sum: two
    experts may change places where their keys are nearer than that."""
    import moe_grouped_matrix_amd as m
    z, valid = _logits(T, E, T + E, off=0.1, pad=0.1)
    bias = torch.randn(E, generator=torch.Generator().manual_seed(E)) * 0.1
    ids, w = m.route(z.cuda(), k, scores=scores, bias=bias.cuda(), valid=valid.cuda())
    want, ww, keys = ref.route(z, k, scores, bias, True, 1.0, valid)
    ids, w = ids.cpu(), w.cpu()
    assert torch.equal(ids < 0, want < 0)
    there = ids >= 0
    slack = (40 + 2 * _range(z)) * U * 2
    got_key = torch.gather(keys, 1, ids.clamp_min(0).long())
    want_key = torch.gather(keys, 1, want.clamp_min(0).long())
    assert bool(((got_key - want_key)[there].abs() <= slack).all())
    assert all(len(set(r[r >= 0].tolist())) == int((r >= 0).sum()) for r in ids)
    ww = ref.weights_of(z, torch.where(there, ids, torch.full_like(ids, -1)), scores, True, 1.0, valid)
    within(w, ww, ww.abs() * (32 + 2 * _range(z)) * U + 1e-37, "weights")


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(8, 4), (128, 8), (300, 12)])
def test_biases_that_are_not_finite(E, k, scores):
    """-inf keeps an expert from being chosen, however few are left; NaN and
    +inf spoil the tokens in which the expert is not switched off."""
    import moe_grouped_matrix_amd as m
    z = _logits(40, E, E)[0]
    z[5, 3] = -math.inf
    bias = torch.full((E,), -math.inf)
    bias[[1, 3, 6]] = 0.25
    ids, w = (t.cpu() for t in m.route(z.cuda(), k, scores=scores, bias=bias.cuda()))
    want = [[int(e) for e in sorted((1, 3, 6), key=lambda e: -float(z[t, e])) if z[t, e] > -math.inf] for t in range(40)]
    assert [r[r >= 0].tolist() for r in ids] == want and bool((ids[:, 3:] == -1).all()) and ids[5, 2] == -1
    assert bool((w[ids < 0] == 0).all()) and bool((w[ids >= 0] > 0).all())
    for far in (math.nan, math.inf):
        bias[3] = far
        ids, w = (t.cpu() for t in m.route(z.cuda(), k, scores=scores, bias=bias.cuda()))
        bad = torch.arange(40) != 5
        assert bool((ids[bad] == -1).all()) and bool(w[bad].isnan().all())
        assert set(ids[5].tolist()) == {1, 6, -1} and bool(w[5].isfinite().all())


def test_route_extremes():
    """Zeros of both signs tie; far logits lose to no rounding; sigmoid scores
    that underflow give weights 0; a NaN or +inf spoils its token only."""
    import moe_grouped_matrix_amd as m
    z = torch.zeros(6, 8)
    z[0, ::2] = -0.0
    z[1] = torch.tensor([-3e38, 3e38, 1e-45, -1e-45, 0.0, 1.0, 1.0, -1.0])
    z[2] = -200.0 - torch.arange(8)
    z[3, 5] = math.nan
    z[4, 2] = math.inf
    z[5] = torch.arange(8) * 30.0
    for scores in ("softmax", "sigmoid"):
        ids, w = (t.cpu() for t in m.route(z.cuda(), 4, scores=scores))
        want, ww, _ = ref.route(z, 4, scores)
        assert torch.equal(ids, want)
        assert ids[0].tolist() == [0, 1, 2, 3] and ids[1].tolist() == [1, 5, 6, 2]
        assert bool(w[3:5].isnan().all()) and bool((ids[3:5] == -1).all())
        if scores == "sigmoid":
            assert bool((w[2] == 0).all())  # exp(-200) is no binary32
        rows = [0, 1, 5] + ([2] if scores == "softmax" else [])
        within(w[rows], ww[rows], ww[rows].abs() * (32 + 2 * 300) * U + 1e-37, scores)
    ids, w = m.route(z[1:2].cuda(), 4, renormalize=False)
    assert w.cpu()[0].tolist() == [1.0, 0.0, 0.0, 0.0]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", SIZES + [(4099, 24, 2)])
def test_balance_loss(T, E, k, scores, dtype):
    import moe_grouped_matrix_amd as m
    for n, (off, pad) in enumerate([(0.0, 0.0), (0.3, 0.2)]):
        z, valid = _logits(T, E, 7 * T + n, dtype, off, pad)
        g = torch.Generator().manual_seed(T)
        ids = torch.randint(-1, E + 1, (T, k), generator=g).to(torch.int64 if n else torch.int32)  # (wild and repeated ones too)
        loss, counts, tokens = m.balance_loss(*_dev(z, ids), scores=scores, coef=0.7, z_coef=0.01, valid=_dev(valid)[0])
        want, wc, wn = ref.balance_loss(z, ids, scores, 0.7, 0.01, valid)
        assert torch.equal(counts.cpu(), wc) and tokens.cpu().tolist() == [wn]
        assert loss.shape == (1,) and loss.dtype == F32
        slack = abs(float(want)) * (64 + 4 * _range(z) + T / 4) * U + 1e-37
        assert abs(float(loss) - float(want)) <= slack, (float(loss), float(want))


def test_balance_loss_of_nothing_and_of_bad_logits():
    import moe_grouped_matrix_amd as m
    z = torch.full((5, 8), -math.inf)
    loss, counts, tokens = m.balance_loss(z.cuda(), torch.full((5, 2), -1, dtype=torch.int32).cuda(), z_coef=1.0)
    assert float(loss) == 0 and not bool(counts.any()) and int(tokens) == 0
    z = torch.zeros(5, 8)
    z[2, 3] = math.nan
    loss, counts, tokens = m.balance_loss(z.cuda(), torch.zeros(5, 2, dtype=torch.int32).cuda())
    assert math.isnan(float(loss)) and int(tokens) == 5 and counts.cpu().tolist() == [10] + [0] * 7


def _grad_case(T, E, k, seed, dtype, off, pad):
    z, valid = _logits(T, E, seed, dtype, off, pad)
    g = torch.Generator().manual_seed(seed + 1)
    ids = ref.route(z, k, valid=valid)[0]
    if T > 2:
        ids[T // 2] = torch.randint(0, E, (k,), generator=g).to(torch.int32)  # repeated experts
        ids[T // 3, 0] = E + 3
    dw = torch.randn(T, k, generator=g)
    counts = torch.randint(0, 50, (E,), generator=g).to(torch.int32)
    return z, valid, ids, dw, counts


@pytest.mark.parametrize("scores,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("T,E,k", [s for s in SIZES if s[0] <= 300])
def test_router_grad(T, E, k, scores, renorm):
    import moe_grouped_matrix_amd as m
    for n, (dtype, off, pad) in enumerate([(F32, 0.0, 0.0), (BF16, 0.3, 0.2), (F32, 0.3, 0.2)]):
        z, valid, ids, dw, counts = _grad_case(T, E, k, 3 * T + n, dtype, off, pad)
        if n == 1:
            dw = dw.to(BF16)
            ids = ids.long()
        dw = torch.where((ids >= 0) & (ids < E), dw, torch.full_like(dw, math.nan))  # not read
        tokens = torch.tensor([max(T, 1)], dtype=torch.int32)
        parts = [dict(dweights=dw), dict(counts=counts, tokens=tokens, dloss=torch.tensor([3.0])),
                 dict(dweights=dw, counts=counts, tokens=tokens)]
        for part in parts:
            coef = dict(coef=0.5, z_coef=0.02) if "counts" in part else {}
            got = m.router_grad(*_dev(z, ids), scores=scores, renormalize=renorm, scale=2.0, valid=_dev(valid)[0],
                                **{k_: v.cuda() for k_, v in part.items()}, **coef)
            assert got.dtype == dtype and got.shape == z.shape
            kw = dict(scores=scores, renormalize=renorm, scale=2.0, valid=valid, **coef)
            if "dweights" in part:
                kw["dweights"] = torch.nan_to_num(part["dweights"].float())
            if "counts" in part:
                kw.update(counts_in=counts, tokens_in=tokens, dloss=float(part.get("dloss", torch.ones(1))))
            want = ref.router_grad(z, ids, **kw)
            # the absolute terms: |g| once for its own score and once in the mean, a and its mean, the logit term
            mag = torch.zeros(T, 1, dtype=torch.float64)
            if "dweights" in part:
                mag = mag + 2 * 2.0 * kw["dweights"].double().abs().sum(1, keepdim=True)
            if "counts" in part:
                f = counts.double() / max(1, int(counts.sum()))
                mag = mag + kw["dloss"] * (2 * 0.5 * E * f.max() + 2 * 0.02 * (_range(z) + 8)) / max(T, 1)
            slack = mag * (64 + 4 * _range(z)) * U
            if dtype == BF16:
                slack = slack + half_step(BF16, want)
            within(got.cpu(), want, slack.expand_as(want) + 1e-37, (scores, renorm, sorted(part)))


@pytest.mark.parametrize("scores,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_router_grad_against_differences(scores, renorm):
    """Central differences of the objective in 64 bits with a step of 1e-4: off
    by some 1e-8 of third derivatives, far below binary32's own error here."""
    import moe_grouped_matrix_amd as m
    T, E, k = 3, 7, 3
    z, _, ids, dw, counts = _grad_case(T, E, k, 5, F32, 0.0, 0.0)
    ids[1] = torch.tensor([4, 4, 0])
    tokens = torch.tensor([T], dtype=torch.int32)
    kw = dict(scores=scores, renormalize=renorm, scale=1.3, coef=0.4, z_coef=0.05)
    there = (ids >= 0) & (ids < E)
    got = m.router_grad(*_dev(z, ids), dweights=dw.cuda(), counts=counts.cuda(), tokens=tokens.cuda(), **kw).cpu().double()
    h = 1e-4
    for t in range(T):
        for e in range(E):
            up, down = z.double().clone(), z.double().clone()
            up[t, e] += h
            down[t, e] -= h
            f = [float(ref.objective(y, ids, torch.where(there, dw, torch.zeros_like(dw)), counts, tokens, 1.0, **kw)) for y in (up, down)]
            assert abs((f[0] - f[1]) / (2 * h) - float(got[t, e])) <= 1e-6 + 1e-7 * dw.abs().sum()


def test_router_grad_of_bad_logits():
    import moe_grouped_matrix_amd as m
    z = torch.zeros(4, 8)
    z[1, 3], z[2, 0] = math.nan, math.inf
    z[3] = -math.inf
    ids, _ = m.route(z.cuda(), 2)
    got = m.router_grad(z.cuda(), ids, dweights=torch.ones(4, 2).cuda()).cpu()
    assert bool(got[1:3].isnan().all()) and not bool(got[3].any()) and bool(torch.isfinite(got[0]).all())


@pytest.mark.parametrize("T", [1, 300, 5000])
def test_captured_and_replayed(T):
    """The router's step in a graph, replayed on new logits with eager work in
    between, gives what the eager calls give, bit for bit."""
    import moe_grouped_matrix_amd as m
    E, k = 64, 4
    z = torch.randn(T, E, device="cuda")

    def step():
        ids, w = m.route(z, k)
        loss, counts, tokens = m.balance_loss(z, ids, coef=0.1, z_coef=0.01)
        return ids, w, loss, counts, tokens, m.router_grad(z, ids, dweights=w, counts=counts, tokens=tokens, coef=0.1, z_coef=0.01)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        made = step()
    for i in range(4):
        z.copy_(torch.randn(T, E, generator=torch.Generator().manual_seed(i)))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(made, step()):
            assert torch.equal(a, b)


def test_offsets_past_31_bits():
    """2^31 - 1024 bf16 logits (4 GiB): the last token's choice, its share of the
    loss and its gradient, all others being switched off."""
    import moe_grouped_matrix_amd as m
    E, k = 1024, 2
    T = 2 ** 21 - 1
    z = torch.full((T, E), -math.inf, dtype=BF16, device="cuda")
    last = torch.randn(E, generator=torch.Generator().manual_seed(1)).to(BF16)
    z[T - 1] = last.cuda()
    ids, w = m.route(z, k)
    want, ww, _ = ref.route(last[None], k)
    assert torch.equal(ids[T - 1:].cpu(), want) and not bool((ids[:T - 1] != -1).any()) and not bool(w[:T - 1].any())
    within(w[T - 1:].cpu(), ww, ww * (32 + 2 * _range(last)) * U, "weights")
    loss, counts, tokens = m.balance_loss(z, ids, coef=0.5, z_coef=0.1)
    lw, cw, _ = ref.balance_loss(last[None], want, coef=0.5, z_coef=0.1)
    assert int(tokens) == 1 and torch.equal(counts.cpu(), cw)
    assert abs(float(loss) - float(lw)) <= float(lw) * (64 + 4 * _range(last)) * U
    dw = torch.zeros(T, k, device="cuda")
    dw[T - 1, 0] = 1
    got = m.router_grad(z, ids, dweights=dw)
    gw = ref.router_grad(last[None], want, dweights=torch.tensor([[1.0, 0.0]]))
    within(got[T - 1:].cpu(), gw, 2 * (64 + 4 * _range(last)) * U + half_step(BF16, gw), "gradient")
    assert not bool(got[:T - 1].any())


@pytest.mark.parametrize("E", [16, 37, 128, 200, 256, 512, 1024])
def test_lowest_and_far_values(E):
    """Masks of the type's lowest finite value are values like any other: chosen
    after all others, with weight 0; sigmoid scores of both far sides."""
    import moe_grouped_matrix_amd as m
    for dtype in (F32, BF16):
        low = torch.finfo(dtype).min
        z = torch.full((3, E), low, dtype=dtype)
        z[0, 5], z[0, 3] = 1.0, 2.0
        z[1] = torch.linspace(-60, 60, E).to(dtype)
        z[2, ::2] = -math.inf
        for scores in ("softmax", "sigmoid"):
            ids, w = (t.cpu() for t in m.route(z.cuda(), 8, scores=scores, renormalize=False))
            want, ww, _ = ref.route(z, 8, scores, renormalize=False)
            assert torch.equal(ids, want)
            within(w, ww, ww * (32 + 2 * 130) * U + 2.0 ** -126, scores)
            loss, _, tokens = m.balance_loss(z.cuda(), ids.cuda(), scores=scores)
            assert int(tokens) == 3 and math.isfinite(float(loss))
            g = m.router_grad(z.cuda(), ids.cuda(), dweights=torch.ones(3, 8).cuda(), scores=scores, renormalize=False).cpu()
            gw = ref.router_grad(z, ids, dweights=torch.ones(3, 8), scores=scores, renormalize=False)
            within(g, gw, (64 + 4 * 130) * U * 9 + half_step(dtype, gw), scores)


def test_two_streams_at_once():
    import moe_grouped_matrix_amd as m
    zs = [torch.randn(3000, 100, generator=torch.Generator().manual_seed(i)).cuda() for i in range(2)]
    ids = [m.route(z, 4)[0] for z in zs]
    want = [m.balance_loss(z, i, z_coef=1.0) for z, i in zip(zs, ids)]
    streams = [torch.cuda.Stream() for _ in zs]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    got = [[m.balance_loss(z, i, z_coef=1.0, stream=st) for z, i, st in zip(zs, ids, streams)] for _ in range(5)]
    torch.cuda.synchronize()
    for pair in got:
        for a, b in zip(pair, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
