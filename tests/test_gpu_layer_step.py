"""A mixture-of-experts layer with its router and its optimizer out of the
library's calls: a training step against the layer written out in 64 bits with
automatic differentiation, the same step captured and replayed, and a decode
step by expert id against the grouped products."""
import pytest
import torch

import layer_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
B = 2.0 ** -8  # half a step of bfloat16, relative
COEF = dict(coef=0.05, z_coef=0.01)


def _inputs(T, G, D, F, seed, pad=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, D, generator=g).to(BF16)
    z = torch.randn(T, G, generator=g)
    valid = torch.rand(T, generator=g) >= (0.15 if pad else 0.0)
    w1 = torch.randn(G, F, D, generator=g) * D ** -0.5
    w2 = torch.randn(G, D, F, generator=g) * F ** -0.5
    return x, z, valid, w1, w2, torch.randn(T, D, generator=g).to(BF16)


def _forward_backward(m, x, z, valid, w1, w2, dout, k, **kw):
    """Products' weights bf16 [G,N,K]; returns what the layer and its router give."""
    G = w1.shape[0]
    ids, weights = m.route(z, k, valid=valid, **kw)
    loss, counts, tokens = m.balance_loss(z, ids, valid=valid, **COEF, **kw)
    sizes, slot_row = m.sort_tokens(ids, G, **kw)
    rows = m.dispatch(x, slot_row, **kw)
    h = m.gmm(rows, w1, sizes, out_dtype=BF16, **kw)
    y = m.gmm(h, w2, sizes, out_dtype=BF16, **kw)
    out = m.combine(y, slot_row, weights, **kw)
    dy, dweights = m.combine_grad(dout, y, slot_row, weights, **kw)
    dz = m.router_grad(z, ids, dweights=dweights, counts=counts, tokens=tokens, valid=valid, **COEF, **kw)
    dh = m.gmm(dy, w2, sizes, out_dtype=BF16, transpose_rhs=True, **kw)
    # (the weights are [G,N,K], so their gradients are tgmm of the output side with the input side)
    dw2 = m.tgmm(dy, h, sizes, out_dtype=BF16, **kw)
    dw1 = m.tgmm(dh, rows, sizes, out_dtype=BF16, **kw)
    return dict(ids=ids, counts=counts, tokens=tokens, sizes=sizes, loss=loss, out=out, dz=dz, dw1=dw1, dw2=dw2)


@pytest.mark.parametrize("T,k,G", [(1, 2, 4), (77, 4, 9), (500, 8, 16)])
def test_training_step(T, k, G):
    """Every bf16 result is off by half a step a rounding on the way, as in the
    layer's own test: out 3, dweights (hence the router's gradient) 2, dw1 and
    dw2 2 and one for their own."""
    import moe_grouped_matrix_amd as m
    D, F = 192, 128
    x, z, valid, w1, w2, dout = _inputs(T, G, D, F, T, T > 1)
    b1, b2 = w1.to(BF16), w2.to(BF16)
    got = _forward_backward(m, *(t.cuda() for t in (x, z, valid, b1, b2, dout)), k)
    ids = got["ids"].cpu()
    assert torch.equal(ids, ref.route(z, k, valid=valid)[0])
    assert torch.equal(got["counts"], got["sizes"]) and int(got["tokens"]) == int(valid.sum())

    zd, w1d, w2d = z.double().requires_grad_(), b1.double().requires_grad_(), b2.double().requires_grad_()
    weights = ref.weights_of(zd, ids, valid=valid)
    out = torch.zeros(T, D, dtype=torch.float64)
    for e in range(G):
        t, j = (ids == e).nonzero(as_tuple=True)
        out = out.index_add(0, t, weights[t, j, None] * (x.double()[t] @ w1d[e].t() @ w2d[e].t()))
    loss = ref.balance_loss(zd, ids, valid=valid, **COEF)[0]
    ((out * dout.double()).sum() + loss).backward()
    assert abs(float(got["loss"]) - float(loss.detach())) <= 1e-5 * abs(float(loss.detach()))
    for name, want, n in (("out", out.detach(), 3), ("dz", zd.grad, 2), ("dw1", w1d.grad, 3), ("dw2", w2d.grad, 3)):
        err = float((got[name].cpu().double() - want).norm())
        assert err <= n * B * float(want.norm()) + 1e-12, (name, err, float(want.norm()))


class Trainer:
    """f32 weights with bf16 copies, eight-bit states, a step counted on the device."""

    def __init__(self, x, z, valid, w1, w2, dout, k):
        self.data, self.k = [t.cuda() for t in (x, z, valid, dout)], k
        self.w = [w1.cuda(), w2.cuda()]
        self.copies = [w.to(BF16) for w in self.w]
        self.m, self.v = ([torch.zeros(w.shape, device="cuda").to(torch.float8_e4m3fn) for w in self.w] for _ in range(2))
        self.ms, self.vs = ([torch.ones(-(-w.numel() // 256), device="cuda") for w in self.w] for _ in range(2))
        self.at = torch.ones(1, dtype=torch.int32, device="cuda")

    def step(self, m, **kw):
        x, z, valid, dout = self.data
        got = _forward_backward(m, x, z, valid, *self.copies, dout, self.k, **kw)
        m.adamw(self.w, [got["dw1"], got["dw2"]], self.m, self.v, self.at, lr=1e-3, weight_decay=0.1, exp_avg_scale=self.ms,
                exp_avg_sq_scale=self.vs, copies=self.copies, **kw)
        return got

    def state(self):
        return [t.clone() for t in self.w + self.copies + [t.view(torch.uint8) for t in self.m + self.v] + self.ms + self.vs]


def test_captured_training_step():
    """A captured step, replayed on new batches, trains as the eager calls do,
    bit for bit."""
    import moe_grouped_matrix_amd as m
    T, k, G, D, F = 200, 4, 8, 192, 128
    eager, caught = (Trainer(*_inputs(T, G, D, F, 1), k) for _ in range(2))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        Trainer(*_inputs(T, G, D, F, 2), k).step(m)  # (a stream's first weight gradient allocates its counters)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        made = caught.step(m)
        caught.at += 1
    for i in range(4):
        x, z, _, _, _, dout = _inputs(T, G, D, F, 10 + i)
        for t in (eager, caught):
            for old, new in zip(t.data, (x, z, None, dout)):
                if new is not None:
                    old.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        want = eager.step(m)
        eager.at += 1
        for name in want:
            assert torch.equal(made[name], want[name]), (i, name)
        for a, b in zip(eager.state(), caught.state()):
            assert torch.equal(a, b), i


def test_step_on_a_stream_of_its_own():
    import moe_grouped_matrix_amd as m
    T, k, G, D, F = 200, 4, 8, 192, 128
    a, b = (Trainer(*_inputs(T, G, D, F, 3), k) for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        a.step(m)
        b.step(m, stream=side)
        a.at += 1
        with torch.cuda.stream(side):
            b.at += 1
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip(a.state(), b.state()):
        assert torch.equal(x, y)


@pytest.mark.parametrize("T", [1, 6])
def test_decode_step(T):
    """A decode step by expert id (route, gmv, gmv with weights) against the
    layer in 64 bits on the same four-bit weights: h and out are rounded to
    bf16 once each."""
    import moe_grouped_matrix_amd as m
    k, G, D, F = 4, 12, 256, 192
    g = torch.Generator().manual_seed(T)
    x, z = torch.randn(T, D, generator=g).to(BF16), torch.randn(T, G, generator=g)
    q1, q2 = torch.randint(0, 256, (G, F, D // 2), generator=g, dtype=torch.uint8), torch.randint(0, 256, (G, D, F // 2), generator=g, dtype=torch.uint8)
    s1, s2 = torch.rand(G, D // 64, 1, F, generator=g) * 0.02, torch.rand(G, F // 32, 1, D, generator=g) * 0.02
    z2 = torch.randint(0, 16, s2.shape, generator=g).float()

    def step(x, z, q1, s1, q2, s2, z2):
        ids, w = m.route(z, k)
        h = m.gmv(x, q1, ids, rhs_format="int4", rhs_scale=s1, out_dtype=BF16)
        return ids, w, h, m.gmv(h, q2, ids, rhs_format="uint4", rhs_scale=s2, rhs_zero=z2, weights=w, out_dtype=BF16)
    dev = [t.cuda() for t in (x, z, q1, s1, q2, s2, z2)]
    ids, w, h, out = step(*dev)
    want_ids, ww, _ = ref.route(z, k)
    assert torch.equal(ids.cpu(), want_ids)
    hd = ref.gmv(x, q1, want_ids, "int4", s1)[0]
    od = ref.gmv(hd, q2, want_ids, "uint4", s2, z2, ww)[0]
    assert float((h.cpu().double() - hd).norm()) <= B * float(hd.norm())
    assert float((out.cpu().double() - od).norm()) <= 2 * B * float(od.norm())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        made = step(*dev)
    for i in range(3):
        dev[0].copy_(torch.randn(T, D, generator=torch.Generator().manual_seed(i)))
        dev[1].copy_(torch.randn(T, G, generator=torch.Generator().manual_seed(i + 9)))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(made, step(*dev)):
            assert torch.equal(a, b)
