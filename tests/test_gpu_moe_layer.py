"""A mixture-of-experts layer out of the library's calls, forward and
backward, against the layer written out in 64 bits; the same calls captured
into graphs and replayed, and run on a stream of their own."""
import pytest
import torch

import moe_reference as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
B = 2.0 ** -8  # half a step of bfloat16, relative


def _layer_inputs(T, k, G, D, F, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, D, generator=g).to(torch.bfloat16)
    scores = torch.randn(T, G, generator=g)
    top = torch.topk(scores, k)
    ids = top.indices.clone()
    ids[torch.rand(T, k, generator=g) < 0.1] = -1  # dropped slots
    w1 = (torch.randn(G, F, D, generator=g) * D ** -0.5).to(torch.bfloat16)
    w2 = (torch.randn(G, D, F, generator=g) * F ** -0.5).to(torch.bfloat16)
    return x, ids, torch.softmax(top.values, 1), w1, w2


def _run_layer(m, x, ids, weights, w1, w2, **kw):
    sizes, slot_row = m.sort_tokens(ids, w1.shape[0], **kw)
    rows = m.dispatch(x, slot_row, **kw)
    h = m.gmm(rows, w1, sizes, out_dtype=torch.bfloat16, **kw)
    y = m.gmm(h, w2, sizes, out_dtype=torch.bfloat16, **kw)
    return sizes, slot_row, rows, h, y, m.combine(y, slot_row, weights, **kw)


def _run_backward(m, dout, weights, w1, w2, state, **kw):
    sizes, slot_row, rows, h, y, _ = state
    dy, dweights = m.combine_grad(dout, y, slot_row, weights, **kw)
    dh = m.gmm(dy, w2, sizes, out_dtype=torch.bfloat16, transpose_rhs=True, **kw)
    dw2 = m.tgmm(dy, h, sizes, **kw)
    drows = m.gmm(dh, w1, sizes, out_dtype=torch.bfloat16, transpose_rhs=True, **kw)
    dw1 = m.tgmm(dh, rows, sizes, **kw)
    return m.combine(drows, slot_row, **kw), dweights, dw1, dw2


@pytest.mark.parametrize("T,k,G", [(1, 2, 5), (70, 4, 9), (600, 8, 16)])
def test_layer_forward_and_backward(T, k, G):
    """Every step rounds to bf16 once, so a result after n roundings is off
    by about n halves of a step of the sizes that go into it: relative
    Frobenius bounds of n * 2^-8 with n the roundings on the way (out: rows are
    exact; h, y, out: 3.  dx: dy, dh, drows, dx over y-independent paths: 4.
    dweights: h, y: 2.  dw1: dy, dh: 2; dw2: dy and h: 2)."""
    import moe_grouped_matrix_amd as m
    D, F = 192, 128
    x, ids, weights, w1, w2 = _layer_inputs(T, k, G, D, F, T)
    dout = torch.randn(T, D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    dev = [t.cuda() for t in (x, ids, weights, w1, w2)]
    state = _run_layer(m, *dev)
    grads = _run_backward(m, dout.cuda(), dev[2], dev[3], dev[4], state)

    xd, wd = x.double().requires_grad_(), weights.double().requires_grad_()
    w1d, w2d = w1.double().requires_grad_(), w2.double().requires_grad_()
    out = torch.zeros(T, D, dtype=torch.float64)
    for e in range(G):
        t, j = (ids == e).nonzero(as_tuple=True)
        out = out.index_add(0, t, wd[t, j, None] * (xd[t] @ w1d[e].t() @ w2d[e].t()))
    out.backward(dout.double())
    for name, got, want, n in (("out", state[-1], out.detach(), 3), ("dx", grads[0], xd.grad, 4),
                               ("dweights", grads[1], wd.grad, 2), ("dw1", grads[2], w1d.grad, 2),
                               ("dw2", grads[3], w2d.grad, 2)):
        err = float((got.cpu().double() - want).norm())
        assert err <= n * B * float(want.norm()) + 1e-12, (name, err, float(want.norm()))


def test_microscaled_layer():
    """Weights in microscaled fp4 with bf16 activations, and with activations
    quantised too (the f8f6f4 product): both against 64 bits on the values that
    the quantised tensors stand for."""
    import moe_grouped_matrix_amd as m
    T, k, G, D, F = 90, 4, 7, 256, 384
    x, ids, weights, w1, _ = _layer_inputs(T, k, G, D, F, 3)
    sizes, slot_row = m.sort_tokens(ids.cuda(), G)
    rows = m.dispatch(x.cuda(), slot_row)
    q, s = m.quant_mxfp4(w1.cuda(), operand="rhs")
    wide = m.widen_mxfp4(q, s, operand="rhs").cpu().double()
    aq, asc = m.quant_mxfp4(rows)
    awide = m.widen_mxfp4(aq, asc).cpu().double()
    y16 = m.gmm(rows, q, sizes, rhs_scale=s, rhs_format="fp4_e2m1")
    y4 = m.gmm(aq, q, sizes, lhs_format="fp4_e2m1", rhs_format="fp4_e2m1", lhs_scale=asc, rhs_scale=s)
    lo = 0
    for h, n in enumerate(sizes.tolist()):
        for got, a in ((y16, rows.cpu().double()), (y4, awide)):
            want, terms = a[lo:lo + n] @ wide[h].t(), a[lo:lo + n].abs() @ wide[h].t().abs()
            ref.within(got.cpu()[lo:lo + n], want, D * U * terms + U * want.abs(), "expert rows")
        lo += n
    out = m.combine(y16, slot_row, weights.cuda(), out_dtype=torch.bfloat16).cpu()
    want, terms = ref.combine(y16.cpu(), slot_row.cpu(), weights)
    ref.within(out, want, k * U * terms + ref.half_step(torch.bfloat16, want.abs() + k * U * terms), "out")
    # the backward pass through frozen fp4 weights reads them widened, in place as [G,K,N]
    dy = torch.randn(T * k, F, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
    dx = m.gmm(dy, m.widen_mxfp4(q, s, operand="rhs"), sizes, transpose_rhs=True).cpu()
    lo = 0
    for h, n in enumerate(sizes.tolist()):
        a = dy.cpu().double()[lo:lo + n]
        ref.within(dx[lo:lo + n], a @ wide[h], F * U * (a.abs() @ wide[h].abs()) * 2, "dx")
        lo += n


def _graph(fn):
    warm = torch.cuda.Stream()
    with torch.cuda.stream(warm):
        fn()
    torch.cuda.current_stream().wait_stream(warm)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = fn()
    return g, out


def test_captured_layers_replay():
    """Two graphs of the whole path over different routings, replayed in turn
    with new inputs and eager calls between: every replay equals the eager
    result bit for bit (the sorts of 5000 and 7001 tokens use a workspace,
    each graph its own)."""
    import moe_grouped_matrix_amd as m
    G, D, F = 12, 128, 64
    made = []
    for T, k, seed in ((5000, 2, 1), (7001, 3, 2)):
        x, ids, weights, w1, _ = _layer_inputs(T, k, G, D, F, seed)
        x, ids, weights = x.cuda(), ids.cuda(), weights.cuda()
        q, s = m.quant_mxfp4(w1.cuda(), operand="rhs")

        def fn(x=x, ids=ids, weights=weights, q=q, s=s):
            sizes, slot_row = m.sort_tokens(ids, G)
            rows = m.dispatch(x, slot_row)
            y = m.gmm(rows, q, sizes, rhs_scale=s, rhs_format="fp4_e2m1", out_dtype=torch.bfloat16)
            out = m.combine(y, slot_row, weights)
            drows, dw = m.combine_grad(out, y, slot_row, weights)
            back = m.widen_mxfp4(*m.quant_mxfp4(drows))
            return sizes, slot_row, rows, y, out, drows, dw, back
        made.append((fn, x, ids) + _graph(fn))
    g = torch.Generator().manual_seed(8)
    for turn in range(4):
        for fn, x, ids, graph, outs in made:
            x.copy_(torch.randn(x.shape, generator=g))
            ids.copy_(torch.randint(-1, G + 1, ids.shape, generator=g))
        for fn, x, ids, graph, outs in made:
            graph.replay()
        want = [[t.clone() for t in fn()] for fn, *_ in made]
        torch.cuda.synchronize()
        for (fn, x, ids, graph, outs), ws in zip(made, want):
            for i, (a, b) in enumerate(zip(outs, ws)):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), (turn, i)


def test_calls_on_a_stream_of_their_own():
    """Two streams run the path at once, the caller's stream waiting for both
    at the end."""
    import moe_grouped_matrix_amd as m
    G, D, F = 8, 256, 128
    ins = [[t.cuda() for t in _layer_inputs(6000, 2, G, D, F, 20 + i)] for i in range(2)]
    want = [[t.clone() for t in _run_layer(m, *a)] for a in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for turn in range(3):
        got = []
        for a, st in zip(ins, streams):
            st.wait_stream(torch.cuda.current_stream())
        for a, st in zip(ins, streams):
            sizes, slot_row = m.sort_tokens(a[1], G, stream=st)
            rows = m.dispatch(a[0], slot_row, stream=st)
            out = m.combine(rows, slot_row, a[2], stream=st)
            drows, dw = m.combine_grad(out, rows, slot_row, a[2], stream=st)
            q, s = m.quant_mxfp4(rows, stream=st)
            got.append((sizes, slot_row, rows, out, drows, dw, m.widen_mxfp4(q, s, stream=st)))
        for st in streams:
            torch.cuda.current_stream().wait_stream(st)
        for a, w, g in zip(ins, want, got):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1]) and torch.equal(g[2], w[2])
            assert torch.equal(g[3], m.combine(w[2], w[1], a[2]))
            dr, dw = m.combine_grad(g[3], w[2], w[1], a[2])
            assert torch.equal(g[4], dr) and torch.equal(g[5], dw)
            assert torch.equal(g[6], m.widen_mxfp4(*m.quant_mxfp4(w[2])))
