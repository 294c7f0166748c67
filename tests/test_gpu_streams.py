"""A layer whose every call, the grouped products included, runs on a stream of
its own, two at once: results equal those of the current stream bit for bit,
with the intermediate tensors dropped as soon as the next call is queued."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _inputs(T, k, G, D, F, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, D, generator=g).to(torch.bfloat16)
    ids = torch.randint(-1, G, (T, k), generator=g)
    w1 = (torch.randn(G, F, D, generator=g) * D ** -0.5).to(torch.bfloat16)
    w2 = (torch.randn(G, D, F, generator=g) * F ** -0.5)
    return [t.cuda() for t in (x, ids, torch.rand(T, k, generator=g), w1, w2)]


def _layer(m, x, ids, weights, w1, w2, **kw):
    G = w1.shape[0]
    sizes, slot_row = m.sort_tokens(ids, G, **kw)
    h = m.gmm(m.dispatch(x, slot_row, **kw), w1, sizes, out_dtype=torch.bfloat16, **kw)
    q, scale = m.quant_mxfp4(w2, operand="rhs", **kw)
    y = m.gmm(h, q, sizes, rhs_scale=scale, rhs_format="fp4_e2m1", out_dtype=torch.bfloat16, **kw)
    out = m.combine(y, slot_row, weights, **kw)
    dy, dweights = m.combine_grad(out, y, slot_row, weights, **kw)
    dh = m.gmm(dy, m.widen_mxfp4(q, scale, operand="rhs", **kw), sizes, transpose_rhs=True, out_dtype=torch.bfloat16, **kw)
    hq, hs = m.quant_fp8(h, **kw)
    return out, dweights, m.gmm(dh, w1, sizes, transpose_rhs=True, **kw), hq, hs


def test_layers_on_two_streams():
    import moe_grouped_matrix_amd as m
    ins = [_inputs(5000 + 700 * i, 2, 8, 256, 384, 30 + i) for i in range(2)]
    want = [_layer(m, *a) for a in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    for turn in range(4):
        for st in streams:
            st.wait_stream(torch.cuda.current_stream())
        got = [_layer(m, *a, stream=st) for a, st in zip(ins, streams)]
        # the current stream allocates meanwhile what a freed block could give it
        junk = [torch.full((5000 * 2, 384), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(8)]
        for st in streams:
            torch.cuda.current_stream().wait_stream(st)
        for i, (ws, gs) in enumerate(zip(want, got)):
            for j, (w, g) in enumerate(zip(ws, gs)):
                assert torch.equal(w.view(torch.uint8), g.view(torch.uint8)), (turn, i, j)
        del junk
    # outputs of the caller's
    a, st = ins[0], streams[0]
    st.wait_stream(torch.cuda.current_stream())
    sizes, slot_row = m.sort_tokens(a[1], 8)
    rows = m.dispatch(a[0], slot_row)
    st.wait_stream(torch.cuda.current_stream())
    out = torch.zeros(rows.shape[0], 384, dtype=torch.bfloat16, device="cuda")
    st.wait_stream(torch.cuda.current_stream())
    assert m.gmm(rows, a[3], sizes, out=out, out_dtype=torch.bfloat16, stream=st) is out
    st.synchronize()
    assert torch.equal(out, m.gmm(rows, a[3], sizes, out_dtype=torch.bfloat16))
    assert m.device_flags() == 0
