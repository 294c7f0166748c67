"""Cases of the mixture-of-experts operators around the grouped matmul: tokens
sorted by expert, dispatched into expert rows and combined back with their
gradient, and microscaled fp4 weights (blocks of 32 with an E8M0 scale each):
quantisation, widening and the grouped product.

With ``own`` false every case runs in elementary torch operations, in 32 bits;
with ``own`` true it makes the package's calls."""
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "i32": torch.int32, "i64": torch.int64}
BYTES = {"bf16": 2, "f32": 4, "i32": 4, "i64": 8}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _lib():
    import moe_grouped_matrix_amd
    return moe_grouped_matrix_amd


# ---------------------------------------------------------------------------
# the cases

def listed():
    return [
        # one token of a chat, its top-8 of 128 experts: a launch and little else
        dict(name="sort_one_token", op="sort", T=1, k=8, G=128, ids="i64", unrouted=0.0),
        # the training batch of the package's own benchmark: 32768 tokens, top-8 of 128
        dict(name="sort_batch", op="sort", T=32768, k=8, G=128, ids="i64", unrouted=0.0),
        # a decode step of 256 sequences on its way into the experts
        dict(name="dispatch_decode", op="dispatch", T=256, k=8, G=128, D=1408, x="bf16", unrouted=0.0),
        # the training batch on its way into the experts
        dict(name="dispatch_batch", op="dispatch", T=32768, k=8, G=128, D=1408, x="bf16", unrouted=0.0),
        # a decode step's expert rows (f32, the product's default output) brought home
        dict(name="combine_decode", op="combine", T=256, k=8, G=128, D=1408, x="f32", out="bf16", weights="f32", unrouted=0.0),
        # the gradient of the training batch's dispatch: the unweighted sum of a token's rows
        dict(name="dispatch_grad_batch", op="combine", T=32768, k=8, G=128, D=1408, x="bf16", out="bf16", weights="none", unrouted=0.0),
        # the gradients of the training batch's combine
        dict(name="combine_grad_batch", op="combine_grad", T=32768, k=8, G=128, D=1408, x="bf16", weights="f32", unrouted=0.0),
        # a ragged f32 layer with dropped slots: odd token count, choices and width
        dict(name="combine_grad_odd", op="combine_grad", T=4099, k=3, G=37, D=1027, x="f32", weights="f32", unrouted=0.1),
        # the down projection of every expert quantised, in the product's weight layout
        dict(name="mxfp4_weights", op="mxfp4", side="rhs", G=128, N=1408, K=704, x="bf16"),
        # a decode step's activations quantised
        dict(name="mxfp4_tokens", op="mxfp4", side="lhs", G=1, N=2048, K=1408, x="bf16"),
        # a decode step of 256 sequences, top-8: every touched expert's weight read once
        dict(name="mxfp4_gmm_decode", op="gmm", M=2048, G=128, N=1408, K=1408, out="bf16"),
        # the training batch's up projection over frozen fp4 weights
        dict(name="mxfp4_gmm_batch", op="gmm", M=262144, G=128, N=1408, K=1408, out="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["sort", "dispatch", "combine", "combine_grad", "mxfp4", "gmm"])
    if op in ("sort", "dispatch", "combine", "combine_grad"):
        T, k, G = _log(rng, 1, 32768), rng.randint(1, 8), _log(rng, 8, 512)
        case = dict(op=op, T=T, k=k, G=G, unrouted=rng.choice([0.0, 0.0, 0.07, 0.5]))
        if op == "sort":
            return dict(case, ids=rng.choice(["i32", "i64"]))
        case["D"] = _log(rng, 16, min(5000, 262144 * 700 // (T * k)))
        if rng.random() < 0.6:
            case["D"] = -(-case["D"] // 64) * 64
        case["x"] = rng.choice(["bf16", "f32"])
        if op == "combine":
            case.update(out=rng.choice(["bf16", "f32"]), weights=rng.choice(["f32", "bf16", "none"]))
        elif op == "combine_grad":
            case["weights"] = rng.choice(["f32", "bf16"])
        return case
    if op == "mxfp4":
        G, N, K = _log(rng, 1, 48), _log(rng, 1, 1400), 32 * rng.randint(1, 40)
        return dict(op=op, side=rng.choice(["lhs", "rhs"]), G=G, N=N, K=K, x=rng.choice(["bf16", "f32"]))
    G, N, K = _log(rng, 1, 128), 8 * rng.randint(1, 176), 64 * rng.randint(1, 22)
    return dict(op=op, M=_log(rng, 1, 131072), G=G, N=N, K=K, out=rng.choice(["bf16", "f32"]))


# ---------------------------------------------------------------------------
# inputs

def _normal(g, shape, scale=1.0):
    return torch.randn(shape, generator=g, device=DEV) * scale


def _router(g, T, k, G):
    """Distinct top-k choices of a softmax router whose experts are drawn with
    Zipf popularity (weight rank^-1.1 over a seeded order of the experts)."""
    rank = torch.randperm(G, generator=g, device=DEV).float() + 1
    noise = -torch.log(-torch.log(torch.rand((T, G), generator=g, device=DEV).clamp(1e-9, 1 - 1e-7)))
    kk = min(k, G)
    top = torch.topk(noise - 1.1 * torch.log(rank), kk, dim=1)
    return top.indices, torch.softmax(top.values, dim=1)


def _routing(case, g):
    """Expert ids (unrouted slots -1) and router weights (NaN there: they count
    for nothing), and the slots' rows after a stable sort by expert."""
    T, k, G = case["T"], case["k"], case["G"]
    ids, w = _router(g, T, k, G)
    off = torch.rand((T, k), generator=g, device=DEV) < case["unrouted"]
    ids = torch.where(off, torch.full_like(ids, -1), ids)
    w = torch.where(off, torch.full_like(w, float("nan")), w)
    return ids, w


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    if op == "mxfp4":
        shape = (case["G"], case["N"], case["K"]) if case["side"] == "rhs" else (case["G"] * case["N"], case["K"])
        # weights of a trained layer: normal, every output row with a size of its own
        x = _normal(g, shape, 0.02) * torch.exp(_normal(g, shape[:-1] + (1,)))
        return dict(case=case, x=x.to(TYPES[case["x"]]))
    if op == "gmm":
        M, G, N, K = case["M"], case["G"], case["N"], case["K"]
        ids, _ = _router(g, M, 1, G)
        sizes = torch.zeros(G, dtype=torch.int64, device=DEV).index_add_(0, ids.flatten(), torch.ones_like(ids.flatten()))
        code, shared = _mx_codes(_normal(g, (G, N, K), 0.02))
        q = code[..., 0::2] | code[..., 1::2] << 4
        scale = (shared + 127).to(torch.uint8).transpose(1, 2).reshape(G, K // 32, 1, N).contiguous()
        return dict(case=case, lhs=_normal(g, (M, K)).to(torch.bfloat16), q=q.to(torch.uint8).contiguous(),
                    scale=scale.view(torch.float8_e8m0fnu), sizes=sizes.to(torch.int32))
    ids, w = _routing(case, g)
    if op == "sort":
        return dict(case=case, ids=ids.to(TYPES[case["ids"]]))
    T, k, D, x = case["T"], case["k"], case["D"], TYPES[case["x"]]
    state = dict(case=case, slot_row=_sort(ids, case["G"])[1])
    if op == "dispatch":
        return dict(state, x=_normal(g, (T, D)).to(x))
    state["rows"] = _normal(g, (T * k, D)).to(x)
    if case["weights"] != "none":
        state["weights"] = w.to(TYPES[case["weights"]])
    if op == "combine_grad":
        state["dout"] = _normal(g, (T, D), 1e-2).to(x)
    return state


# ---------------------------------------------------------------------------
# the plain forms

def _sort(ids, G):
    """group_sizes [G], slot_row [T,k]: the row of each slot when slots are
    sorted by expert, equal experts in slot order, unrouted slots last (and
    given as the complement of their row)."""
    key = torch.where((ids >= 0) & (ids < G), ids, torch.full_like(ids, G)).flatten()
    ordered, slot = torch.sort(key, stable=True)
    row = torch.empty_like(slot)
    row[slot] = torch.arange(slot.numel(), device=slot.device)
    row = torch.where(key < G, row, -1 - row).reshape(ids.shape)
    edge = torch.searchsorted(ordered, torch.arange(G + 1, device=ids.device, dtype=ordered.dtype))
    return (edge[1:] - edge[:-1]).to(torch.int32), row.to(torch.int32)


def _row_of(slot_row):
    """Every slot's row as an index, and whether the slot is routed."""
    routed = slot_row >= 0
    return torch.where(routed, slot_row, -1 - slot_row).long(), routed


def _dispatch(x, slot_row):
    row, routed = _row_of(slot_row)
    slot = torch.empty(row.numel(), dtype=torch.int64, device=x.device)
    slot[row.flatten()] = torch.arange(row.numel(), device=x.device)
    rows = x[slot // slot_row.shape[1]]
    return torch.where(routed.flatten()[slot][:, None], rows, torch.zeros_like(rows))


def _combine(rows, slot_row, weights, out):
    row, routed = _row_of(slot_row)
    w = routed.float() if weights is None else torch.where(routed, weights.float(), torch.zeros((), device=rows.device))
    return (rows[row].float() * w[..., None]).sum(1).to(out)


def _combine_grad(dout, rows, slot_row, weights):
    row, routed = _row_of(slot_row)
    d = dout.float()[:, None, :]
    w = torch.where(routed, weights.float(), torch.zeros((), device=rows.device))
    drows = torch.empty_like(rows)
    drows[row.flatten()] = (w[..., None] * d).to(rows.dtype).reshape(-1, rows.shape[1])
    dweights = (rows[row].float() * d).sum(-1)
    return drows, torch.where(routed, dweights, torch.zeros_like(dweights)).to(weights.dtype)


def _mx_codes(x):
    """e2m1 codes (0..15) and the block exponents of x [..., K] in blocks of 32."""
    b = x.float().reshape(x.shape[:-1] + (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    shared = torch.where(amax > 0, (torch.frexp(amax)[1] - 3).clamp(-127, 125), torch.zeros((), dtype=torch.int32, device=x.device))
    t = torch.ldexp(b, -shared)
    a = t.abs()
    code = (a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
    code = code + 8 * torch.signbit(t)
    return code.reshape(x.shape).to(torch.uint8), shared[..., 0]


def _mx_values(code, shared):
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=code.device)
    return torch.ldexp(table[code.int()].reshape(shared.shape + (32,)), shared[..., None]).reshape(code.shape)


def _gmm_mxfp4(lhs, q, scale, sizes, out):
    """Rows in tiles of one group each (32 or 256 rows, the last of a group
    part empty), every tile a product with its group's widened weight."""
    (M, K), (G, N) = lhs.shape, q.shape[:2]
    code = torch.stack((q & 15, q >> 4), -1).reshape(G, N, K)
    shared = scale.view(torch.uint8).int().reshape(G, K // 32, N).transpose(1, 2) - 127
    w = _mx_values(code, shared).transpose(1, 2).contiguous()
    high = 256 if M >= 64 * G else 32
    sizes = sizes.long()
    first = torch.cumsum(sizes, 0) - sizes
    tiles = torch.cumsum((sizes + high - 1) // high, 0)
    tile = torch.arange(M // high + G, device=lhs.device)
    group = torch.searchsorted(tiles, tile, right=True).clamp(max=G - 1)
    at = tile - (tiles - (sizes + high - 1) // high)[group]
    inside = at[:, None] * high + torch.arange(high, device=lhs.device)
    live = inside < sizes[group][:, None]
    row = torch.where(live, first[group][:, None] + inside, torch.full_like(inside, M))
    a = torch.cat((lhs, lhs.new_zeros(1, K)))[row].float()
    result = torch.zeros((M + 1, N), dtype=out, device=lhs.device)
    result[row.flatten()] = torch.bmm(a, w[group]).reshape(-1, N).to(out)
    return result[:M]


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        m = _lib()
        if op == "sort":
            return m.sort_tokens(state["ids"], c["G"])
        if op == "dispatch":
            return m.dispatch(state["x"], state["slot_row"])
        if op == "combine":
            return m.combine(state["rows"], state["slot_row"], state.get("weights"), out_dtype=TYPES[c["out"]])
        if op == "combine_grad":
            return m.combine_grad(state["dout"], state["rows"], state["slot_row"], state["weights"])
        if op == "mxfp4":
            q, scale = m.quant_mxfp4(state["x"], operand=c["side"])
            return m.widen_mxfp4(q, scale, operand=c["side"], out_dtype=torch.bfloat16)
        return m.gmm(state["lhs"], state["q"], state["sizes"], rhs_scale=state["scale"], rhs_format="fp4_e2m1",
                     out_dtype=TYPES[c["out"]])
    if op == "sort":
        return _sort(state["ids"], c["G"])
    if op == "dispatch":
        return _dispatch(state["x"], state["slot_row"])
    if op == "combine":
        return _combine(state["rows"], state["slot_row"], state.get("weights"), TYPES[c["out"]])
    if op == "combine_grad":
        return _combine_grad(state["dout"], state["rows"], state["slot_row"], state["weights"])
    if op == "mxfp4":
        return _mx_values(*_mx_codes(state["x"])).to(torch.bfloat16)
    return _gmm_mxfp4(state["lhs"], state["q"], state["scale"], state["sizes"], TYPES[c["out"]])


def work(case):
    op = case["op"]
    if op == "mxfp4":
        # quantised and widened again: x read, the values written (the codes between them are not counted)
        return {"bytes": case["G"] * case["N"] * case["K"] * (BYTES[case["x"]] + 2), "flops": 0}
    if op == "gmm":
        M, G, N, K = case["M"], case["G"], case["N"], case["K"]
        return {"bytes": M * K * 2 + min(M, G) * N * K * (0.5 + 1 / 32) + M * N * BYTES[case["out"]], "flops": 2.0 * M * N * K}
    n = case["T"] * case["k"]
    if op == "sort":
        return {"bytes": n * (BYTES[case["ids"]] + 4) + 4 * case["G"], "flops": 0}
    big, small = n * case["D"], case["T"] * case["D"]
    es, routed = BYTES[case["x"]], 1 - case["unrouted"]
    if op == "dispatch":
        return {"bytes": 4 * n + (big + small) * es, "flops": 0}
    wb = 0 if case["weights"] == "none" else BYTES[case["weights"]] * n
    if op == "combine":
        return {"bytes": 4 * n + wb + big * routed * es + small * BYTES[case["out"]], "flops": 2.0 * big * routed}
    return {"bytes": 4 * n + 2 * wb + (big + big * routed + small) * es, "flops": 3.0 * big * routed}


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "sort":
        return None
    if op == "mxfp4":
        x = s["x"].double()
        parts = []
        for block in x.reshape(-1, 32).split(1 << 20):
            top = block.abs().amax(1, keepdim=True)
            e = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top))))
            e = torch.where(torch.exp2(e) > top, e - 1, e)  # log2 next to a power of two
            unit = torch.exp2((torch.where(top > 0, e, e + 2) - 2).clamp(-127, 125))
            t = (block / unit).abs()
            # the grid's step is 1/2 below 2, 1 below 4 and 2 above; round() takes ties to even
            step = torch.where(t < 2, 0.5, torch.where(t < 4, 1.0, 2.0))
            parts.append(torch.sign(block) * torch.clamp(torch.round(t / step) * step, max=6.0) * unit)
        return torch.cat(parts).reshape(x.shape)
    if op == "gmm":
        G, N, K = case["G"], case["N"], case["K"]
        out = torch.zeros((case["M"], N), dtype=torch.float64, device=DEV)
        pairs = torch.tensor([[(-1.0 if c & 8 else 1.0) * E2M1[c & 7] for c in (b & 15, b >> 4)] for b in range(256)],
                             dtype=torch.float64, device=DEV)
        unit = torch.exp2(s["scale"].view(torch.uint8).double() - 127).reshape(G, K // 32, N)
        lo = 0
        for h, size in enumerate(s["sizes"].tolist()):
            w = pairs[s["q"][h].long()].reshape(N, K) * unit[h].t().repeat_interleave(32, 1)
            out[lo:lo + size] = s["lhs"][lo:lo + size].double() @ w.t().contiguous()
            lo += size
        return out
    T, k, D = case["T"], case["k"], case["D"]
    slot_row = s["slot_row"].cpu()
    routed = slot_row >= 0
    row = torch.where(routed, slot_row, ~slot_row).long().to(DEV)
    routed = routed.to(DEV)
    if op == "dispatch":
        out = torch.zeros((T * k, D), dtype=torch.float64, device=DEV)
        for j in range(k):
            out.index_copy_(0, row[:, j], torch.where(routed[:, j, None], s["x"].double(), 0.0))
        return out
    w = s["weights"].double() if "weights" in s else torch.ones((T, k), dtype=torch.float64, device=DEV)
    if op == "combine":
        out = torch.zeros((T, D), dtype=torch.float64, device=DEV)
        for j in range(k):
            out += torch.where(routed[:, j, None], s["rows"][row[:, j]].double() * w[:, j, None], 0.0)
        return out
    drows = torch.zeros((T * k, D), dtype=torch.float64, device=DEV)
    dweights = torch.zeros((T, k), dtype=torch.float64, device=DEV)
    d = s["dout"].double()
    for j in range(k):
        drows.index_copy_(0, row[:, j], torch.where(routed[:, j, None], d * w[:, j, None], 0.0))
        dweights[:, j] = torch.where(routed[:, j], (s["rows"][row[:, j]].double() * d).sum(1), 0.0)
    return drows, dweights
