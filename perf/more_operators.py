"""Cases of the operators at both ends of a mixture-of-experts layer: the router
(its choice of experts, the balance loss with per-expert counts, and the
gradient of both), the experts' products of a few tokens by expert id over
four-bit weights, and the AdamW step of the layer's weights.

With ``own`` false every case runs in elementary torch operations, in 32 bits;
with ``own`` true it makes the package's calls."""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4, "e8m0": 1}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = 256  # elements of an eight-bit state that share a scale
ROOM = 1024  # the tensors of a step start at multiples of this in their buffers
COEF, Z_COEF = 0.01, 0.001  # of the balance loss and of its logit term
LR, BETAS, EPS, DECAY, STEP = 1e-4, (0.9, 0.95), 1e-8, 0.1, 100


def _lib():
    import moe_grouped_matrix_amd
    return moe_grouped_matrix_amd


# ---------------------------------------------------------------------------
# the cases

def listed():
    return [
        # one token of a chat chooses its top-8 of 128 experts: a launch and little else
        dict(name="route_one_token", op="route", T=1, E=128, k=8, x="f32", scores="softmax", renorm=True, pad=0.0, off=0.0),
        # the training batch of the package's own benchmark: 32768 tokens, top-8 of 128
        dict(name="route_batch", op="route", T=32768, E=128, k=8, x="f32", scores="softmax", renorm=True, pad=0.0, off=0.0),
        # the load-balancing loss of that batch
        dict(name="balance_batch", op="balance", T=32768, E=128, k=8, x="f32", scores="softmax", pad=0.0, off=0.0),
        # a ragged batch with padded rows and experts that are switched off, bf16 logits, sigmoid scores
        dict(name="balance_odd", op="balance", T=4099, E=37, k=3, x="bf16", scores="sigmoid", pad=0.1, off=0.05),
        # the router's backward pass in that training batch, through the weights and the balance loss
        dict(name="router_grad_batch", op="router_grad", T=32768, E=128, k=8, x="f32", scores="softmax", renorm=True, pad=0.0, off=0.0),
        # the same in the ragged batch
        dict(name="router_grad_odd", op="router_grad", T=4099, E=37, k=3, x="bf16", scores="sigmoid", renorm=True, pad=0.1, off=0.05),
        # one token of a chat through the up projections of its 8 experts (int4, groups of 128)
        dict(name="gmv_one_token", op="gmv", T=1, k=8, G=128, N=1408, K=1408, fmt="int4", block=128, scale="f32", zero=False,
             per_slot=False, weights=False, out="bf16", unrouted=0.0),
        # and back through their down projections, summed with the router's weights (uint4, groups of 32 with zero points)
        dict(name="gmv_down_one_token", op="gmv", T=1, k=8, G=128, N=1408, K=704, fmt="uint4", block=32, scale="bf16", zero=True,
             per_slot=True, weights=True, out="bf16", unrouted=0.0),
        # a decode step of 32 sequences: most experts touched, few rows each
        dict(name="gmv_decode", op="gmv", T=32, k=8, G=128, N=1408, K=1408, fmt="int4", block=128, scale="f32", zero=False,
             per_slot=False, weights=False, out="bf16", unrouted=0.0),
        # a dense layer (one expert) for four sequences, microscaled fp4 weights
        dict(name="gmv_dense", op="gmv", T=4, k=1, G=1, N=8192, K=4096, fmt="fp4_e2m1", block=32, scale="e8m0", zero=False,
             per_slot=False, weights=False, out="f32", unrouted=0.0),
        # the optimizer step of every expert's up and down projection of the benchmark's layer: f32 weights with the
        # bf16 copies that the products read, bf16 gradients, eight-bit states
        dict(name="adamw_experts", op="adamw", sizes="128x1408x1408,128x1408x704", p="f32", g="bf16", bits=8, copies=True),
        # the small tensors of 24 layers (routers, norms, biases): launches and many ends
        dict(name="adamw_small", op="adamw", sizes=",".join(["128x1408", "1408", "704", "37", "1"] * 24), p="f32", g="f32",
             bits=32, copies=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["route", "balance", "router_grad", "gmv", "gmv", "adamw"])
    if op == "gmv":
        T, G = _log(rng, 1, 32), _log(rng, 1, 128)
        K = 32 * _log(rng, 1, 44)
        fmt = rng.choice(["int4", "uint4", "fp4_e2m1"])
        scale = "e8m0" if fmt == "fp4_e2m1" and rng.random() < 0.7 else rng.choice(["f32", "bf16"])
        block = 32 if scale == "e8m0" else rng.choice([b for b in (32, 64, 128, K) if K % b == 0])
        return dict(op=op, T=T, k=rng.randint(1, min(8, G)), G=G, N=_log(rng, 1, 1408), K=K, fmt=fmt, block=block, scale=scale,
                    zero=fmt != "fp4_e2m1" and rng.random() < 0.5, per_slot=rng.random() < 0.5, weights=rng.random() < 0.5,
                    out=rng.choice(["bf16", "f32"]), unrouted=rng.choice([0.0, 0.0, 0.1]))
    if op == "adamw":
        total, count = _log(rng, 1000, 20000000), _log(rng, 1, 150)
        sizes = [max(1, int(total / count * rng.uniform(0.1, 1.9))) for _ in range(count)]
        return dict(op=op, sizes=",".join(map(str, sizes)), p=rng.choice(["f32", "f32", "bf16"]), g=rng.choice(["f32", "bf16"]),
                    bits=rng.choice([8, 32]), copies=rng.random() < 0.5)
    E = _log(rng, 2, 512)
    case = dict(op=op, T=_log(rng, 1, 32768), E=E, k=rng.randint(1, min(8, E)), x=rng.choice(["f32", "bf16"]),
                scores=rng.choice(["softmax", "sigmoid"]), pad=rng.choice([0.0, 0.1]), off=rng.choice([0.0, 0.05, 0.5]))
    if op != "balance":
        case["renorm"] = rng.random() < 0.6
    return case


# ---------------------------------------------------------------------------
# inputs

def _normal(g, shape, scale=1.0):
    return torch.randn(shape, generator=g, device=DEV) * scale


def _uniform(g, shape):
    return torch.rand(shape, generator=g, device=DEV)


def _logits(case, g):
    """A router's logits, its experts with Zipf popularity (rank^-1.1 over a
    seeded order); some experts switched off a token, and some tokens with none
    left, by logits of -inf; padded rows hold NaN."""
    T, E = case["T"], case["E"]
    rank = torch.randperm(E, generator=g, device=DEV).float() + 1
    z = _normal(g, (T, E), 1.5) - 1.1 * torch.log(rank)
    if case["off"]:
        away = (_uniform(g, (T, E)) < case["off"]) | (_uniform(g, (T, 1)) < 0.02)
        z = torch.where(away, torch.full_like(z, -math.inf), z)
    valid = None
    if case["pad"]:
        valid = _uniform(g, (T,)) >= case["pad"]
        z = torch.where(valid[:, None], z, torch.full_like(z, math.nan))
    return z.to(TYPES[case["x"]]), valid


def _quantise(w, case):
    """Codes 0..15, scales and zero points of w [G,N,K] in blocks of K."""
    G, N, K = w.shape
    b = w.reshape(G, N, K // case["block"], case["block"])
    fmt = case["fmt"]
    zero = None
    if fmt == "fp4_e2m1":
        amax = b.abs().amax(-1, keepdim=True)
        s = amax / 6
        if case["scale"] == "e8m0":
            s = torch.exp2(torch.floor(torch.log2(amax.clamp_min(1e-20))) - 2)
        elif case["scale"] == "bf16":
            s = s.bfloat16().float()
        t = (b / s).abs()
        code = (t > 0.25).int() + (t >= 0.75) + (t > 1.25) + (t >= 1.75) + (t > 2.5) + (t >= 3.5) + (t > 5)
        code = code + 8 * (b < 0)
    else:
        low, high = b.amin(-1, keepdim=True), b.amax(-1, keepdim=True)
        s = (high - low) / 15 if case["zero"] else b.abs().amax(-1, keepdim=True) / 7
        s = s.clamp_min(1e-20)
        if case["scale"] == "bf16":
            s = s.bfloat16().float()
        least = 0 if fmt == "uint4" else -8
        if case["zero"]:
            zero = torch.round(least - low / s)
            code = torch.clamp(torch.round(b / s) + zero, least, least + 15)
        else:  # uint4 without zero points: magnitudes
            code = torch.clamp(torch.round((b.abs() if fmt == "uint4" else b) / s), least, least + 15)
        code = code.int() & 15
    lay = lambda t: t[..., 0].transpose(1, 2).unsqueeze(2).contiguous()  # noqa: E731  [G,N,nb,1] -> [G,nb,1,N]
    if case["scale"] == "e8m0":
        s = lay(torch.log2(s) + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    else:
        s = lay(s).to(TYPES[case["scale"]])
    return code.to(torch.uint8).reshape(G, N, K), s, None if zero is None else lay(zero).to(s.dtype)


def _shapes(case):
    return [tuple(int(n) for n in s.split("x")) for s in case["sizes"].split(",")]


def _places(case):
    """Where each tensor starts in its buffer, its elements, and the buffer's length."""
    at, places = 0, []
    for shape in _shapes(case):
        n = math.prod(shape)
        places.append((at, n, shape))
        at += -(-n // ROOM) * ROOM
    return places, at


def _views(buffer, places):
    return [buffer[at:at + n].view(shape) for at, n, shape in places]


def _blocks(buffer, places):
    return [buffer[at // BLOCK:at // BLOCK + -(-n // BLOCK)] for at, n, _ in places]


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    if op == "adamw":
        places, total = _places(case)
        inside = torch.zeros(total, dtype=torch.bool, device=DEV)
        for at, n, _ in places:
            inside[at:at + n] = True
        fill = lambda t: torch.where(inside, t, torch.zeros((), device=DEV))  # noqa: E731
        size = torch.exp(_normal(g, (total // BLOCK, 1), 0.5)).expand(-1, BLOCK).reshape(-1)  # gradients of this block
        state = dict(case=case, p=fill(_normal(g, total, 0.02)).to(TYPES[case["p"]]),
                     g=fill(_normal(g, total, 1e-3) * size).to(TYPES[case["g"]]))
        m, v = fill(_normal(g, total, 3e-4) * size), fill((1e-3 * size * torch.exp(_normal(g, total, 0.3))) ** 2)
        if case["bits"] == 8:
            state["m"], state["ms"] = _eight_bits(m, False)
            state["v"], state["vs"] = _eight_bits(torch.sqrt(v), True)
        else:
            state["m"], state["v"] = m, v
        if case["copies"]:
            state["c"] = torch.zeros(total, dtype=torch.bfloat16, device=DEV)
        state["lists"] = {n: _views(state[n], places) for n in ("p", "g", "m", "v", "c") if n in state}
        state["lists"].update({n: _blocks(state[n], places) for n in ("ms", "vs") if n in state})
        return state
    if op == "gmv":
        T, k, G, N, K = case["T"], case["k"], case["G"], case["N"], case["K"]
        rank = torch.randperm(G, generator=g, device=DEV).float() + 1
        noise = -torch.log(-torch.log(_uniform(g, (T, G)).clamp(1e-9, 1 - 1e-7)))
        top = torch.topk(noise - 1.1 * torch.log(rank), k, dim=1)
        ids = torch.where(_uniform(g, (T, k)) < case["unrouted"], torch.full_like(top.indices, -1), top.indices)
        code, scale, zero = _quantise(_normal(g, (G, N, K), 0.02) * torch.exp(_normal(g, (G, N, 1), 0.3)), case)
        q = (code[..., 0::2] | code[..., 1::2] << 4).contiguous()
        state = dict(case=case, x=_normal(g, (T, k, K) if case["per_slot"] else (T, K)).to(torch.bfloat16), q=q, scale=scale,
                     zero=zero, ids=ids.to(torch.int32))
        if case["weights"]:
            state["w"] = torch.softmax(top.values, dim=1)
        return state
    z, valid = _logits(case, g)
    state = dict(case=case, z=z, valid=valid)
    if op != "route":
        state["ids"] = _route(z, valid, case["k"], case["scores"], case.get("renorm", True))[0]
    if op == "router_grad":
        _, state["counts"], state["tokens"] = _balance(z, state["ids"], valid, case["scores"])
        state["dw"] = _normal(g, (case["T"], case["k"]), 1e-2)
        state["dloss"] = torch.ones(1, device=DEV)
    return state


# ---------------------------------------------------------------------------
# the plain forms

def _live(z, valid):
    """The logits in 32 bits, those that count, and the rows that do."""
    z = z.float()
    row = (z > -math.inf).any(1) | z.isnan().any(1)
    if valid is not None:
        row = row & valid
    z = torch.where(row[:, None], z, torch.zeros_like(z))
    return z, (z > -math.inf) & row[:, None], row


def _scores(z, kind):
    """Scores of the logits, and their logarithm of summed exponentials."""
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    s = e / total if kind == "softmax" else 1 / (1 + torch.exp(-z))
    return s, (top + torch.log(total))[:, 0]


def _route(z, valid, k, kind, renorm):
    """expert_ids [T,k] int32 and weights [T,k] of the k largest logits, equal
    ones in the order of their experts."""
    z, live, row = _live(z, valid)
    order = torch.sort(torch.where(live, z, torch.full_like(z, -math.inf)), dim=1, descending=True, stable=True)
    ids, value = order.indices[:, :k], order.values[:, :k]
    there = torch.gather(live, 1, ids)
    if kind == "softmax" and renorm:
        s = torch.exp(value - torch.where(row, value[:, 0], torch.zeros_like(value[:, 0]))[:, None])
    else:
        s = torch.gather(_scores(z, kind)[0], 1, ids)
    s = torch.where(there, s, torch.zeros_like(s))
    if renorm:
        total = s.sum(1, keepdim=True)
        s = torch.where(total > 0, s / total, torch.zeros_like(s))
    return torch.where(there, ids, torch.full_like(ids, -1)).to(torch.int32), s


def _balance(z, ids, valid, kind):
    """loss [1], counts int32 [E], tokens int32 [1]."""
    E = z.shape[1]
    z, _, row = _live(z, valid)
    s, lse = _scores(z, kind)
    p = torch.where(row[:, None], s / s.sum(1, keepdim=True), torch.zeros_like(s))
    flat = ids.flatten().long()
    counts = torch.zeros(E + 1, dtype=torch.int32, device=z.device)
    counts.index_add_(0, torch.where(flat >= 0, flat, torch.full_like(flat, E)), torch.ones_like(flat, dtype=torch.int32))
    counts, tokens = counts[:E], row.sum().to(torch.int32).reshape(1)
    n = tokens.clamp_min(1).double()
    share = counts.double() / counts.sum().clamp_min(1)
    loss = COEF * E * (share * p.sum(0, dtype=torch.float64) / n).sum()
    loss = loss + Z_COEF * (torch.where(row, lse, torch.zeros_like(lse)).double() ** 2).sum() / n
    return loss.float().reshape(1), counts, tokens


def _router_grad(z, ids, valid, kind, renorm, dw, counts, tokens, dloss):
    dtype, E = z.dtype, z.shape[1]
    z, _, row = _live(z, valid)
    s, lse = _scores(z, kind)
    total = s.sum(1, keepdim=True)
    p = s / total
    n = tokens.clamp_min(1).float()
    a = dloss * COEF * E / n * (counts.float() / counts.sum().clamp_min(1))
    about = (p * a).sum(1, keepdim=True)
    # the weights: ds of the chosen scores
    there = ids >= 0
    at = torch.where(there, ids, torch.zeros_like(ids)).long()
    chosen = torch.where(there, torch.gather(s, 1, at), torch.zeros_like(dw))
    g = torch.where(there, dw, torch.zeros_like(dw))
    if renorm:
        S = chosen.sum(1, keepdim=True)
        share = torch.where(S > 0, chosen / S, torch.zeros_like(S))
        chosen_dz = share * (g - (share * g).sum(1, keepdim=True))  # s ds
    else:
        chosen_dz = chosen * g
    if kind == "sigmoid":
        dz = p * (1 - s) * (a - about)
        chosen_dz = chosen_dz * (1 - chosen)
    else:
        dz = p * (a - about)
        if not renorm:
            dz = dz - s * chosen_dz.sum(1, keepdim=True)
    dz = dz + (2 * Z_COEF) * dloss / n * (lse[:, None] * torch.exp(z - lse[:, None]))
    dz = dz.scatter_add(1, at, chosen_dz)
    return torch.where(row[:, None], dz, torch.zeros_like(dz)).to(dtype)


def _widen(q, scale, zero, case):
    """Weights [..., N, K] in 32 bits of packed codes [..., N, K/2], their scales and zero points [..., nb, 1, N]."""
    code = torch.stack((q & 15, q >> 4), -1).reshape(q.shape[:-1] + (-1, case["block"])).int()  # [..., N, nb, block]
    if case["fmt"] == "fp4_e2m1":
        value = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=q.device)[code]
    else:
        value = (code - 16 * (code >= 8) if case["fmt"] == "int4" else code).float()
    lay = lambda t: t.squeeze(-2).transpose(-1, -2).unsqueeze(-1)  # noqa: E731
    if zero is not None:
        value = value - lay(zero).float()
    unit = torch.exp2(scale.view(torch.uint8).float() - 127) if case["scale"] == "e8m0" else scale.float()
    return (value * lay(unit)).reshape(q.shape[:-1] + (-1,))


def _gmv(x, q, scale, zero, ids, w, case):
    T, k = ids.shape
    there = ids >= 0
    at = torch.where(there, ids, torch.zeros_like(ids)).long().flatten()
    wide = _widen(q[at], scale.view(torch.uint8)[at] if case["scale"] == "e8m0" else scale[at],
                  None if zero is None else zero[at], case)
    x = (x if case["per_slot"] else x[:, None].expand(-1, k, -1)).float().reshape(T * k, -1, 1)
    y = torch.bmm(wide, x.contiguous()).reshape(T, k, -1)
    y = torch.where(there[..., None], y, torch.zeros_like(y))
    if w is not None:
        y = (y * torch.where(there, w, torch.zeros_like(w))[..., None]).sum(1)
    return y.to(TYPES[case["out"]])


def _eight_bits(x, positive):
    """e4m3 codes and the scales of blocks of BLOCK; a positive value is never 0."""
    b = x.reshape(-1, BLOCK)
    top = b.abs().amax(1, keepdim=True)
    scale = torch.where(top > 0, (top / 448).clamp_min(2.0 ** -126), torch.ones_like(top))
    t = b / scale
    if positive:
        t = torch.where(b > 0, t.clamp_min(2.0 ** -9), t)
    return t.to(torch.float8_e4m3fn).reshape(-1), scale[:, 0]


def _from_eight_bits(q, scale):
    return (q.float().reshape(-1, BLOCK) * scale[:, None]).reshape(-1)


def _adamw(s):
    """One step over whole buffers (what lies between their tensors stays zero);
    every operation rounded to 32 bits."""
    b1, b2 = BETAS
    eight = s["case"]["bits"] == 8
    p, g = s["p"].float(), s["g"].float()
    m = _from_eight_bits(s["m"], s["ms"]) if eight else s["m"]
    v = _from_eight_bits(s["v"], s["vs"]) ** 2 if eight else s["v"]
    m = m * b1 + g * (1 - b1)
    v = v * b2 + (g * g) * (1 - b2)
    root = torch.sqrt(v)
    p = p * (1 - LR * DECAY) - (LR / (1 - b1 ** STEP)) * (m / (root * (1 / math.sqrt(1 - b2 ** STEP)) + EPS))
    s["p"].copy_(p)
    if "c" in s:
        s["c"].copy_(p)
    if eight:
        for name, (code, scale) in (("m", _eight_bits(m, False)), ("v", _eight_bits(root, True))):
            s[name].copy_(code)
            s[name + "s"].copy_(scale)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if op == "route":
        if own:
            return _lib().route(s["z"], c["k"], scores=c["scores"], renormalize=c["renorm"], valid=s["valid"])
        return _route(s["z"], s["valid"], c["k"], c["scores"], c["renorm"])
    if op == "balance":
        if own:
            return _lib().balance_loss(s["z"], s["ids"], scores=c["scores"], coef=COEF, z_coef=Z_COEF, valid=s["valid"])
        return _balance(s["z"], s["ids"], s["valid"], c["scores"])
    if op == "router_grad":
        if own:
            return _lib().router_grad(s["z"], s["ids"], dweights=s["dw"], scores=c["scores"], renormalize=c["renorm"],
                                      counts=s["counts"], tokens=s["tokens"], dloss=s["dloss"], coef=COEF, z_coef=Z_COEF,
                                      valid=s["valid"])
        return _router_grad(s["z"], s["ids"], s["valid"], c["scores"], c["renorm"], s["dw"], s["counts"], s["tokens"], s["dloss"])
    if op == "gmv":
        if own:
            return _lib().gmv(s["x"], s["q"], s["ids"], rhs_format=c["fmt"], rhs_scale=s["scale"], rhs_zero=s["zero"],
                              weights=s.get("w"), out_dtype=TYPES[c["out"]])
        return _gmv(s["x"], s["q"], s["scale"], s["zero"], s["ids"], s.get("w"), c)
    if own:
        n = s["lists"]
        _lib().adamw(n["p"], n["g"], n["m"], n["v"], STEP, lr=LR, betas=BETAS, eps=EPS, weight_decay=DECAY,
                     exp_avg_scale=n.get("ms"), exp_avg_sq_scale=n.get("vs"), copies=n.get("c"))
    else:
        _adamw(s)
    return {n: s[n] for n in ("p", "m", "v", "ms", "vs", "c") if n in s}


def work(case):
    op = case["op"]
    if op == "adamw":
        n = sum(math.prod(s) for s in _shapes(case))
        state = 4 * (1 + 4 / BLOCK) if case["bits"] == 8 else 16
        return {"bytes": n * (2 * BYTES[case["p"]] + BYTES[case["g"]] + state + 2 * case["copies"]), "flops": 14.0 * n}
    if op == "gmv":
        T, k, G, N, K = case["T"], case["k"], case["G"], case["N"], case["K"]
        slots = T * k
        # experts that a step touches: with every one as likely, G (1 - (1 - k/G)^T)
        touched = G * (1 - (1 - min(1.0, k / G)) ** T)
        scales = K // case["block"] * BYTES[case["scale"]] * (2 if case["zero"] else 1)
        return {"bytes": touched * N * (K / 2 + scales) + (slots if case["per_slot"] else T) * K * 2 + 4 * slots +
                (T if case["weights"] else slots) * N * BYTES[case["out"]] + 4 * slots * case["weights"],
                "flops": 2.0 * slots * N * K}
    T, E, k = case["T"], case["E"], case["k"]
    read = T * E * BYTES[case["x"]] + (T if case["pad"] else 0)
    if op == "route":
        return {"bytes": read + 8 * T * k, "flops": 4.0 * T * E}
    if op == "balance":
        return {"bytes": read + 4 * T * k + 4 * E + 8, "flops": 6.0 * T * E}
    return {"bytes": read + T * E * BYTES[case["x"]] + 8 * T * k + 4 * E, "flops": 10.0 * T * E}


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_softmax(z, row):
    z = torch.where(row[:, None], z, torch.zeros_like(z))
    lse = torch.logsumexp(z, 1)
    return torch.exp(z - lse[:, None]), lse


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "adamw":
        b1, b2 = BETAS
        eight = case["bits"] == 8
        widen = lambda q, sc: q.double() * sc.double().repeat_interleave(BLOCK)  # noqa: E731
        m = (widen(s["m"], s["ms"]) if eight else s["m"].double()) * b1
        m += (1 - b1) * s["g"].double()
        v = (widen(s["v"], s["vs"]).square_() if eight else s["v"].double()) * b2
        v += (1 - b2) * s["g"].double().square_()
        p = s["p"].double() * (1 - LR * DECAY) - LR * (m / (1 - b1 ** STEP)) / (torch.sqrt(v / (1 - b2 ** STEP)) + EPS)
        out = {"p": p, "m": m, "v": v, "c": p} if case["copies"] else {"p": p, "m": m, "v": v}
        if eight:
            for name, x in (("m", m), ("v", v.sqrt_())):
                top = x.abs().reshape(-1, BLOCK).amax(1)
                unit = torch.where(top > 0, (top / 448).clamp_min(2.0 ** -126), torch.ones_like(top))
                t = x / unit.repeat_interleave(BLOCK)
                # the grid of e4m3: steps of 2^(e-3) from 2^e on, of 2^-9 below 2^-6
                step = torch.exp2(torch.floor(torch.log2(t.abs().clamp_min(2.0 ** -6))) - 3)
                t = torch.round(t / step) * step
                out[name], out[name + "s"] = torch.where((x > 0) & (t == 0), 2.0 ** -9, t) if name == "v" else t, unit
        return out
    if op == "gmv":
        T, k, N, K = case["T"], case["k"], case["N"], case["K"]
        ids = s["ids"].tolist()
        out = torch.zeros((T, k, N), dtype=torch.float64, device=DEV)
        table = list(E2M1) + [-v for v in E2M1] if case["fmt"] == "fp4_e2m1" else \
            [float(c - 16 if c >= 8 and case["fmt"] == "int4" else c) for c in range(16)]
        pairs = torch.tensor([[table[b & 15], table[b >> 4]] for b in range(256)], dtype=torch.float64, device=DEV)
        unit = torch.exp2(s["scale"].view(torch.uint8).double() - 127) if case["scale"] == "e8m0" else s["scale"].double()
        for t in range(T):
            for j in range(k):
                e = ids[t][j]
                if e < 0:
                    continue
                w = pairs[s["q"][e].long()].reshape(N, -1, case["block"])
                if s["zero"] is not None:
                    w = w - s["zero"][e, :, 0].double().t()[..., None]
                x = (s["x"][t, j] if case["per_slot"] else s["x"][t]).double()
                out[t, j] = (w * unit[e, :, 0].t()[..., None]).reshape(N, K) @ x
        if not case["weights"]:
            return out
        w = torch.where(s["ids"] >= 0, s["w"].double(), 0.0)
        return (out * w[..., None]).sum(1)
    z = s["z"].double()
    valid = s["valid"] if s["valid"] is not None else torch.ones(case["T"], dtype=torch.bool, device=DEV)
    row = valid & (z > -math.inf).any(1)
    soft, lse = _exact_softmax(z, row)
    score = soft if case["scores"] == "softmax" else torch.sigmoid(torch.where(row[:, None], z, 0.0))
    experts = torch.arange(case["E"], device=DEV)
    if op == "route":
        left, parts = torch.where(row[:, None], z, -math.inf), []
        for _ in range(case["k"]):
            best = left.amax(1, keepdim=True)
            first = torch.where(left == best, experts, case["E"]).amin(1, keepdim=True)
            parts.append(torch.where(best > -math.inf, torch.gather(score, 1, first), 0.0))
            left = left.scatter(1, first, -math.inf)
        w = torch.cat(parts, 1)
        return None, (w / w.sum(1, keepdim=True).clamp_min(1e-300) if case["renorm"] else w)
    prob = torch.where(row[:, None], score / score.sum(1, keepdim=True), 0.0)
    ids = s["ids"].long()
    picked = (ids[..., None] == experts).double()  # [T,k,E]
    share = picked.sum((0, 1)) / max(1.0, float((ids >= 0).sum()))
    n = max(1.0, float(row.sum()))
    if op == "balance":
        loss = COEF * case["E"] * (share * prob.sum(0)).sum() / n + Z_COEF * torch.where(row, lse, 0.0).square().sum() / n
        return loss.reshape(1), None, None
    # by the chain rule, a factor at a time: weights -> scores -> logits
    dscore = torch.zeros_like(z)
    chosen = (picked * score[:, None, :]).sum(-1)
    g = torch.where(ids >= 0, s["dw"].double(), 0.0)
    if case["renorm"]:
        S = chosen.sum(1, keepdim=True).clamp_min(1e-300)
        g = g / S - (g * chosen).sum(1, keepdim=True) / (S * S) * (ids >= 0)
    dscore += (picked * g[..., None]).sum(1)
    total = score.sum(1, keepdim=True)
    dprob = COEF * case["E"] / n * share
    dscore += (dprob - (dprob * prob).sum(1, keepdim=True)) / total
    if case["scores"] == "softmax":
        dz = score * (dscore - (dscore * score).sum(1, keepdim=True))
    else:
        dz = dscore * score * (1 - score)
    dz += 2 * Z_COEF / n * lse[:, None] * soft
    return torch.where(row[:, None], dz, 0.0)
