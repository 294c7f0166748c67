"""Plain 64-bit forms of the operators of include/gmm_layer.h, for the tests
(CPU tensors in, float64 tensors out), written as loops over the definitions;
the AdamW step also in binary32 with every operation rounded."""
import math

import numpy as np
import torch

from moe_reference import E2M1, unpack

INF = math.inf


def score(z, scores):
    """Scores of one token's logits (a float64 vector with something above -inf)."""
    if scores == "sigmoid":
        return torch.sigmoid(z)  # 1 / (1 + exp(-z)), with a gradient of 0 where that exponential overflows
    e = torch.exp(z - z.max())
    return e / e.sum()


def counts_rows(logits, valid):
    z = logits.double()
    ok = (z > -INF).any(1) | z.isnan().any(1)
    return ok if valid is None else ok & valid.bool()


def route(logits, k, scores="softmax", bias=None, renormalize=True, scale=1.0, valid=None):
    """(expert_ids int32, weights float64, the keys that ranked the choices)."""
    T, E = logits.shape
    ids = torch.full((T, k), -1, dtype=torch.int32)
    weights = torch.zeros(T, k, dtype=torch.float64)
    keys = torch.full((T, E), -INF, dtype=torch.float64)
    for t in torch.nonzero(counts_rows(logits, valid))[:, 0].tolist():
        z = logits[t].double()
        if bool((~(z < INF)).any()):
            weights[t] = math.nan
            continue
        s = score(z, scores)
        key = torch.where(z > -INF, z if bias is None else s + bias.double(), torch.full_like(z, -INF))
        keys[t] = key
        order = sorted((e for e in range(E) if z[e] > -INF), key=lambda e: (-float(key[e]), e))[:k]
        for j, e in enumerate(order):
            ids[t, j] = e
        if order:
            chosen = s[order]
            if renormalize:
                chosen = chosen / chosen.sum()
            weights[t, :len(order)] = scale * chosen
    return ids, weights, keys


def balance_loss(logits, ids, scores="softmax", coef=1.0, z_coef=0.0, valid=None):
    """(loss, counts int32 [E], n); loss is differentiable in float64 logits."""
    T, E = logits.shape
    rows = counts_rows(logits.detach(), valid)
    counts = torch.zeros(E, dtype=torch.int64)
    for e in ids.reshape(-1).tolist():
        if 0 <= e < E:
            counts[e] += 1
    n = int(rows.sum())
    total, z2 = torch.zeros(E, dtype=torch.float64), torch.zeros((), dtype=torch.float64)
    for t in torch.nonzero(rows)[:, 0].tolist():
        z = logits[t].double()
        s = score(z, scores)
        total = total + s / s.sum()
        z2 = z2 + torch.logsumexp(z, 0) ** 2
    f = counts.double() / max(1, int(counts.sum()))
    loss = coef * E * (f * total).sum() / max(1, n) + z_coef * z2 / max(1, n)
    return loss, counts.to(torch.int32), n


def weights_of(logits, ids, scores="softmax", renormalize=True, scale=1.0, valid=None):
    """route()'s weights for given choices (0 where there is none), differentiable."""
    T, E = logits.shape
    rows = counts_rows(logits.detach(), valid)
    out = []
    for t in range(T):
        there = [j for j in range(ids.shape[1]) if 0 <= int(ids[t, j]) < E] if rows[t] else []
        w = torch.zeros(ids.shape[1], dtype=torch.float64)
        if there:
            s = score(logits[t].double(), scores)[ids[t, there].long()]
            w = w.index_put((torch.tensor(there),), scale * (s / s.sum() if renormalize else s))
        out.append(w)
    return torch.stack(out) if out else torch.zeros(0, ids.shape[1], dtype=torch.float64)


def objective(logits, ids, dweights=None, counts_in=None, tokens_in=None, dloss=1.0, scores="softmax", renormalize=True, scale=1.0,
              coef=1.0, z_coef=0.0, valid=None):
    """What router_grad() is the gradient of, in float64 logits."""
    total = torch.zeros((), dtype=torch.float64)
    if dweights is not None:
        g = torch.where((ids >= 0) & (ids < logits.shape[1]), dweights.double(), torch.zeros((), dtype=torch.float64))
        total = total + (g * weights_of(logits, ids, scores, renormalize, scale, valid)).sum()
    if counts_in is not None:
        E = logits.shape[1]
        f = counts_in.double() / max(1, int(counts_in.sum()))
        n = max(1, int(tokens_in))
        for t in torch.nonzero(counts_rows(logits.detach(), valid))[:, 0].tolist():
            z = logits[t].double()
            s = score(z, scores)
            total = total + dloss * (coef * E * (f * s / s.sum()).sum() / n + z_coef * torch.logsumexp(z, 0) ** 2 / n)
    return total


def router_grad(logits, ids, **kw):
    """The gradient by automatic differentiation of objective(), with the
    switched-off experts' logits left out of it."""
    z = logits.double().clone()
    off = z == -INF
    # (an expert at -inf has score 0 and no gradient; a number far below every binary32 stands in for it, so that no 0 * inf arises)
    rows = counts_rows(logits, kw.get("valid"))
    z = torch.where(off, torch.full_like(z, -1e300), z)
    z = torch.where(rows[:, None], z, torch.zeros_like(z)).requires_grad_()
    valid = rows
    kw = dict(kw, valid=valid)
    value = objective(z, ids, **kw)
    if not value.requires_grad:
        return torch.zeros_like(z)
    value.backward()
    return torch.where(off | ~rows[:, None], torch.zeros_like(z), z.grad)


def code_values(fmt):
    if fmt == "fp4_e2m1":
        return torch.from_numpy(E2M1)
    return torch.tensor([float(c - 16 if fmt == "int4" and c >= 8 else c) for c in range(16)], dtype=torch.float64)


def wide_scale(scale):
    return torch.exp2(scale.view(torch.uint8).double() - 127) if scale.dtype == torch.float8_e8m0fnu else scale.double()


def gmv(x, q, ids, fmt, scale, zero=None, weights=None):
    """(float64 result, the sum of the absolute terms) of gmv()."""
    G, N, nb = q.shape[0], q.shape[1], scale.shape[1]
    T, k = ids.shape
    K = 2 * q.shape[2]
    value = code_values(fmt)[unpack(q).long()].reshape(G, N, nb, K // nb)
    unit = wide_scale(scale)[:, :, 0].transpose(1, 2)[..., None]
    z = zero.double()[:, :, 0].transpose(1, 2)[..., None] if zero is not None else torch.zeros(())
    w, size = ((value - z) * unit).reshape(G, N, K), ((value.abs() + z.abs()) * unit.abs()).reshape(G, N, K)
    out, mag = torch.zeros(T, k, N, dtype=torch.float64), torch.zeros(T, k, N, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if 0 <= e < G:
                v = (x[t, j] if x.dim() == 3 else x[t]).double()
                out[t, j], mag[t, j] = w[e] @ v, size[e] @ v.abs()
    if weights is None:
        return out, mag
    there = (ids >= 0) & (ids < G)
    r = torch.where(there, weights.double(), torch.zeros((), dtype=torch.float64))[..., None]
    return (out * r).sum(1), (mag * r.abs()).sum(1)


def factors(step, lr, betas, weight_decay):
    b1, b2 = betas
    return np.float32(1 - lr * weight_decay), np.float32(lr / (1 - b1 ** step)), np.float32(1 / math.sqrt(1 - b2 ** step))


def quantise_state(x, positive):
    """(codes float8_e4m3fn, scales float32) of a binary32 vector, in blocks of 256."""
    n = len(x)
    pad = np.zeros(-(-n // 256) * 256, np.float32)
    pad[:n] = x
    b = pad.reshape(-1, 256)
    bad = ~np.isfinite(b).all(1)
    b = np.where(bad[:, None], np.float32(0), b)
    top = np.abs(b).max(1)
    s = np.where(top > 0, np.maximum(top * np.float32(1 / 448), np.float32(2.0 ** -126)), np.float32(1)).astype(np.float32)
    t = b / s[:, None]
    assert t.dtype == np.float32
    if positive:
        t = np.where(b > 0, np.maximum(t, np.float32(2.0 ** -9)), t)
    t = np.clip(t, np.float32(-448), np.float32(448))
    codes = torch.from_numpy(t.reshape(-1)[:n].copy()).to(torch.float8_e4m3fn)
    return codes, torch.from_numpy(np.where(bad, np.float32(np.nan), s))


def widen_state(codes, scale):
    n = codes.numel()
    return codes.reshape(-1).float().numpy() * scale.numpy().repeat(256)[:n]


def adamw_f32(p, g, m, v, step, lr, betas, eps, weight_decay, grad_scale=None, root_of_v=None):
    """The step in binary32, every operation rounded: (p, m, v, sqrt v) as numpy
    float32.  root_of_v: sqrt(v) of an eight-bit state, in place of v."""
    f = np.float32
    decay, rate, unit = factors(step, lr, betas, weight_decay)
    b1, b2 = betas
    with np.errstate(all="ignore"):
        if grad_scale is not None:
            g = g * f(grad_scale)
        if root_of_v is not None:
            v = root_of_v * root_of_v
        m = m * f(b1) + g * f(1 - b1)
        v = v * f(b2) + (g * g) * f(1 - b2)
        root = np.sqrt(v)
        p = p * decay - rate * (m / (root * unit + f(eps)))
    assert p.dtype == m.dtype == v.dtype == root.dtype == np.float32
    return p, m, v, root


def adamw_f64(p, g, m, v, step, lr, betas, eps, weight_decay):
    b1, b2 = betas
    m = b1 * m.double() + (1 - b1) * g.double()
    v = b2 * v.double() + (1 - b2) * g.double() ** 2
    p = p.double() * (1 - lr * weight_decay) - lr * (m / (1 - b1 ** step)) / ((v / (1 - b2 ** step)).sqrt() + eps)
    return p, m, v
