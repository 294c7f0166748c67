"""Plain 64-bit forms of the operators of include/gmm_moe.h, for the tests
(CPU tensors in, numpy or float64 tensors out)."""
import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E2M1 = np.concatenate([E2M1, -E2M1])


def sort_tokens(ids, G):
    """(group_sizes int32 [G], slot_row int32 of ids' shape)."""
    flat = ids.reshape(-1).tolist()
    keys = [e if 0 <= e < G else G for e in flat]
    sizes = [0] * (G + 1)
    for e in keys:
        sizes[e] += 1
    at = [0] * (G + 1)
    for g in range(G):
        at[g + 1] = at[g] + sizes[g]
    out = []
    for e in keys:
        out.append(at[e] if e < G else ~at[e])
        at[e] += 1
    return (torch.tensor(sizes[:G], dtype=torch.int32),
            torch.tensor(out, dtype=torch.int32).reshape(ids.shape))


def dispatch(x, slot_row):
    T, k = slot_row.shape
    out = torch.full((T * k, x.shape[1]), -77.0).to(x.dtype)
    for t in range(T):
        for j in range(k):
            r = int(slot_row[t, j])
            out[r if r >= 0 else ~r] = x[t] if r >= 0 else torch.zeros_like(x[t])
    return out


def _split(slot_row):
    routed = slot_row >= 0
    return torch.where(routed, slot_row, ~slot_row).long(), routed


def combine(rows, slot_row, weights=None):
    """(out float64 [T,D], the sum of the absolute terms)."""
    row, routed = _split(slot_row)
    w = torch.ones(slot_row.shape, dtype=torch.float64) if weights is None else weights.double()
    terms = torch.where(routed[..., None], rows.double()[row] * w[..., None], torch.zeros((), dtype=torch.float64))
    return terms.sum(1), terms.abs().sum(1)


def combine_grad(dout, rows, slot_row, weights):
    """(drows float64 [T*k,D], dweights float64 [T,k], the latter's sum of absolute terms)."""
    row, routed = _split(slot_row)
    zero = torch.zeros((), dtype=torch.float64)
    d = dout.double()[:, None, :]
    drows = torch.full(rows.shape, float("nan"), dtype=torch.float64)
    drows[row.flatten()] = torch.where(routed[..., None], d * weights.double()[..., None], zero).reshape(-1, rows.shape[1])
    terms = torch.where(routed[..., None], d * rows.double()[row], zero)
    return drows, terms.sum(-1), terms.abs().sum(-1)


def quant_mxfp4(x):
    """(codes uint8 [...,K], scale bytes uint8 [...,K/32]) of x [...,K], by the
    definition: nearest of the sixteen values, ties to the even code."""
    a = x.double().numpy().reshape(x.shape[:-1] + (-1, 32))
    finite = np.isfinite(a).all(-1)
    amax = np.where(finite, np.abs(np.where(np.isfinite(a), a, 0)).max(-1), 0.0)
    _, e = np.frexp(amax)
    E = np.where(amax > 0, np.clip(e - 1 - 2, -127, 125), 0)
    byte = np.where(finite, E + 127, 255)
    t = np.ldexp(np.where(finite[..., None], a, 0.0), -E[..., None])
    mag = np.minimum(np.abs(t), 6.0)
    dist = np.abs(mag[..., None] - E2M1[:8])
    best = dist.min(-1, keepdims=True)
    # at a tie the two nearest are neighbours, and one of them is even
    code = np.where((dist == best)[..., ::2].any(-1), 2 * (dist == best)[..., ::2].argmax(-1), dist.argmin(-1))
    code = code + 8 * (np.signbit(t) & finite[..., None])
    return torch.from_numpy(code.reshape(x.shape).astype(np.uint8)), torch.from_numpy(byte.astype(np.uint8))


def pack(codes):
    return codes[..., 0::2] | codes[..., 1::2] << 4


def unpack(q):
    return torch.stack((q & 15, q >> 4), -1).reshape(q.shape[:-1] + (2 * q.shape[-1],))


def values(codes, byte):
    """float64 values of codes [...,K] under scale bytes [...,K/32] (NaN for byte 255)."""
    v = torch.from_numpy(E2M1)[codes.long()].reshape(byte.shape + (32,))
    unit = torch.exp2(byte.double() - 127)
    unit = torch.where(byte == 255, torch.full_like(unit, float("nan")), unit)
    return (v * unit[..., None]).reshape(codes.shape)


def rhs_layout(byte):
    """[Ga,N,nb] -> the weight layout [Ga,nb,1,N]."""
    return byte.transpose(1, 2).unsqueeze(2).contiguous()


def within(got, want, slack, what):
    """|got - want| <= slack elementwise (NaN and infinities refused)."""
    d = (got.double() - want).abs()
    bad = ~(d <= slack)
    assert not bool(bad.any()), (what, int(bad.sum()), float(d.max()), bad.nonzero()[0].tolist())


def half_step(t, value):
    """Half a rounding step of type t around value (subnormals included)."""
    f = torch.finfo(t)
    return value.abs() * (f.eps / 2) + f.tiny * f.eps / 2
