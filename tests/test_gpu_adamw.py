"""GPU parity of the AdamW step (include/gmm_layer.h, gmm_adamw_run): bit for
bit against the formula in binary32 with every operation rounded (numpy), and
against the formula in 64 bits."""
import math

import numpy as np
import pytest
import torch

import layer_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16, E4 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
HYPER = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
SHAPES = [(1,), (2,), (3,), (4,), (5,), (255,), (256,), (257,), (37, 11), (4095,), (4096,), (4097,), (3, 5, 7, 11), (8, 64, 96), (1,), (70001,)]


def _same(a, b, what):
    """Equal bits, NaN to NaN."""
    a, b = np.asarray(a), np.asarray(b)
    same = (a.view(np.uint32) == b.view(np.uint32)) | (np.isnan(a) & np.isnan(b))
    assert same.all(), (what, int((~same).sum()), np.nonzero(~same)[0][:4], a[~same][:4], b[~same][:4])


def _tensors(shapes, seed, pd, gd, eight):
    g = torch.Generator().manual_seed(seed)
    made = []
    for shape in shapes:
        n = math.prod(shape)
        p = (torch.randn(shape, generator=g) * 0.05).to(pd)
        grad = (torch.randn(shape, generator=g) * 10.0 ** float(torch.randint(-6, 1, (), generator=g))).to(gd)
        grad.view(-1)[torch.rand(n, generator=g) < 0.2] = 0
        m = torch.randn(n, generator=g).numpy() * np.float32(1e-3)
        v = (torch.randn(n, generator=g).numpy() * np.float32(1e-3)) ** 2
        v[::3] = 0
        t = dict(p=p, g=grad)
        if eight:
            t["m"], t["ms"] = ref.quantise_state(m, False)
            t["v"], t["vs"] = ref.quantise_state(np.sqrt(v), True)
        else:
            t["m"], t["v"] = torch.from_numpy(m), torch.from_numpy(v)
        t["m"], t["v"] = t["m"].reshape(shape), t["v"].reshape(shape)
        made.append(t)
    return made


def _call(m, ts, step, copies=False, **kw):
    """The step on device copies of ts; returns them (with copies as "c")."""
    dev = [{n: x.cuda() for n, x in t.items()} for t in ts]
    if copies:
        for t in dev:
            t["c"] = torch.full(t["p"].shape, 7.0, dtype=BF16, device="cuda")
    col = lambda n: [t[n] for t in dev] if n in dev[0] else None  # noqa: E731
    m.adamw(col("p"), col("g"), col("m"), col("v"), step, exp_avg_scale=col("ms"), exp_avg_sq_scale=col("vs"), copies=col("c"), **kw)
    return dev


def _compare(ts, dev, step, lr, betas, eps, weight_decay, grad_scale=None):
    for i, (t, d) in enumerate(zip(ts, dev)):
        p, g = (t[n].reshape(-1).float().numpy() for n in ("p", "g"))
        eight = "ms" in t
        if eight:
            m0, v0, root = ref.widen_state(t["m"], t["ms"]), None, ref.widen_state(t["v"], t["vs"])
        else:
            m0, v0, root = t["m"].reshape(-1).numpy(), t["v"].reshape(-1).numpy(), None
        p, m, v, r = ref.adamw_f32(p, g, m0, v0, step, lr, betas, eps, weight_decay, grad_scale, root)
        got = {n: x.cpu().reshape(-1) for n, x in d.items()}
        want = torch.from_numpy(p).to(t["p"].dtype).float().numpy()
        _same(got["p"].float().numpy(), want, ("p", i))
        if "c" in got:
            _same(got["c"].float().numpy(), torch.from_numpy(p).to(BF16).float().numpy(), ("c", i))
        if eight:
            for name, x, positive in (("m", m, False), ("v", r, True)):
                codes, scale = ref.quantise_state(x, positive)
                _same(got[name + "s"].numpy(), scale.numpy(), (name + "s", i))
                ok = ~np.isnan(scale.numpy()).repeat(256)[:len(x)]
                assert np.array_equal(got[name].view(torch.uint8).numpy()[ok], codes.view(torch.uint8).numpy()[ok]), (name, i)
        else:
            _same(got["m"].numpy(), m, ("m", i))
            _same(got["v"].numpy(), v, ("v", i))


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("pd,gd,copies", [(F32, F32, False), (F32, BF16, True), (BF16, BF16, False), (BF16, F32, True)])
def test_step(pd, gd, copies, eight):
    import moe_grouped_matrix_amd as m
    for step in (1, 2, 1000):
        ts = _tensors(SHAPES, step, pd, gd, eight)
        _compare(ts, _call(m, ts, step, copies, **HYPER), step, **HYPER)


@pytest.mark.parametrize("eight", [False, True])
def test_many_tensors(eight):
    """More tensors than a launch takes, empty ones among them."""
    import moe_grouped_matrix_amd as m
    shapes = [((i * 37) % 700,) for i in range(131)] + [(0, 5)]
    ts = _tensors(shapes, 3, F32, F32, eight)
    _compare(ts, _call(m, ts, 7, True, **HYPER), 7, **HYPER)


def test_hyperparameters():
    import moe_grouped_matrix_amd as m
    ts = _tensors([(1000,)], 4, F32, F32, False)
    for kw in (dict(lr=0.0), dict(betas=(0.0, 0.0)), dict(weight_decay=0.0), dict(eps=1.0), dict(betas=(0.99, 0.999999), lr=100.0)):
        h = dict(HYPER, **kw)
        _compare(ts, _call(m, ts, 12345, **h), 12345, **h)


@pytest.mark.parametrize("eight", [False, True])
def test_against_the_formula_in_64_bits(eight):
    """m: three roundings (u of each term, 2u of the sum), v: five; the step is
    lr times a quotient whose denominator is within some 8 u of itself, and p
    two roundings more."""
    import moe_grouped_matrix_amd as m
    u = 2.0 ** -24
    t, = ts = _tensors([(20000,)], 5, F32, F32, eight)
    d, = _call(m, ts, 10, **HYPER)
    if eight:
        m0, v0 = torch.from_numpy(ref.widen_state(t["m"], t["ms"])), torch.from_numpy(ref.widen_state(t["v"], t["vs"])).double() ** 2
    else:
        m0, v0 = t["m"], t["v"]
    p, mm, vv = ref.adamw_f64(t["p"], t["g"], m0, v0, 10, **HYPER)
    moved = HYPER["lr"] * (0.9 * m0.double().abs() + 0.1 * t["g"].double().abs()) / (1 - 0.9 ** 10) / ((vv / (1 - 0.95 ** 10)).sqrt() + 1e-8)
    slack = 4 * u * t["p"].double().abs() + 16 * u * moved + 1e-30
    assert bool(((d["p"].cpu().double() - p).abs() <= slack).all())
    if not eight:
        assert bool(((d["m"].cpu().double() - mm).abs() <= 4 * u * (m0.double().abs() + t["g"].double().abs())).all())
        assert bool(((d["v"].cpu().double() - vv).abs() <= 8 * u * vv + 1e-44).all())


def test_states_that_end_and_begin():
    """Zero states with scales of 1 begin; tiny and huge values, an infinity
    and a NaN of one block; a positive v never turns to code 0."""
    import moe_grouped_matrix_amd as m
    n = 256 * 6 + 5
    t = dict(p=torch.zeros(n), g=torch.randn(n, generator=torch.Generator().manual_seed(0)),
             m=torch.zeros(n).to(E4), v=torch.zeros(n).to(E4), ms=torch.ones(7), vs=torch.ones(7))
    t["g"][256:512] = 0
    t["g"][512:768] *= 1e-38
    t["g"][768:1024] *= 1e18
    t["g"][1030] = math.inf
    t["g"][1290] = math.nan
    t["g"][3] = 1e6  # the others of its block are far below it
    d, = dev = _call(m, [t], 1, **HYPER)
    _compare([t], dev, 1, **HYPER)
    v, vs, ms = d["v"].cpu().float(), d["vs"].cpu(), d["ms"].cpu()
    assert bool((v[:256] > 0).all()) and not bool(v[256:512].any()) and float(vs[1]) == 1 == float(ms[1])
    assert vs.isnan().tolist() == ms.isnan().tolist() == [False] * 4 + [True, True, False]
    assert not bool(d["v"].cpu().view(torch.uint8)[1024:1536].any())


def test_step_rate_and_scale_on_the_device():
    """Read when the step runs: a captured step, replayed, goes on counting; and
    it gives what numbers on the host give, bit for bit."""
    import moe_grouped_matrix_amd as m
    ts = _tensors([(300,), (5000,)], 6, F32, BF16, True)
    a, b = ([{n: x.cuda() for n, x in t.items()} for t in ts] for _ in range(2))
    cols = lambda dev: [[t[n] for t in dev] for n in ("p", "g", "m", "v")]  # noqa: E731
    more = lambda dev: dict(exp_avg_scale=[t["ms"] for t in dev], exp_avg_sq_scale=[t["vs"] for t in dev])  # noqa: E731
    step = torch.tensor([5], dtype=torch.int32, device="cuda")
    lr, gs = torch.tensor([1e-3], device="cuda"), torch.tensor([0.5], device="cuda")
    rest = dict(betas=(0.9, 0.99), eps=1e-8, weight_decay=0.01)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.adamw(*cols(a), step, lr=lr, grad_scale=gs, **more(a), **rest)
        step += 1
    for i in range(4):
        lr.fill_(1e-3 * (i + 1))
        gs.fill_(0.5 + i)
        for x, y in zip(a, b):
            x["g"].normal_()
            y["g"].copy_(x["g"])
        graph.replay()
        m.adamw(*cols(b), 5 + i, lr=float(lr), grad_scale=gs.clone(), **more(b), **rest)
        for x, y in zip(a, b):
            for name in x:
                assert torch.equal(x[name].view(torch.uint8), y[name].view(torch.uint8)), (i, name)


def test_rows_of_a_buffer_are_left_alone():
    """What lies behind a tensor's last element stays as it was."""
    import moe_grouped_matrix_amd as m
    for eight in (False, True):
        n = 1021
        buf = {k: torch.full((1100,), 3.0, device="cuda") for k in ("p", "g")}
        st = {k: torch.full((1100,), 2.0, device="cuda").to(E4 if eight else F32) for k in ("m", "v")}
        sc = {k: torch.full((8,), 0.5, device="cuda") for k in ("ms", "vs")}
        cp = torch.full((1100,), 9.0, dtype=BF16, device="cuda")
        kw = dict(exp_avg_scale=[sc["ms"][:4]], exp_avg_sq_scale=[sc["vs"][:4]]) if eight else {}
        m.adamw([buf["p"][:n]], [buf["g"][:n]], [st["m"][:n]], [st["v"][:n]], 1, lr=0.1, copies=[cp[:n]], **kw)
        assert bool((buf["p"][n:] == 3).all()) and bool((buf["p"][:n] != 3).all()) and bool((cp[n:] == 9).all())
        assert all(bool((t.float()[n:] == 2).all()) for t in st.values()) and all(bool((t[4:] == 0.5).all()) for t in sc.values())


def test_lazy_copies_become_their_own():
    """A step on lazy copies leaves what they were copied from as it was."""
    import moe_grouped_matrix_amd as m
    old = [torch.full((300,), v, device="cuda") for v in (3.0, 0.5, 0.25)]
    p, a, v = (torch._lazy_clone(t) for t in old)
    m.adamw([p], [torch.ones(300, device="cuda")], [a], [v], 1, lr=0.1)
    assert bool((p != 3).all()) and [t.unique().tolist() for t in old] == [[3.0], [0.5], [0.25]]


def test_offsets_past_32_bits():
    """A tensor of 2^32 + 1000 weights with eight-bit states: its first and last
    elements step like a tensor of their own (they lie in blocks of their own)."""
    import moe_grouped_matrix_amd as m
    n = 2 ** 32 + 1000
    blocks = -(-n // 256)
    big = dict(p=torch.zeros(n, dtype=BF16, device="cuda"), g=torch.zeros(n, dtype=BF16, device="cuda"),
               m=torch.zeros(n, dtype=torch.uint8, device="cuda").view(E4), v=torch.zeros(n, dtype=torch.uint8, device="cuda").view(E4),
               ms=torch.ones(blocks, device="cuda"), vs=torch.ones(blocks, device="cuda"))
    t, = _tensors([(1000,)], 8, BF16, BF16, True)
    for lo in (0, 2 ** 32):
        for name in ("p", "g"):
            big[name][lo:lo + 1000] = t[name].cuda()
        for name in ("m", "v"):
            big[name].view(torch.uint8)[lo:lo + 1000] = t[name].view(torch.uint8).cuda()
        for name in ("ms", "vs"):
            big[name][lo // 256:lo // 256 + 4] = t[name].cuda()
    m.adamw([big["p"]], [big["g"]], [big["m"]], [big["v"]], 3, exp_avg_scale=[big["ms"]], exp_avg_sq_scale=[big["vs"]], **HYPER)
    for lo in (0, 2 ** 32):
        d = {name: big[name][lo:lo + 1000].contiguous() for name in ("p", "m", "v")}
        d.update({name: big[name][lo // 256:lo // 256 + 4].contiguous() for name in ("ms", "vs")})
        _compare([t], [d], 3, **HYPER)


def test_a_thousand_steps_of_one_tensor():
    """The device's factors (powers by squaring in double) are the host's, for
    steps up to the largest."""
    import moe_grouped_matrix_amd as m
    ts = _tensors([(300,)], 9, F32, F32, False)
    for step in (1, 2, 3, 10, 255, 256, 1000, 123457, 2 ** 31 - 1):
        at = torch.tensor([step], dtype=torch.int32, device="cuda")
        a, b = _call(m, ts, step, **HYPER), _call(m, ts, at, **HYPER)
        for name in ("p", "m", "v"):
            assert torch.equal(a[0][name], b[0][name]), (step, name)
    a, b = _call(m, ts, 1, **HYPER), _call(m, ts, torch.tensor([0], dtype=torch.int32, device="cuda"), **HYPER)
    assert torch.equal(a[0]["p"], b[0]["p"])  # (a step below 1 counts as 1)
