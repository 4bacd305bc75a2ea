"""AdamW over many tensors at once against the formula in 64 bits, states in 32 and 8 bits.

Tolerances: float32 states take three roundings of 2^-24 each; a parameter takes the
rounding of its own type, of lr, weight decay and the quotient (eight roundings at most
of the update).  Codes of 8-bit states are compared exactly, as the values they stand
for: the moments are formed in float64 on both sides, and inputs lie off the borders.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

import torch  # noqa: E402

import semi_markov_crf_prefix_b200 as sc  # noqa: E402

BLOCK = 256


def decode(codes, scale, second):
    """The values of codes, from the format's definition."""
    bias = 31 if second else 15
    out = []
    for c in range(256):
        mag = c if second else c & 127
        e, f = mag >> 3, mag & 7
        v = f / 8 * 2.0 ** (1 - bias) if e == 0 else (1 + f / 8) * 2.0 ** (e - bias)
        out.append(-v if not second and c & 128 else v)
    table = torch.tensor(out, dtype=torch.float64, device="cuda")
    flat = codes.reshape(-1).long()
    return (table[flat] * scale.double().repeat_interleave(BLOCK)[:flat.numel()]).view(codes.shape)


def nearest(x, second):
    """The values of x's codes: nearest in the table of all codes (inputs off the borders)."""
    flat = x.reshape(-1)
    n, pad = flat.numel(), -flat.numel() % BLOCK
    blocks = torch.nn.functional.pad(flat, (0, pad)).view(-1, BLOCK)
    scale = (blocks.abs().amax(1).float().double() / 1.875).float()
    every = torch.arange(256 if second else 128, dtype=torch.uint8, device="cuda")
    table = decode(every, torch.ones(1, device="cuda"), second)
    y = torch.where(scale[:, None] > 0, blocks.abs() / scale.double()[:, None], 0.0)
    at = torch.bucketize(y, (table[1:] + table[:-1]) / 2)
    if second:
        at = torch.where((blocks > 0) & (scale[:, None] > 0), at.clamp_min(1), at)
    return (table[at] * scale.double()[:, None] * blocks.sign()).reshape(-1)[:n].view(x.shape), scale


def formula(p, g, m, v, t, lr, b1, b2, eps, wd):
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    move = lr * (m / (1 - b1 ** t)) / (torch.sqrt(v / (1 - b2 ** t)) + eps)
    return p * (1 - lr * wd) - move, m, v, move


SIZES = [(1,), (7,), (255,), (256,), (257,), (64, 64), (4096,), (8193,), (3, 5, 11), (0,), (100_003,)]
KINDS = [(torch.float32, torch.float32), (torch.float32, torch.float64), (torch.bfloat16, torch.bfloat16),
         (torch.float16, torch.float16), (torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)]


def make(sizes, kinds, seed=0, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda s, t: (torch.randn(*s, generator=g, device="cuda", dtype=torch.float64)  # noqa: E731
                        * torch.exp(spread * torch.randn(*s, generator=g, device="cuda", dtype=torch.float64))).to(t)
    params, grads = [], []
    for i, s in enumerate(sizes):
        pt, gt = kinds[i % len(kinds)]
        params.append(rnd(s, pt))
        grads.append((rnd(s, torch.float64) * 1e-2).to(gt))
    return params, grads


def close(got, want, move, dtype, old):
    lim = (torch.finfo(dtype).eps / 2 * 1.001 * want.abs() + 8 * 2.0 ** -24 * (move.abs() + old.abs())
           + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps)
    return torch.all((got.double() - want).abs() <= lim)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("kinds", [KINDS, KINDS[:1], KINDS[2:3]])
def test_steps_against_formula(bits, kinds):
    params, grads = make(SIZES, kinds)
    m, v, ms, vs = sc.new_adamw_state(params, bits)
    hyper = dict(lr=3e-3, betas=(0.9, 0.99), eps=1e-6, weight_decay=0.1)
    for t in range(1, 5):
        old = [(p.double(), a.double() if bits == 32 else decode(a, s, False), c.double() if bits == 32 else decode(c, r, True))
               for p, a, c, s, r in zip(params, m, v, ms or m, vs or v)]
        sc.adamw_step(params, grads, m, v, t, exp_avg_scale=ms, exp_avg_sq_scale=vs, **hyper)
        got_m = m if bits == 32 else sc.adamw_state_values(m, ms, "exp_avg")
        got_v = v if bits == 32 else sc.adamw_state_values(v, vs, "exp_avg_sq")
        for i, (p, g) in enumerate(zip(params, grads)):
            ep, em, ev, move = formula(old[i][0], g.double(), old[i][1], old[i][2], t, hyper["lr"], 0.9, 0.99, 1e-6, 0.1)
            assert close(p, ep, move, p.dtype, old[i][0]), (t, i)
            if bits == 32:
                size = old[i][1].abs() * 0.9 + 0.1 * g.double().abs()
                assert torch.all((got_m[i].double() - em).abs() <= 3 * 2.0 ** -24 * size + 1e-44)
                assert torch.all((got_v[i].double() - ev).abs() <= 4 * 2.0 ** -24 * ev + 1e-44)
            elif p.numel():
                qm, sm = nearest(em, False)
                qv, sv = nearest(ev, True)
                assert torch.equal(ms[i], sm) and torch.equal(vs[i], sv)
                assert torch.equal(got_m[i], qm.float()) and torch.equal(got_v[i], qv.float())
                assert torch.equal(got_m[i].double(), decode(m[i], ms[i], False).float().double())
        # gradients of another size each time, so that codes move
        grads = [(g * (1.7 + i % 3)).to(g.dtype) for i, g in enumerate(grads)]


def test_small_values_in_8_bits():
    # a block that spans many magnitudes: nothing that is not zero reads as a second moment of zero
    p = [torch.zeros(512, device="cuda")]
    g = [torch.logspace(0, -20, 512, device="cuda")]
    g[0][5] = 0.0
    m, v, ms, vs = sc.new_adamw_state(p, 8)
    sc.adamw_step(p, g, m, v, 1, exp_avg_scale=ms, exp_avg_sq_scale=vs)
    got = sc.adamw_state_values(v, vs, "exp_avg_sq")[0]
    assert torch.all((got > 0) == (g[0].double() ** 2 * 0.001 > 0)) and got[5] == 0
    assert torch.all(torch.isfinite(p[0])) and p[0].abs().max() <= 1.01e-3
    # all zeros stay zeros, and the parameter only decays
    p = [torch.ones(300, device="cuda")]
    m, v, ms, vs = sc.new_adamw_state(p, 8)
    sc.adamw_step(p, [torch.zeros(300, device="cuda")], m, v, 1, lr=0.5, weight_decay=0.5, exp_avg_scale=ms, exp_avg_sq_scale=vs)
    assert not m[0].any() and not v[0].any() and torch.all(p[0] == 0.75)


@pytest.mark.parametrize("bits", [32, 8])
def test_not_finite_stays_in_its_place(bits):
    p, g = make([(700,), (300,)], KINDS[:1])
    want = [t.clone() for t in p]
    g[0][300] = float("inf")
    g[0][301] = float("nan")
    m, v, ms, vs = sc.new_adamw_state(p, bits)
    sc.adamw_step(p, g, m, v, 1, exp_avg_scale=ms, exp_avg_sq_scale=vs)
    bad = ~torch.isfinite(p[0])
    assert bad[300] and bad[301] and bad.sum() == 2 and torch.isfinite(p[1]).all()
    assert not torch.equal(p[1], want[1])
    if bits == 8:
        values = sc.adamw_state_values(m, ms, "exp_avg")[0]
        assert torch.isnan(values[256:512]).any() and torch.isfinite(values[:256]).all() and torch.isfinite(values[512:]).all()


def test_scale_step_and_rate_on_the_device():
    p, g = make(SIZES, KINDS)
    q = [t.clone() for t in p]
    a, b = sc.new_adamw_state(p), sc.new_adamw_state(q)
    step = torch.tensor(7, device="cuda")
    lr = torch.tensor(2e-3, device="cuda")
    sc.adamw_step(p, g, a[0], a[1], step, lr=lr, grad_scale=0.25)
    # (0.25 scales a float32 exactly; in float16 it would round the smallest values)
    sc.adamw_step(q, [t.float() * 0.25 for t in g], b[0], b[1], 7, lr=float(lr))
    assert all(torch.equal(x, y) for x, y in zip(p, q))
    assert all(torch.equal(x, y) for x, y in zip(a[0] + a[1], b[0] + b[1]))


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps_follow_the_counter(bits):
    p, g = make(SIZES, KINDS)
    q = [t.clone() for t in p]
    a, b = sc.new_adamw_state(p, bits), sc.new_adamw_state(q, bits)
    step, lr = torch.tensor(0, device="cuda"), torch.tensor(1e-3, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.add_(1)
        sc.adamw_step(p, g, a[0], a[1], step, lr=lr, exp_avg_scale=a[2], exp_avg_sq_scale=a[3])
    for t in range(1, 4):
        lr.fill_(1e-3 / t)
        graph.replay()
        sc.adamw_step(q, g, b[0], b[1], t, lr=float(torch.tensor(1e-3 / t)), exp_avg_scale=b[2], exp_avg_sq_scale=b[3])
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(p, q))
    for x, y in zip(a, b):
        assert x is None or all(torch.equal(s, t) for s, t in zip(x, y))


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors_and_odd_places(bits):
    # more tensors than one launch holds, in one buffer at every alignment
    g = torch.Generator(device="cuda").manual_seed(9)
    sizes = [int(n) for n in torch.randint(0, 700, (1000,), generator=torch.Generator().manual_seed(1))]
    flat = torch.randn(sum(sizes), generator=g, device="cuda")
    grad = torch.randn(sum(sizes), generator=g, device="cuda")
    p, gr = list(flat.clone().split(sizes)), list(grad.split(sizes))
    m, v, ms, vs = sc.new_adamw_state(p, bits)
    if bits == 32:       # states at every alignment too
        m, v = list(torch.zeros_like(flat).split(sizes)), list(torch.zeros_like(flat).split(sizes))
    else:
        m, v = (list(torch.zeros_like(flat, dtype=torch.uint8).split(sizes)) for _ in range(2))
    sc.adamw_step(p, gr, m, v, 1, exp_avg_scale=ms, exp_avg_sq_scale=vs)
    ep, _, _, move = formula(flat.double(), grad.double(), torch.zeros_like(flat, dtype=torch.float64),
                             torch.zeros_like(flat, dtype=torch.float64), 1, 1e-3, 0.9, 0.999, 1e-8, 0.01)
    assert close(torch.cat(p), ep, move, torch.float32, flat.double())


def test_overwritten_parameters_are_noticed():
    w = torch.randn(8, device="cuda", requires_grad=True)
    y = (w * w).sum()
    m, v, _, _ = sc.new_adamw_state([w])
    sc.adamw_step([w], [torch.ones(8, device="cuda")], m, v, 1)
    with pytest.raises(RuntimeError):
        y.backward()


def test_leaves_stay_leaves():
    # parameters as a model holds them, with gradients recorded around the call
    w = torch.randn(300, device="cuda", requires_grad=True)
    for bits in (32, 8):
        m, v, ms, vs = sc.new_adamw_state([w], bits)
        old = w.detach().clone()
        sc.adamw_step([w], [torch.ones_like(w)], m, v, 1, exp_avg_scale=ms, exp_avg_sq_scale=vs)
        assert w.is_leaf and w.requires_grad and not torch.equal(w, old)
        if bits == 8:
            assert not sc.adamw_state_values(m, ms, "exp_avg")[0].requires_grad


def test_refusals():
    p, g = make([(8, 4), (5,)], KINDS[:1])
    m, v, _, _ = sc.new_adamw_state(p)
    c, w, cs, ws = sc.new_adamw_state(p, 8)
    f = sc.adamw_step
    for bad in (lambda: f(p, g[:1], m, v, 1), lambda: f(p, [g[0].t(), g[1]], m, v, 1), lambda: f([p[0].t(), p[1]], g, m, v, 1),
                lambda: f(p, g, m[:1], v, 1), lambda: f(p, g, c, w, 1, exp_avg_scale=cs),
                lambda: f(p, g, c, w, 1, exp_avg_scale=cs, exp_avg_sq_scale=[ws[0], ws[1][:0]]),
                lambda: f([p[0], p[0]], [g[0], g[0]], [m[0], m[0]], [v[0], v[0]], 1),
                lambda: f([p[0], p[1]], [g[0].reshape(4, 8), g[1]], m, v, 1)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: f(p, g, c, w, 1), lambda: f(p, g, m, v, 1, exp_avg_scale=cs, exp_avg_sq_scale=ws),
                lambda: f([t.double() for t in p], g, m, v, 1), lambda: f(p, [t.int() for t in g], m, v, 1),
                lambda: f(p, g, m, v, torch.tensor(1.0, device="cuda")),
                lambda: f(p, g, m, v, 1, lr=torch.tensor(1e-3, dtype=torch.float64, device="cuda")),
                lambda: f(p, g, m, v, torch.tensor(1))):
        with pytest.raises(TypeError):
            bad()
    for kw in (dict(betas=(1.0, 0.9)), dict(eps=-1.0), dict(lr=math.nan), dict(weight_decay=-0.1)):
        with pytest.raises(sc.SemiCRFError):
            f(p, g, m, v, 1, **kw)
    with pytest.raises(sc.SemiCRFError):
        f(p, g, m, v, 0)
