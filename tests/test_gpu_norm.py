"""Group norm with an activation, channels last, against its definition in 64 bits.

Tolerances, from the arithmetic (float32 inside; u = 2^-24).  Sums of n values in
float32 runs of at most 128 and shuffles, then float64: 2^-17 of the absolute sum at
most.  So mean and 1/std are off by 2^-17 of (|x| + |mean|) / std at the largest x,
which enters y by |w|, and exp, reciprocal and the normal tail (1.5e-7 = 2^-22.7) add
2^-21: y within 2^-16 (|w| spread + |b| + 1) plus half a step, spread = max |x - 0| / std
of the row block and group.  dx likewise by the size of its terms; dw, db by 2^-16 of
their absolute sums times the spread.
"""
import pytest

pytestmark = pytest.mark.gpu

import torch  # noqa: E402

import semi_markov_crf_prefix_b200 as sc  # noqa: E402

TYPES = [torch.float32, torch.bfloat16, torch.float16]
# (N, S, C, G): registers (one and several rows), single positions, two passes, odd channels,
# one channel, one group, a group a channel, more columns than a block
SHAPES = [(3, 50, 17, 1), (2, 4000, 128, 8), (700, 1, 512, 8), (9, 1, 24, 3), (5, 3, 24, 3), (2, 3001, 20, 4),
          (1, 1, 1, 1), (1, 7, 2000, 2000), (2, 9, 4096, 4), (40, 33, 64, 64), (3, 700, 6, 2), (1, 70000, 8, 1)]


def act64(z, kind):
    if kind == "silu":
        return z * torch.sigmoid(z)
    if kind == "gelu":
        return 0.5 * z * torch.special.erfc(-z * 0.5 ** 0.5)
    return z


def definition(x, G, w, b, lengths, eps, kind):
    """(y, xh, spread) in float64; differentiable."""
    N, S, C = x.shape
    L = torch.full((N,), S, device=x.device) if lengths is None else lengths.long()
    ok = (torch.arange(S, device=x.device) < L[:, None])[:, :, None, None]
    u = torch.where(ok, x.view(N, S, G, C // G), 0.0)
    n = (L.double() * (C // G)).clamp_min(1)[:, None, None, None]
    mean = u.sum((1, 3), keepdim=True) / n
    d = torch.where(ok, u - mean, 0.0)
    std = torch.sqrt((d * d).sum((1, 3), keepdim=True) / n + eps)
    xh = d / std
    z = xh * w.view(G, -1) + b.view(G, -1)
    spread = (u.abs().amax((1, 3), keepdim=True) / std).detach().expand_as(u)
    return torch.where(ok, act64(z, kind), 0.0).reshape(N, S, C), xh.reshape(N, S, C), spread.reshape(N, S, C), std


def half_step(t):
    return torch.finfo(t).eps / 2


def check(x, G, w=None, b=None, lengths=None, eps=1e-5, kind="none", seed=2, dy=None):
    N, S, C = x.shape
    g = torch.Generator(device="cuda").manual_seed(seed)
    dy = torch.randn(N, S, C, generator=g, device="cuda").to(x.dtype) if dy is None else dy
    leaves = [x.clone().requires_grad_(True)] + [t.clone().requires_grad_(True) for t in (w, b) if t is not None]
    it = iter(leaves[1:])
    lw, lb = (next(it) if w is not None else None), (next(it) if b is not None else None)
    y = sc.group_norm(leaves[0], G, lw, lb, lengths=lengths, eps=eps, activation=kind)
    got = torch.autograd.grad(y, leaves, dy)
    x64 = torch.nan_to_num(x.double(), nan=0.0).requires_grad_(True)
    w64 = (torch.ones(C, device="cuda") if w is None else w).double().requires_grad_(True)
    b64 = (torch.zeros(C, device="cuda") if b is None else b).double().requires_grad_(True)
    ey, xh, spread, std = definition(x64, G, w64, b64, lengths, eps, kind)
    ex, ew, eb = torch.autograd.grad(ey, (x64, w64, b64), torch.nan_to_num(dy.double(), nan=0.0))
    # 1.2: the largest slope of the activations, rounded up
    zsize = w64.abs() * (spread + xh.abs()) + b64.abs() + 1
    e = 2.0 ** -16
    assert y.dtype == x.dtype
    assert torch.all((y.double() - ey).abs() <= 1.2 * e * zsize + half_step(x.dtype) * ey.abs() * 1.001 + 1e-7)
    d64 = torch.nan_to_num(dy.double(), nan=0.0).abs() * 1.2
    terms = (d64 * (w64.abs() + 1) * (1 + zsize)).view(N, S, G, -1)
    most = terms.amax((1, 3), keepdim=True) * (1 + xh.abs().view(N, S, G, -1)) * (1 + xh.abs().amax())
    bound = (e * most / std).reshape(N, S, C)
    assert torch.all((got[0].double() - ex).abs() <= bound + half_step(x.dtype) * ex.abs() * 1.001 + 1e-7)
    if w is not None:
        lim = e * (d64 * (1 + xh.abs()) * (1 + zsize)).sum((0, 1))
        assert got[1].dtype == w.dtype
        assert torch.all((got[1].double() - ew).abs() <= lim + half_step(w.dtype) * ew.abs() * 1.001)
    if b is not None:
        lim = e * (d64 * (1 + zsize)).sum((0, 1))
        assert torch.all((got[-1].double() - eb).abs() <= lim + half_step(b.dtype) * eb.abs() * 1.001)
    if lengths is not None:
        for n, L in enumerate(lengths.tolist()):
            assert torch.all(y[n, L:] == 0) and torch.all(got[0][n, L:] == 0)
    return y


def inputs(N, S, C, dtype, seed=0, shift=0.5, wtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(N, S, C, generator=g, device="cuda") + shift).to(dtype)
    w = (1 + 0.2 * torch.randn(C, generator=g, device="cuda")).to(wtype)
    b = (0.2 * torch.randn(C, generator=g, device="cuda")).to(wtype)
    return x, w, b


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
@pytest.mark.parametrize("shape", SHAPES)
def test_against_definition(shape, kind, dtype):
    N, S, C, G = shape
    x, w, b = inputs(N, S, C, dtype)
    check(x, G, w, b, kind=kind)


@pytest.mark.parametrize("shape", [(6, 300, 17, 1), (6, 3000, 64, 4), (6, 1, 64, 4), (6, 9000, 32, 8)])
@pytest.mark.parametrize("dtype", TYPES)
def test_lengths(shape, dtype):
    N, S, C, G = shape
    x, w, b = inputs(N, S, C, dtype)
    lengths = torch.tensor([0, 1, S, max(S - 1, 0), S // 2, min(2, S)], dtype=torch.int32, device="cuda")
    dy = torch.randn(N, S, C, device="cuda").to(dtype)
    for n, L in enumerate(lengths.tolist()):
        x[n, L:] = float("nan")       # not read
        dy[n, L:] = float("nan")
    check(x, G, w, b, lengths=lengths, kind="silu", dy=dy)


@pytest.mark.parametrize("shape", [(3, 50, 16, 2), (2, 4000, 64, 8), (300, 1, 64, 8)])
def test_weights(shape):
    N, S, C, G = shape
    x, w, b = inputs(N, S, C, torch.bfloat16, wtype=torch.bfloat16)
    check(x, G, w, b, kind="gelu")               # in x's type
    check(x, G, None, None, kind="silu")
    check(x, G, w, None)
    check(x, G, None, b)
    # neither asked for
    y = sc.group_norm(x.clone().requires_grad_(True), G, w, b)
    assert y.grad_fn is not None


@pytest.mark.parametrize("shape", [(2, 60, 32, 4), (2, 20000, 32, 4), (64, 1, 32, 4)])
def test_mean_far_from_zero_and_outliers(shape):
    N, S, C, G = shape
    x, w, b = inputs(N, S, C, torch.float32, shift=1e4)
    check(x, G, w, b)                            # the tolerance grows with |x| / std
    x, w, b = inputs(N, S, C, torch.float32)
    x[:, 0] = 1e4                                # the first row of every group
    check(x, G, w, b)
    x[:] = 3.0                                   # no variance at all
    y = sc.group_norm(x, G, w, b)
    assert torch.all(y == b)


def test_not_aligned():
    for C, G in ((64, 8), (24, 3), (16, 2)):
        for dtype in TYPES:
            x, w, b = inputs(4, 33, C, dtype)
            off = torch.empty(x.numel() + 1, dtype=dtype, device="cuda")[1:].view_as(x)
            off.copy_(x)
            assert not off.data_ptr() % 16 == 0
            check(off, G, w, b, kind="silu")


def test_more_axes_and_rows():
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(3, 5, 7, 24, generator=g, device="cuda")
    y = sc.group_norm(x, 4, activation="gelu")
    assert torch.equal(y, sc.group_norm(x.view(3, 35, 24), 4, activation="gelu").view_as(x))
    x = torch.randn(100, 24, generator=g, device="cuda")
    assert torch.equal(sc.group_norm(x, 4), sc.group_norm(x.view(100, 1, 24), 4).view(100, 24))
    x = torch.randn(70000, 2, 8, generator=g, device="cuda")      # more row blocks than a grid axis holds
    check(x, 2)


def test_gradient_against_differences():
    # central differences of the definition in float64 (h = 1e-6: off by h^2 and 1e-16 / h,
    # 1e-9 of the sums' size); the kernel's gradient in float32 by its own tolerance, 2^-12
    # of the absolute sum here
    for shape, G in (((2, 40, 12), 3), ((2, 3000, 12), 3), ((50, 1, 16), 2)):
        x, w, b = inputs(*shape, torch.float32)
        g = torch.Generator(device="cuda").manual_seed(6)
        dy = torch.randn(*shape, generator=g, device="cuda")
        leaves = [t.clone().requires_grad_(True) for t in (x, w, b)]
        y = sc.group_norm(leaves[0], G, leaves[1], leaves[2], activation="silu")
        for i, grad in enumerate(torch.autograd.grad(y, leaves, dy)):
            u = torch.randn(grad.shape, generator=g, device="cuda").double()
            value = []
            for h in (1e-6, -1e-6):
                t = [v.detach().double() for v in leaves]
                t[i] = t[i] + h * u
                value.append((definition(t[0], G, t[1], t[2], None, 1e-5, "silu")[0] * dy.double()).sum())
            slope = (value[0] - value[1]) / 2e-6
            terms = (grad.double() * u).abs().sum()
            assert abs((grad.double() * u).sum() - slope) <= 2.0 ** -12 * terms


def test_same_call_same_bits_stream_and_graph():
    for shape, G in (((3, 60, 32), 4), ((3, 6000, 32), 4), ((3000, 1, 32), 4)):
        x, w, b = inputs(*shape, torch.bfloat16)
        run = lambda t: sc.group_norm_forward(t, G, w, b, activation="silu")  # noqa: E731
        y, st = run(x)
        back = sc.group_norm_backward(x, x, st, G, w, b, activation="silu")
        y2, st2 = run(x)
        assert torch.equal(y, y2) and torch.equal(st, st2)
        assert all(torch.equal(a, c) for a, c in zip(back, sc.group_norm_backward(x, x, st, G, w, b, activation="silu")))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            y3, _ = run(x)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(y, y3)
        x2 = x.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y4, st4 = run(x2)
            back4 = sc.group_norm_backward(x2, x2, st4, G, w, b, activation="silu")
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y4) and all(torch.equal(a, c) for a, c in zip(back, back4))


def test_rows_past_32_bits():
    # 2^31 + 2^20 elements: the last row block lies behind 32-bit offsets
    C, S = 1 << 10, 1 << 15
    N = 64 + 1
    x = torch.zeros(N, S, C, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(8)
    x[-1] = torch.randn(S, C, generator=g, device="cuda").bfloat16()
    y = sc.group_norm(x, 4, activation="silu")
    assert torch.equal(y[-1:], sc.group_norm(x[-1:].clone(), 4, activation="silu")) or \
        (y[-1] - sc.group_norm(x[-1:].clone(), 4, activation="silu")[0]).abs().max() <= 2.0 ** -6
    assert torch.all(y[:-1] == 0)


def test_bad_lengths_are_reported():
    x, w, b = inputs(3, 40, 8, torch.float32)
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    lengths = torch.tensor([41, -1, 40], dtype=torch.int32, device="cuda")
    y, _ = sc.group_norm_forward(x, 2, w, b, lengths=lengths, ws=ws)
    assert sc.device_status(ws) == sc._lib.SEMICRF_ERR_INVALID_LENGTH
    assert torch.equal(y[0], sc.group_norm(x[:1], 2, w, b)[0]) and torch.all(y[1] == 0)


def test_second_derivatives_are_refused():
    x, w, b = inputs(2, 9, 8, torch.float32)
    x.requires_grad_(True)
    first = torch.autograd.grad(sc.group_norm(x, 2, w, b).square().sum(), x, create_graph=True)[0]
    with pytest.raises(RuntimeError):
        first.sum().backward()


def test_refusals():
    x, w, b = inputs(3, 40, 8, torch.bfloat16)
    f = sc.group_norm
    for bad in (lambda: f(x, 3), lambda: f(x, 0), lambda: f(x, 2, w[:4]), lambda: f(x.transpose(0, 1), 2),
                lambda: f(x, 2, activation="relu"), lambda: f(x[0, 0], 2), lambda: f(x[:0], 2),
                lambda: f(x[0], 2, lengths=torch.ones(40, dtype=torch.int32, device="cuda")),
                lambda: f(x, 2, lengths=torch.ones(2, dtype=torch.int32, device="cuda")), lambda: f(x, 2, eps=-1.0)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: f(x.double(), 2), lambda: f(x, 2, w.half()), lambda: f(x, 2, w, b.bfloat16()),
                lambda: f(x, 2, lengths=torch.ones(3, device="cuda"))):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(sc.SemiCRFError):
        sc.group_norm_forward(x, 2, ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))
