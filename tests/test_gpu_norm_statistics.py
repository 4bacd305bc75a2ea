"""The statistics of group norm on values that are hard for them.

Where rows do not fit a thread block's registers, means and squares about them come from
runs of at most 128 values in float32, eight at a time: of a batch's squares, about the mean
of the values before it, at least half stays in the sum, so its ten roundings of 2^-24 count
twice, and sixteen batches are added: 36 roundings, below 2^-18.8 of the sum of squares;
behind that float64.  So 1/std is right to 2^-19.8 and its rounding, and a mean to 2^-20 of a
run's range.  y takes four roundings of 2^-24 more.
"""
import pytest

pytestmark = pytest.mark.gpu

import torch  # noqa: E402

import semi_markov_crf_prefix_b200 as sc  # noqa: E402
from test_gpu_norm import check  # noqa: E402


def rnd(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def exact(x, G, w, b, eps=1e-5):
    N, S, C = x.shape
    u = x.double().view(N, S, G, C // G)
    mean = u.mean((1, 3), keepdim=True)
    d = u - mean
    rstd = torch.rsqrt((d * d).mean((1, 3), keepdim=True) + eps)
    xh = (d * rstd).view(N, S, C)
    return xh * w.double() + b.double(), xh, mean.view(N, G), rstd.view(N, G)


# (the last one: 128 values a run)
@pytest.mark.parametrize("shape,groups", [((2, 20000, 32), 4), ((1, 5000, 64), 64), ((3, 9000, 6), 1), ((1, 3001, 20), 4),
                                          ((1184, 128, 520), 2)])
@pytest.mark.parametrize("outlier", [10.0, -1e3, 1e5])
@pytest.mark.parametrize("rows", [1, 4, 8])
def test_outliers_at_the_start(shape, groups, outlier, rows):
    x, w, b = rnd(1, *shape), 1 + 0.2 * rnd(2, shape[2]), 0.2 * rnd(3, shape[2])
    x[:, :rows] = outlier
    y, stats = sc.group_norm_forward(x, groups, w, b)
    want, xh, mean, rstd = exact(x, groups, w, b)
    assert torch.all((stats[..., 1].double() / rstd - 1).abs() <= 2.0 ** -19.8 + 2.0 ** -23)
    # a run's range is |outlier| + 10 and at most 128 of S values are in it
    run = 2.0 ** -20 * (abs(outlier) + 10) * min(1.0, 128 * max(1, 256 // shape[2]) / shape[1])
    assert torch.all((stats[..., 0].double() - mean).abs() <= run + 2.0 ** -23 * mean.abs())
    off = (run * rstd.amax() + (2.0 ** -19.8 + 2.0 ** -23) * xh.abs() + 4 * 2.0 ** -24 * xh.abs()) * w.double().abs() + 2.0 ** -24 * want.abs()
    off = off + 2.0 ** -23 * (mean.abs() * rstd).amax() * w.double().abs()
    assert torch.all((y.double() - want).abs() <= off)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape,groups", [((2, 20000, 32), 4), ((1, 7001, 33), 3)])
def test_deviations_of_shifted_values(shape, groups, dtype):
    # a mean of 1e6 deviations
    x = (rnd(4, *shape) + (1e6 if dtype == torch.float32 else 100.0)).to(dtype)
    _, stats = sc.group_norm_forward(x, groups)
    _, _, mean, rstd = exact(x, groups, torch.ones(shape[2], device="cuda"), torch.zeros(shape[2], device="cuda"))
    assert torch.all((stats[..., 1].double() / rstd - 1).abs() <= 2.0 ** -19.8 + 2.0 ** -23)
    assert torch.all((stats[..., 0].double() / mean - 1).abs() <= 2.0 ** -23)


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("shape,groups", [((2, 9000, 16), 4), ((2, 30, 16), 4), ((2, 1, 16), 4)])
def test_values_that_are_not_finite(shape, groups, value):
    # the statistics of their row block and group are NaN, and so is all of it
    x = rnd(5, *shape)
    for at in (0, shape[1] // 2, shape[1] - 1):
        t = x.clone()
        t[1, at, 5] = value
        y = sc.group_norm(t, groups)
        assert torch.isnan(y[1, :, 4:8]).all()
        y[1, :, 4:8] = 0
        assert torch.isfinite(y).all()


@pytest.mark.parametrize("shape,groups", [((9001, 1, 520), 8), ((9000, 2, 1030), 2), ((300, 3, 40000), 4), ((1000, 2, 8200), 1),
                                          ((700, 1, 8001), 9), ((90, 30, 2400), 400)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ragged", [False, True])
def test_many_wide_row_blocks(shape, groups, dtype, ragged):
    # rows in slices of groups, and more row blocks than one piece of scratch holds; against 64
    # bits, and some of them alone
    N, S, C = shape
    x, w, b, dy = rnd(6, *shape).add_(0.3).to(dtype), 1 + 0.2 * rnd(7, C), 0.2 * rnd(8, C), rnd(9, *shape).to(dtype)
    lengths = torch.arange(N, device="cuda", dtype=torch.int32).remainder_(S + 1) if ragged else None
    check(x, groups, w, b, lengths=lengths, kind="silu", dy=dy)
    y, stats = sc.group_norm_forward(x, groups, w, b, lengths=lengths, activation="silu")
    dx, dw, db = sc.group_norm_backward(dy, x, stats, groups, w, b, lengths=lengths, activation="silu")
    for at in (slice(0, 100), slice(N // 2 - 7, N // 2 + 93), slice(N - 100, N)):
        some = None if lengths is None else lengths[at].clone()
        t, st = sc.group_norm_forward(x[at].clone(), groups, w, b, lengths=some, activation="silu")
        assert torch.all((t.double() - y[at].double()).abs() <= 2.0 ** -7 * t.double().abs() + 1e-5)
        u, _, _ = sc.group_norm_backward(dy[at].clone(), x[at].clone(), st, groups, w, b, lengths=some, activation="silu")
        assert torch.all((u.double() - dx[at].double()).abs() <= 2.0 ** -7 * u.double().abs() + 1e-5 * u.abs().max())
    again = sc.group_norm_backward(dy, x, stats, groups, w, b, lengths=lengths, activation="silu")
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw) and torch.equal(again[2], db)


@pytest.mark.parametrize("shape,groups", [((2, 4000, 128), 8), ((1, 70000, 8), 1), ((2, 3001, 20), 4), ((1, 9000, 1040), 1),
                                          ((3, 50, 16), 2), ((4, 9, 2000), 5), ((700, 1, 512), 8)])
@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_every_term_of_the_gradient(shape, groups, kind, dtype):
    # an upstream gradient with a mean and a part along xh, so that both means that dx takes
    # away are as large as what stays, against bounds made of dx's own terms: xh, z and the
    # slopes to 2^-20 of their parts, means to 2^-17 of the absolute mean (float32 runs of 128)
    N, S, C = shape
    x, w, b = rnd(10, *shape).to(dtype), 1 + 0.2 * rnd(11, C), 0.2 * rnd(12, C)
    grp = lambda t: t.view(N, S, groups, C // groups)  # noqa: E731
    mean_of = lambda t: grp(t).mean((1, 3), keepdim=True).expand(N, S, groups, C // groups).reshape(N, S, C)  # noqa: E731
    x64, w64, b64 = x.double(), w.double(), b.double()
    d = x64 - mean_of(x64)
    rstd = torch.rsqrt(mean_of(d * d) + 1e-5)
    xh = d * rstd
    z = xh * w64 + b64
    dy = (1.0 + 0.8 * xh + 0.5 * rnd(13, *shape)).to(dtype)
    if kind == "silu":
        slope = torch.sigmoid(z) * (1 + z * (1 - torch.sigmoid(z)))
    elif kind == "gelu":
        slope = 0.5 * torch.special.erfc(-z * 0.5 ** 0.5) + z * torch.exp(-z * z / 2) * 0.3989422804014327
    else:
        slope = torch.ones_like(z)
    dz = dy.double() * slope
    g = dz * w64
    m1, m2 = mean_of(g), mean_of(g * xh)
    want = rstd * (g - m1 - xh * m2)
    leaves = [t.clone().requires_grad_(True) for t in (x, w, b)]
    y = sc.group_norm(leaves[0], groups, leaves[1], leaves[2], activation=kind)
    dx, dw, db = torch.autograd.grad(y, leaves, dy)
    u = 2.0 ** -20
    ez = dy.double().abs() * u * (1 + (w64 * xh).abs() + w64.abs() + b64.abs())      # of dz
    e1 = mean_of(w64.abs() * ez) + 2.0 ** -17 * mean_of(g.abs())
    e2 = mean_of((w64 * xh).abs() * ez) + 2.0 ** -17 * mean_of((g * xh).abs())
    step = torch.finfo(dtype).eps / 2 * 1.001
    bound = rstd * (w64.abs() * ez + e1 + xh.abs() * e2 + u * (g.abs() + m1.abs() + (xh * m2).abs())) + step * want.abs()
    assert torch.all((dx.double() - want).abs() <= bound)
    # either mean left out would be far outside
    if S * (C // groups) > 8:
        assert ((rstd * m1).abs() > 2 * bound).double().mean() > 0.9
        assert ((rstd * xh * m2).abs() > 2 * bound).double().mean() > 0.7
    flat = lambda t: t.abs().sum((0, 1))  # noqa: E731
    assert torch.all((dw.double() - (dz * xh).sum((0, 1))).abs() <= 2.0 ** -17 * flat(dz * xh) + flat(ez * (1 + xh.abs())))
    assert torch.all((db.double() - dz.sum((0, 1))).abs() <= 2.0 ** -17 * flat(dz) + flat(ez))


@pytest.mark.parametrize("shape,groups", [((2, 9000, 16), 4), ((2, 30, 16), 4), ((3, 1, 512), 8), ((2, 2, 8200), 1), ((1184, 128, 520), 2)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_lowest_value_of_the_type(shape, groups, dtype):
    # its square passes float32: an infinite variance, not a NaN
    N, S, C = shape
    per = C // groups
    for at in {0, min(5, S - 1), S - 1}:
        x, b = rnd(14, *shape).to(dtype), rnd(15, C)
        x[-1, at, per + 1 if groups > 1 else 3] = torch.finfo(dtype).min
        y = sc.group_norm(x, groups, None, b)
        some = slice(per, 2 * per) if groups > 1 else slice(0, per)
        assert torch.equal(y[-1, :, some], b.to(dtype)[some].expand(S, per))
        assert torch.isfinite(y).all()


@pytest.mark.parametrize("value", [3.0, -1e30, 1e-30, 2e38])
@pytest.mark.parametrize("shape,groups", [((2, 9000, 16), 4), ((1184, 128, 520), 2)])
def test_constants(shape, groups, value):
    b = rnd(16, shape[2])
    y = sc.group_norm(torch.full(shape, value, device="cuda"), groups, None, b)
    assert torch.equal(y, b.expand(shape))
