"""AdamW's states where they leave the ordinary range: blocks of 8-bit codes with values that
are not finite or pass float32."""
import pytest

pytestmark = pytest.mark.gpu

import torch  # noqa: E402

import semi_markov_crf_prefix_b200 as sc  # noqa: E402


@pytest.mark.parametrize("dtype,value", [(torch.float32, 1e21), (torch.bfloat16, 1e21), (torch.float64, 1e25),
                                         (torch.float32, float("inf")), (torch.float32, -float("inf")),
                                         (torch.float32, float("nan")), (torch.float64, 1e300)])
def test_a_block_that_overflows_reads_as_nan(dtype, value):
    gen = torch.Generator(device="cuda").manual_seed(3)
    p = [torch.randn(1000, generator=gen, device="cuda")]
    g = (torch.randn(1000, generator=gen, device="cuda") * 1e-2).to(dtype)
    g[300] = value                     # in the second block of 256
    m, v, ms, vs = sc.new_adamw_state(p, 8)
    inside = torch.zeros(1000, dtype=torch.bool, device="cuda")
    inside[256:512] = True
    sc.adamw_step(p, [g], m, v, 1, exp_avg_scale=ms, exp_avg_sq_scale=vs)
    second = sc.adamw_state_values(v, vs, "exp_avg_sq")[0]
    assert torch.equal(torch.isnan(second), inside) and torch.isfinite(second[~inside]).all()
    first = sc.adamw_state_values(m, ms, "exp_avg")[0]
    # the first moment passes float32 only where 0.1 of the gradient does
    if abs(0.1 * value) < torch.finfo(torch.float32).max:
        assert torch.isfinite(first).all()
    else:
        assert torch.equal(torch.isnan(first), inside) and torch.isfinite(first[~inside]).all()
    # ordinary gradients afterwards: the block's parameters say so, the others go on
    g.fill_(1e-2)
    before = p[0].clone()
    sc.adamw_step(p, [g], m, v, 2, exp_avg_scale=ms, exp_avg_sq_scale=vs)
    assert torch.equal(torch.isnan(p[0]), inside)
    assert torch.all(p[0][~inside] != before[~inside])
    second = sc.adamw_state_values(v, vs, "exp_avg_sq")[0]
    assert torch.equal(torch.isnan(second), inside)


def test_a_moment_that_is_infinite_already():
    # float32 states allow it; here a code's scale does
    p = [torch.ones(512, device="cuda")]
    m, v, ms, vs = sc.new_adamw_state(p, 8)
    m[0].fill_(100)
    ms[0].fill_(1.0)
    ms[0][1] = float("inf")
    sc.adamw_step(p, [torch.full((512,), 1e-2, device="cuda")], m, v, 1, exp_avg_scale=ms, exp_avg_sq_scale=vs)
    first = sc.adamw_state_values(m, ms, "exp_avg")[0]
    assert torch.isfinite(first[:256]).all() and torch.isnan(first[256:]).all()


def test_the_largest_moments_that_float32_holds():
    # a block's largest value at float32's end is no overflow
    top = 1.8e19
    p = [torch.zeros(256, device="cuda")]
    g = torch.full((256,), top, device="cuda")
    m, v, ms, vs = sc.new_adamw_state(p, 8)
    sc.adamw_step(p, [g], m, v, 1, betas=(0.9, 0.0), exp_avg_scale=ms, exp_avg_sq_scale=vs)
    second = sc.adamw_state_values(v, vs, "exp_avg_sq")[0]
    assert torch.allclose(second, torch.full_like(second, top ** 2), rtol=2.0 ** -4)
    assert torch.allclose(p[0], torch.full_like(p[0], -1e-3), rtol=1e-5)


@pytest.mark.parametrize("bits", [32, 8])
def test_large_float64_gradients_are_scaled_before_they_are_rounded(bits):
    # the gradients pass float32, scaled ones do not
    gen = torch.Generator(device="cuda").manual_seed(4)
    g = torch.randn(777, generator=gen, device="cuda", dtype=torch.float64)
    p = [torch.randn(777, generator=gen, device="cuda")]
    q = [p[0].clone()]
    a, b = sc.new_adamw_state(p, bits), sc.new_adamw_state(q, bits)
    scale = 2.0 ** -120
    sc.adamw_step(p, [g * 2.0 ** 130], a[0], a[1], 1, grad_scale=scale, exp_avg_scale=a[2], exp_avg_sq_scale=a[3])
    sc.adamw_step(q, [g * 2.0 ** 10], b[0], b[1], 1, exp_avg_scale=b[2], exp_avg_sq_scale=b[3])
    assert torch.isfinite(p[0]).all() and torch.equal(p[0], q[0])
    assert all(torch.equal(x, y) for x, y in zip(a[0] + a[1], b[0] + b[1]))


@pytest.mark.parametrize("bits", [32, 8])
def test_overlaps_are_refused_and_neighbours_are_not(bits):
    flat, g = torch.randn(1024, device="cuda"), torch.randn(512, device="cuda")
    p = [flat[:512], flat[512:]]
    m, v, ms, vs = sc.new_adamw_state(p, bits)
    how = dict(exp_avg_scale=ms, exp_avg_sq_scale=vs)
    sc.adamw_step(p, [g, g], m, v, 1, **how)                # one gradient for both
    want = flat.clone()
    bad = [lambda: sc.adamw_step([flat[:512], flat[511:1023]], [g, g], m, v, 2, **how),
           lambda: sc.adamw_step([p[0], p[0]], [g, g], m, v, 2, **how),
           lambda: sc.adamw_step(p, [g, g], [m[0], m[0]], v, 2, **how),
           lambda: sc.adamw_step(p, [g, g], m, [v[0], m[1]], 2, **how),
           lambda: sc.adamw_step(p, [g, flat[:512]], m, v, 2, **how)]
    if bits == 8:
        bad.append(lambda: sc.adamw_step(p, [g, g], m, v, 2, exp_avg_scale=[ms[0], ms[0]], exp_avg_sq_scale=vs))
    for call in bad:
        with pytest.raises(ValueError):
            call()
    assert torch.equal(flat, want)


@pytest.mark.parametrize("bits", [32, 8])
def test_everything_written_is_reported_to_autograd(bits):
    p = [torch.randn(300, device="cuda"), torch.randn(5, device="cuda")]
    m, v, ms, vs = sc.new_adamw_state(p, bits)
    g = [torch.ones_like(t) for t in p]
    written = [*p, *m, *v, *(ms or ()), *(vs or ())]
    before = [t._version for t in written]
    sc.adamw_step(p, g, m, v, 1, exp_avg_scale=ms, exp_avg_sq_scale=vs)
    assert all(t._version > n for t, n in zip(written, before)) and all(t._version == 0 for t in g)


@pytest.mark.parametrize("bits", [32, 8])
def test_parameters_without_a_gradient_stay(bits):
    # as torch.autograd.grad(..., allow_unused=True) gives them
    gen = torch.Generator(device="cuda").manual_seed(5)
    p = [torch.randn(n, generator=gen, device="cuda") for n in (300, 5, 700)]
    q = [t.clone() for t in p]
    a, b = sc.new_adamw_state(p, bits), sc.new_adamw_state(q, bits)
    g = [torch.randn(300, generator=gen, device="cuda"), None, torch.randn(700, generator=gen, device="cuda")]
    sc.adamw_step(p, g, a[0], a[1], 1, exp_avg_scale=a[2], exp_avg_sq_scale=a[3])
    some = lambda ts: ts and [ts[0], ts[2]]  # noqa: E731
    sc.adamw_step(some(q), some(g), some(b[0]), some(b[1]), 1, exp_avg_scale=some(b[2]), exp_avg_sq_scale=some(b[3]))
    for x, y in zip((p, *a), (q, *b)):
        assert x is None or all(torch.equal(s, t) for s, t in zip(x, y))
    assert not torch.equal(p[0], torch.zeros(300, device="cuda")) and not a[0][1].any()
    assert sc.adamw_step(p, [None] * 3, a[0], a[1], 2, exp_avg_scale=a[2], exp_avg_sq_scale=a[3]) is None
    assert all(torch.equal(s, t) for s, t in zip(p, q))
