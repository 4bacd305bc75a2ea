"""What linear attention rounds inside a call, at sizes where nothing averages out.

For 16-bit operands the scores times their decays and the state as q's operand enter the
matrix unit in two bf16 terms, each nearest: 2^-17 of the value at most.  float16 operands
are two terms themselves, exactly, and the product of both second terms (2^-8 of each
operand) is left out: 2^-16 of a product, of q and k and of P and v.  Everything else is
float32: a few roundings of 2^-24 and accumulators that cut at 2^-23, below 2^-20 of the
absolute sum M at these lengths.  The state's keys are held to 24 bits.  All outputs are
independent of which of them are asked for.
"""
import pytest

pytestmark = pytest.mark.gpu

import torch  # noqa: E402

import semi_markov_crf_prefix_b200 as sc  # noqa: E402


def half_step(t):
    return torch.finfo(t).eps / 2


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("state", [False, True])
def test_products_to_their_bits(dtype, d, state):
    # values of opposite sign, so that o is far smaller than the two terms it is made of and
    # what those lost shows behind o's own rounding; q has few components, so that little is
    # lost in the scores themselves
    B, H = 64, 8
    g = torch.Generator(device="cuda").manual_seed(11)
    q, k, v = (torch.randn(B, 2, H, d, generator=g, device="cuda").to(dtype) for _ in range(3))
    q[..., 2:] = 0
    v[:, 1] = -v[:, 0]
    k[:, 1] = k[:, 0]
    k[:, 1, :, 0] += 0.25 * k[:, 0, :, 1]
    ld = torch.linspace(-0.01, -0.0001, H, device="cuda")
    s0 = None
    if state:
        q[:, 0, :, 1:] = 0      # o of the first position: one row of the state against one product
        s0 = torch.randn(B, H, d, d, generator=g, device="cuda")
        s0[:, :, 0] = -(k[:, 0, :, :1].float() * v[:, 0].float()) * (1 + 0.01 * torch.rand(B, H, d, generator=g, device="cuda"))
    o = sc.linear_attention(q, k, v, ld, scale=1.0, initial_state=s0)
    lam = torch.exp(ld.double())[:, None]
    q, k, v = q.double(), k.double(), v.double()
    sum_of = lambda x, y: (x * y).sum(-1, keepdim=True)  # noqa: E731
    size = lambda x, y: sum_of(x.abs(), y.abs())  # noqa: E731
    lead = lambda x: torch.exp2(torch.floor(torch.log2(x.abs())))  # noqa: E731  (2^-17 of this is half a step of two terms)
    if state:
        s0 = s0[:, :, 0].double()
        row, p = q[:, 0, :, :1] * lam, sum_of(q[:, 0], k[:, 0])
        want, M, got = row * s0 + p * v[:, 0], (row * s0).abs() + (p * v[:, 0]).abs(), o[:, 0]
        held = row.abs() * lead(s0) + lead(p) * v[:, 0].abs()
    else:
        a, b = sum_of(q[:, 1], k[:, 0]) * lam, sum_of(q[:, 1], k[:, 1])
        want, got = a * v[:, 0] + b * v[:, 1], o[:, 1]
        M = (size(q[:, 1], k[:, 0]) + size(q[:, 1], k[:, 1])) * v[:, 0].abs()
        held = (lead(a) + lead(b)) * v[:, 0].abs()
    tiny = torch.finfo(dtype).smallest_normal * half_step(dtype)
    off = (got.double() - want).abs() - half_step(dtype) * want.abs() * 1.001 - tiny
    lost = 2.0 ** -20 + (2.0 ** -15 if dtype == torch.float16 else 0.0)
    assert torch.all(off <= 2.0 ** -17 * held + lost * M)
    assert (want.abs() < M / 32).float().mean() > 0.05          # there are such values


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [2, 16, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_state_is_held_to_24_bits(dtype, T, d):
    # one-signed products of few positions; 128 positions: 24 cut sums of 2^-23 are 2^-18.4
    B, H = 32, 4
    g = torch.Generator(device="cuda").manual_seed(12)
    q, k, v = (torch.rand(B, T, H, d, generator=g, device="cuda").to(dtype) for _ in range(3))
    ld = torch.tensor([-0.3, -0.05, -0.007, -0.001], device="cuda")
    _, s = sc.linear_attention(q, k, v, ld, return_state=True)
    left = torch.exp(ld.double()[None, :] * (T - 1 - torch.arange(T, device="cuda"))[:, None])[None, :, :, None]
    want = torch.einsum("bthk,bthv->bhkv", k.double() * left, v.double())
    assert torch.all((s.double() - want).abs() <= (2.0 ** -20 if T <= 16 else 2.0 ** -18) * want)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [300, 4000])
@pytest.mark.parametrize("reverse", [False, True])
def test_outputs_do_not_depend_on_what_is_asked_for(d, T, reverse):
    g = torch.Generator(device="cuda").manual_seed(13)
    q, k, v, do = (torch.randn(2, T, 2, d, generator=g, device="cuda").bfloat16() for _ in range(4))
    s0 = torch.randn(2, 2, d, d, generator=g, device="cuda")
    ld = torch.tensor([-0.02, -0.0005], device="cuda")
    for initial in (None, s0):
        how = dict(initial_state=initial, reverse=reverse)
        a, none = sc.linear_attention_forward(q, k, v, ld, **how)
        b, _ = sc.linear_attention_forward(q, k, v, ld, return_state=True, **how)
        assert none is None and torch.equal(a, b)
        ga = sc.linear_attention_backward(do, q, k, v, ld, **how)
        gb = sc.linear_attention_backward(do, q, k, v, ld, want_initial_state=True, **how)
        assert all(torch.equal(x, y) for x, y in zip(ga[:3], gb[:3]))


@pytest.mark.parametrize("dk,dv", [(64, 64), (16, 40), (130, 70)])
@pytest.mark.parametrize("T", [2, 130])
def test_the_largest_values_of_float32(dk, dv, T):
    # finite operands at the type's end (what is infinite may spread, as documented)
    top = torch.finfo(torch.float32).max
    g = torch.Generator(device="cuda").manual_seed(14)
    ld = torch.tensor([-0.5], device="cuda")
    for value in (top, -top):
        q, k = (torch.zeros(1, T, 1, dk, device="cuda") for _ in range(2))
        v = torch.rand(1, T, 1, dv, generator=g, device="cuda")
        q[..., 0], k[..., 0] = 0.5, 0.25
        v[0, T - 1, 0, 3] = value
        o, s = sc.linear_attention(q, k, v, ld, scale=1.0, return_state=True)
        left = torch.exp(ld.double() * torch.arange(T - 1, -1, -1, device="cuda"))
        want = 0.25 * (left[:, None] * v[0, :, 0].double()).sum(0)
        assert torch.allclose(s[0, 0, 0].double(), want, rtol=2.0 ** -16)
        assert torch.allclose(o[0, -1, 0].double(), 0.5 * want, rtol=2.0 ** -16)
        # the same of a given state
        s0 = torch.zeros(1, 1, dk, dv, device="cuda")
        s0[0, 0, 0, 5] = value
        v[0, T - 1, 0, 3] = 1.0
        o, s = sc.linear_attention(q, k, v, ld, scale=1.0, initial_state=s0, return_state=True)
        assert torch.allclose(s[0, 0, 0, 5].double(), s0[0, 0, 0, 5].double() * torch.exp(ld.double() * T)[0], rtol=2.0 ** -16)
        assert torch.allclose(o[0, 0, 0, 5].double(), 0.5 * s0[0, 0, 0, 5].double() * torch.exp(ld.double())[0], rtol=2.0 ** -16)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [3, 300])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_what_is_not_finite_is_not_lost(dtype, d, T, value):
    # wherever it stands in a valid position, its own outputs and the state show it, and other
    # sequences and heads do not
    g = torch.Generator(device="cuda").manual_seed(15)
    ld = torch.tensor([-0.1, -0.001], device="cuda")
    for which in range(4):
        x = [torch.randn(2, T, 2, d, generator=g, device="cuda").to(dtype) for _ in range(3)]
        s0 = torch.randn(2, 2, d, d, generator=g, device="cuda")
        if which < 3:
            x[which][1, T - 2, 1, 5] = value
        else:
            s0[1, 1, 5, 7] = value
        o, s = sc.linear_attention(*x, ld, initial_state=s0, return_state=True)
        bad = o[1, T - 2, 1]
        assert not torch.isfinite(bad).all()
        if which > 0:
            assert not torch.isfinite(s[1, 1]).all()
        assert torch.isfinite(o[0]).all() and torch.isfinite(o[1, :, 0]).all()
        assert torch.isfinite(s[0]).all() and torch.isfinite(s[1, 0]).all()
