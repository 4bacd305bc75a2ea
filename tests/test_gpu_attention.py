"""Linear attention with a decay for each head against its definition in 64 bits.

Tolerances, from the arithmetic.  Let M be the same sums with every factor's absolute
value.  float32: sums of exact products in 24 bits, rounded (or cut, by the matrix
unit) at most 2^-23 of a partial sum in each of at most 128 steps of accumulation
(scores 24, products with V 48, with the state 24, the state's own 48, fewer at each
once terms of size 2^-8 are left out), so 2^-23 * 128 = 2^-16 of M.  16 bits: half a
step of the result, plus 2^-16 M, plus the second factors' two terms (P, the state and
the decayed keys, 2^-16 each at most): 2^-14 M covers them.  States are float32 from
three terms: 2^-16 M.
"""
import pytest

pytestmark = pytest.mark.gpu

import torch  # noqa: E402

import semi_markov_crf_prefix_b200 as sc  # noqa: E402

TYPES = [torch.float32, torch.bfloat16, torch.float16]


def half_step(t):
    return torch.finfo(t).eps / 2


def tol(exact, M, dtype):
    if dtype == torch.float32:
        return 2.0 ** -16 * M + 1e-30
    tiny = torch.finfo(dtype).smallest_normal * half_step(dtype)   # subnormal halves round by this much
    return half_step(dtype) * exact.abs() * 1.001 + 2.0 ** -14 * M + 2 * tiny


def definition(q, k, v, ld, lengths, scale, s0, reverse):
    """(o, state) in float64 by the sum over pairs; differentiable."""
    B, T, H, _ = q.shape
    L = torch.full((B,), T, device=q.device) if lengths is None else lengths.long().clamp(0, T)
    t = torch.arange(T, device=q.device)
    ok = (t < L[:, None])[:, :, None, None]
    q, k, v = (torch.where(ok, x, torch.zeros_like(x)) for x in (q, k, v))
    at = torch.where(ok[..., 0, 0], (L[:, None] - 1 - t) if reverse else t.expand(B, T), 0)
    far = at[:, :, None] - at[:, None, :]
    power = lambda n: torch.where(n == 0, 1.0, torch.exp(ld.double()[None, :, None, None] * n.clamp_min(0)))  # noqa: E731
    w = torch.where(far[:, None] >= 0, power(far[:, None]), 0.0)
    o = scale * torch.einsum("bthk,bjhk,bhtj,bjhv->bthv", q, k, w, v)
    left = power((L[:, None] - 1 - at).clamp_min(0)[:, None, :, None])
    state = torch.einsum("bthk,bhtx,bthv->bhkv", k, left, v)
    if s0 is not None:
        state = state + power(L[:, None, None, None].expand(B, 1, 1, 1)) * s0
        since = power((at + 1)[:, None, :, None]).permute(0, 2, 1, 3)
        o = o + scale * torch.einsum("bthk,bhkv->bthv", q * since, s0)
    return torch.where(ok, o, torch.zeros_like(o)), state


def inputs(B, T, H, dk, dv, dtype, seed=0, lengths=None, state=False, decay=None, layout="dense"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    if layout == "packed":            # views of one projection's output
        both = rnd(B, T, H * (2 * dk + dv)).to(dtype)
        q, k, v = both.split([H * dk, H * dk, H * dv], -1)
        q, k, v = q.unflatten(-1, (H, dk)), k.unflatten(-1, (H, dk)), v.unflatten(-1, (H, dv))
    elif layout == "heads first":     # [B,H,T,d] in memory
        q, k, v = (rnd(B, H, T, d).to(dtype).transpose(1, 2) for d in (dk, dk, dv))
    elif layout == "off":             # no 16-byte alignment
        q, k, v = (rnd(B * T * H * d + 1).to(dtype)[1:].view(B, T, H, d) for d in (dk, dk, dv))
    else:
        q, k, v = (rnd(B, T, H, d).to(dtype) for d in (dk, dk, dv))
    ld = torch.linspace(-0.2, -0.001, H, device="cuda") if decay is None else torch.full((H,), decay, device="cuda")
    return q, k, v, ld, (rnd(B, H, dk, dv) if state else None)


def check(q, k, v, ld, s0=None, lengths=None, reverse=False, scale=None, seed=1, train=True):
    dk, dv = q.shape[-1], v.shape[-1]
    sc_ = dk ** -0.5 if scale is None else scale
    g = torch.Generator(device="cuda").manual_seed(seed)
    do = torch.randn(*q.shape[:3], dv, generator=g, device="cuda").to(q.dtype)
    ds = torch.randn(q.shape[0], q.shape[2], dk, dv, generator=g, device="cuda")
    leaves = [x.detach().requires_grad_(True) for x in (q, k, v)] + ([s0.clone().requires_grad_(True)] if s0 is not None else [])
    a = leaves[3] if s0 is not None else None
    o, s = sc.linear_attention(*leaves[:3], ld, lengths=lengths, scale=scale, initial_state=a, return_state=True,
                               reverse=reverse)
    clean = lambda x: torch.nan_to_num(x.detach().double(), nan=0.0)  # noqa: E731  (padding may hold NaN)
    x64 = [clean(x).requires_grad_(True) for x in leaves]
    eo, es = definition(*x64[:3], ld, lengths, sc_, x64[3] if s0 is not None else None, reverse)
    absolute = [x.detach().abs().requires_grad_(True) for x in x64]
    mo, ms = definition(*absolute[:3], ld, lengths, abs(sc_), absolute[3] if s0 is not None else None, reverse)
    assert o.dtype == q.dtype and s.dtype == torch.float32
    assert torch.all((o.double() - eo).abs() <= tol(eo, mo, q.dtype))
    assert torch.all((s.double() - es).abs() <= 2.0 ** -16 * ms + 1e-30)
    if lengths is not None:
        for b, n in enumerate(lengths.tolist()):
            assert torch.all(o[b, n:] == 0)
    if not train:
        return o, s
    grads = torch.autograd.grad((o, s), leaves, (do, ds))
    exact = torch.autograd.grad((eo, es), x64, (do.double(), ds.double()))
    bound = torch.autograd.grad((mo, ms), absolute, (do.double().abs(), ds.double().abs()))
    for got, want, M in zip(grads, exact, bound):
        t = tol(want, M, got.dtype) if got.dtype != torch.float32 or q.dtype == torch.float32 else 2.0 ** -16 * M + 1e-30
        assert torch.all((got.double() - want).abs() <= t)
    return o, s


SHAPES = [(1, 1, 1, 64, 64), (2, 127, 2, 64, 64), (1, 128, 2, 64, 64), (1, 129, 2, 64, 48), (2, 300, 2, 32, 64),
          (1, 1030, 2, 16, 8), (2, 257, 1, 128, 128), (1, 384, 2, 128, 72), (1, 140, 2, 33, 20), (1, 40, 1, 7, 1),
          (1, 70, 1, 200, 130), (1, 2, 3, 256, 256)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("reverse", [False, True])
def test_against_definition(shape, dtype, reverse):
    q, k, v, ld, s0 = inputs(*shape, dtype, state=True)
    check(q, k, v, ld, s0, reverse=reverse)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("layout", ["packed", "heads first", "off"])
@pytest.mark.parametrize("d", [64, 128])
def test_layouts(layout, dtype, d):
    q, k, v, ld, s0 = inputs(2, 200, 3, d, d, dtype, layout=layout, state=True)
    check(q, k, v, ld, s0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("d", [64, 100, 128])
def test_lengths(dtype, reverse, d):
    # none, one, a chunk, one more, all; what lies behind the end is NaN and must not be read
    lengths = torch.tensor([0, 1, 128, 129, 300, 255], dtype=torch.int32, device="cuda")
    q, k, v, ld, s0 = inputs(6, 300, 2, d, d, dtype, state=True)
    for b, n in enumerate(lengths.tolist()):
        for x in (q, k, v):
            x[b, n:] = float("nan")
    check(q, k, v, ld, s0, lengths=lengths, reverse=reverse)
    check(q, k, v, ld, None, lengths=lengths, reverse=reverse)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("decay", [0.0, -1e-4, -0.5, -3.0, -50.0, float("-inf")])
@pytest.mark.parametrize("d", [64, 100])
def test_decays(dtype, decay, d):
    q, k, v, ld, s0 = inputs(1, 300, 2, d, d, dtype, state=True, decay=decay)
    check(q, k, v, ld, s0, train=decay > -1e30)


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 64), (torch.bfloat16, 128), (torch.float32, 64), (torch.float32, 96),
                                     (torch.float16, 64)])
@pytest.mark.parametrize("reverse", [False, True])
def test_segments(dtype, d, reverse):
    # one long sequence is walked in segments that are joined; lengths that end in the
    # first, in the middle of one, at a segment's end, in the last
    T = 5000
    q, k, v, ld, s0 = inputs(4, T, 1, d, d, dtype, state=True, decay=-0.002)
    from semi_markov_crf_prefix_b200 import encoder
    assert encoder.linear_attention_workspace_bytes(q, v) > 256   # it is walked in segments
    check(q, k, v, ld, s0, reverse=reverse, lengths=torch.tensor([T, 3, 2944, 1409], dtype=torch.int32, device="cuda"))
    check(q[:1], k[:1], v[:1], ld, None, reverse=reverse)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("reverse", [False, True])
def test_segments_without_a_state(d, reverse):
    # no state leaves (fewer terms); a segment's end, one more, one less, and NaN behind the ends
    T = 4000
    q, k, v, ld, s0 = inputs(4, T, 1, d, d, torch.bfloat16, state=True, decay=-0.002)
    lengths = torch.tensor([T, 1024, 1025, 1023], dtype=torch.int32, device="cuda")
    for b, n in enumerate(lengths.tolist()):
        for x in (q, k, v):
            x[b, n:] = float("nan")
    o = sc.linear_attention(q, k, v, ld, lengths=lengths, initial_state=s0, reverse=reverse)
    args = [torch.nan_to_num(x.double(), nan=0.0) for x in (q, k, v)]
    want, _ = definition(*args, ld, lengths, d ** -0.5, s0.double(), reverse)
    M, _ = definition(*[x.abs() for x in args], ld, lengths, d ** -0.5, s0.double().abs(), reverse)
    assert torch.all((o.double() - want).abs() <= tol(want, M, torch.bfloat16))


def test_second_derivatives_are_refused():
    q, k, v, ld, _ = inputs(1, 9, 1, 16, 16, torch.float32)
    q.requires_grad_(True)
    first = torch.autograd.grad(sc.linear_attention(q, k, v, ld).square().sum(), q, create_graph=True)[0]
    with pytest.raises(RuntimeError):
        first.sum().backward()


def test_pieces_equal_the_whole():
    # a sequence read in pieces with the state handed on, then position by position
    q, k, v, ld, _ = inputs(2, 400, 2, 64, 64, torch.float32)
    whole, end = sc.linear_attention(q, k, v, ld, return_state=True)
    a, s = sc.linear_attention(q[:, :150], k[:, :150], v[:, :150], ld, return_state=True)
    b, s = sc.linear_attention(q[:, 150:390], k[:, 150:390], v[:, 150:390], ld, initial_state=s, return_state=True)
    steps = []
    for t in range(390, 400):
        steps.append(sc.linear_attention_step(q[:, t], k[:, t], v[:, t], ld, s))
    got = torch.cat([a, b, torch.stack(steps, 1)], 1)
    one = lambda x: x.double().abs()  # noqa: E731
    M, Ms = definition(one(q), one(k), one(v), ld, None, 64 ** -0.5, None, False)
    assert torch.all((got - whole).abs() <= 2 * 2.0 ** -16 * M)
    assert torch.all((s - end).abs() <= 2 * 2.0 ** -16 * Ms)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(1, 4, 64, 64), (3, 2, 128, 128), (2, 1, 33, 20), (1, 1, 1, 1), (2, 3, 256, 256),
                                   (5, 2, 8, 130), (2, 2, 100, 4)])
def test_step(shape, dtype):
    B, H, dk, dv = shape
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(B, 2, H * (2 * dk + dv), generator=g, device="cuda").to(dtype)[:, 1]
    q, k, v = x.split([H * dk, H * dk, H * dv], -1)
    q, k, v = q.unflatten(-1, (H, dk)), k.unflatten(-1, (H, dk)), v.unflatten(-1, (H, dv))
    ld = torch.linspace(-2.0, -0.001, H, device="cuda")
    s = torch.randn(B, H, dk, dv, generator=g, device="cuda")
    want = torch.exp(ld.double())[:, None, None] * s.double() + k.double()[..., None] * v.double()[..., None, :]
    eo = torch.einsum("bhk,bhkv->bhv", q.double(), want) * 0.25
    Ms = s.double().abs() + k.double().abs()[..., None] * v.double().abs()[..., None, :]
    M = torch.einsum("bhk,bhkv->bhv", q.double().abs(), Ms) * 0.25
    o = sc.linear_attention_step(q, k, v, ld, s, scale=0.25)
    # three roundings of the state; dk + 3 of the sum at most
    assert torch.all((s.double() - want).abs() <= 3 * 2.0 ** -24 * Ms)
    assert torch.all((o.double() - eo).abs() <= half_step(dtype) * eo.abs() * 1.001 + (dk + 8) * 2.0 ** -24 * M
                     + torch.finfo(dtype).smallest_normal * half_step(dtype))


def test_gradient_against_differences():
    # the output is linear in q, in k, in v and in the state, so a central difference of any
    # width is the derivative itself, but for rounding: twice the output's tolerance
    q, k, v, ld, s0 = inputs(2, 150, 2, 64, 40, torch.float32, state=True)
    g = torch.Generator(device="cuda").manual_seed(5)
    do = torch.randn(2, 150, 2, 40, generator=g, device="cuda")
    leaves = [x.clone().requires_grad_(True) for x in (q, k, v, s0)]
    o = sc.linear_attention(*leaves[:3], ld, initial_state=leaves[3])
    grads = torch.autograd.grad(o, leaves, do)
    for i, grad in enumerate(grads):
        u = torch.randn(grad.shape, generator=g, device="cuda")
        value = []
        M = 0.0
        for sign in (1.0, -1.0):
            x = [t.detach().clone() for t in leaves]
            x[i] += sign * u
            y = sc.linear_attention(*x[:3], ld, initial_state=x[3])
            value.append((y.double() * do.double()).sum())
            a = [t.double().abs() for t in x]
            mo, _ = definition(*a[:3], ld, None, 64 ** -0.5, a[3], False)
            M = M + (mo * do.double().abs()).sum()
        slope = (value[0] - value[1]) / 2
        a = [t.detach().double().abs().requires_grad_(True) for t in leaves]
        mo, _ = definition(*a[:3], ld, None, 64 ** -0.5, a[3], False)
        mg, = torch.autograd.grad(mo, a[i], do.double().abs())
        got = (grad.double() * u.double()).sum()
        assert abs(got - slope) <= 2.0 ** -16 * (M + (mg * u.double().abs()).sum())


def test_gradient_of_a_sum_and_of_the_state_alone():
    q, k, v, ld, s0 = inputs(2, 130, 2, 64, 64, torch.bfloat16, state=True)
    leaves = [x.clone().requires_grad_(True) for x in (q, k, v, s0)]
    # an upstream gradient without memory of its own (all strides 0)
    sc.linear_attention(*leaves[:3], ld, initial_state=leaves[3]).sum().backward()
    ones = torch.autograd.grad(sc.linear_attention(*leaves[:3], ld, initial_state=leaves[3]), leaves,
                               torch.ones(2, 130, 2, 64, dtype=torch.bfloat16, device="cuda"))
    assert all(torch.equal(x.grad, g) for x, g in zip(leaves, ones))
    _, s = sc.linear_attention(*leaves[:3], ld, initial_state=leaves[3], return_state=True)
    dq, dk, dv, ds = torch.autograd.grad(s.sum(), leaves)
    assert torch.all(dq == 0)
    assert torch.allclose(ds, torch.exp(ld * 130)[None, :, None, None].expand_as(ds), rtol=2 ** -20)
    # q alone wants a gradient
    o = sc.linear_attention(leaves[0], k, v, ld)
    assert torch.autograd.grad(o.float().sum(), leaves[0])[0].shape == q.shape


@pytest.mark.parametrize("dtype", TYPES)
def test_shared_heads_by_expanding(dtype):
    # one key and value head for all query heads, one query for all sequences: strides of 0
    q, k, v, ld, _ = inputs(2, 200, 3, 64, 64, dtype)
    one_q, one_k, one_v = (x.detach().clone().requires_grad_(True) for x in (q[:1], k[:, :, :1], v[:, :, :1]))
    full = [x.detach().expand(2, 200, 3, 64).contiguous().requires_grad_(True) for x in (one_q, one_k, one_v)]
    do = torch.randn(2, 200, 3, 64, device="cuda").to(dtype)
    o = sc.linear_attention(one_q.expand(2, -1, 3, -1), one_k.expand(-1, -1, 3, -1), one_v.expand(-1, -1, 3, -1), ld)
    w = sc.linear_attention(*full, ld)
    # (two kernels may serve the two, each right to its tolerance)
    M, _ = definition(*[x.detach().double().abs() for x in full], ld, None, 0.125, None, False)
    assert torch.all((o.double() - w.double()).abs() <= 2 * tol(w.double(), M, dtype))
    got = torch.autograd.grad(o, (one_q, one_k, one_v), do)
    want = torch.autograd.grad(w, full, do)
    a = [x.detach().double().abs().requires_grad_(True) for x in full]
    mo, _ = definition(*a, ld, None, 0.125, None, False)
    bound = torch.autograd.grad(mo, a, do.double().abs())
    for g, h, m, axis in zip(got, want, bound, (0, 2, 2)):
        lim = 2 * tol(h.double(), m, dtype).sum(axis, keepdim=True)      # autograd adds the heads' shares in dtype
        lim = lim + 4 * half_step(dtype) * h.double().abs().sum(axis, keepdim=True)
        assert torch.all((g.double() - h.double().sum(axis, keepdim=True)).abs() <= lim)


def test_overwritten_state_is_noticed():
    q, k, v, ld, s0 = inputs(1, 3, 1, 16, 16, torch.float32, state=True)
    s0.requires_grad_(True)
    held = s0 * 1.0
    o = sc.linear_attention(q, k, v, ld, initial_state=held)
    sc.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], ld, held.detach())
    with pytest.raises(RuntimeError):
        o.sum().backward()


def test_axes_of_length_one():
    # their strides say nothing
    q, k, v, ld, _ = inputs(1, 150, 1, 64, 64, torch.bfloat16)
    odd = [x.as_strided(x.shape, (7, 64, 3, 1)) for x in (q, k, v)]
    assert torch.equal(sc.linear_attention(*odd, ld), sc.linear_attention(q, k, v, ld))


def test_same_call_same_bits():
    for dtype, d in ((torch.bfloat16, 64), (torch.bfloat16, 128), (torch.float32, 64), (torch.float32, 80)):
        q, k, v, ld, s0 = inputs(2, 1500, 2, d, d, dtype, state=True)
        a = sc.linear_attention_forward(q, k, v, ld, initial_state=s0, return_state=True)
        b = sc.linear_attention_forward(q, k, v, ld, initial_state=s0, return_state=True)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        ga = sc.linear_attention_backward(q, q, k, v, ld)
        gb = sc.linear_attention_backward(q, q, k, v, ld)
        assert all(torch.equal(x, y) for x, y in zip(ga[:3], gb[:3]))


def test_far_apart_sequences():
    # strides that pass 2^31 elements
    big = torch.empty(2 ** 31 + 2 ** 20, dtype=torch.bfloat16, device="cuda")
    for dtype, d in ((torch.bfloat16, 64), (torch.bfloat16, 20)):
        q, k, v, ld, _ = inputs(2, 130, 2, d, d, dtype)
        views = []
        for i, x in enumerate((q, k, v)):
            view = big.as_strided(x.shape, (2 ** 31, 2 * d, d, 1), 2 ** 16 * i)
            view.copy_(x)
            views.append(view)
        assert torch.equal(sc.linear_attention(*views, ld), sc.linear_attention(q, k, v, ld))


def test_captured_and_on_another_stream():
    q, k, v, ld, s0 = inputs(1, 3000, 2, 64, 64, torch.bfloat16, state=True)
    want, end = sc.linear_attention(q, k, v, ld, initial_state=s0, return_state=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sc.linear_attention(q, k, v, ld)                     # first call outside of the capture
        o2, _ = sc.linear_attention(q, k, v, ld, initial_state=s0, return_state=True)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o2, want)
    graphs = []
    for _ in range(2):                                       # two graphs, each with its own workspace
        x = [t.clone() for t in (q, k, v)]
        state = s0.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o, s = sc.linear_attention(*x, ld, initial_state=s0, return_state=True)
            step = sc.linear_attention_step(x[0][:, 0], x[1][:, 0], x[2][:, 0], ld, state)
        graphs.append((g, x, o, s, state, step))
    for g, x, o, s, state, step in graphs:
        x[2].mul_(2.0)
        state.copy_(s0)
    for g, *_ in graphs:
        g.replay()
    torch.cuda.synchronize()
    s2 = s0.clone()
    w2, e2 = sc.linear_attention(q, k, v * 2, ld, initial_state=s0, return_state=True)
    st2 = sc.linear_attention_step(q[:, 0], k[:, 0], v[:, 0] * 2, ld, s2)
    for _, _, o, s, state, step in graphs:
        assert torch.equal(o, w2) and torch.equal(s, e2) and torch.equal(state, s2) and torch.equal(step, st2)


def test_bad_lengths_are_reported():
    q, k, v, ld, _ = inputs(3, 140, 1, 64, 64, torch.bfloat16)
    ws = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    lengths = torch.tensor([141, -1, 140], dtype=torch.int32, device="cuda")
    o, _ = sc.linear_attention_forward(q, k, v, ld, lengths=lengths, ws=ws)
    assert sc.device_status(ws) == sc._lib.SEMICRF_ERR_INVALID_LENGTH
    assert torch.equal(o[0], sc.linear_attention(q[:1], k[:1], v[:1], ld)[0]) and torch.all(o[1] == 0)
    sc.clear_device_status(ws)
    sc.linear_attention_forward(q, k, v, ld, ws=ws)
    assert sc.device_status(ws) == 0


def test_refusals():
    q, k, v, ld, s0 = inputs(2, 10, 2, 16, 24, torch.bfloat16, state=True)
    f = sc.linear_attention
    for bad in (lambda: f(q, k[:, :9], v, ld), lambda: f(q, k, v[:, :, :1], ld), lambda: f(q, k, v, ld[:1]),
                lambda: f(q, k, v, ld, lengths=torch.ones(3, dtype=torch.int32, device="cuda")),
                lambda: f(q, k, v, ld, initial_state=s0[:1]), lambda: f(q, k, v, ld, initial_state=s0.transpose(0, 1)),
                lambda: f(q.transpose(1, 3).contiguous().transpose(1, 3), k, v, ld),
                lambda: f(q[0], k[0], v[0], ld), lambda: f(q, k, v, ld.clone().requires_grad_(True)),
                lambda: f(q[:, :0], k[:, :0], v[:, :0], ld),
                lambda: f(*(torch.zeros(1, 2, 1, 300, device="cuda") for _ in range(3)), ld[:1]),
                lambda: sc.linear_attention_step(q[:, 0].clone().requires_grad_(True), k[:, 0], v[:, 0], ld, s0)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: f(q, k.float(), v, ld), lambda: f(q.double(), k, v, ld), lambda: f(q, k, v, ld.double()),
                lambda: f(q, k, v, ld, lengths=torch.ones(2, dtype=torch.int64, device="cuda")),
                lambda: f(q, k, v, ld, initial_state=s0.double()), lambda: f(q, k, None, ld)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(sc.SemiCRFError):
        sc.linear_attention_forward(q, k, v, ld, ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))
