"""One training step of a sequence labeller, as its parts are used together: linear
attention in both directions of time, group norm with an activation for each position,
emissions, the semi-CRF loss, gradients, AdamW."""
import pytest

pytestmark = pytest.mark.gpu

import torch  # noqa: E402

import semi_markov_crf_prefix_b200 as sc  # noqa: E402

B, T, H, d, C, K = 3, 150, 2, 32, 5, 6


def make(seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s, k=0.2: (k * torch.randn(*s, generator=g, device="cuda")).requires_grad_(True)  # noqa: E731
    E = H * d
    params = dict(qkv=rnd(3 * E, 8), w=torch.ones(2 * E, device="cuda", requires_grad=True), b=rnd(2 * E), head=rnd(C, 2 * E),
                  A=rnd(C, C), D=rnd(K, C))
    x = torch.randn(B, T, 8, generator=g, device="cuda")
    lengths = torch.tensor([T, 1, 97], dtype=torch.int32, device="cuda")
    labels = torch.full((B, T), -1, dtype=torch.int32, device="cuda")
    starts = torch.zeros((B, T), dtype=torch.uint8, device="cuda")
    for i, L in enumerate(lengths.tolist()):
        for s in range(0, L, 4):
            labels[i, s:min(s + 4, L)] = (s // 4) % C
            starts[i, s] = 1
    return params, x, lengths, labels, starts, torch.tensor([-0.05, -0.01], device="cuda")


def loss(p, x, lengths, labels, starts, decay, norm=None, attention=None):
    attention = attention or (lambda *a, reverse: sc.linear_attention(*a, decay, lengths=lengths, reverse=reverse))
    norm = norm or (lambda y: sc.group_norm(y.view(B * T, 2 * H * d), 2 * H, p["w"], p["b"], activation="silu").view(B, T, -1))
    q, k, v = (x @ p["qkv"].t()).unflatten(-1, (3, H, d)).unbind(2)
    y = torch.cat([attention(q, k, v, reverse=r).reshape(B, T, H * d) for r in (False, True)], -1)
    emissions = norm(y) @ p["head"].t()
    return sc.semicrf_nll(emissions, p["A"], p["D"], lengths, labels, starts).sum()


def test_step_of_the_whole():
    p, *data = make()
    value = loss(p, *data)
    grads = torch.autograd.grad(value, list(p.values()))
    assert torch.isfinite(value) and all(torch.isfinite(g).all() for g in grads)

    # the same with plain operations around the loss
    lengths = data[1]
    ok = (torch.arange(T, device="cuda") < lengths[:, None])[:, :, None, None]
    t = torch.arange(T, device="cuda")
    ld = data[4].double()

    def attention(q, k, v, reverse):
        far = (t[None, :] - t[:, None]) if reverse else (t[:, None] - t[None, :])
        w = torch.where(far >= 0, torch.exp(ld[:, None, None] * far.clamp_min(0)), 0.0)
        q, k, v = (torch.where(ok, u, 0.0).double() for u in (q, k, v))
        return torch.where(ok, torch.einsum("bihk,bjhk,hij,bjhv->bihv", q, k, w, v) * d ** -0.5, 0.0).float()

    def norm(y):
        u = y.double().view(B, T, 2 * H, d)
        u = (u - u.mean(-1, keepdim=True)) / torch.sqrt(u.var(-1, unbiased=False, keepdim=True) + 1e-5)
        z = u.reshape(B, T, -1) * p["w"].double() + p["b"].double()
        return (z * torch.sigmoid(z)).float()

    plain = loss(p, *data, norm=norm, attention=attention)
    want = torch.autograd.grad(plain, list(p.values()))
    # the parts differ by float32 roundings (2^-16 of their terms, see their own tests); a few
    # products later 1e-3 of each gradient's norm is far above that and far below a wrong term
    assert abs(value - plain) <= 1e-4 * abs(plain)
    for g, w in zip(grads, want):
        assert (g - w).norm() <= 1e-3 * w.norm()

    # gradients as they come, the CRF's in float64, to new parameters
    params = [t.detach().clone() for t in p.values()]
    gs = [g.double() if n in ("A", "D") else g for n, g in zip(p, grads)]
    for bits in (32, 8):
        ps = [t.clone() for t in params]
        m, v, ms, vs = sc.new_adamw_state(ps, bits)
        sc.adamw_step(ps, gs, m, v, 1, lr=1e-3, weight_decay=0.0, exp_avg_scale=ms, exp_avg_sq_scale=vs)
        for new, old, g in zip(ps, params, grads):
            # the first step moves by lr against the gradient's sign where that is not tiny
            big = g.abs() > 1e-4
            assert torch.allclose((new - old)[big], -1e-3 * g.sign()[big], rtol=1e-3, atol=1e-6)


def test_captured_training_step():
    # forward, backward and step in one graph, with the same parameters' eager graph alive
    p, *data = make(1)
    eager = loss(p, *data)
    names = list(p)
    state = sc.new_adamw_state([p[n] for n in names])
    step = torch.zeros((), dtype=torch.int64, device="cuda")
    leaves = {n: t.detach().clone().requires_grad_(True) for n, t in p.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(loss(leaves, *data), list(leaves.values()))
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        value = loss(leaves, *data)
        grads = torch.autograd.grad(value, list(leaves.values()))
        step.add_(1)
        sc.adamw_step([leaves[n].detach() for n in names], list(grads), state[0], state[1], step, lr=1e-2)
    want = {n: t.detach().clone() for n, t in p.items()}
    m, v = [torch.zeros_like(t) for t in state[0]], [torch.zeros_like(t) for t in state[1]]
    for i in range(1, 4):
        graph.replay()
        w = {n: t.clone().requires_grad_(True) for n, t in want.items()}
        g = torch.autograd.grad(loss(w, *data), list(w.values()))
        sc.adamw_step(list(want.values()), list(g), m, v, i, lr=1e-2)
    torch.cuda.synchronize()
    for n in names:
        assert torch.allclose(leaves[n], want[n], rtol=1e-5, atol=1e-6), n
    assert torch.equal(eager, loss(p, *data))
    del graph
