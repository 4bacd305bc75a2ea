"""Calls of the operators around the loss as programs make them: parameters held by a model,
inference, layouts, sizes."""
import pytest

pytestmark = pytest.mark.gpu

import torch  # noqa: E402

import semi_markov_crf_prefix_b200 as sc  # noqa: E402


def rnd(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def test_decays_held_as_a_parameter():
    q, k, v = (rnd(i, 2, 9, 2, 16) for i in range(3))
    decay = torch.nn.Parameter(torch.tensor([-0.1, -0.01], device="cuda"))
    want = sc.linear_attention(q, k, v, decay.detach())
    for mode in (torch.no_grad, torch.inference_mode):
        with mode():
            assert torch.equal(sc.linear_attention(q, k, v, decay), want)
            assert torch.equal(sc.linear_attention_forward(q, k, v, decay)[0], want)
            state = torch.zeros(2, 2, 16, 16, device="cuda")
            for t in range(9):
                o = sc.linear_attention_step(q[:, t], k[:, t], v[:, t], decay, state)
            assert torch.allclose(o, want[:, -1], rtol=1e-4, atol=1e-5)
    # where a gradient would be lost it is refused, whatever else asks for one
    with pytest.raises(ValueError):
        sc.linear_attention(q, k, v, decay)
    with pytest.raises(ValueError):
        sc.linear_attention(q.requires_grad_(True), k, v, decay)
    with pytest.raises(ValueError):
        sc.linear_attention_forward(q.detach(), k, v, decay)
    with pytest.raises(ValueError), torch.enable_grad():
        sc.linear_attention_step(q.detach()[:, 0], k[:, 0], v[:, 0], decay, torch.zeros(2, 2, 16, 16, device="cuda"))
    with pytest.raises(TypeError):
        sc.linear_attention(q.detach(), k, v, None)
