"""Calls of the operators around the loss as programs make them: parameters held by a model,
inference, layouts, sizes."""
import pytest

pytestmark = pytest.mark.gpu

import torch  # noqa: E402

import semi_markov_crf_prefix_b200 as sc  # noqa: E402
from test_gpu_attention import check as attention_check, inputs as attention_inputs  # noqa: E402


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


def test_workspace_follows_the_operands():
    # widths over 64 in bf16: partial sums only where the copy engine cannot address the operands
    from semi_markov_crf_prefix_b200 import encoder
    B, T, H, d = 4, 20000, 4, 128
    q = torch.zeros(B, T, H, d, dtype=torch.bfloat16, device="cuda")
    ld = torch.full((H,), -0.01, device="cuda")
    size = q.numel() * 2

    def used(f):
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        f()
        return torch.cuda.max_memory_allocated() - before

    assert used(lambda: sc.linear_attention_forward(q, q, q, ld)) < size + (64 << 20)
    assert used(lambda: sc.linear_attention_backward(q, q, q, q, ld)) < 3 * size + (64 << 20)
    # the size for any operands is what it was, and serves
    need = encoder.linear_attention_workspace_bytes(q, q)
    assert need > 2 * size
    odd = torch.zeros(q.numel() + 1, dtype=torch.bfloat16, device="cuda")[1:].view_as(q)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    sc.linear_attention_forward(odd, q, q, ld, ws=ws)
    with pytest.raises(sc.SemiCRFError):
        sc.linear_attention_forward(odd, q, q, ld, ws=ws[:need // 2])
    sc.linear_attention_forward(q, q, q, ld, ws=ws[:need // 2])


def test_a_workspace_that_turns_out_too_small(monkeypatch):
    # the library's call has the last word on its plan
    from semi_markov_crf_prefix_b200 import encoder
    q, k, v, do = (rnd(i, 1, 4000, 2, 64).bfloat16() for i in range(4))
    ld = torch.tensor([-0.1, -0.001], device="cuda")
    want = sc.linear_attention_forward(q, k, v, ld)[0]
    grads = sc.linear_attention_backward(do, q, k, v, ld)
    monkeypatch.setattr(encoder, "_attention_ws_at", lambda *a: 256)
    assert torch.equal(sc.linear_attention_forward(q, k, v, ld)[0], want)
    assert all(torch.equal(a, b) for a, b in zip(sc.linear_attention_backward(do, q, k, v, ld)[:3], grads))
    with pytest.raises(sc.SemiCRFError):
        sc.linear_attention_forward(q, k, v, ld, ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("strides", ["sliding", "heads apart", "positions and heads out of proportion", "positions first"])
def test_strides_of_any_order(strides, d, dtype):
    B, T, H = 2, 300, 3
    buf = rnd(7, 4 * B * T * H * d + 4096).to(dtype)
    st = {"sliding": (T * 8 + 8 * H, 8, 16, 1),                    # windows of one row that overlap
          "heads apart": (H * T * d, d, T * d, 1),
          "positions and heads out of proportion": (T * (H * d + 24), H * d + 24, d + 8, 1),
          "positions first": (H * d, B * H * d, d, 1)}[strides]
    x = [buf.as_strided((B, T, H, d), st, i * 512) for i in range(3)]
    ld = torch.tensor([-0.2, -0.02, -0.002], device="cuda")
    dense = [t.contiguous() for t in x]
    assert torch.equal(sc.linear_attention(*x, ld), sc.linear_attention(*dense, ld))
    do = rnd(8, B, T, H, d).to(dtype)
    for got, want in zip(sc.linear_attention_backward(do, *x, ld)[:3], sc.linear_attention_backward(do, *dense, ld)[:3]):
        assert torch.equal(got, want)


@pytest.mark.parametrize("dtype,dk,dv", [(torch.float16, 128, 128), (torch.float16, 200, 130), (torch.bfloat16, 200, 130),
                                         (torch.bfloat16, 130, 200), (torch.float32, 130, 70), (torch.float16, 64, 65)])
@pytest.mark.parametrize("reverse", [False, True])
def test_wide_heads_in_segments(dtype, dk, dv, reverse):
    # blocks of the contraction, slices of the values and joined segments in one call
    T = 2500
    q, k, v, ld, s0 = attention_inputs(2, T, 1, dk, dv, dtype, state=True, decay=-0.003)
    assert sc.linear_attention_workspace_bytes(q, v) > 256
    attention_check(q, k, v, ld, s0, reverse=reverse, lengths=torch.tensor([T, 1300], dtype=torch.int32, device="cuda"))
    attention_check(q[:1], k[:1], v[:1], ld, None, reverse=reverse)


@pytest.mark.parametrize("d", [64, 100])
def test_rows_off_the_copy_engine_in_segments(d):
    # bf16 without 16-byte alignment
    q, k, v, ld, s0 = attention_inputs(1, 3100, 1, d, d, torch.bfloat16, state=True, decay=-0.003, layout="off")
    attention_check(q, k, v, ld, s0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 100, 128])
@pytest.mark.parametrize("T", [1, 2, 300, 2500])
def test_no_memory_at_all(dtype, d, T):
    # log_decay of minus infinity: each position alone, gradients too
    q, k, v, ld, s0 = attention_inputs(1, T, 2, d, d, dtype, state=True, decay=float("-inf"))
    attention_check(q, k, v, ld, s0)
    attention_check(q, k, v, ld, s0, reverse=True)


def test_calls_from_several_threads():
    # each with its own stream and tensors, at the same time
    import threading
    ld = torch.tensor([-0.1, -0.001], device="cuda")

    def work(seed):
        q, k, v, do = (rnd(4 * seed + i, 2, 1500, 2, 64).bfloat16() for i in range(4))
        x = rnd(seed + 100, 4, 700, 32)
        p, g = [rnd(seed + 200, 5000)], [rnd(seed + 300, 5000)]
        m, w, ms, ws = sc.new_adamw_state(p, 8)
        out = []
        for i in range(1, 6):
            leaves = [t.clone().requires_grad_(True) for t in (q, k, v)]
            o = sc.linear_attention(*leaves, ld)
            out += [o.detach(), *torch.autograd.grad(o, leaves, do)]
            y = x.clone().requires_grad_(True)
            z = sc.group_norm(y, 4, activation="silu")
            out += [z.detach(), *torch.autograd.grad(z, y, x)]
            sc.adamw_step(p, g, m, w, i, exp_avg_scale=ms, exp_avg_sq_scale=ws)
        return out + [p[0].clone(), *sc.adamw_state_values(m, ms, "exp_avg")]

    want = [work(s) for s in range(4)]
    torch.cuda.synchronize()
    got = [None] * 4

    def run(s):
        with torch.cuda.stream(torch.cuda.Stream()):
            got[s] = work(s)
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=run, args=(s,)) for s in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
