"""What linear attention and group norm find on the device reaches who calls them without a
workspace of their own."""
import pytest

pytestmark = pytest.mark.gpu

import torch  # noqa: E402

import semi_markov_crf_prefix_b200 as sc  # noqa: E402

BAD = sc._lib.SEMICRF_ERR_INVALID_LENGTH


@pytest.fixture(autouse=True)
def cleared():
    sc.clear_device_status()
    yield
    sc.clear_device_status()


def attention(dtype, T, lengths, grad=False):
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(2, T, 2, 64, generator=g, device="cuda").to(dtype).requires_grad_(grad) for _ in range(3))
    ld = torch.tensor([-0.1, -0.01], device="cuda")
    o = sc.linear_attention(q, k, v, ld, lengths=torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    return o, (q, k, v)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [1, 150, 3000])
def test_lengths_of_linear_attention(dtype, T):
    attention(dtype, T, [T, 0])
    assert sc.device_status() == 0
    attention(dtype, T, [T, T + 1])
    assert sc.device_status() == BAD and sc.device_status() == BAD     # until it is cleared
    attention(dtype, T, [T, 0])
    assert sc.device_status(device="cuda") == BAD
    sc.clear_device_status()
    assert sc.device_status() == 0
    o, leaves = attention(dtype, T, [-1, T], grad=True)
    sc.clear_device_status()
    torch.autograd.grad(o.float().sum(), leaves)
    assert sc.device_status() == BAD


@pytest.mark.parametrize("shape,groups", [((2, 40, 8), 2), ((2, 9000, 8), 2), ((2, 1, 8), 2)])
def test_lengths_of_group_norm(shape, groups):
    x = torch.randn(*shape, device="cuda", requires_grad=True)
    good = torch.tensor([shape[1], 0], dtype=torch.int32, device="cuda")
    y = sc.group_norm(x, groups, lengths=good)
    torch.autograd.grad(y.sum(), x)
    assert sc.device_status() == 0
    y = sc.group_norm(x, groups, lengths=good + 1)
    assert sc.device_status() == BAD
    sc.clear_device_status()
    torch.autograd.grad(y.sum(), x)
    assert sc.device_status() == BAD
    sc.clear_device_status()
    with torch.no_grad():
        sc.group_norm(x, groups, lengths=good - 1)
    assert sc.device_status() == BAD


def test_captured_and_on_another_stream():
    x = torch.randn(2, 40, 8, device="cuda")
    lengths = torch.tensor([40, 40], dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sc.group_norm(x, 2, lengths=lengths)
    graph.replay()
    assert sc.device_status() == 0
    lengths[0] = 41
    graph.replay()
    assert sc.device_status() == BAD
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        sc.clear_device_status()
        sc.group_norm(x, 2, lengths=lengths)
        assert sc.device_status() == BAD


def test_a_workspace_keeps_its_own_word():
    x = torch.randn(2, 40, 8, device="cuda")
    lengths = torch.tensor([41, 40], dtype=torch.int32, device="cuda")
    ws, other = (torch.zeros(1 << 16, dtype=torch.uint8, device="cuda") for _ in range(2))
    sc.group_norm_forward(x, 2, lengths=lengths, ws=ws)
    sc.group_norm_forward(x, 2, ws=other)
    assert sc.device_status(ws) == BAD and sc.device_status(other) == 0 and sc.device_status() == BAD
    sc.clear_device_status(ws)
    assert sc.device_status(ws) == 0 and sc.device_status() == BAD
