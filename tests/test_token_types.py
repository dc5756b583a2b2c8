"""Tokens of any whole type: those outside [0, V) stay outside, the others keep
their value, on the host and through the differentiable operators."""
import pytest
import torch

from block_planner_amd import nn as htnn

WHOLE = [torch.uint8, torch.int8, torch.int16, torch.int32, torch.int64, torch.uint16, torch.uint32, torch.uint64]


def values(dtype, V):
    """Every kind of value the type has: ordinary, the borders of [0, V), its own."""
    info = torch.iinfo(dtype)
    v = {0, 1, 5, 77, V - 1, V, V + 1, -1, -2, info.min, info.max, 2 ** 32 + 3, 2 ** 63 + 1}
    return sorted(x for x in v if info.min <= x <= info.max)


def tensor(v, dtype):
    if dtype is torch.uint64:
        return torch.tensor([x - 2 ** 64 if x >= 2 ** 63 else x for x in v]).view(dtype)
    return torch.tensor(v, dtype=torch.int64).to(dtype)


@pytest.mark.parametrize("dtype", WHOLE)
@pytest.mark.parametrize("V", [1, 100, 127, 128, 255, 256, 1003, 32767, 50001, 1 << 29])
def test_values_on_the_host(dtype, V):
    v = values(dtype, V)
    got = htnn._int32(tensor(v, dtype), V)
    assert got.dtype == torch.int32 and got.is_contiguous()
    for x, y in zip(v, got.tolist()):
        assert y == x if 0 <= x < V else not 0 <= y < V, (dtype, V, x, y)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.bool, torch.complex64])
def test_other_types_are_refused(dtype):
    with pytest.raises(ValueError, match="whole numbers"):
        htnn._int32(torch.zeros(3, dtype=dtype), 10)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.uint8, torch.int8, torch.int16, torch.int64])
@pytest.mark.parametrize("V", [100, 1003, 50001])
def test_through_the_operators(dtype, V):
    print(dtype, V, flush=True)
    v = [x for x in values(dtype, V) if abs(x) < 2 ** 40]
    tokens = tensor(v, dtype).cuda()
    x = torch.randn(len(v), V, device="cuda", requires_grad=True)
    logp, _ = htnn.token_logprobs(x, tokens)
    want = torch.log_softmax(x.detach().double(), -1)
    for i, t in enumerate(v):
        assert logp[i].item() == pytest.approx(want[i, t].item() if 0 <= t < V else 0.0, abs=1e-4)
    logp.sum().backward()
    live = torch.tensor([0 <= t < V for t in v])
    assert torch.equal((x.grad != 0).any(1).cpu(), live)
    y = torch.randn(len(v), V, device="cuda", requires_grad=True)
    teacher = torch.zeros(len(v), 1, device="cuda")
    loss = htnn.distill_loss(y, tokens[:, None], teacher, torch.ones(len(v), device="cuda"))
    want = -sum(torch.log_softmax(y.detach().double(), -1)[i, t].item() for i, t in enumerate(v) if 0 <= t < V)
    assert loss.item() == pytest.approx(want, rel=1e-5)
