"""Gradients of AddRMSNorm's leaves over several backward calls: x and residual
have one gradient, but their .grad are tensors of their own."""
import pytest
import torch

from block_planner_amd import nn as htnn

pytestmark = pytest.mark.gpu
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.mark.parametrize("shape", [(5, 64), (2, 3, 64), (1, 64), (64,)])
@pytest.mark.parametrize("xt,rt", [("fp32", "fp32"), ("bf16", "bf16"), ("fp32", "bf16"), ("bf16", "fp32")])
@pytest.mark.parametrize("use", ["y", "h", "both"])
def test_leaves_over_several_backward_calls(shape, xt, rt, use):
    print(shape, xt, rt, use, flush=True)
    torch.manual_seed(len(shape))
    x = torch.randn(shape, device="cuda").to(TYPES[xt]).requires_grad_()
    r = torch.randn(shape, device="cuda").to(TYPES[rt]).requires_grad_()
    w = torch.rand(shape[-1], device="cuda").requires_grad_()
    gy, gh = torch.randn(shape, device="cuda"), torch.randn(shape, device="cuda")

    def backward():
        y, h = htnn.add_rms_norm(x, w, r, out_dtype=torch.float32)
        loss = (y * gy).sum() if use != "h" else 0.0
        (loss + ((h.float() * gh).sum() if use != "y" else 0.0)).backward()

    backward()
    assert x.grad.dtype == x.dtype and r.grad.dtype == r.dtype and x.grad.shape == r.grad.shape == shape
    assert x.grad.untyped_storage().data_ptr() != r.grad.untyped_storage().data_ptr()
    once = [t.grad.clone() for t in (x, r)]
    backward()
    backward()
    for t, g in zip((x, r), once):           # 2 g is exact, 3 g is rounded once
        assert torch.equal(t.grad, (3 * g.double()).to(t.dtype))
    r.grad.zero_()
    assert torch.equal(x.grad, (3 * once[0].double()).to(x.dtype))


def test_one_tensor_as_both():
    x = torch.randn(7, 64, device="cuda", requires_grad=True)
    w = torch.rand(64, device="cuda")
    y, _ = htnn.add_rms_norm(x, w, x, out_dtype=torch.float32)
    y.sum().backward()
    z = (2 * x.detach()).requires_grad_()
    y, _ = htnn.add_rms_norm(z, w, out_dtype=torch.float32)
    y.sum().backward()
    assert torch.equal(x.grad, 2 * z.grad)


@pytest.mark.parametrize("shape", [(5, 64), (2, 3, 64), (64,), (0, 64)])
def test_the_norm_may_be_changed_in_place(shape):
    x, r = (torch.randn(shape, device="cuda", requires_grad=True) for _ in range(2))
    w = torch.rand(64, device="cuda")
    y, h = htnn.add_rms_norm(x, w, r, out_dtype=torch.float32)
    y.mul_(2)
    (y.sum() + h.sum()).backward()
    got, x.grad = x.grad, None
    y, h = htnn.add_rms_norm(x, w, r, out_dtype=torch.float32)
    (2 * y.sum() + h.sum()).backward()
    assert torch.equal(got, x.grad)
    y, h = htnn.add_rms_norm(x, w, r)
    with pytest.raises(RuntimeError, match="modified by an inplace"):        # the backward pass reads it
        h.mul_(2)
        (y.sum() + h.sum()).backward()
