"""nn.qk_norm_rope's backward pass without norms: the rotation of the gradient
alone, with no memory but the gradients it returns."""
import pytest
import torch

from block_planner_amd import api
from block_planner_amd import nn as htnn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("x,y", [("float32", "float32"), ("float32", "bfloat16"), ("bfloat16", "float32")])
@pytest.mark.parametrize("with_k", [True, False])
def test_backward_without_norms_allocates_its_gradients_only(x, y, with_k):
    T, n, m, d = 2000, 8, 4, 128
    x, y = getattr(torch, x), getattr(torch, y)
    torch.manual_seed(7)
    q = torch.randn(T, n, d, device="cuda").to(x).requires_grad_(True)
    k = torch.randn(T, m, d, device="cuda").to(x).requires_grad_(True) if with_k else None
    pos, inv = torch.arange(T, dtype=torch.int32, device="cuda"), api.rope_inv_freq(d, device="cuda")
    yq, yk = htnn.qk_norm_rope(q, k, pos, inv, out_dtype=y)
    gq, gk = torch.randn(T, n, d, device="cuda").to(y), torch.randn(T, m, d, device="cuda").to(y)
    leaves, outs, grads = ([q, k], [yq, yk], [gq, gk]) if with_k else ([q], [yq], [gq])
    torch.cuda.synchronize()
    asked = lambda: torch.cuda.memory_stats()["requested_bytes.all.allocated"]  # noqa: E731  (all calls so far)
    before = asked()
    got = torch.autograd.grad(outs, leaves, grads)
    torch.cuda.synchronize()
    size = sum(t.numel() * t.element_size() for t in got)
    assert asked() - before <= size + 4096
    # the inverse rotation: forward at the negative positions
    want = api.qk_norm_rope(gq, gk if with_k else None, -pos, inv, out_dtype=x)
    for a, b in zip(got, want):
        assert a.dtype == x and torch.equal(a, b)
