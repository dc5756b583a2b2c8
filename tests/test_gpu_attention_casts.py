"""HyperAttention as a module among others: casts, gradients."""
import pytest
import torch

from block_planner_amd import nn as htnn

pytestmark = pytest.mark.gpu


def dev():
    return torch.device("cuda:0")


class Same(torch.nn.Module):
    def forward(self, o):
        return o.float()


def layer(seed=3, **kw):
    torch.manual_seed(seed)
    lin = torch.nn.Linear(128, (8 + 2 * 2) * 64, bias=False, device=dev())
    return htnn.HyperAttention(htnn.HyperLinear.from_linear(lin), Same(), 8, 2, 64, **kw)


def step(att, x, q_len=(70, 3)):
    pool = htnn.KVPool(1, 12, 2, 64, len(q_len), 6, dev())
    with torch.no_grad():
        return att(x, pool, 0, pool.plan(list(q_len)))


@pytest.mark.parametrize("cast", ["float", "half", "bfloat16", "to", "double"])
@pytest.mark.parametrize("qk_norm", [True, False])
def test_casts_of_the_module(cast, qk_norm):
    """The frequencies stay in 64 bits (a cast would lose the phase of far
    positions); the norm's weights are cast like any weight and used in 32 bits."""
    x = torch.randn(73, 128, device=dev())
    att = layer(qk_norm=qk_norm, base=500000.0)
    if qk_norm:
        with torch.no_grad():   # values that every type holds
            att.q_weight.copy_(torch.randint(8, 24, (64,), device=dev()) / 16)
            att.k_weight.copy_(torch.randint(8, 24, (64,), device=dev()) / 16)
    want, freq = step(att, x), att.inv_freq.clone()
    moved = torch.nn.Sequential(att)
    moved = moved.to(torch.bfloat16) if cast == "to" else getattr(moved, cast)()
    assert moved[0] is att and att.inv_freq.dtype == torch.float64 and torch.equal(att.inv_freq, freq)
    assert torch.equal(step(att, x), want)


def test_moves_of_the_module():
    """To the host and back: the frequencies move, and are the same."""
    att = layer()
    freq = att.inv_freq.clone()
    att.cpu()
    assert att.inv_freq.device.type == "cpu" and torch.equal(att.inv_freq, freq.cpu())
    att.to(dev())
    assert att.inv_freq.is_cuda and torch.equal(att.inv_freq, freq)


def test_a_module_made_without_memory():
    """Moved from the meta device by to_empty, as any module."""
    att = layer()
    att.to("meta")
    assert att.inv_freq.is_meta
    att.to_empty(device=dev())
    assert att.inv_freq.is_cuda and att.inv_freq.dtype == torch.float64


def test_gradients_are_refused():
    """No backward pass goes through the cache: where something asks for
    gradients the call raises, instead of returning an output that none reach.
    Under no_grad, and where nothing asks, it runs."""
    x = torch.randn(73, 128, device=dev())
    pool = htnn.KVPool(1, 12, 2, 64, 2, 6, dev())
    att = layer(qk_norm=True)
    want = step(att, x)
    assert torch.equal(att(x, pool, 0, pool.plan([70, 3])), want)   # the norm's weights do not ask by themselves
    trained = layer(qk_norm=True)
    trained.q_weight.requires_grad_(True)
    lin = torch.nn.Linear(128, (8 + 2 * 2) * 64, bias=False, device=dev())
    for a, y in ((att, x.clone().requires_grad_(True)), (trained, x),
                 (htnn.HyperAttention(lin, Same(), 8, 2, 64), x),
                 (htnn.HyperAttention(htnn.HyperLinear.from_linear(lin, inference_only=False), Same(), 8, 2, 64), x)):
        with pytest.raises(RuntimeError, match="no_grad"):
            a(y, pool, 0, pool.plan([1, 72]))
        pool.release([True, True])
        plan = pool.plan([70, 3])
        with torch.no_grad():
            out = a(y, pool, 0, plan)
        assert not out.requires_grad
        with torch.inference_mode():
            assert torch.equal(a(y, pool, 0, plan), out)
