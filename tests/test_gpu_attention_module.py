"""HyperAttention over a KVPool, qk_norm_rope's autograd, and the operators in
HIP graphs, on the GPU."""
import numpy as np
import pytest
import torch

import kv_reference as ref
from block_planner_amd import api
from block_planner_amd import nn as htnn

pytestmark = pytest.mark.gpu


def dev():
    return torch.device("cuda:0")


class Tap(torch.nn.Module):
    """An output linear that keeps what it is given."""

    def forward(self, o):
        self.seen = o
        return o.float()


@pytest.mark.parametrize("qk_norm,window", [(True, 0), (False, 50)])
def test_attention_over_steps(qk_norm, window):
    """Prompts, single tokens, a release with a new prompt in its place: the
    cache equals the host's bit for bit, the attention is within the host's
    bound for it, pages are accounted for."""
    torch.manual_seed(1)
    R, n, m, d, hidden = 4, 8, 2, 64, 128
    lin = torch.nn.Linear(hidden, (n + 2 * m) * d, bias=False, device=dev())
    att = htnn.HyperAttention(htnn.HyperLinear.from_linear(lin), Tap(), n, m, d, qk_norm=qk_norm, window=window)
    if qk_norm:
        with torch.no_grad():
            att.q_weight.add_(0.2 * torch.randn(d, device=dev()))
            att.k_weight.add_(0.2 * torch.randn(d, device=dev()))
    pool = htnn.KVPool(1, 20, m, d, R, 8, dev())
    codes, scales = (t.cpu().numpy() for t in pool.caches[0])
    steps = [[70, 3, 0, 130], [1, 1, 0, 1], [1, 1, 64, 1], [1, 60, 1, 1], None, [1, 5, 20, 1], [1, 1, 1, 1]]
    for q_len in steps:
        if q_len is None:
            pool.release([False, True, True, False])
            continue
        step = pool.plan(q_len)
        x = torch.randn(sum(q_len), hidden, device=dev())
        out = att(x, pool, 0, step)
        assert int(step.status[1]) == 0 and out.shape == (sum(q_len), n * d)
        y = att.qkv(x).detach().unflatten(1, (n + 2 * m, d))
        q, k = api.qk_norm_rope(y[:, :n], y[:, n:n + m], step.positions, att.inv_freq, att.q_weight, att.k_weight,
                                att.eps, out_dtype=torch.bfloat16)
        codes, scales = ref.write(k.float().cpu().numpy(), y[:, n + m:].cpu().numpy(), step.slots.cpu().numpy(), codes,
                                  scales)
        np.testing.assert_array_equal(pool.caches[0][0].cpu().numpy(), codes)
        np.testing.assert_array_equal(pool.caches[0][1].cpu().numpy(), scales)
        want, tol = ref.attention(q.float().cpu().numpy(), codes, scales, pool.table.cpu().numpy(),
                                  step.cu_q.cpu().numpy(), step.kv_len.cpu().numpy(), 1 / np.sqrt(d), True, window)
        got = att.out.seen.unflatten(1, (n, d)).double().cpu().numpy()
        assert np.all(np.abs(got - want) <= tol)
        held = [int(p) for r in range(R) for p in pool.table[r, :int(pool.owned[r])]]
        free = pool.free_pages[:int(pool.n_free)].tolist()
        assert sorted(held + free) == list(range(20))


def test_pool_refuses_and_recovers():
    """A request that finds no pages stores nothing and keeps its length."""
    pool = htnn.KVPool(1, 3, 1, 64, 2, 4, dev())
    step = pool.plan([100, 100])
    assert step.status.tolist() == [1, 1] and pool.kv_len.tolist() == [100, 0]
    assert torch.all(step.slots[100:] == -1)
    pool.release([True, False])
    step = pool.plan([0, 100])
    assert step.status.tolist() == [1, 0] and pool.kv_len.tolist() == [0, 100]
    with pytest.raises(ValueError):
        pool.plan([1])
    with pytest.raises(ValueError):
        pool.plan(torch.ones(2, dtype=torch.int32, device=dev()))


@pytest.mark.parametrize("x,y,norm", [("fp32", "fp32", True), ("fp32", "bf16", True), ("fp32", "fp32", False)])
def test_autograd(x, y, norm):
    """Gradients through autograd equal the backward call's; a k that is not
    used gets zeros; a broadcast upstream gradient is read correctly."""
    types = {"fp32": torch.float32, "bf16": torch.bfloat16}
    torch.manual_seed(2)
    T, n, m, d = 21, 4, 2, 64
    q = torch.randn(T, n, d, device=dev(), dtype=types[x], requires_grad=True)
    k = torch.randn(T, m, d, device=dev(), dtype=types[x], requires_grad=True)
    w = [torch.randn(d, device=dev(), requires_grad=True) if norm else None for _ in range(2)]
    pos, inv = torch.arange(T, dtype=torch.int32, device=dev()), api.rope_inv_freq(d, device=dev())
    yq, yk = htnn.qk_norm_rope(q, k, pos, inv, *w, out_dtype=types[y])
    gq, gk = torch.randn_like(yq), torch.randn_like(yk)
    leaves = [q, k] + (w if norm else [])
    got = torch.autograd.grad([yq, yk], leaves, [gq, gk], retain_graph=True)
    want = api.qk_norm_rope_backward(gq, gk, q.detach(), k.detach(), pos, inv,
                                     *(t.detach() if norm else None for t in w))
    for g, v in zip(got, want):
        assert torch.equal(g, v)
    assert torch.all(torch.autograd.grad(yq.sum(), k, retain_graph=True)[0] == 0)
    one = torch.autograd.grad(yq.sum(), q)[0]           # gradient of a sum: an expanded tensor of ones
    flat = api.qk_norm_rope_backward(torch.ones_like(yq), torch.zeros_like(yk), q.detach(), k.detach(), pos, inv,
                                     *(t.detach() if norm else None for t in w))[0]
    assert torch.equal(one, flat)


def test_calls_on_a_given_stream():
    """stream= with inputs that are copied first (misaligned), while the
    current stream reuses memory: the same bits as on the current stream."""
    torch.manual_seed(4)
    T, n, m, d = 300, 8, 2, 64
    odd = lambda h: torch.randn(T * h * d + 1, device=dev())[1:].view(T, h, d)  # noqa: E731
    q, k, v, dq, dk = odd(n), odd(m), odd(m), odd(n), odd(m)
    w = [torch.randn(d, device=dev()) for _ in range(2)]
    pos, inv = torch.arange(T, dtype=torch.int32, device=dev()), api.rope_inv_freq(d, device=dev())
    ints = lambda a: torch.tensor(a, dtype=torch.int32, device=dev())  # noqa: E731
    got = []
    for side in (None, torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        codes, scales = api.kv_cache(12, m, d, dev())
        table = torch.full((2, 6), -1, dtype=torch.int32, device=dev())
        torch.cuda.synchronize()
        step = api.kv_plan(ints([100, 200]), ints([0, 0]), ints([0, 0]), table, ints(list(range(12))), ints([12]), T,
                           stream=side)
        yq, yk = api.qk_norm_rope(q, k, pos, inv, *w, out_dtype=torch.bfloat16, stream=side)
        api.kv_write(yk, v, step.slots, codes, scales, stream=side)
        o = api.kv_attention(yq, codes, scales, table, step.cu_q, step.kv_len, 200, stream=side)
        g = api.qk_norm_rope_backward(dq, dk, q, k, pos, inv, *w, stream=side)
        junk = [torch.full((T, n, d), 9.0, device=dev()) for _ in range(8)]   # what the copies' memory would become
        torch.cuda.synchronize()
        del junk
        got.append([t.clone() for t in (*step, table, yq, yk, codes, scales, o, *g)])
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert torch.equal(a, b)


def test_decode_step_in_a_graph():
    """Norm, write and attention of a decode step in one HIP graph, replayed
    with other inputs and lengths, against the same calls made eagerly; the
    program's own work in between."""
    rng = np.random.default_rng(3)
    R, n, m, d, width = 5, 8, 2, 128, 40
    kv = np.array([3, 2000, 64, 700, 1], np.int32)
    codes, scales = (torch.from_numpy(a).to(dev()) for a in ref.random_cache(rng, 120, m, d))
    table = torch.from_numpy(ref.random_table(rng, kv + 40, 120, width)).to(dev())
    cu = torch.arange(R + 1, dtype=torch.int32, device=dev())
    y = torch.randn(R, n + 2 * m, d, device=dev())
    lens = torch.from_numpy(kv).to(dev())
    slots, pos = torch.zeros(R, dtype=torch.int32, device=dev()), torch.zeros(R, dtype=torch.int32, device=dev())
    inv = api.rope_inv_freq(d, device=dev())

    def step(c, s):
        q, k = api.qk_norm_rope(y[:, :n], y[:, n:n + m], pos, inv, out_dtype=torch.bfloat16)
        api.kv_write(k, y[:, n + m:], slots, c, s)
        return api.kv_attention(q, c, s, table, cu, lens, 1)

    def place(i):
        y.copy_(torch.randn(R, n + 2 * m, d, generator=torch.Generator(device=dev()).manual_seed(i), device=dev()))
        at = torch.from_numpy(kv).to(dev()) + i
        pos.copy_(at)
        slots.copy_(table.gather(1, (at // 64).long()[:, None])[:, 0] * 64 + at % 64)
        lens.copy_(at + 1)

    place(0)
    c2, s2 = codes.clone(), scales.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(c2, s2)
    torch.cuda.current_stream().wait_stream(side)
    c2.copy_(codes)
    s2.copy_(scales)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(c2, s2)
    for i in range(6):
        place(i)
        graph.replay()
        torch.cuda.synchronize()
        want = step(codes, scales)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(c2, codes) and torch.equal(s2, scales), i


def test_plan_and_backward_in_a_graph():
    """The page plan and the backward call (which adds partial sums) captured
    and replayed."""
    T, n, m, d = 300, 8, 2, 64
    q, k = torch.randn(T, n, d, device=dev()), torch.randn(T, m, d, device=dev())
    dq, dk = torch.randn_like(q), torch.randn_like(k)
    w = [torch.randn(d, device=dev()) for _ in range(2)]
    pos, inv = torch.arange(T, dtype=torch.int32, device=dev()), api.rope_inv_freq(d, device=dev())
    ints = lambda a: torch.tensor(a, dtype=torch.int32, device=dev())  # noqa: E731
    q_len, kv, owned, free, n_free = ints([100, 0, 200]), ints([0, 3, 64]), ints([0, 1, 1]), ints(list(range(9))), ints([9])
    table = torch.full((3, 6), -1, dtype=torch.int32, device=dev())
    step = api.kv_step(3, T, dev())

    def call():
        api.kv_plan(q_len, kv, owned, table, free, n_free, T, out=step)
        return api.qk_norm_rope_backward(dq, dk, q, k, pos, inv, *w)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for i in range(5):
        dq.normal_(), dk.normal_(), q.normal_(), k.normal_()
        q_len.copy_(ints([100 - 7 * i, i, 200 + 6 * i]))
        graph.replay()
        torch.cuda.synchronize()
        seen = [t.clone() for t in (*out, *step, table)]
        want = call()
        torch.cuda.synchronize()
        for a, b in zip(seen, (*want, *step, table)):
            assert torch.equal(a, b), i
