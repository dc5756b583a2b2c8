"""AddRMSNorm, token_logprobs and distill_loss as modules: autograd against the
formulas in 64 bits, chains of them with the quantised linears, HIP graphs,
streams."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import logits_reference as ref
from block_planner_amd import api
from block_planner_amd import binding as B
from block_planner_amd import nn as htnn

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def dev():
    return torch.device("cuda:0")


def host(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("x,r,y", [("fp32", "fp32", "bf16"), ("bf16", "fp32", "fp32"), ("fp32", "bf16", "bf16"), ("fp32", None, "fp32")])
def test_norm_autograd(x, r, y):
    """Both outputs used, leading dims, the expanded gradient of a sum; the
    formulas' gradients as in the operator's own test."""
    T = ref.TYPES
    torch.manual_seed(0)
    xs = torch.randn(2, 9, 136, device=dev()).to(T[x]).requires_grad_()
    rs = torch.randn(2, 9, 136, device=dev()).to(T[r]).requires_grad_() if r else None
    norm = htnn.AddRMSNorm(136, eps=1e-5, out_dtype=T[y])
    with torch.no_grad():
        norm.weight.add_(0.3 * torch.randn(136, device=dev()))
    out, h = norm(xs, rs)
    assert out.dtype == T[y] and out.shape == xs.shape
    dy = torch.randn_like(out)
    if r:
        assert h.dtype == T[r] and h.shape == xs.shape
        ((out * dy).sum() + 0.5 * h.sum()).backward()
    else:
        assert h is None
        (out * dy).sum().backward()
    hn = host(h if r else xs).reshape(-1, 136)
    dh = np.full_like(hn, 0.5) if r else None
    w = host(norm.weight)
    d, dw = ref.norm_backward(host(dy).reshape(-1, 136), hn, w, dh, 1e-5)
    for leaf, t in ((xs, x), (rs, r)):
        if leaf is not None:
            assert leaf.grad.dtype == T[t]
            tol = 512 * U * np.abs(d).max() + (ref.HALF[t] * np.abs(d) if t == "bf16" else 0)
            assert np.all(np.abs(host(leaf.grad).reshape(-1, 136) - d) <= tol)
    assert np.all(np.abs(host(norm.weight.grad) - dw) <= 512 * U * np.abs(dw).max() + 1e-30)


def test_norm_with_one_output_used():
    """Gradients where only the sum, or only the norm, is used."""
    x, r = (torch.randn(5, 64, device=dev(), requires_grad=True) for _ in range(2))
    norm = htnn.AddRMSNorm(64, out_dtype=torch.float32)
    norm(x, r)[1].sum().backward()
    assert torch.all(x.grad == 1) and torch.all(r.grad == 1) and norm.weight.grad is None
    x.grad = r.grad = None
    norm(x, r)[0].square().sum().backward()
    assert torch.equal(x.grad, r.grad) and norm.weight.grad is not None
    norm.bfloat16()                                     # casts of the module: the kernels still read fp32
    y, _ = norm(x, r)
    y.sum().backward()
    assert torch.isfinite(y).all() and norm.weight.grad.dtype == torch.bfloat16


def test_token_logprobs_autograd():
    torch.manual_seed(1)
    V = 777
    x = (3 * torch.randn(2, 5, V, device=dev())).requires_grad_()
    for tokens in (torch.randint(0, V, (2, 5), device=dev()), torch.randint(0, V, (2, 5, 3), device=dev(), dtype=torch.int16)):
        tokens.view(-1)[0] = -100
        g, e = torch.randn(tokens.shape, device=dev()), torch.randn(2, 5, device=dev())
        logp, ent = htnn.token_logprobs(x, tokens, temperature=0.9)
        assert logp.shape == tokens.shape and ent.shape == (2, 5)
        flat = host(tokens).astype(int).reshape(10, -1)
        want, went, _, _, b1, b2, _ = ref.token_logprobs(host(x).reshape(10, V), flat, 0, 0.9)
        assert np.all(np.abs(host(logp).reshape(10, -1) - want) <= b1 * U) and np.all(np.abs(host(ent).reshape(-1) - went) <= b2 * U)
        x.grad = None
        ((logp * g).sum() + (ent * e).sum()).backward()
        dx, tol = ref.gradient(host(x).reshape(10, V), 0.9, flat, host(g).reshape(10, -1), host(e).reshape(-1))
        assert np.all(np.abs(host(x.grad).reshape(10, V) - dx) <= tol * U)
        x.grad = None
        htnn.token_logprobs(x, tokens)[0].neg_().sum().backward()        # one output, changed in place
        dx, tol = ref.gradient(host(x).reshape(10, V), 1.0, flat, -np.ones(flat.shape), np.zeros(10))
        assert np.all(np.abs(host(x.grad).reshape(10, V) - dx) <= tol * U)


@pytest.mark.parametrize("t", ["fp32", "bf16"])
def test_distill_autograd(t):
    """The gradient under an upstream factor, a second backward call, no
    gradient, the mean over rows."""
    torch.manual_seed(2)
    V, k = 5003, 9
    x = (3 * torch.randn(3, 4, V, device=dev())).to(ref.TYPES[t]).requires_grad_()
    ids = torch.randint(0, V, (3, 4, k), device=dev())
    ids[0, 0, 3:] = -1
    tv = torch.randn(3, 4, k, device=dev())
    w = torch.rand(3, 4, device=dev())
    w[1, 1] = 0
    want, dx, bl, bx = ref.distill(host(x).reshape(12, V), host(ids).astype(int).reshape(12, k), host(tv).reshape(12, k), 2.0,
                                   host(w).reshape(-1))
    total = (host(w).reshape(-1) * want).sum()
    loss = htnn.distill_loss(x, ids, tv, w, temperature=2.0)
    with torch.no_grad():
        alone = htnn.distill_loss(x, ids, tv, w, temperature=2.0)
    bound = (np.abs(host(w).reshape(-1)) * (bl + 16 * np.abs(want))).sum() * U
    assert abs(loss.item() - total) <= bound and abs(alone.item() - total) <= bound
    for factor in (1.0, 3.0):                           # the kept gradient, then one from the statistics
        x.grad = None
        (loss * factor).backward(retain_graph=True)
        extra = ref.HALF[t] * 2 * factor * np.abs(dx) if t == "bf16" else 2 * U * factor * np.abs(dx)
        assert x.grad.dtype == x.dtype
        assert np.all(np.abs(host(x.grad).reshape(12, V) - factor * dx) <= factor * bx * U + extra + 2.0 ** -120)
    x.grad = None
    (htnn.distill_loss(x, ids, tv, w, temperature=2.0) * 3.0).backward()   # the kept one, scaled: rounded twice in bf16
    extra = 2.01 * ref.HALF[t] * 3 * np.abs(dx) if t == "bf16" else 4 * U * 3 * np.abs(dx)
    assert np.all(np.abs(host(x.grad).reshape(12, V) - 3 * dx) <= 3 * bx * U + extra + 2.0 ** -120)
    mean = htnn.distill_loss(x.detach(), ids, tv, temperature=2.0).item()
    full, _, bl, _ = ref.distill(host(x).reshape(12, V), host(ids).astype(int).reshape(12, k), host(tv).reshape(12, k), 2.0, np.ones(12))
    assert abs(mean - full.mean()) <= (bl + 16 * np.abs(full)).mean() * U


def test_scale_rows():
    for dt in (torch.float32, torch.bfloat16):
        for V, pad in ((7, 0), (1003, 1), (40000, 0)):
            wide = torch.randn(5, V + pad, device=dev()).to(dt)
            x = wide[:, pad:]
            want = (x.float() * 0.37).to(dt)
            keep = x.clone()
            api.scale_rows(x, torch.ones(1, device=dev()))
            assert torch.equal(x, keep)
            api.scale_rows(x, torch.full((1,), 0.37, device=dev()))
            assert torch.equal(x, want)


def models(seed=3, hidden=256, vocab=1200):
    torch.manual_seed(seed)
    teacher = torch.nn.Linear(hidden, vocab, bias=False, device=dev())
    with torch.no_grad():
        teacher.weight.mul_(4)
    student = htnn.HyperLinear.from_linear(teacher, inference_only=False, eps_int4=0.5)
    return teacher, student, htnn.AddRMSNorm(hidden)


def test_a_training_step_from_the_teacher_to_the_norm():
    """Residual and norm, the quantised linear, the teacher's alternatives, the
    loss, and back: every gradient against the chain of formulas in 64 bits
    (the linear's backward kernels are good to 1e-3 of the largest entry)."""
    hidden, M, k = 256, 70, 16
    teacher, student, norm = models(hidden=hidden)
    x, r = (torch.randn(M, hidden, device=dev(), requires_grad=True) for _ in range(2))
    with torch.no_grad():
        h = x + r
        kept = api.token_logprobs(teacher(h), top=k)
    y, h = norm(x, r)
    logits = student(y)
    w = torch.rand(M, device=dev())
    loss = htnn.distill_loss(logits, kept.top_tokens, kept.top_logprobs, w, temperature=1.5)
    (loss + 0.1 * h.sum()).backward()
    What = host(api_dequant(student))
    _, dl, _, bl = ref.distill(host(logits), host(kept.top_tokens).astype(int), host(kept.top_logprobs), 1.5, host(w))
    dy = dl @ What
    dW = dl.T @ host(y)
    d, dw = ref.norm_backward(dy, host(h), host(norm.weight), np.full((M, hidden), 0.1), norm.eps)
    assert np.abs(host(student.weight.grad) - dW).max() <= 1e-3 * np.abs(dW).max()
    # dy reaches the norm rounded to y's type, bf16
    scale = np.abs(dy).max() * (1e-3 + 2.0 ** -8) * np.abs(host(norm.weight)).max()
    rn = 1 / np.sqrt((host(h) ** 2).mean(-1, keepdims=True) + norm.eps)
    assert np.all(np.abs(host(x.grad) - d) <= 4 * scale * rn + 1e-6) and torch.equal(x.grad, r.grad)
    assert np.abs(host(norm.weight.grad) - dw).max() <= (1e-3 + 2.0 ** -8) * np.abs(dy).max() * np.abs(host(h) * rn).sum(0).max()


def api_dequant(layer):
    """W_hat of a HyperLinear: the linear of the unit rows."""
    eye = torch.eye(layer.in_features, device=dev(), dtype=torch.bfloat16)
    with torch.no_grad():
        return api.linear(layer.packed, eye).t().contiguous()


def test_serving_in_8_bits():
    """Norms in 8 bits into quantised linears, layer after layer, and what the
    last one says: against the same rows' values through the bf16 paths."""
    torch.manual_seed(4)
    hidden, M = 512, 96
    lins = [htnn.HyperLinear.from_linear(torch.nn.Linear(hidden, n, bias=False, device=dev())) for n in (hidden, hidden, 1500)]
    norms = [htnn.AddRMSNorm(hidden, bits8=True) for _ in lins]
    x = torch.randn(M, hidden, device=dev())
    with torch.no_grad():
        h, out = None, x
        for norm, lin in zip(norms, lins):
            rows, h2 = norm(out, h)
            seen = out if h is None else out + h
            want, _ = api.add_rms_norm_q8(seen, norm.weight)
            assert torch.equal(api.q8_values(rows), api.q8_values(want))
            h = seen if h2 is None else h2
            out = lin(rows)
            plain = api.linear(lin.packed, api.q8_values(rows))
            assert (out - plain).abs().max() <= 1e-3 * plain.abs().max()
        r = api.token_logprobs(out, top=10)
    assert r.top_tokens.shape == (M, 10) and torch.isfinite(r.entropy).all()
    lin = htnn.HyperLinear.from_linear(torch.nn.Linear(hidden, 64, bias=False, device=dev()), inference_only=False)
    with pytest.raises(RuntimeError, match="no backward pass"):
        lin(rows)
    with torch.no_grad(), pytest.raises(ValueError, match="input features"):
        htnn.HyperLinear.from_linear(torch.nn.Linear(256, 64, bias=False, device=dev()))(rows)


def captured(call, refill, rounds=6):
    """call() captured once and replayed, inputs changed between, with eager
    work beside it; every replay against the eager result."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for i in range(rounds):
        refill(i)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = call()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), i


def test_operators_in_graphs():
    """Serving (norm in 8 bits, linear, log probabilities of rows in parts) and
    training calls (norm and its gradients' partial sums, the step, both
    gradients) captured, two graphs of the first kind replayed in turn."""
    torch.manual_seed(5)
    hidden, V, M = 256, 40000, 40
    pw = api.pack(W := torch.randn(V, hidden, device=dev()) / 16, api.plan(W))
    x, r = torch.randn(M, hidden, device=dev()), torch.randn(M, hidden, device=dev())
    w = torch.rand(hidden, device=dev())
    ids = torch.randint(0, V, (M,), dtype=torch.int32, device=dev())

    def serve():
        rows, h = api.add_rms_norm_q8(x, w, r)
        o = api.token_logprobs(api.linear(pw, rows), ids, top=8)
        return h, o.logprobs, o.entropy, o.top_logprobs, o.top_tokens

    def refill(i):
        x.normal_(), r.normal_(), ids.random_(0, V)

    captured(serve, refill)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = serve()
        graphs.append((g, out))
    refill(0)
    want = serve()
    for _ in range(3):
        for g, out in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))

    M, V, k = 300, 20011, 6
    lg, t2 = torch.randn(M, V, device=dev()) * 2, torch.randn(M, k, device=dev())
    i2 = torch.randint(0, V, (M, k), dtype=torch.int32, device=dev())
    wt, tok = torch.rand(M, device=dev()), torch.randint(0, V, (M,), dtype=torch.int32, device=dev())
    dy, h = torch.randn(900, hidden, device=dev()), torch.randn(900, hidden, device=dev())
    ge = torch.randn(M, device=dev())

    def train():
        loss, d = api.distill_step(lg, i2, t2, wt, temperature=2.0)
        l2, st = api.distill_loss(lg, i2, t2, temperature=2.0)
        o = api.token_logprobs(lg, tok)
        return (loss, d, l2, api.distill_backward(wt, lg, i2, t2, st, temperature=2.0), o.logprobs,
                api.token_logprobs_backward(wt, ge, lg, tok, o.stats, o.entropy), *api.add_rms_norm_backward(dy, h, w))

    captured(train, lambda i: (lg.normal_(), t2.normal_(), i2.random_(0, V), wt.uniform_(), dy.normal_(), h.normal_()))


def test_training_loss_in_a_graph():
    """Loss and gradient of the module, forward and backward captured, over more
    rows than one workgroup adds; the loss within its sum's rounding (four
    stages of at most 256 entries, 1024 in the last, and the product)."""
    torch.manual_seed(7)
    M, V, k = 70001, 40, 5
    x = torch.randn(M, V, device=dev()).requires_grad_()
    t, ids = torch.randn(M, k, device=dev()), torch.randint(0, V, (M, k), device=dev())
    w = torch.rand(M, device=dev())
    with torch.no_grad():
        eager = htnn.distill_loss(x, ids, t, w)

    def call():
        loss = htnn.distill_loss(x, ids, t, w)
        return loss.detach(), torch.autograd.grad(loss, x)[0]

    captured(call, lambda i: (x.detach().normal_(), t.normal_(), ids.random_(0, V), w.uniform_()))
    got, _ = call()
    terms = host(w) * host(api.distill_loss(x.detach(), ids.int(), t)[0])
    assert abs(got.item() - terms.sum()) <= (3 * 256 + 1024 + 1) * U * np.abs(terms).sum() and got != eager


def test_no_tokens_a_row():
    x = torch.randn(3, 2, 50, device=dev()).requires_grad_()
    lp, ent = htnn.token_logprobs(x, torch.empty(3, 2, 0, dtype=torch.long, device=dev()))
    assert lp.shape == (3, 2, 0) and ent.shape == (3, 2)
    ent.sum().backward()
    assert torch.isfinite(x.grad).all()


def test_two_streams_at_once():
    """Calls of the same kind on two streams, each with its own temporaries."""
    torch.manual_seed(6)
    x = [torch.randn(8, 70000, device=dev()) for _ in range(2)]
    want = [api.token_logprobs(t, top=20) for t in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        got = [api.token_logprobs(t, top=20, stream=s) for t, s in zip(x, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.top_tokens, b.top_tokens) and torch.equal(a.entropy, b.entropy)


def test_the_example_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "distill_head.py"), "--steps", "6", "--rows", "256",
                        "--vocab", "4000", "--hidden", "512"], capture_output=True, text=True, timeout=110)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "rows/s" in r.stdout
