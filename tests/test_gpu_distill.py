"""The distillation loss, its gradient and the step on the GPU against the
formulas in 64 bits; tolerances are derived in logits_reference."""
import numpy as np
import pytest
import torch

import logits_reference as ref
from block_planner_amd import api
from test_gpu_logprobs import INF, check, dev, logits, put

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES, HALF = ref.TYPES, ref.HALF


def teacher(rng, h, k):
    """Ids among the student's likely and other entries, some twice, some not
    kept; a row that keeps nothing, one whose kept entries have no weight."""
    M, V = h.shape
    ids = rng.integers(0, V, size=(M, k)).astype(np.int32)
    ids[:, 0] = h.argmax(1)
    if k > 2:
        ids[:, 2] = ids[:, 1]
        ids[:, -1] = rng.choice([-1, V, -100], M)
    t = (rng.normal(size=(M, k)) * 3).astype(np.float32)
    if M > 4:
        ids[3] = -1
        t[4] = -INF
    if k > 4:
        t[:, 3] = -INF
    return ids, t


CASES = [  # M, V, k, T
    (1, 1, 1, 1.0), (2, 3, 2, 2.0), (6, 7, 3, 1.0), (5, 64, 8, 1.0), (33, 1003, 8, 1.0), (7, 1024, 64, 4.0), (6, 4096, 65, 1.0),
    (5, 4100, 5, 0.5), (300, 515, 20, 1.0), (5, 16385, 20, 2.0), (2, 32000, 1024, 1.0), (2, 32771, 31, 1.0),
    (5, 65536, 20, 1.0), (3, 70001, 20, 1.0), (2, 131072, 20, 1.0), (2, 140003, 20, 1.0), (1030, 77, 5, 1.0),
    (1030, 1003, 70, 2.0), (1027, 1900, 9, 1.0)]


@pytest.mark.parametrize("M,V,k,T", CASES)
@pytest.mark.parametrize("t", ["fp32", "bf16"])
@pytest.mark.parametrize("kind", ["normal", "masked", "lowest", "sure", "huge"])
def test_loss_backward_and_step(M, V, k, T, t, kind):
    print(M, V, k, T, t, kind, flush=True)
    rng = np.random.default_rng(M + V + k)
    x, h = put(logits(rng, kind, M, V, t), t, pad=rng.integers(0, 3), shift=rng.integers(0, 9))
    ids, tv = teacher(rng, h, k)
    w = rng.normal(size=M).astype(np.float32)
    if M > 1:
        w[M // 2] = 0
    ig, tg, wg = (torch.from_numpy(a).to(dev()) for a in (ids, tv, w))
    loss, stats = api.distill_loss(x, ig, tg, temperature=T)
    d = api.distill_backward(wg, x, ig, tg, stats, temperature=T)
    step = api.distill_step(x, ig, tg, wg, temperature=T)
    one = api.distill_step(x, ig, tg, temperature=T)
    torch.cuda.synchronize()
    want, dx, bl, bx = ref.distill(h, ids, tv.astype(np.float64), T, w.astype(np.float64))
    full, d1, bl1, bx1 = ref.distill(h, ids, tv.astype(np.float64), T, np.ones(M))
    check(loss, full, bl1, "loss")
    check(step[0], want, bl, "the step's loss")
    check(one[0], full, bl1, "the step's loss without weights")
    for o, g, b in ((d, dx, bx), (step[1], dx, bx), (one[1], d1, bx1)):
        assert o.dtype == TYPES[t]
        extra = HALF[t] * np.abs(g) if t == "bf16" else 0
        off = np.abs(o.double().cpu().numpy() - g) - (b * U + extra + 2.0 ** -120)
        assert np.all(off <= 0), off.max()
    again = api.distill_step(x, ig, tg, wg, temperature=T)
    assert torch.equal(again[0], step[0]) and torch.equal(again[1], step[1])
    odd = torch.empty(M, V + 1, dtype=TYPES[t], device=dev())[:, 1:]     # other rows' alignment
    assert torch.equal(api.distill_step(x, ig, tg, wg, temperature=T, out=odd)[1], step[1])
    assert torch.equal(api.distill_backward(wg, x, ig, tg, stats, temperature=T, out=odd), d)
    for f in (lambda y, s: api.distill_step(y, ig, tg, wg, temperature=T, out=y, stats=s)[1],
              lambda y, s: api.distill_backward(wg, y, ig, tg, stats, temperature=T, out=y)):
        wide = torch.empty(M, V + 16, dtype=TYPES[t], device=dev())
        off = (x.data_ptr() - wide.data_ptr()) % 16 // wide.element_size()
        over = wide[:, off:off + V] if x.stride(0) % (16 // wide.element_size()) == wide.stride(0) % (16 // wide.element_size()) \
            else x.clone()
        over.copy_(x)
        s = torch.empty(M, 2, device=dev())
        got = f(over, s)
        g = got.double().cpu().numpy()
        extra = HALF[t] * np.abs(dx) if t == "bf16" else 0
        assert got.data_ptr() == over.data_ptr() and np.all(np.abs(g - dx) <= bx * U + extra + 2.0 ** -120)


def test_stats_of_the_step_serve_the_backward_pass():
    rng = np.random.default_rng(0)
    x, h = put(logits(rng, "normal", 6, 5003), "fp32")
    ids, tv = (torch.from_numpy(a).to(dev()) for a in teacher(rng, h, 9))
    stats = torch.empty(6, 2, device=dev())
    w = torch.tensor([1.0, 0.5, 0, 2, 1, 1], device=dev())
    _, d = api.distill_step(x, ids, tv, w, stats=stats)
    other = api.distill_backward(w, x, ids, tv, stats)
    assert torch.allclose(d, other, rtol=1e-5, atol=1e-8)


def test_idle_rows_are_not_read():
    """A row of weight 0 may hold anything."""
    x = torch.randn(4, 999, device=dev())
    x[1] = float("nan")
    ids = torch.zeros(4, 2, dtype=torch.int32, device=dev())
    t = torch.zeros(4, 2, device=dev())
    w = torch.tensor([1.0, 0.0, 1.0, 1.0], device=dev())
    loss, d = api.distill_step(x, ids, t, w)
    assert loss[1] == 0 and torch.all(d[1] == 0) and torch.isfinite(d).all() and torch.isfinite(loss).all()
    loss, stats = api.distill_loss(x, ids, t)
    assert torch.isnan(loss[1]) and torch.isfinite(loss[[0, 2, 3]]).all()
    d = api.distill_backward(w, x, ids, t, stats)
    assert torch.all(d[1] == 0) and torch.isfinite(d).all()


def test_no_rows_and_other_stream():
    x = torch.randn(5, 3001, device=dev(), dtype=torch.bfloat16)
    ids = torch.randint(0, 3001, (5, 7), dtype=torch.int32, device=dev())
    t = torch.randn(5, 7, device=dev())
    loss, d = api.distill_step(x[:0], ids[:0], t[:0])
    assert loss.shape == (0,) and d.shape == (0, 3001)
    want = api.distill_step(x, ids, t)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    got = api.distill_step(x, ids, t, stream=other)
    other.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_gradient_against_differences():
    """Central differences, step 2^-10, of the loss in 64 bits along random
    directions: 1e-4 of the gradient's size against the direction's."""
    rng = np.random.default_rng(11)
    M, V, T, step = 5, 257, 1.5, 2.0 ** -10
    x, h = put(logits(rng, "normal", M, V), "fp32")
    ids, tv = teacher(rng, h, 6)
    tv = np.where(np.isfinite(tv), tv, -3.0).astype(np.float32)
    w = rng.normal(size=M).astype(np.float32)
    _, d = api.distill_step(x, *(torch.from_numpy(a).to(dev()) for a in (ids, tv, w)), temperature=T)
    d = d.double().cpu().numpy()
    f = lambda a: (ref.distill(a, ids, tv.astype(np.float64), T, np.ones(M))[0] * w).sum()  # noqa: E731
    for _ in range(4):
        u = rng.normal(size=h.shape)
        num = (f(h + step * u) - f(h - step * u)) / (2 * step)
        assert abs(num - (d * u).sum()) <= 1e-4 * np.linalg.norm(d) * np.linalg.norm(u)


def test_a_row_of_more_than_a_gigabyte():
    """Offsets within a row past 2^30 bytes: zeros with a few others."""
    V = 300_000_007
    x = torch.zeros(1, V, device=dev())
    x[0, 5], x[0, V - 2], x[0, V - 1] = 12.0, 14.0, 13.0
    s = np.exp(12.0) + np.exp(14.0) + np.exp(13.0) + V - 3
    ids = torch.tensor([[V - 2, 5, 1 << 28]], dtype=torch.int32, device=dev())
    r = api.token_logprobs(x, ids, top=5)
    assert r.top_tokens[0].tolist() == [V - 2, V - 1, 5, 0, 1]
    want = np.array([14.0, 12.0, 0.0]) - np.log(s)
    assert np.abs(r.logprobs[0].double().cpu().numpy() - want).max() < 1e-5
    t = torch.zeros(1, 3, device=dev())
    loss, d = api.distill_step(x, ids, t)
    assert abs(loss.item() - (-np.log(3) - want.mean())) < 1e-4
    g = api.distill_backward(torch.ones(1, device=dev()), x, ids, t, api.distill_loss(x, ids, t)[1])
    for grad in (d, g):
        assert abs(grad[0, V - 2].item() - (np.exp(14.0) / s - 1 / 3)) < 1e-6 and abs(grad[0, 5].item() - (np.exp(12.0) / s - 1 / 3)) < 1e-6
        assert abs(grad[0, V - 1].item() * s / np.exp(13.0) - 1) < 1e-4 and abs(grad[0, 1 << 27].item() * s - 1) < 1e-4
        assert abs(grad[0, 1 << 28].item() - (1 / s - 1 / 3)) < 1e-6
