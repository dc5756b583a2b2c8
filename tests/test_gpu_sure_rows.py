"""Rows whose likeliest token is nearly certain: log probabilities close to 0,
entropies, losses and gradients of such rows against 64 bits, with tolerances
relative to the results.

In units of u = 2^-24, z an entry's distance from the largest over the
temperature, tail the sum of exp(-z) over the others:
  an exponential: its difference, the scaling's constants and product, 4 z, and its
  own rounding, 2; scaled to larger maxima, 4 z in all and 3 for each of 32 steps
  and two joins, 102;
  the tail: 8 of its mean z and 170 (62 additions at most); a thread's part of a
  tail over 2^-4 may be added up with the largest's 1 in it: 64 (1 + tail) / tail more;
  log1p and its products, 10: relative, as log1p's own slope is at most 1;
  the entropy's sum of e z: 8 of its mean z and 240, two additions a step more, and
  the division by 1 + tail."""
import numpy as np
import pytest
import torch

import logits_reference as ref
from block_planner_amd import api

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES, HALF = ref.TYPES, ref.HALF


def dev():
    return torch.device("cuda:0")


def sure(rng, M, V, t, T, gap):
    """Rows whose largest is exp(gap) times as likely as the others together."""
    x = rng.normal(size=(M, V)) * 2
    at = rng.integers(0, V, M)
    at[:4] = [0, V - 1, V // 2, 1][:min(M, 4)]          # single entries before and after the whole pieces
    rows = np.arange(M)
    x[rows, at] = -np.inf
    if V > 1:
        x[rows, at] = T * (gap + np.log(np.exp(x / T).sum(1)))
    else:
        x[rows, at] = 3.0
    wide = torch.zeros(M, V + 3, dtype=TYPES[t], device=dev())[:, 1:V + 1]
    wide.copy_(torch.from_numpy(x))
    return wide, wide.double().cpu().numpy(), at


def parts(h, at, T):
    """(tail, relative bounds of the largest's log p and of H)."""
    rows = np.arange(len(h))
    z = (h[rows, at][:, None] - h) / T
    e = np.exp(-z)
    e[rows, at] = 0
    tail = e.sum(1)
    some = np.maximum(tail, 1e-300)
    z1 = (e * z).sum(1) / some
    z2 = (e * z * z).sum(1) / np.maximum((e * z).sum(1), 1e-300)
    rel = 8 * z1 + 180 + np.where(tail >= 2.0 ** -4, 64 * (1 + tail) / some, 0)
    return tail, rel, np.maximum(rel, 8 * z2 + 260) + tail / (1 + tail) * rel


CASES = [(1, 1), (2, 2), (3, 9), (5, 65), (7, 1003), (5, 4001), (300, 515), (1100, 301), (1030, 1203), (1, 32000),
         (9, 20001), (2, 50001), (1, 70000), (1, 128000)]
GAPS = [0.5, 2.0, 4.0, 7.0, 10.0, 15.0, 25.0, 50.0]


def near(got, want, rel, what, extra=0.0):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    off = np.abs(got - want) - (np.abs(want) * rel * U + extra + 2.0 ** -120)
    assert np.all(off <= 0), (what, off.max(), (np.abs(got - want) / np.maximum(np.abs(want), 1e-300)).max())


@pytest.mark.parametrize("M,V", CASES)
@pytest.mark.parametrize("t", ["fp32", "bf16"])
@pytest.mark.parametrize("T", [1.0, 0.7])
@pytest.mark.parametrize("gap", GAPS)
def test_log_probabilities(M, V, t, T, gap):
    print(M, V, t, T, gap, flush=True)
    rng = np.random.default_rng(M + V + int(10 * gap))
    x, h, at = sure(rng, M, V, t, T, gap)
    tail, rel, rel_h = parts(h, at, T)
    tokens = torch.from_numpy(at.astype(np.int32)).to(dev())
    logp = -np.log1p(tail)
    rows = np.arange(M)
    z = (h[rows, at][:, None] - h) / T
    p = np.exp(-z + logp[:, None])
    p[rows, at] = 0
    H = -np.exp(logp) * logp + (p * (z - logp[:, None])).sum(1)
    g, e = rng.normal(size=M).astype(np.float32), rng.normal(size=M).astype(np.float32)
    for k in (0, min(V, 5)):
        r = api.token_logprobs(x, tokens, top=k, temperature=T)
        near(r.logprobs.cpu(), logp, rel, "logp")
        near(r.entropy.cpu(), H, rel_h, "entropy")
        if k:
            near(r.top_logprobs[:, 0].cpu(), logp, rel, "top")
    # the gradient of g log p: g (1 - p) at the token
    d = api.token_logprobs_backward(torch.from_numpy(g).to(dev()), None, x, tokens, r.stats, r.entropy, temperature=T)
    d = d.double().cpu().numpy()
    near(d[rows, at], g * -np.expm1(logp) / T, rel + 40, "given", HALF[t] * np.abs(g * np.expm1(logp) / T) if t == "bf16" else 0)
    # of e H: -e p (log p + H), two terms of either sign
    d = api.token_logprobs_backward(None, torch.from_numpy(e).to(dev()), x, None, r.stats, r.entropy, temperature=T)
    want = -e * np.exp(logp) * (logp + H) / T
    near(d.double().cpu().numpy()[rows, at], want, 40, "entropy's",
         np.abs(e) / T * U * ((rel + 40) * np.abs(logp) + (rel_h + 40) * H) + (HALF[t] * np.abs(want) if t == "bf16" else 0))


@pytest.mark.parametrize("M,V", CASES[1:])
@pytest.mark.parametrize("t", ["fp32", "bf16"])
@pytest.mark.parametrize("gap", GAPS)
@pytest.mark.parametrize("k", [1, 6])
def test_distillation(M, V, t, gap, k):
    print(M, V, t, gap, k, flush=True)
    rng = np.random.default_rng(3 * M + V + int(10 * gap) + k)
    T, k, rows = 1.0, min(k, V), np.arange(M)
    x, h, at = sure(rng, M, V, t, T, gap)
    tail, rel, _ = parts(h, at, T)
    # the teacher is about as sure of the same token, its first before they are mixed
    ids = np.stack([np.r_[a, rng.permutation(np.delete(np.arange(V), a))[:k - 1]] for a in at]).astype(np.int32)
    teacher = (rng.normal(size=(M, k)) * 0.5).astype(np.float32)
    teacher[:, 0] = 0.9 * gap + (teacher[:, 1:].max(1) if k > 1 else 1)
    order = rng.permutation(k)
    ids, teacher = np.ascontiguousarray(ids[:, order]), np.ascontiguousarray(teacher[:, order])
    own = int(np.flatnonzero(order == 0)[0])
    zt = teacher[:, own][:, None] - teacher.astype(np.float64)
    et = np.exp(-zt)
    et[:, own] = 0
    tt = et.sum(1)
    lt = -zt - np.log1p(tt)[:, None]
    p = np.exp(lt)
    logq = -np.log1p(tail)
    zs = (h[rows, at][:, None] - h)[rows[:, None], ids]
    lq = -zs + logq[:, None]
    want = (p * (lt - lq)).sum(1)
    rt = 8 * zt.max(1) + 60                                     # the teacher's p and log p of its largest
    size = (p * (np.abs(lt) * (rt[:, None] + 40) + np.abs(lq) * (rel[:, None] + 40) +
                 np.abs(lt - lq) * (rt[:, None] + 40))).sum(1)
    w = (rng.random(M) + 0.5).astype(np.float32)
    a = (torch.from_numpy(ids).to(dev()), torch.from_numpy(teacher).to(dev()))
    gw = torch.from_numpy(w).to(dev())
    loss, stats = api.distill_loss(x, *a, temperature=T)
    near(loss.cpu(), want, 0, "loss", size * U)
    loss, dx = api.distill_step(x, *a, gw, temperature=T)
    near(loss.cpu(), want, 0, "step's loss", size * U)
    # at the certain token: w (q - p) = w (p' q - q' p) with q' = 1 - q, p' = 1 - p
    p1 = et.sum(1) / (1 + tt)
    q1 = -np.expm1(logq)
    at_top = w * (p1 * np.exp(logq) - q1 * p[:, own])
    bound = w * U * (p1 * np.exp(logq) * (rt + k + 60) + q1 * p[:, own] * (rel + 60))
    for d in (dx, api.distill_backward(gw, x, *a, stats, temperature=T)):
        near(d.double().cpu().numpy()[rows, at], at_top, 0, "gradient", bound + (HALF[t] * np.abs(at_top) if t == "bf16" else 0))
