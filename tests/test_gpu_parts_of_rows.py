"""Long rows whose parts differ in what they allow: parts of nothing but -Inf, one
entry in a whole row, the type's lowest beside -Inf, NaN and +Inf in one part."""
import math

import pytest
import torch

from block_planner_amd import api

pytestmark = pytest.mark.gpu
INF, LOWEST = math.inf, torch.finfo(torch.float32).min
V = 128000            # seven parts of 18288 columns


def plain(x):
    """(entropy, log softmax) in 64 bits."""
    logp = torch.log_softmax(x.double(), -1)
    p = logp.exp()
    return -(p * torch.where(p > 0, logp, 0.0)).sum(-1), logp


def compare(x, k, places):
    tokens = torch.tensor([places] * len(x), dtype=torch.int32, device="cuda")
    r = api.token_logprobs(x, tokens, top=k)
    H, logp = plain(x)
    want = torch.gather(logp, 1, tokens.long())
    assert torch.allclose(r.entropy.double(), H, rtol=2e-5, atol=1e-30)
    for a, b in ((r.logprobs, want), (r.top_logprobs, torch.gather(logp, 1, r.top_tokens.long()))):
        fine = torch.isfinite(b)
        assert torch.equal(torch.isfinite(a), fine) and torch.equal(a[~fine].double(), b[~fine])
        assert torch.allclose(a[fine].double(), b[fine], rtol=2e-5, atol=1e-6)
    best = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k].int()
    assert torch.equal(r.top_tokens, best)
    return r


@pytest.mark.parametrize("M", [1, 2, 60])
@pytest.mark.parametrize("k", [0, 3, 64])
def test_parts_that_allow_nothing(M, k):
    print(M, k, flush=True)
    torch.manual_seed(M + k)
    x = torch.randn(M, V, device="cuda")
    x[:, 18288:90000] = -INF
    compare(x, k, [0, 20000, V - 1])
    x[:, :18288] = -INF                                   # the last two parts are left, the cut within one
    compare(x, k, [0, 20000, V - 1])


@pytest.mark.parametrize("M", [1, 60])
@pytest.mark.parametrize("at", [0, 1, 18287, 18288, 64000, V - 1])
@pytest.mark.parametrize("value", [3.0, LOWEST, 0.0])
def test_one_entry_is_allowed(M, at, value):
    print(M, at, value, flush=True)
    x = torch.full((M, V), -INF, device="cuda")
    x[:, at] = value
    r = compare(x, 2, [at, (at + 7) % V])
    assert (r.logprobs[:, 0] == 0).all() and (r.entropy == 0).all() and (r.stats[:, 0] == value).all() and (r.stats[:, 1] == 0).all()


@pytest.mark.parametrize("M", [1, 60])
def test_nothing_is_allowed_and_the_lowest_value(M):
    x = torch.full((M, V), -INF, device="cuda")
    r = api.token_logprobs(x, torch.zeros(M, dtype=torch.int32, device="cuda"), top=3)
    assert (r.logprobs == -INF).all() and (r.entropy == 0).all() and (r.top_logprobs == -INF).all()
    assert (r.stats[:, 0] == -INF).all() and r.top_tokens.tolist() == [[0, 1, 2]] * M
    x[:, 30000:30008] = LOWEST
    r = api.token_logprobs(x, torch.full((M,), 30000, dtype=torch.int32, device="cuda"), top=9)
    assert torch.allclose(r.logprobs, torch.full((M,), -math.log(8), device="cuda"), rtol=1e-6)
    assert torch.allclose(r.entropy, torch.full((M,), math.log(8), device="cuda"), rtol=1e-6)
    assert r.top_tokens.tolist() == [[*range(30000, 30008), 0]] * M


@pytest.mark.parametrize("bad", [math.nan, INF])
@pytest.mark.parametrize("at", [0, 18288, 18300, V - 1])
def test_nan_and_inf_in_one_part(bad, at):
    print(bad, at, flush=True)
    x = torch.randn(3, V, device="cuda")
    x[1, at] = bad
    r = api.token_logprobs(x, torch.zeros(3, dtype=torch.int32, device="cuda"), top=4)
    for v in (r.logprobs, r.entropy, r.top_logprobs):
        assert torch.isnan(v[1]).all() and torch.isfinite(v[[0, 2]]).all()
    assert (r.top_tokens[1] == -1).all() and (r.top_tokens[[0, 2]] >= 0).all()
    ids, teacher = torch.randint(0, V, (3, 5), device="cuda", dtype=torch.int32), torch.randn(3, 5, device="cuda")
    loss, d = api.distill_step(x, ids, teacher)
    alone, _ = api.distill_loss(x, ids, teacher)
    for v in (loss, d, alone):
        assert torch.isnan(v[1]).all() and torch.isfinite(v[[0, 2]]).all()


@pytest.mark.parametrize("k", [1, 7, 64, 65, 300])
def test_teachers_of_every_kind(k):
    """Rows that keep nothing, one entry, equal ones, the lowest value; NaN and +Inf
    stay in their rows."""
    print(k, flush=True)
    x = torch.randn(9, 2000, device="cuda")
    ids = torch.stack([torch.randperm(2000, device="cuda")[:k] for _ in range(9)]).int()
    t = torch.randn(9, k, device="cuda")
    ids[0] = -1
    t[1] = -INF
    t[2] = LOWEST
    t[3] = 5.0
    t[4, 1:] = -INF
    t[5, k // 2] = math.nan
    t[6, k // 2] = INF
    ids[7, k // 2:] = 2000
    loss, d = api.distill_step(x, ids, t)
    alone, stats = api.distill_loss(x, ids, t)
    back = api.distill_backward(torch.ones(9, device="cuda"), x, ids, t, stats)
    keep = (ids >= 0) & (ids < 2000) & (t != -INF)
    logq = torch.log_softmax(x.double(), -1)
    for m in range(9):
        if not keep[m].any():
            want, dw = 0.0, torch.zeros(2000, dtype=torch.float64, device="cuda")
        else:
            lp = torch.log_softmax(t[m][keep[m]].double(), -1)
            at = ids[m][keep[m]].long()
            want = (lp.exp() * (lp - logq[m][at])).sum().item()
            dw = logq[m].exp().index_add(0, at, -lp.exp())
        for got in (loss, alone):
            assert got[m].item() == pytest.approx(want, rel=2e-5, abs=2e-6, nan_ok=True)
        if m not in (5, 6):
            assert torch.allclose(d[m].double(), dw, rtol=2e-5, atol=1e-6) and torch.allclose(back[m].double(), dw, rtol=2e-5, atol=1e-6)
        else:
            assert math.isnan(want) and torch.isnan(d[m][ids[m].long()]).all()
