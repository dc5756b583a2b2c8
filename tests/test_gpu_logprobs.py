"""ht_token_logprobs and its backward pass on the GPU against the formulas in
64 bits; tolerances are derived in logits_reference (units of 2^-24)."""
import numpy as np
import pytest
import torch

import logits_reference as ref
from block_planner_amd import api
from block_planner_amd import binding as B

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES, HALF = ref.TYPES, ref.HALF
INF = float("inf")


def dev():
    return torch.device("cuda:0")


def put(a, t, pad=0, shift=0):
    """Rows on the GPU inside wider ones, `shift` entries from their start."""
    M, V = a.shape
    wide = torch.full((M, V + pad + shift), 7.0, dtype=TYPES[t], device=dev())
    x = wide[:, shift:shift + V]
    x.copy_(torch.from_numpy(a.astype(np.float32)))
    return x, x.double().cpu().numpy()


def logits(rng, kind, M, V, t="fp32"):
    x = rng.normal(size=(M, V)) * 2.5
    x[np.arange(M), rng.integers(0, V, M)] = 11.0
    if kind == "ties":
        x = np.floor(rng.normal(size=(M, V)) * 1.5)
    elif kind == "zeros":
        x = np.where(rng.random((M, V)) < 0.5, 0.0, -0.0)
    elif kind == "up":
        x = np.sort(x, 1)
    elif kind == "down":
        x = -np.sort(-x, 1)
    elif kind == "masked":
        x[:, rng.random(V) < 0.5] = -INF
        x[0] = -INF                                     # nothing is allowed
        x[-1, 1:] = -INF                                # one entry is, if there are two rows
    elif kind == "lowest":
        x[:, rng.random(V) < 0.5] = torch.finfo(TYPES[t]).min
        x[0] = torch.finfo(TYPES[t]).min
    elif kind == "huge":
        x = x * 1e30
    elif kind == "sure":
        x[:, 0] = 200.0
    return x


def check(o, want, bound, name):
    got = o.double().cpu().numpy()
    want = np.where(np.abs(want) > np.finfo(np.float32).max, np.copysign(INF, want), want)     # past fp32's range
    both = np.isfinite(want)
    assert np.array_equal(np.isfinite(got), both) and np.array_equal(got[~both], want[~both]), name
    off = np.abs(got[both] - want[both]) - bound[both] * U
    assert np.all(off <= 0), (name, off.max())


def run(x, h, tokens, k, T):
    g = torch.from_numpy(tokens.astype(np.int32)).to(dev())
    r = api.token_logprobs(x, g, top=k, temperature=T)
    torch.cuda.synchronize()
    logp, ent, top, ids, b1, b2, b3 = ref.token_logprobs(h, tokens, k, T)
    assert r.top_tokens.dtype == torch.int32 and np.array_equal(r.top_tokens.cpu().numpy(), ids)
    check(r.logprobs, logp, b1, "logprobs")
    check(r.entropy, ent, b2, "entropy")
    check(r.top_logprobs, top, b3, "top")
    again = api.token_logprobs(x, g, top=k, temperature=T)
    for a, b in zip(r, again):
        assert torch.equal(a, b)
    return r


CASES = [  # M, V, k, n, T
    (1, 1, 1, 1, 1.0), (3, 2, 2, 2, 0.5), (2, 7, 5, 1, 1.0), (5, 8, 8, 3, 1.0), (4, 63, 63, 1, 2.0), (4, 64, 64, 1, 1.0),
    (3, 65, 64, 1, 1.0), (9, 1000, 20, 1, 0.7), (2, 1003, 1, 2, 1.0), (3, 4095, 64, 1, 1.0), (2, 4096, 5, 1, 1.0),
    (300, 515, 5, 1, 1.0), (1, 8193, 64, 1, 1.3), (1, 32000, 20, 4, 1.0), (7, 50001, 33, 1, 1.0), (1, 128000, 64, 1, 1.0)]
KINDS = ["normal", "ties", "zeros", "up", "down", "masked", "lowest", "huge", "sure"]


@pytest.mark.parametrize("M,V,k,n,T", CASES)
@pytest.mark.parametrize("t", ["fp32", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
def test_rows(M, V, k, n, T, t, kind):
    print(M, V, k, n, T, t, kind, flush=True)
    rng = np.random.default_rng(M * 7 + V)
    x, h = put(logits(rng, kind, M, V, t), t, pad=rng.integers(0, 3), shift=rng.integers(0, 9))
    tokens = rng.integers(-1, V + 1, size=(M, n))
    tokens[0, 0] = h[0].argmax()
    run(x, h, tokens, k, T)


@pytest.mark.parametrize("M", [1, 2, 17, 64, 255, 256, 257])
@pytest.mark.parametrize("V", [4099, 12289, 40000])
def test_parts_of_rows(M, V):
    """Rows cut into parts and whole ones, either side of the rules, with ties
    across the cuts."""
    print(M, V, flush=True)
    rng = np.random.default_rng(M + V)
    few = min(M, 20)
    x, h = put(np.floor(rng.normal(size=(M, V)) * 3), "fp32", shift=1)
    tokens = rng.integers(0, V, size=(M, 1)).astype(np.int32)
    r = api.token_logprobs(x, torch.from_numpy(tokens).to(dev()), top=40)
    logp, ent, top, ids, b1, b2, b3 = ref.token_logprobs(h[:few], tokens[:few], 40, 1.0)
    assert np.array_equal(r.top_tokens[:few].cpu().numpy(), ids)
    check(r.logprobs[:few], logp, b1, "logprobs")
    check(r.entropy[:few], ent, b2, "entropy")
    check(r.top_logprobs[:few], top, b3, "top")


@pytest.mark.parametrize("M,k", [(256, 20), (257, 20), (600, 64), (1025, 64), (1025, 32), (1100, 3)])
@pytest.mark.parametrize("t", ["fp32", "bf16"])
@pytest.mark.parametrize("kind", ["normal", "ties", "zeros", "up", "masked"])
def test_many_rows(M, k, t, kind):
    """Either side of the rules on threads per row, with more equal entries than
    are counted at the end and rows that put everything aside."""
    print(M, k, t, kind, flush=True)
    rng = np.random.default_rng(M + k)
    x, h = put(np.resize(logits(rng, kind, 12, 14001, t), (M, 14001)), t, shift=3)
    rows = [0, 1, M - 1]
    run(x[rows], h[rows], np.zeros((3, 1), int), k, 1.0)
    r = api.token_logprobs(x, top=k)
    want = ref.token_logprobs(h[:12], np.zeros((12, 1), int), k, 1.0)[3]
    assert np.array_equal(r.top_tokens.cpu().numpy(), np.resize(want, (M, k)))


def test_no_tokens_no_top_no_rows_other_stream():
    rng = np.random.default_rng(0)
    x, h = put(logits(rng, "normal", 5, 999), "fp32")
    r = api.token_logprobs(x)
    assert r.logprobs is None and r.top_logprobs.shape == (5, 0) and r.top_tokens.shape == (5, 0)
    _, ent, _, _, _, b2, _ = ref.token_logprobs(h, np.zeros((5, 1), int), 0, 1.0)
    check(r.entropy, ent, b2, "entropy")
    a, b = r.stats.double().cpu().numpy().T
    assert np.array_equal(a, h.max(1))
    assert np.allclose(a + b * np.log(2), [np.log(np.exp(v - v.max()).sum()) + v.max() for v in h], rtol=1e-5)
    none = api.token_logprobs(x[:0], torch.empty(0, dtype=torch.int32, device=dev()), top=3)
    assert none.top_logprobs.shape == (0, 3) and none.logprobs.shape == (0,)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    s = api.token_logprobs(x, top=5, stream=other)
    other.synchronize()
    assert torch.equal(s.top_tokens, api.token_logprobs(x, top=5).top_tokens)
    turned = x.t().contiguous().t()                     # columns apart: read from a copy
    assert torch.equal(api.token_logprobs(turned, top=5).top_tokens, s.top_tokens)


def test_nan_and_inf_stay_in_their_rows():
    x = torch.randn(300, 2003, device=dev())
    want = api.token_logprobs(x, torch.zeros(300, dtype=torch.int32, device=dev()), top=4)
    y = x.clone()
    y[3, 100], y[5, 2002], y[7] = float("nan"), INF, float("nan")
    for rows in (y, y[:9]):                             # whole rows, parts of rows
        r = api.token_logprobs(rows, torch.zeros(len(rows), dtype=torch.int32, device=dev()), top=4)
        bad = torch.tensor([3, 5, 7], device=dev())
        for v in (r.logprobs, r.entropy, r.top_logprobs):
            assert torch.isnan(v[bad]).all()
        assert (r.top_tokens[bad] == -1).all()
        good = torch.tensor([0, 1, 2, 4, 6, 8], device=dev())
        assert torch.equal(r.top_tokens[good], want.top_tokens[good])
        assert torch.allclose(r.entropy[good], want.entropy[good], rtol=1e-5)


def test_a_cache_of_logits_past_4_gib():
    """Rows whose offsets pass 32 bits."""
    M, V = 9000, 128008
    x = torch.zeros(M, V, dtype=torch.float32, device=dev())
    x[-1, 77], x[-1, V - 1] = 9.0, 8.0
    r = api.token_logprobs(x, torch.full((M,), 77, dtype=torch.int32, device=dev()), top=3)
    assert r.top_tokens[-1].tolist() == [77, V - 1, 0] and r.top_tokens[0].tolist() == [0, 1, 2]
    s = np.exp(9.0) + np.exp(8.0) + V - 2
    assert abs(r.logprobs[-1].item() - (9 - np.log(s))) < 1e-5
    d = api.token_logprobs_backward(torch.ones(M, device=dev()), None, x, torch.full((M,), 77, dtype=torch.int32, device=dev()),
                                    r.stats, out=x)
    assert abs(d[-1, 77].item() - (1 - np.exp(9.0) / s)) < 1e-5 and abs(d[-1, 5].item() * s + 1) < 1e-4


GRADS = [(1, 1, 1, 1.0), (3, 7, 2, 0.5), (2, 64, 1, 1.0), (5, 1003, 3, 1.0), (40, 515, 1, 2.0), (2, 16384, 1, 1.0),
         (3, 16385, 2, 0.7), (600, 33, 1, 1.0), (2, 50001, 70, 1.0)]


@pytest.mark.parametrize("M,V,n,T", GRADS)
@pytest.mark.parametrize("t", ["fp32", "bf16"])
@pytest.mark.parametrize("kind", ["normal", "masked", "lowest", "sure", "huge"])
@pytest.mark.parametrize("what", ["logp", "entropy", "both"])
def test_backward(M, V, n, T, t, kind, what):
    print(M, V, n, T, t, kind, what, flush=True)
    rng = np.random.default_rng(M + V + n)
    x, h = put(logits(rng, kind, M, V, t), t, pad=rng.integers(0, 3), shift=rng.integers(0, 9))
    tokens = rng.integers(-1, V, size=(M, n)).astype(np.int32)
    if n > 1:
        tokens[:, 1] = tokens[:, 0]                     # the same token twice
    g = rng.normal(size=(M, n)).astype(np.float32) * (what != "entropy")
    e = rng.normal(size=M).astype(np.float32) * (what != "logp")
    g[M // 2], e[M // 2] = 0, 0                         # a row without a gradient
    tg, gg, eg = (torch.from_numpy(a).to(dev()) for a in (tokens, g, e))
    r = api.token_logprobs(x, tg, temperature=T)
    args = (None if what == "entropy" else gg, None if what == "logp" else eg, x, None if what == "entropy" else tg,
            r.stats, r.entropy)
    d = api.token_logprobs_backward(*args, temperature=T)
    torch.cuda.synchronize()
    dx, tol = ref.gradient(h, T, tokens if what != "entropy" else tokens[:, :0], g.astype(np.float64), e.astype(np.float64))
    extra = HALF[t] * np.abs(dx) if t == "bf16" else 0
    assert d.dtype == TYPES[t] and np.all(np.abs(d.double().cpu().numpy() - dx) <= tol * U + extra + 2.0 ** -120)
    assert torch.all(d[M // 2] == 0)
    odd = torch.empty(M, V + 1, dtype=TYPES[t], device=dev())[:, 1:]     # other rows' alignment
    assert torch.equal(api.token_logprobs_backward(*args, temperature=T, out=odd), d)
    over = x.clone()
    args = (*args[:2], over, *args[3:])
    got = api.token_logprobs_backward(*args, temperature=T, out=over)
    assert got.data_ptr() == over.data_ptr()
    same = got.double().cpu().numpy()                   # other alignment: other pieces, the same values
    assert np.array_equal(same, d.double().cpu().numpy())


def test_gradient_against_differences():
    """Central differences, step 2^-10, of the forward in 64 bits along random
    directions: 1e-4 of the gradient's size against the direction's."""
    rng = np.random.default_rng(9)
    M, V, T, step = 4, 301, 0.8, 2.0 ** -10
    x, h = put(logits(rng, "normal", M, V), "fp32")
    tokens = rng.integers(0, V, size=(M, 2))
    g, e = rng.normal(size=(M, 2)).astype(np.float32), rng.normal(size=M).astype(np.float32)
    tg = torch.from_numpy(tokens.astype(np.int32)).to(dev())
    r = api.token_logprobs(x, tg, temperature=T)
    d = api.token_logprobs_backward(torch.from_numpy(g).to(dev()), torch.from_numpy(e).to(dev()), x, tg, r.stats, r.entropy,
                                    temperature=T).double().cpu().numpy()

    def f(a):
        logp, ent = ref.token_logprobs(a, tokens, 0, T)[:2]
        return (logp * g).sum() + (ent * e).sum()

    for _ in range(4):
        u = rng.normal(size=h.shape)
        num = (f(h + step * u) - f(h - step * u)) / (2 * step)
        assert abs(num - (d * u).sum()) <= 1e-4 * np.linalg.norm(d) * np.linalg.norm(u)
