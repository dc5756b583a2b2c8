"""Alternatives of rows with many equal entries: equal ones by lower token, also
where a wavefront sorts a part of what it has put aside before the row's end."""
import numpy as np
import pytest
import torch

from block_planner_amd import api

pytestmark = pytest.mark.gpu
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


def first_of(x, k):
    """The k largest of every row, equal ones by lower token."""
    return torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, :k].int()


def straddling(V, threads, k, t, start=0):
    """A row for `threads` threads that reads two steps of 16 entries a thread from `start`
    on: fewer than 64 pieces reach the first bound, then one step's 64 lanes of the first
    wavefront tie, the low lanes in their second piece, the high ones, which hold the
    lower tokens, in their first."""
    vec = 4 if t == "fp32" else 8
    row = np.zeros(V)
    waves = threads // 64
    for w in range(waves):
        for lane in range(40 if w == 0 else -(-k // waves)):
            row[start + vec * (64 * w + lane)] = 1.0
    step = 16 * threads
    for lane in range(64):
        piece = lane if lane >= 24 else threads + lane
        row[start + step + vec * piece] = 5.0
    return row


@pytest.mark.parametrize("M,V,threads,start", [(1100, 4096, 64, 0), (1030, 30000, 64, 0), (300, 8192, 256, 0), (257, 32000, 256, 0),
                                               (3, 16384, 512, 0), (256, 32000, 512, 0), (2, 40000, 512, 0),
                                               (2, 40000, 512, 20000), (1, 128000, 512, 2 * 18288)])
@pytest.mark.parametrize("t", ["fp32", "bf16"])
@pytest.mark.parametrize("k", [1, 5, 20, 24])
def test_a_step_that_is_sorted_in_two_parts(M, V, threads, start, t, k):
    print(M, V, threads, start, t, k, flush=True)
    x = torch.from_numpy(np.resize(straddling(V, threads, k, t, start), (M, V))).to(TYPES[t]).cuda()
    want = first_of(x, k)
    for _ in range(3):
        assert torch.equal(api.token_logprobs(x, top=k).top_tokens, want)


@pytest.mark.parametrize("M,V", [(1, 128000), (2, 50000), (4, 8000), (64, 32000), (300, 32000), (1100, 8000), (2000, 30000)])
@pytest.mark.parametrize("t", ["fp32", "bf16"])
@pytest.mark.parametrize("k", [1, 20, 32, 64])
@pytest.mark.parametrize("trend", [1.0, 4.0, 20.0, 100.0, -4.0])
def test_whole_numbers_with_a_trend(M, V, t, k, trend):
    print(M, V, t, k, trend, flush=True)
    g = torch.Generator(device="cuda").manual_seed(V + k)
    x = torch.randn(M, V, generator=g, device="cuda") + torch.linspace(0, trend, V, device="cuda")
    x = x.floor().to(TYPES[t])
    want = first_of(x, k)
    r = api.token_logprobs(x, top=k)
    assert torch.equal(r.top_tokens, want)
    for _ in range(3):
        again = api.token_logprobs(x, top=k)
        assert torch.equal(again.top_tokens, r.top_tokens) and torch.equal(again.top_logprobs, r.top_logprobs)
