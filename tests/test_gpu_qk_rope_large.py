"""ht_qk_norm_rope and its backward pass on more data than the Infinity Cache
holds (256 MiB and more moved, read with the hint not to keep it there): every
row equal, bit for bit, to the same row in a small call, and the weights'
gradients against sums in 64 bits."""
import pytest
import torch

from block_planner_amd import api

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


def inputs(T, n_q, n_k, D, x, norm):
    g = torch.Generator(device="cuda").manual_seed(T + D)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    rows = rand(T, (n_q + n_k) * D).to(x)
    q, k = rows[:, :n_q * D].unflatten(1, (n_q, D)), rows[:, n_q * D:].unflatten(1, (n_k, D))
    w = [1 + 0.3 * rand(D) if norm else None for _ in range(2)]
    pos = torch.randint(0, 100000, (T,), generator=g, device="cuda", dtype=torch.int32)
    return rand, q, k, pos, w


# T, n_q, n_k, D, rot: just over 256 MiB of fp32 in and bf16 out
SHAPES = [(9001, 32, 8, 128, 128), (40003, 14, 4, 64, 32), (5003, 32, 4, 256, 256)]


@pytest.mark.parametrize("T,n_q,n_k,D,rot", SHAPES)
@pytest.mark.parametrize("y,norm,interleaved", [("bf16", True, False), ("fp32", True, True), ("bf16", False, True),
                                                ("fp32", False, False)])
def test_forward(T, n_q, n_k, D, rot, y, norm, interleaved):
    print(T, n_q, n_k, D, rot, y, flush=True)
    _, q, k, pos, w = inputs(T, n_q, n_k, D, torch.float32, norm)
    assert T * (n_q + n_k) * D * (4 + TYPES[y].itemsize) >= 256 << 20
    inv = api.rope_inv_freq(rot, device="cuda")
    big = api.qk_norm_rope(q, k, pos, inv, *w, interleaved=interleaved, out_dtype=TYPES[y])
    for at in (slice(0, 40), slice(T // 2, T // 2 + 300), slice(T - 41, T)):
        small = api.qk_norm_rope(q[at], k[at], pos[at], inv, *w, interleaved=interleaved, out_dtype=TYPES[y])
        assert torch.equal(big[0][at], small[0]) and torch.equal(big[1][at], small[1])


@pytest.mark.parametrize("T,n_q,n_k,D,rot", SHAPES)
@pytest.mark.parametrize("y,norm", [("fp32", True), ("bf16", True), ("bf16", False)])
def test_backward(T, n_q, n_k, D, rot, y, norm):
    print(T, n_q, n_k, D, rot, y, flush=True)
    rand, q, k, pos, w = inputs(T, n_q, n_k, D, torch.float32, norm)
    inv = api.rope_inv_freq(rot, device="cuda")
    dq, dk = rand(T, n_q, D).to(TYPES[y]), rand(T, n_k, D).to(TYPES[y])
    big = api.qk_norm_rope_backward(dq, dk, q, k, pos, inv, *w)
    for at in (slice(0, 40), slice(T // 2, T // 2 + 300), slice(T - 41, T)):
        small = api.qk_norm_rope_backward(dq[at], dk[at], q[at], k[at], pos[at], inv, *w)
        assert torch.equal(big[0][at], small[0]) and torch.equal(big[1][at], small[1])
    if not norm:
        assert big[2] is None and big[3] is None
        return
    a = pos.double()[:, None, None] * inv
    for dy, x, got in ((dq, q, big[2]), (dk, k, big[3])):
        n = x.double()
        n = n / (n.square().mean(-1, keepdim=True) + 1e-6).sqrt()
        g = dy.double()
        lo, hi = g[..., :rot // 2].clone(), g[..., rot // 2:rot].clone()
        g[..., :rot // 2] = lo * a.cos() + hi * a.sin()
        g[..., rot // 2:rot] = hi * a.cos() - lo * a.sin()
        terms = (g * n).flatten(0, 1)
        # a term is off by 40 u of (|g_i| + |g_j|) |n|, a sum of m terms in chains of c
        # additions by c u of the terms' sizes: at most (rows per lane + 64 + 20) deep
        chain = T * (n_q + n_k) // 512 // 8 + 84
        lo, hi = g[..., :rot // 2].abs(), g[..., rot // 2:rot].abs()
        pair = torch.cat([lo + hi, lo + hi, g[..., rot:].abs()], -1).flatten(0, 1)
        tol = U * (40 * (pair * n.flatten(0, 1).abs()).sum(0) + chain * terms.abs().sum(0))
        assert torch.all((got.double() - terms.sum(0)).abs() <= tol)
        del n, g, terms, pair, lo, hi
