"""ht_qk_norm_rope and its backward pass on the GPU against the formulas in 64
bits; the gradient also against differences.

Tolerances, in units of u = 2^-24: a normed entry has the sum of squares (13
additions deep), a square root, a division and two products behind it, the
rotation two products and a sum, and sine and cosine are good to 2 u beside
the argument's rounding (a turn in [-1/2, 1/2] to 2^-26, 4 u of a radian):
under 32 u of |n_i| + |n_j|.  A bf16 result adds half its step, 2^-8."""
import numpy as np
import pytest
import torch

import kv_reference as ref
from block_planner_amd import api

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


def dev():
    return torch.device("cuda:0")


def case(seed, T, n_q, n_k, D, rot, x, norm, far=4096):
    """q and k as slices of wider rows, positions, frequencies, weights (the
    host copies hold the values after rounding to the type)."""
    rng = np.random.default_rng(seed)
    rows = torch.from_numpy((rng.normal(size=(T, (n_q + 2 * n_k + 1) * D)) * 2).astype(np.float32)).to(TYPES[x])
    gpu = rows.to(dev())
    f = rows.float().numpy()
    cut = lambda a: (a[:, :n_q * D].reshape(T, n_q, D), a[:, n_q * D:(n_q + n_k) * D].reshape(T, n_k, D))  # noqa: E731
    pos = rng.integers(0, far, T).astype(np.int32)
    inv = 10000.0 ** (-2.0 * np.arange(rot // 2) / max(rot, 1))
    w = [(1 + 0.3 * rng.normal(size=D)).astype(np.float32) for _ in range(2)] if norm else [None, None]
    q, k = (gpu[:, :n_q * D].unflatten(1, (n_q, D)), gpu[:, n_q * D:(n_q + n_k) * D].unflatten(1, (n_k, D)))
    put = lambda a: None if a is None else torch.from_numpy(a).to(dev())  # noqa: E731
    return rng, (q, k, put(pos), put(inv), put(w[0]), put(w[1])), (*cut(f), pos, inv, w[0], w[1])


def pair_sum(n, half, interleaved):
    """|n_i| + |n_j| of each entry's pair."""
    a = np.abs(n)
    i = np.arange(half)
    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    s = a.copy()
    s[..., lo] = s[..., hi] = a[..., lo] + a[..., hi]
    return s


def normed(x, w, eps):
    x = x.astype(np.float64)
    return x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w


SHAPES = [  # T, n_q, n_k, D, rot
    (1, 32, 8, 128, 128), (1, 1, 1, 64, 64), (5, 4, 1, 64, 64), (37, 8, 2, 128, 64), (3, 5, 3, 80, 80),
    (7, 2, 1, 96, 48), (9, 3, 3, 256, 256), (2, 4, 2, 8, 8), (11, 2, 2, 16, 8), (6, 3, 1, 200, 40), (4, 2, 1, 64, 0),
    (700, 9, 3, 128, 128), (3000, 2, 1, 64, 32), (4099, 32, 4, 64, 64)]


@pytest.mark.parametrize("T,n_q,n_k,D,rot", SHAPES)
@pytest.mark.parametrize("x,y,norm,interleaved", [("fp32", "bf16", True, False), ("bf16", "bf16", False, True),
                                                  ("fp32", "fp32", True, True), ("bf16", "fp32", True, False),
                                                  ("fp32", "fp32", False, False)])
def test_forward(T, n_q, n_k, D, rot, x, y, norm, interleaved):
    print(T, n_q, n_k, D, rot, x, y, flush=True)
    eps = 1e-6
    _, g, h = case(T + D, T, n_q, n_k, D, rot, x, norm)
    out = api.qk_norm_rope(*g[:4], q_weight=g[4], k_weight=g[5], eps=eps, interleaved=interleaved, out_dtype=TYPES[y])
    torch.cuda.synchronize()
    for o, xi, w in zip(out, h[:2], h[4:]):
        want = ref.norm_rope(xi, w, h[2], h[3], eps, interleaved)
        tol = 32 * U * pair_sum(normed(xi, w, eps), rot // 2, interleaved)
        if y == "bf16":
            tol = tol + 2.0 ** -8 * np.abs(want)
        assert o.dtype == TYPES[y]
        assert np.all(np.abs(o.double().cpu().numpy() - want) <= tol + 1e-38)


def test_far_positions_keep_their_phase():
    """Positions up to 2^31 - 1: the angle is reduced in fp64 (an error of
    2^-53 of 2^31 radians, 2^-22, joins the tolerance)."""
    T = 64
    _, g, h = case(1, T, 4, 2, 64, 64, "fp32", False)
    pos = np.linspace(0, 2 ** 31 - 1, T).astype(np.int64).astype(np.int32)
    out = api.qk_norm_rope(g[0], g[1], torch.from_numpy(pos).to(dev()), g[3])
    want = ref.norm_rope(h[0], None, pos, h[3], 0, False)
    tol = (32 * U + 4 * U) * pair_sum(normed(h[0], None, 0), 32, False)
    assert np.all(np.abs(out[0].double().cpu().numpy() - want) <= tol)


def test_zero_rows_and_in_place():
    """A zero head gives zeros (eps keeps the norm finite); y may be x itself;
    k may be left out; rows may lie inside heads."""
    _, g, h = case(2, 9, 4, 2, 128, 128, "fp32", True)
    q = g[0].clone()
    q[3, 2] = 0
    want = api.qk_norm_rope(q, g[1], *g[2:4], q_weight=g[4], k_weight=g[5])
    assert torch.all(want[0][3, 2] == 0)
    k = g[1].clone()
    got = api.qk_norm_rope(q, k, *g[2:4], q_weight=g[4], k_weight=g[5], out=(q, k))
    assert got[0].data_ptr() == q.data_ptr() and torch.equal(q, want[0]) and torch.equal(k, want[1])
    alone = api.qk_norm_rope(g[0], None, *g[2:4])
    both = api.qk_norm_rope(g[0], g[1], *g[2:4])
    assert alone[1] is None and torch.equal(alone[0], both[0])
    inside = g[0].transpose(0, 1).contiguous().transpose(0, 1)      # [T, H, D] stored [H, T, D]
    assert inside.stride(1) > inside.stride(0)
    assert torch.equal(api.qk_norm_rope(inside, g[1], *g[2:4])[0], both[0])
    odd = torch.empty(9, 4, 130, device=dev())[:, :, 1:129]         # misaligned: read from a copy
    odd.copy_(g[0])
    assert torch.equal(api.qk_norm_rope(odd, g[1], *g[2:4])[0], both[0])
    none = api.qk_norm_rope(g[0][:0], g[1][:0], g[2][:0], g[3])
    assert none[0].shape == (0, 4, 128)


def backward_tol(dy, x, w, pos, inv, eps, interleaved):
    """g is as exact as a rotation (32 u of its pair); dx = r (w g - xhat m)
    carries that twice, the mean's 13 additions and the norm's: 64 u of the
    terms' sizes.  dw: the same per term, and its sum is under 40 additions
    deep for these sizes: 128 u of the sum of |terms|."""
    half = len(inv)
    g = ref.rotate(dy.astype(np.float64), pos, inv, interleaved, -1.0)
    size = pair_sum(g, half, interleaved)
    size = np.maximum(size, pair_sum(dy.astype(np.float64), half, interleaved))
    if w is None:
        return 32 * U * size, None
    x, w = x.astype(np.float64), np.abs(w.astype(np.float64))
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = np.abs(x * r)
    return 64 * U * r * (w * size + xh * (w * size * xh).mean(-1, keepdims=True)), 128 * U * (size * xh).sum((0, 1))


@pytest.mark.parametrize("T,n_q,n_k,D,rot", SHAPES)
@pytest.mark.parametrize("x,y,norm,interleaved", [("fp32", "fp32", True, False), ("bf16", "fp32", True, True),
                                                  ("fp32", "bf16", True, True), ("bf16", "bf16", False, False)])
def test_backward(T, n_q, n_k, D, rot, x, y, norm, interleaved):
    print(T, n_q, n_k, D, rot, x, y, flush=True)
    eps = 1e-5
    rng, g, h = case(T + D + 1, T, n_q, n_k, D, rot, x, norm)
    dy = [torch.from_numpy(rng.normal(size=(T, n, D)).astype(np.float32)).to(TYPES[y]) for n in (n_q, n_k)]
    got = api.qk_norm_rope_backward(dy[0].to(dev()), dy[1].to(dev()), *g[:4], q_weight=g[4], k_weight=g[5], eps=eps,
                                    interleaved=interleaved)
    again = api.qk_norm_rope_backward(dy[0].to(dev()), dy[1].to(dev()), *g[:4], q_weight=g[4], k_weight=g[5], eps=eps,
                                      interleaved=interleaved)
    torch.cuda.synchronize()
    for i in range(2):
        d = dy[i].float().numpy()
        dx, dw = ref.norm_rope_backward(d, h[i], h[4 + i], h[2], h[3], eps, interleaved)
        tx, tw = backward_tol(d, h[i], h[4 + i], h[2], h[3], eps, interleaved)
        if x == "bf16":
            tx = tx + 2.0 ** -8 * np.abs(dx)
        assert got[i].dtype == TYPES[x]
        assert np.all(np.abs(got[i].double().cpu().numpy() - dx) <= tx + 1e-38)
        assert torch.equal(got[i], again[i])
        if norm:
            assert np.all(np.abs(got[2 + i].double().cpu().numpy() - dw) <= tw)
            assert torch.equal(got[2 + i], again[2 + i])
        else:
            assert got[2 + i] is None


def test_backward_without_rows_gives_zero_weight_gradients():
    _, g, h = case(3, 2, 4, 2, 64, 64, "fp32", True)
    q, k, p = g[0][:0], g[1][:0], g[2][:0]
    got = api.qk_norm_rope_backward(q, k, q, k, p, g[3], q_weight=g[4], k_weight=g[5])
    torch.cuda.synchronize()
    assert torch.all(got[2] == 0) and torch.all(got[3] == 0)


def test_gradient_against_differences():
    """Central differences, step h = 2^-10, of the forward in 64 bits along
    random directions: off by h^2 / 6 of a third derivative (under 2^-20 times
    some tens here) beside the kernel's own rounding; 1e-4 of the gradient's
    size against the direction's."""
    eps, step = 1e-5, 2.0 ** -10
    rng, g, h = case(4, 13, 3, 2, 64, 32, "fp32", True)
    dy = [rng.normal(size=(13, n, 64)).astype(np.float32) for n in (3, 2)]
    got = api.qk_norm_rope_backward(*(torch.from_numpy(d).to(dev()) for d in dy), *g[:4], q_weight=g[4],
                                    k_weight=g[5], eps=eps)
    for i in range(2):
        f = lambda x, w: (ref.norm_rope(x, w, h[2], h[3], eps, False) * dy[i]).sum()  # noqa: E731
        x, w = h[i].astype(np.float64), h[4 + i].astype(np.float64)
        for _ in range(4):
            u, v = rng.normal(size=x.shape), rng.normal(size=w.shape)
            num = (f(x + step * u, w) - f(x - step * u, w)) / (2 * step)
            dx = got[i].double().cpu().numpy()
            assert abs(num - (dx * u).sum()) <= 1e-4 * np.linalg.norm(dx) * np.linalg.norm(u)
            num = (f(x, w + step * v) - f(x, w - step * v)) / (2 * step)
            dw = got[2 + i].double().cpu().numpy()
            assert abs(num - (dw * v).sum()) <= 1e-4 * np.linalg.norm(dw) * np.linalg.norm(v)
