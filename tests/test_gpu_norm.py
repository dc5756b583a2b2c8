"""ht_add_rms_norm, its backward pass and 8-bit rows on the GPU against the
formulas in 64 bits; the gradient also against differences.

Tolerances, in units of u = 2^-24 (half an fp32 step, relative).  A row's sum of
squares: each lane adds at most 32 products (K <= 32768 on 1024 threads), a
wavefront adds 6 deep, the workgroup 16: 55 roundings, halved by the square
root; then its rounding, the division's and the products by r and w: 32 u of
|y| is beyond them.  h is the fp32 sum of x and res, rounded to res's type: equal."""
import numpy as np
import pytest
import torch

import logits_reference as ref
from block_planner_amd import api
from block_planner_amd import binding as B

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES, HALF = ref.TYPES, ref.HALF


def dev():
    return torch.device("cuda:0")


def rows(rng, M, K, t, scale=1.0):
    x = torch.from_numpy((rng.normal(size=(M, K)) * scale).astype(np.float32)).to(TYPES[t])
    return x.to(dev()), x.double().numpy()


def host(t):
    return t.double().cpu().numpy()


SHAPES = [(1, 64), (1, 4096), (1, 8), (3, 8), (5, 72), (17, 512), (2, 520), (33, 1024), (9, 1032), (7, 2048),
          (130, 2056), (6, 4096), (5, 4104), (3, 8192), (2, 8200), (3, 16384), (2, 16392), (2, 32768), (1031, 64),
          (700, 640)]


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("x,r,y", [("fp32", "fp32", "bf16"), ("bf16", "fp32", "fp32"), ("fp32", "bf16", "fp32"),
                                   ("bf16", "bf16", "bf16"), ("fp32", None, "fp32"), ("bf16", None, "bf16")])
def test_forward(M, K, x, r, y):
    print(M, K, x, r, y, flush=True)
    rng = np.random.default_rng(M * 131 + K)
    xg, xh = rows(rng, M, K, x)
    rg, rh = rows(rng, M, K, r, 2.0) if r else (None, 0.0)
    w = (1 + 0.3 * rng.normal(size=K)).astype(np.float32)
    out, h = api.add_rms_norm(xg, torch.from_numpy(w).to(dev()), rg, eps=1e-5, out_dtype=TYPES[y])
    torch.cuda.synchronize()
    hw = ref.rounded((xh + rh).astype(np.float32), r) if r else xh
    if r:
        assert h.dtype == TYPES[r] and np.array_equal(host(h), hw)
    else:
        assert h is None
    want = ref.norm(hw, w.astype(np.float64), 1e-5)
    tol = (32 * U + (HALF[y] if y == "bf16" else 0)) * np.abs(want) + 1e-38
    assert out.dtype == TYPES[y] and np.all(np.abs(host(out) - want) <= tol)


def test_strides_in_place_streams_and_no_rows():
    """Parts of wider rows; misaligned ones (read from a copy); outputs over
    the inputs; another stream; no rows; one row of any stride."""
    rng = np.random.default_rng(1)
    M, K = 37, 264
    wide, _ = rows(rng, M, 3 * K, "fp32")
    x, res = wide[:, :K], wide[:, K:2 * K]
    w = torch.rand(K, device=dev()) + 0.5
    want = api.add_rms_norm(x.contiguous(), w, res.contiguous(), out_dtype=torch.float32)
    got = api.add_rms_norm(x, w, res, out_dtype=torch.float32)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    odd = torch.empty(M, K + 1, device=dev())[:, 1:]
    odd.copy_(x)
    assert torch.equal(api.add_rms_norm(odd, w, res, out_dtype=torch.float32)[0], want[0])
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    third = api.add_rms_norm(x, w, res, out_dtype=torch.float32, stream=other)
    other.synchronize()
    assert torch.equal(third[0], want[0])
    got = api.add_rms_norm(x, w, res, out_dtype=torch.float32, out=(x, res))
    assert got[0].data_ptr() == x.data_ptr() and torch.equal(x, want[0]) and torch.equal(res, want[1])
    assert api.add_rms_norm(x[:0], w, res[:0])[0].shape == (0, K)
    one = api.add_rms_norm(wide[5:6, 2 * K:], w)
    assert torch.equal(one[0], api.add_rms_norm(wide[:, 2 * K:], w)[0][5:6])


def test_zero_and_non_finite_rows():
    """A zero row gives zeros; Inf or NaN stay in their row."""
    x = torch.randn(8, 512, device=dev())
    x[2] = 0
    x[4, 7] = float("inf")
    x[5, 9] = float("nan")
    w = torch.ones(512, device=dev())
    y, _ = api.add_rms_norm(x, w, out_dtype=torch.float32)
    assert torch.all(y[2] == 0) and torch.isnan(y[4, 7]) and torch.all(torch.isnan(y[5]))
    assert torch.isfinite(y[[0, 1, 2, 3, 6, 7]]).all()
    q, _ = api.add_rms_norm_q8(x, w)
    v = api.q8_values(q, torch.float32)
    assert torch.all(v[2] == 0) and torch.isnan(v[4, :64]).all() and torch.all(torch.isnan(v[5]))
    assert torch.isfinite(v[[0, 1, 2, 3, 6, 7]]).all() and torch.all(v[4, 64:] == 0)


@pytest.mark.parametrize("M,K", [(1, 64), (15, 128), (16, 512), (17, 1024), (33, 2048), (128, 4096), (5, 8192), (3, 16384)])
@pytest.mark.parametrize("x,r", [("fp32", "fp32"), ("bf16", "bf16"), ("fp32", None)])
def test_q8(M, K, x, r):
    """The codes are those of the norm in 64 bits, in the documented places, their
    values exact.  The host's 64 bits differ from the kernel's by some 2^-50: a code
    may differ only where the scaled value lies within 2^-40 of a border, and a
    scale only where the largest value lies that near a power of two (no case
    here has either: the count is asserted)."""
    print(M, K, x, r, flush=True)
    rng = np.random.default_rng(M + K)
    xg, xh = rows(rng, M, K, x, 3.0)
    rg, rh = rows(rng, M, K, r) if r else (None, 0.0)
    w = torch.rand(K, device=dev()) * 4
    w[:64] = 0 if K > 64 else w[:64]          # a block of zeros
    q, h = api.add_rms_norm_q8(xg, w, rg, eps=1e-6)
    values = api.q8_values(q), api.q8_values(q, torch.float32)
    torch.cuda.synchronize()
    hw = ref.rounded((xh + rh).astype(np.float32), r) if r else xh
    assert h is None if r is None else np.array_equal(host(h), hw)
    codes, scales = ref.q8_encode(ref.norm(hw, host(w), float(np.float32(1e-6))))
    ci, si = ref.q8_index(M, K)
    assert np.array_equal(q.codes.cpu().numpy().reshape(-1)[ci], codes)
    assert np.array_equal(q.scales.cpu().numpy().reshape(-1)[si[:, ::64]], scales)
    want = codes * np.repeat(scales, 64, 1)
    for v in values:
        assert np.array_equal(host(v), want)


def test_q8_of_tiny_and_huge_values():
    """Blocks around the smallest scale, and past fp32's range."""
    x = torch.ones(4, 256, device=dev())
    w = torch.ones(256, device=dev())
    w[:64], w[64:128], w[128:192], w[192:] = 2.0 ** -126, 2.0 ** -149, 3e38, 1.0
    q, _ = api.add_rms_norm_q8(x, w, eps=0.0)
    v = api.q8_values(q, torch.float32)
    assert torch.all(v[:, :64] == 2.0 ** -126) and torch.all(v[:, 64:128] == 0) and torch.all(v[:, 192:] == 1)
    assert torch.isfinite(v[:, 128:192]).all() and torch.all((v[:, 128:192] / 3e38 - 1).abs() <= 2.0 ** -7)
    # h r below fp32's normal numbers, brought back by the weight: 64-bit values of
    # this row, which 32 bits lose, and zeros beside them
    y = torch.zeros(1, 256, device=dev())
    y[0, :64], y[0, 64:128], y[0, 128] = torch.arange(1, 65, device=dev()) * 3e-14, 3e-14, 3e30
    w[:64], w[64:128] = 3e38, 1e37
    q, _ = api.add_rms_norm_q8(y, w, eps=0.0)
    v = host(api.q8_values(q, torch.float32))
    h = host(y)
    want = h / np.sqrt(np.mean(h * h)) * host(w)
    for b in range(2):
        blk = want[:, 64 * b:64 * b + 64]
        E = np.frexp(np.abs(blk).max())[1]
        assert np.array_equal(v[:, 64 * b:64 * b + 64], np.rint(np.ldexp(blk, 7 - E)).clip(-127, 127) * 2.0 ** (E - 7))
    x[:, 128:192] = 4.0
    assert torch.isnan(api.q8_values(api.add_rms_norm_q8(x, w, eps=0.0)[0])[:, 128:192]).all()


def weight(rng, N, K, int8):
    W = rng.standard_t(4.0, size=(N, K)).astype(np.float32) / 64
    W[:, rng.integers(0, K, K // 100 + 1)] *= 8
    Wg = torch.from_numpy(W).to(dev())
    fmt = api.plan(Wg)
    if int8 == "all":
        fmt.fill_(B.HT_INT8)
    elif int8 == "tile":
        fmt[:256] = B.HT_INT8
    return W, api.pack(Wg, fmt), fmt


@pytest.mark.parametrize("M", [1, 3, 20, 33, 100, 129, 700])
@pytest.mark.parametrize("N,K,int8", [(512, 512, "all"), (304, 1024, "all"), (512, 512, "tile"), (96, 256, "none")])
def test_linear_over_q8_rows(M, N, K, int8, orc):
    """y = x_hat . W_hat^T: where every block is INT8 and there are more than 32
    rows it is HT_PATH_W8A8 of x_hat bit for bit (x_hat's own codes are the
    rows'); elsewhere within the linear's 1e-3 of the largest entry."""
    print(M, N, K, int8, flush=True)
    rng = np.random.default_rng(M + N)
    W, pw, fmt = weight(rng, N, K, int8)
    x = torch.from_numpy(rng.normal(size=(M, K)).astype(np.float32)).to(dev())
    q, _ = api.add_rms_norm_q8(x, torch.ones(K, device=dev()))
    xh = api.q8_values(q)
    y = api.linear(pw, q)
    want = host(xh) @ orc.dequant(W, fmt.cpu().numpy()).astype(np.float64).T
    assert np.abs(host(y) - want).max() <= 1e-3 * np.abs(want).max()
    assert torch.equal(api.linear(pw, q), y)
    if int8 == "all" and M > 32:
        assert torch.equal(y, api.linear(pw, xh, path=B.HT_PATH_W8A8))
    relu = api.linear(pw, q, act=B.HT_ACT_RELU)
    assert torch.equal(relu, y.clamp(min=0))


def test_linear_over_q8_rows_past_a_launch():
    """More rows than one launch of the int8 kernel takes (8192): the last rows
    come out as they do alone."""
    rng = np.random.default_rng(3)
    M, K = 8192 + 200, 1024
    _, pw, _ = weight(rng, 272, K, "all")
    x = torch.randn(M, K, device=dev())
    w = torch.ones(K, device=dev())
    y = api.linear(pw, api.add_rms_norm_q8(x, w)[0])
    last = api.linear(pw, api.add_rms_norm_q8(x[8192:], w)[0])
    first = api.linear(pw, api.add_rms_norm_q8(x[:8192], w)[0])
    torch.cuda.synchronize()
    assert torch.equal(y[8192:], last) and torch.equal(y[:8192], first)
    assert torch.isfinite(y).all()


def backward_tol(dy, h, w, dh, eps):
    """The sums (55 roundings, the dot's products two more) reach d through
    r, r^3 and products: 128 u of the sizes of its terms; dw: a term is good to
    40 u, and a column adds at most 4 rows a step of 512 workgroups, then 8
    parts and 6 halvings: under 40 additions more here."""
    r = 1 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    g = np.abs(dy * w)
    size = r * g + np.abs(h) * r ** 3 * (g * np.abs(h)).sum(-1, keepdims=True) / h.shape[-1]
    size = size + (0 if dh is None else np.abs(dh))
    return 128 * U * size, 96 * U * np.abs(dy * h * r).sum(0)


@pytest.mark.parametrize("M,K", SHAPES + [(3000, 256), (2500, 2056)])
@pytest.mark.parametrize("y,t,x,res", [("fp32", "fp32", "fp32", True), ("bf16", "fp32", "bf16", True),
                                       ("bf16", "bf16", "bf16", False), ("fp32", "bf16", "fp32", True)])
def test_backward(M, K, y, t, x, res):
    print(M, K, y, t, x, flush=True)
    eps = 1e-5
    rng = np.random.default_rng(M + 7 * K)
    dyg, dy = rows(rng, M, K, y)
    hg, h = rows(rng, M, K, t, 2.0)
    dhg, dh = rows(rng, M, K, t) if res else (None, None)
    w = (1 + 0.3 * rng.normal(size=K)).astype(np.float32)
    wg = torch.from_numpy(w).to(dev())
    got = api.add_rms_norm_backward(dyg, hg, wg, dhg, eps=eps, x_dtype=TYPES[x])
    again = api.add_rms_norm_backward(dyg, hg, wg, dhg, eps=eps, x_dtype=TYPES[x])
    torch.cuda.synchronize()
    d, dw = ref.norm_backward(dy, h, w.astype(np.float64), dh, eps)
    tol, tol_w = backward_tol(dy, h, w.astype(np.float64), dh, eps)
    for o, name in ((got[0], x), (got[1], t)):
        assert o.dtype == TYPES[name]
        extra = HALF[name] * np.abs(d) if name == "bf16" else 0
        assert np.all(np.abs(host(o) - d) <= tol + extra + 1e-38)
    assert (got[0] is got[1]) == (x == t)
    assert np.all(np.abs(host(got[2]) - dw) <= tol_w + 1e-38)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_backward_without_rows_and_in_place():
    w = torch.rand(72, device=dev())
    e = torch.empty(0, 72, device=dev())
    assert torch.all(api.add_rms_norm_backward(e, e, w)[2] == 0)
    dy, h, dh = (torch.randn(50, 72, device=dev()) for _ in range(3))
    want = api.add_rms_norm_backward(dy, h, w, dh)
    for i, over in enumerate((dy.clone(), h.clone(), dh.clone())):
        args = [dy, h, dh]
        args[i] = over
        got = api.add_rms_norm_backward(args[0], args[1], w, args[2], out=over)
        assert got[1].data_ptr() == over.data_ptr()
        assert torch.equal(over, want[1]) and torch.equal(got[2], want[2])


@pytest.mark.parametrize("M,K,t,y", [(8300, 4104, "fp32", "bf16"), (16400, 4096, "bf16", "bf16"), (9001, 2040, "fp32", "fp32"),
                                     (3000, 16392, "bf16", "fp32")])
def test_more_than_the_caches_hold(M, K, t, y):
    """Matrices of more than 256 MiB: every row equals that of a small call, and
    the weight's gradient the formula's (a workgroup adds at most 33 rows here, in
    turn, then 12 parts and 6 halvings: backward_tol's 96 u hold 40 a term)."""
    print(M, K, t, y, flush=True)
    torch.manual_seed(M)
    x, r = (torch.randn(M, K, device=dev()).to(TYPES[t]) for _ in range(2))
    w = torch.rand(K, device=dev()) + 0.5
    out, h = api.add_rms_norm(x, w, r, out_dtype=TYPES[y])
    dy = torch.randn(M, K, device=dev()).to(TYPES[y])
    dx, dres, dw = api.add_rms_norm_backward(dy, h, w, r)
    for i in (0, M // 2 - 7, M - 40):
        c = slice(i, i + 40)
        o, s = api.add_rms_norm(x[c], w, r[c], out_dtype=TYPES[y])
        assert torch.equal(o, out[c]) and torch.equal(s, h[c])
        assert torch.equal(api.add_rms_norm_backward(dy[c], h[c], w, r[c])[1], dres[c])
    want, size = torch.zeros(2, K, device=dev(), dtype=torch.float64)
    for i in range(0, M, 1000):
        d = h[i:i + 1000].double()
        d = dy[i:i + 1000].double() * d / (d.square().mean(1, keepdim=True) + 1e-6).sqrt()
        want += d.sum(0)
        size += d.abs().sum(0)
    assert torch.all((dw.double() - want).abs() <= 96 * U * size)


def test_gradient_against_differences():
    """Central differences, step 2^-10, of the forward in 64 bits along random
    directions: off by a third derivative times 2^-20 / 6, under 1e-4 of the
    gradient's size against the direction's."""
    rng = np.random.default_rng(5)
    M, K, eps, step = 11, 128, 1e-5, 2.0 ** -10
    hg, h = rows(rng, M, K, "fp32")
    dyg, dy = rows(rng, M, K, "fp32")
    dhg, dh = rows(rng, M, K, "fp32")
    w = (1 + 0.3 * rng.normal(size=K)).astype(np.float32)
    dx, _, dw = (host(t) for t in api.add_rms_norm_backward(dyg, hg, torch.from_numpy(w).to(dev()), dhg, eps=eps))
    f = lambda a, b: (ref.norm(a, b, eps) * dy).sum() + (a * dh).sum()  # noqa: E731
    w = w.astype(np.float64)
    for _ in range(4):
        u, v = rng.normal(size=h.shape), rng.normal(size=K)
        num = (f(h + step * u, w) - f(h - step * u, w)) / (2 * step)
        assert abs(num - (dx * u).sum()) <= 1e-4 * np.linalg.norm(dx) * np.linalg.norm(u)
        num = (f(h, w + step * v) - f(h, w - step * v)) / (2 * step)
        assert abs(num - (dw * v).sum()) <= 1e-4 * np.linalg.norm(dw) * np.linalg.norm(v)
