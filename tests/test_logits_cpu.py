"""The norm with the residual's addition, 8-bit rows, token log probabilities and
distillation without a GPU: host checks of every entry point (only invalid or
empty calls are made, so nothing is launched), the Python layers' refusals,
sizes, and the host reference against torch in 64 bits."""
import ctypes

import numpy as np
import pytest
import torch

import logits_reference as ref
from block_planner_amd import api
from block_planner_amd import binding as B
from block_planner_amd import nn as htnn

A = 0x10000   # an aligned address nobody reads
OK, EINVAL, ESHAPE, EALIGN, ESMALL = 0, 1, 2, 3, 4
BF, F32 = B.HT_BF16, B.HT_FP32


def call(name, base, **change):
    """Status of the entry point with some of its arguments replaced."""
    args = dict(base)
    assert set(change) <= set(args), set(change) - set(args)
    args.update(change)
    return getattr(B.load(), name)(*args.values())


def q8(codes=A, scales=A, M=5, K=128):
    return ctypes.byref(B.Q8Desc(codes, scales, M, K))


NORM = dict(x=A, ldx=128, xt=F32, res=A, ldr=128, rt=BF, M=5, K=128, w=A, eps=1e-6, h=A, ldh=128, y=A, ldy=128, yt=BF,
            q=None, stream=None)


@pytest.mark.parametrize("change,code", [
    *[({k: None}, EINVAL) for k in ("x", "w")], (dict(y=None), EINVAL), (dict(res=None), EINVAL),   # h without res
    *[({k: A + 8}, EALIGN) for k in ("x", "res", "w", "h", "y")],
    (dict(xt=1), EINVAL), (dict(rt=0), EINVAL), (dict(yt=3), EINVAL), (dict(eps=-1e-9), EINVAL), (dict(eps=float("nan")), EINVAL),
    (dict(M=-1), ESHAPE), (dict(K=0), ESHAPE), (dict(K=132), ESHAPE), (dict(K=32776), ESHAPE), (dict(M=1 << 22), ESHAPE),
    (dict(ldx=120), ESHAPE), (dict(ldy=64), ESHAPE), (dict(ldx=130), EALIGN), (dict(ldh=132), EALIGN),
    (dict(q=q8(M=4)), ESHAPE), (dict(q=q8(K=64)), ESHAPE), (dict(q=q8(codes=None)), EINVAL), (dict(q=q8(codes=A + 4)), EALIGN),
    (dict(q=q8(M=5, K=136), K=136, ldx=136, ldr=136, ldh=136, ldy=136), ESHAPE)])
def test_norm_argument_checks(change, code):
    assert call("ht_add_rms_norm", NORM, **change) == code


def test_norm_without_rows_launches_nothing():
    assert call("ht_add_rms_norm", NORM, M=0, x=None, res=None, h=None, y=None, w=None) == OK


NBACK = dict(dy=A, lddy=128, yt=BF, h=A, ldh=128, ht=F32, dh=A, lddh=128, M=3000, K=128, w=A, eps=1e-6, dres=A, lddres=128,
             dx=A, lddx=128, dw=A, ws=A, ws_bytes=1 << 24, stream=None)


@pytest.mark.parametrize("change,code", [
    *[({k: None}, EINVAL) for k in ("dy", "h", "w", "dres", "dw")],
    *[({k: A + 8}, EALIGN) for k in ("dy", "h", "dh", "w", "dres", "dx", "dw", "ws")],
    (dict(ws=None), ESMALL), (dict(ws_bytes=16), ESMALL), (dict(yt=1), EINVAL), (dict(ht=3), EINVAL), (dict(K=12), ESHAPE),
    (dict(M=-1), ESHAPE), (dict(lddh=64), ESHAPE), (dict(lddx=132), EALIGN), (dict(eps=-1.0), EINVAL)])
def test_norm_backward_argument_checks(change, code):
    assert call("ht_add_rms_norm_backward", NBACK, **change) == code


def test_norm_workspace():
    assert B.ht_add_rms_norm_workspace(0, 128) == 0 and B.ht_add_rms_norm_workspace(1, 4096) == 0
    assert 0 < B.ht_add_rms_norm_workspace(8192, 4096) <= 768 * 4096 * 4
    assert 0 < B.ht_add_rms_norm_workspace(1 << 20, 32768) <= 512 * 32768 * 4
    for bad in ((1, 12), (-1, 64), (1, 40000)):
        with pytest.raises(B.HTError):
            B.ht_add_rms_norm_workspace(*bad)


def test_q8_sizes_and_checks():
    assert B.ht_q8_bytes(17, 192) == (2 * 3 * 1024, 2 * 3 * 64)
    assert B.ht_q8_bytes(0, 64) == (0, 0)
    for bad in ((1, 100), (-1, 64), ((1 << 30) + 1, 64), (1, (1 << 20) + 64)):
        with pytest.raises(B.HTError) as e:
            B.ht_q8_bytes(*bad)
        assert e.value.code == ESHAPE
    v = dict(q=q8(), y=A, ldy=128, yt=BF, stream=None)
    for change, code in ((dict(q=None), EINVAL), (dict(q=q8(scales=None)), EINVAL), (dict(y=None), EINVAL), (dict(yt=0), EINVAL),
                         (dict(ldy=64), ESHAPE), (dict(ldy=130), EALIGN), (dict(y=A + 8), EALIGN), (dict(q=q8(M=0), y=None), OK)):
        assert call("ht_q8_values", v, **change) == code


def all_int8(N=512, K=128, tile=16):
    return B.ht_refresh_desc(N, K, tile, [0, N * K // 64, 0, 0, 0], A, buf_bytes=1 << 32)


def test_linear_q8_checks():
    w = all_int8()
    v = dict(w=ctypes.byref(w), x=q8(M=100), y=A, ldy=512, act=0, ws=A, ws_bytes=1 << 30, stream=None)
    assert B.ht_linear_q8_workspace(w, 5) >= 5 * 128 * 2                  # few rows: their values
    small = v | dict(x=q8(M=5))
    for base, change, code in ((v, dict(w=None), EINVAL), (v, dict(x=None), EINVAL), (v, dict(x=q8(codes=None)), EINVAL),
                               (v, dict(y=None), EINVAL), (v, dict(act=2), EINVAL), (v, dict(x=q8(K=64, M=100)), ESHAPE),
                               (v, dict(x=q8(M=0)), ESHAPE), (v, dict(ldy=500), ESHAPE), (v, dict(y=A + 4), EALIGN),
                               (v, dict(x=q8(scales=A + 8, M=100)), EALIGN), (small, dict(ws=None), ESMALL),
                               (small, dict(ws_bytes=64), ESMALL), (small, dict(ws=A + 8), EALIGN)):
        assert call("ht_linear_forward_q8", base, **change) == code
    with pytest.raises(B.HTError):
        B.ht_linear_q8_workspace(w, 0)


def test_linear_q8_workspace_holds_the_last_launch():
    """Rows past 8192 run as a further launch, which may be split where the
    first is not."""
    w = all_int8(38400, 1024)
    for last in (33, 128, 5000):
        assert B.ht_linear_q8_workspace(w, 8192 + last) >= B.ht_linear_workspace(w, last, B.HT_PATH_W8A8) - last * 1024 * 2 - 65536


LOGP = dict(x=A + 2, ld=1001, type=BF, M=3, V=1000, tokens=A, n_tok=2, k=5, t=1.0, logp=A, entropy=A, top=A, ids=A, stats=A, ws=A,
            ws_bytes=1 << 30, stream=None)
WRONG_ROWS = [(dict(M=-1), ESHAPE), (dict(M=(1 << 22) + 1), ESHAPE), (dict(V=0), ESHAPE), (dict(V=(1 << 29) + 1, ld=1 << 30), ESHAPE),
              (dict(ld=999), ESHAPE), (dict(type=0), EINVAL), (dict(x=A + 1), EALIGN), (dict(x=A + 2, type=F32), EALIGN),
              (dict(t=0.0), EINVAL), (dict(t=-1.0), EINVAL), (dict(t=float("nan")), EINVAL), (dict(t=float("inf")), EINVAL),
              (dict(t=1e-31), EINVAL)]


@pytest.mark.parametrize("change,code", [
    *WRONG_ROWS, *[({k: None}, EINVAL) for k in ("x", "tokens", "logp", "top", "ids")],
    *[({k: A + 2}, EALIGN) for k in ("tokens", "logp", "entropy", "top", "ids", "stats")], (dict(ws=A + 8), EALIGN),
    (dict(k=-1), ESHAPE), (dict(k=65), ESHAPE), (dict(V=4, k=5), ESHAPE), (dict(n_tok=-1), ESHAPE), (dict(n_tok=1025), ESHAPE),
    (dict(V=128000, ld=128000, ws=None), ESMALL), (dict(V=128000, ld=128000, ws_bytes=64), ESMALL)])
def test_logprobs_argument_checks(change, code):
    assert call("ht_token_logprobs", LOGP, **change) == code


def test_logprobs_workspace():
    assert B.ht_token_logprobs_workspace(0, 128000, 5) == 0
    assert B.ht_token_logprobs_workspace(4096, 128000, 64) == 0            # whole rows
    assert B.ht_token_logprobs_workspace(64, 8000, 64) == 0
    assert 0 < B.ht_token_logprobs_workspace(1, 128000, 5) <= 16 * (12 + 40) + 256


LBACK = dict(g=A, e=A, x=A + 2, ld=1001, type=BF, M=3, V=1000, tokens=A, n_tok=2, stats=A, entropy=A, t=1.0, dx=A + 2, ldd=1000,
             stream=None)


@pytest.mark.parametrize("change,code", [
    *WRONG_ROWS, *[({k: None}, EINVAL) for k in ("x", "tokens", "g", "stats", "entropy", "dx")],
    *[({k: A + 2}, EALIGN) for k in ("g", "e", "tokens", "stats", "entropy")], (dict(dx=A + 1), EALIGN), (dict(ldd=999), ESHAPE),
    (dict(n_tok=1025), ESHAPE)])
def test_logprobs_backward_argument_checks(change, code):
    assert call("ht_token_logprobs_backward", LBACK, **change) == code


DLOSS = dict(x=A + 2, ld=1001, type=BF, M=3, V=1000, ids=A, teacher=A, k=4, t=1.0, loss=A, stats=A, stream=None)
DBACK = dict(g=A, x=A + 2, ld=1001, type=BF, M=3, V=1000, ids=A, teacher=A, k=4, stats=A, t=1.0, dx=A + 2, ldd=1000, stream=None)
DSTEP = dict(x=A + 2, ld=1001, type=BF, M=3, V=1000, ids=A, teacher=A, k=4, w=A, t=1.0, loss=A, stats=A, dx=A + 2, ldd=1000,
             stream=None)
ENTRIES = [(dict(k=0), ESHAPE), (dict(k=1025), ESHAPE), (dict(ids=None), EINVAL), (dict(teacher=None), EINVAL),
           (dict(ids=A + 2), EALIGN), (dict(teacher=A + 1), EALIGN), (dict(x=None), EINVAL), (dict(stats=A + 2), EALIGN)]


@pytest.mark.parametrize("name,base,more", [
    ("ht_distill_loss", DLOSS, [(dict(loss=None), EINVAL), (dict(loss=A + 2), EALIGN)]),
    ("ht_distill_backward", DBACK, [(dict(g=None), EINVAL), (dict(stats=None), EINVAL), (dict(dx=None), EINVAL),
                                    (dict(ldd=10), ESHAPE), (dict(g=A + 2), EALIGN)]),
    ("ht_distill_step", DSTEP, [(dict(loss=None), EINVAL), (dict(dx=None), EINVAL), (dict(dx=A + 1), EALIGN), (dict(w=A + 2), EALIGN),
                                (dict(ldd=10), ESHAPE)])])
def test_distill_argument_checks(name, base, more):
    for change, code in WRONG_ROWS + ENTRIES + more:
        assert call(name, base, **change) == code, change


def test_scale_rows_checks():
    v = dict(dx=A, ld=1000, type=BF, M=3, V=1000, g=A, stream=None)
    for change, code in ((dict(dx=None), EINVAL), (dict(g=None), EINVAL), (dict(g=A + 2), EALIGN), (dict(ld=9), ESHAPE), (dict(M=0), OK),
                         (dict(type=1), EINVAL)):
        assert call("ht_scale_rows", v, **change) == code


def test_nothing_is_launched_without_rows():
    assert call("ht_token_logprobs", LOGP, M=0, x=None) == OK
    assert call("ht_token_logprobs_backward", LBACK, M=0, x=None) == OK
    for name, base in (("ht_distill_loss", DLOSS), ("ht_distill_backward", DBACK), ("ht_distill_step", DSTEP)):
        assert call(name, base, M=0, x=None) == OK


# -- the Python layers --------------------------------------------------------
def t(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


I32 = torch.int32


def test_python_refusals():
    """Types, shapes and host tensors, before anything is launched."""
    x, w = t(3, 64), t(64)
    for f in (api.add_rms_norm, api.add_rms_norm_q8):
        for args, kw in (((x.half(), w), {}), ((x, w.bfloat16()), {}), ((x, w[:60]), {}), ((x[0], w), {}), ((x, w, x[:2]), {}),
                         ((x, w, x.half()), {})):
            with pytest.raises(ValueError, match="expected"):
                f(*args, **kw)
        with pytest.raises(ValueError, match="on the GPU"):
            f(x, w)
    for kw in (dict(out_dtype=torch.float16), dict(out=(t(3, 64), None)), dict(out=(t(3, 60, dtype=torch.bfloat16), None))):
        with pytest.raises(ValueError, match="expected"):
            api.add_rms_norm(x, w, **kw)
    for args, kw in (((x, x, w, x.bfloat16()), {}), ((x[:2], x, w), {}), ((x, x, w), dict(x_dtype=torch.float16)),
                     ((x, x, w), dict(out=x.bfloat16()))):
        with pytest.raises(ValueError, match="expected"):
            api.add_rms_norm_backward(*args, **kw)
    q = api.q8_rows(3, 64, "cpu")
    assert q.codes.shape == (1, 1, 64, 16) and q.scales.shape == (1, 16)
    with pytest.raises(B.HTError):
        api.q8_rows(3, 60, "cpu")
    for bad in (q._replace(M=40), q._replace(codes=q.codes.float()), q._replace(scales=q.scales[0])):
        with pytest.raises(ValueError, match="expected"):
            api.q8_values(bad)
    with pytest.raises(ValueError, match="path"):
        api.linear(None, q, path=B.HT_PATH_W8A8)
    l, ids = t(3, 50), t(3, dtype=I32)
    for args, kw in (((l.half(), ids), {}), ((l[0], ids), {}), ((l, ids.long()), {}), ((l, ids[:2]), {}), ((l,), dict(top=65)),
                     ((l,), dict(top=51)), ((l,), dict(top=-1)), ((l, t(3, 4, dtype=I32)[:, ::2]), {})):
        with pytest.raises(ValueError, match="expected"):
            api.token_logprobs(*args, **kw)
    with pytest.raises(ValueError, match="on the GPU"):
        api.token_logprobs(l, ids)
    g, s = t(3), t(3, 2)
    for args in ((g, None, l, None, s), (None, None, l, ids, s), (g, g, l, ids, s), (g, None, l, ids, t(3)), (g.double(), None, l, ids, s),
                 (g[:2], None, l, ids, s)):
        with pytest.raises(ValueError, match="expected|both or neither"):
            api.token_logprobs_backward(*args)
    i2, t2 = t(3, 4, dtype=I32), t(3, 4)
    for args in ((l, i2.long(), t2), (l, i2, t2[:, :3]), (l, i2, t2.double()), (l, ids, g), (l, i2[:2], t2[:2]), (l, t(3, 1025, dtype=I32), t(3, 1025))):
        with pytest.raises(ValueError, match="expected"):
            api.distill_loss(*args)
        with pytest.raises(ValueError, match="expected"):
            api.distill_step(*args)
    for kw in (dict(weight=t(2)), dict(weight=t(3).double()), dict(out=l.bfloat16()), dict(stats=t(3))):
        with pytest.raises(ValueError, match="expected"):
            api.distill_step(l, i2, t2, **kw)
    with pytest.raises(ValueError, match="on the GPU"):
        api.distill_step(l, i2, t2)
    with pytest.raises(ValueError, match="expected"):
        api.distill_backward(t(2), l, i2, t2, s)
    with pytest.raises(ValueError, match="expected"):
        api.scale_rows(l, t(2))


def test_module_refusals():
    with pytest.raises(ValueError, match="multiple of 64"):
        htnn.AddRMSNorm(72, bits8=True, device="cpu")
    with pytest.raises(ValueError, match="multiple of 8"):
        htnn.AddRMSNorm(36, device="cpu")
    n = htnn.AddRMSNorm(64, bits8=True, device="cpu")
    with pytest.raises(RuntimeError, match="no backward pass"):
        n(t(3, 64))
    with pytest.raises(ValueError, match="expected"):
        htnn.add_rms_norm(t(3, 64), t(64), t(4, 64))
    with pytest.raises(ValueError, match="expected"):
        htnn.token_logprobs(t(3, 50), t(4, dtype=torch.long))
    with pytest.raises(ValueError, match="whole numbers"):
        htnn.token_logprobs(t(3, 50), t(3))
    for args in ((t(3, 50), t(3, 4, dtype=I32), t(3, 5)), (t(3, 50), t(2, 4, dtype=I32), t(2, 4))):
        with pytest.raises(ValueError, match="expected"):
            htnn.distill_loss(*args)
    with pytest.raises(ValueError, match="expected"):
        htnn.distill_loss(t(3, 50), t(3, 4, dtype=I32), t(3, 4), weight=t(2))


# -- the reference ------------------------------------------------------------
def test_reference_against_torch():
    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.normal(size=(4, 30)) * 3).requires_grad_()
    tok = torch.from_numpy(rng.integers(0, 30, size=(4, 2)))
    g, e = torch.from_numpy(rng.normal(size=(4, 2))), torch.from_numpy(rng.normal(size=4))
    lp = torch.log_softmax(x / 0.7, -1)
    H = -(lp.exp() * lp).sum(-1)
    logp, ent, top, ids, *_ = ref.token_logprobs(x.detach().numpy(), tok.numpy(), 5, 0.7)
    assert np.allclose(logp, lp.gather(1, tok).detach()) and np.allclose(ent, H.detach())
    assert np.allclose(top, lp.topk(5).values.detach()) and np.array_equal(ids, lp.topk(5).indices)
    ((lp.gather(1, tok) * g).sum() + (H * e).sum()).backward()
    assert np.allclose(ref.gradient(x.detach().numpy(), 0.7, tok.numpy(), g.numpy(), e.numpy())[0], x.grad)
    x.grad = None
    tv, w = torch.from_numpy(rng.normal(size=(4, 2))), torch.from_numpy(rng.normal(size=4))
    p = torch.softmax(tv / 2, -1)
    loss = (p * (p.log() - torch.log_softmax(x / 2, -1).gather(1, tok))).sum(-1)
    (w * loss).sum().backward()
    got, dx, _, _ = ref.distill(x.detach().numpy(), tok.numpy(), tv.numpy(), 2.0, w.numpy())
    assert np.allclose(got, loss.detach()) and np.allclose(dx, x.grad)
    h = torch.from_numpy(rng.normal(size=(4, 16))).requires_grad_()
    wt = torch.from_numpy(rng.normal(size=16)).requires_grad_()
    y = torch.nn.functional.rms_norm(h, (16,), wt, 1e-3)
    assert np.allclose(ref.norm(h.detach().numpy(), wt.detach().numpy(), 1e-3), y.detach())
    dy, dh = torch.from_numpy(rng.normal(size=(4, 16))), torch.from_numpy(rng.normal(size=(4, 16)))
    ((y * dy).sum() + (h * dh).sum()).backward()
    d, dw = ref.norm_backward(dy.numpy(), h.detach().numpy(), wt.detach().numpy(), dh.numpy(), 1e-3)
    assert np.allclose(d, h.grad) and np.allclose(dw, wt.grad)


def test_reference_rounding_and_codes():
    rng = np.random.default_rng(1)
    x = (rng.normal(size=1000) * 10.0 ** rng.integers(-3, 4, 1000)).astype(np.float32)
    assert np.array_equal(ref.rounded(x, "bf16"), torch.from_numpy(x).bfloat16().double().numpy())
    codes, scales = ref.q8_encode(np.array([[1.0, -1.99, 0.0] + [0.25] * 61]))
    assert scales[0, 0] == 2.0 ** -6 and codes[0, 0] == 64 and codes[0, 1] == -127 and codes[0, 3] == 16
    i, s = ref.q8_index(33, 128)
    assert len(np.unique(i)) == 33 * 128 and i.max() < B.ht_q8_bytes(33, 128)[0]
    assert len(np.unique(s)) == 33 * 2 and 4 * s.max() < B.ht_q8_bytes(33, 128)[1]
