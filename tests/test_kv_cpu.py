"""The cache operators without a GPU: host checks of every entry point (only
invalid or empty calls are made, so nothing is launched), the Python layer's
refusals, sizes, and the host reference itself against closed forms."""
import ctypes

import numpy as np
import pytest
import torch

import kv_reference as ref
from block_planner_amd import api
from block_planner_amd import binding as B

A = 0x10000   # an aligned address nobody reads
OK, EINVAL, ESHAPE, EALIGN, ESMALL = 0, 1, 2, 3, 4
BF, F32 = B.HT_BF16, B.HT_FP32


def call(name, base, **change):
    """Status of the entry point with some of its arguments replaced."""
    args = dict(base)
    assert set(change) <= set(args), set(change) - set(args)
    args.update(change)
    return getattr(B.load(), name)(*args.values())


def cache(codes=A, scales=A, n_pages=10, heads=2, dim=128):
    return ctypes.byref(B.KVCacheDesc(codes, scales, n_pages, heads, dim))


BAD_CACHES = [(dict(codes=None), EINVAL), (dict(scales=None), EINVAL), (dict(n_pages=0), ESHAPE),
              (dict(n_pages=1 << 25), ESHAPE), (dict(heads=0), ESHAPE), (dict(dim=0), ESHAPE), (dict(dim=96), ESHAPE),
              (dict(dim=320), ESHAPE), (dict(codes=A + 8), EALIGN), (dict(scales=A + 2), EALIGN)]


def test_cache_bytes():
    assert B.ht_kv_cache_bytes(10, 8, 128) == (10 * 8 * 2 * 64 * 128, 10 * 8 * 2 * 4)
    assert B.ht_kv_cache_bytes(100000, 8, 128)[0] > 2 ** 32
    for bad in ((0, 8, 128), (10, 0, 128), (10, 8, 100), (1 << 25, 8, 128)):
        with pytest.raises(B.HTError) as e:
            B.ht_kv_cache_bytes(*bad)
        assert e.value.code == ESHAPE
    assert B.load().ht_kv_cache_bytes(1, 1, 64, None, None) == EINVAL


PLAN = dict(q_len=A, kv_len=A + 64, owned=A + 128, R=4, table=A + 256, P=8, ldt=8, free=A + 512, cap=16, n_free=A + 640,
            T=4, cu_q=A + 1024, slots=A + 1088, positions=A + 1152, kv_out=A + 1216, owned_out=A + 1280,
            status=A + 1344, stream=None)


@pytest.mark.parametrize("change,code", [
    *[({k: None}, EINVAL) for k in ("q_len", "kv_len", "owned", "table", "free", "n_free", "cu_q", "slots",
                                    "positions", "kv_out", "owned_out", "status")],
    *[({k: A + 1}, EALIGN) for k in ("q_len", "kv_len", "owned", "table", "free", "n_free", "cu_q", "slots",
                                     "positions", "kv_out", "owned_out", "status")],
    (dict(R=0), ESHAPE), (dict(R=-1), ESHAPE), (dict(T=-1), ESHAPE), (dict(P=0), ESHAPE), (dict(ldt=7), ESHAPE),
    (dict(cap=0), ESHAPE), (dict(R=1 << 31), ESHAPE), (dict(T=1 << 31), ESHAPE), (dict(P=1 << 25, ldt=1 << 25), ESHAPE),
    (dict(kv_out=A + 64), EINVAL), (dict(owned_out=A + 128), EINVAL), (dict(status=A + 640), EINVAL),
    (dict(cu_q=A), EINVAL), (dict(slots=A + 1152), EINVAL)])
def test_plan_argument_checks(change, code):
    assert call("ht_kv_plan", PLAN, **change) == code


RELEASE = dict(which=A, R=4, kv_len=A, owned=A, table=A, P=8, ldt=8, free=A, cap=16, n_free=A, stream=None)


@pytest.mark.parametrize("change,code", [
    *[({k: None}, EINVAL) for k in ("which", "kv_len", "owned", "table", "free", "n_free")],
    *[({k: A + 2}, EALIGN) for k in ("kv_len", "owned", "table", "free", "n_free")],
    (dict(R=0), ESHAPE), (dict(P=0), ESHAPE), (dict(ldt=4), ESHAPE), (dict(cap=0), ESHAPE)])
def test_release_argument_checks(change, code):
    assert call("ht_kv_release", RELEASE, **change) == code


ROPE = dict(q=A, ldq=512, hsq=64, k=A, ldk=512, hsk=64, xt=F32, T=3, n_q=4, n_k=2, D=64, rot=64, inter=0, pos=A, inv=A,
            wq=A, wk=A, eps=1e-6, yq=A, ldyq=256, hsyq=64, yk=A, ldyk=128, hsyk=64, yt=BF, stream=None)


@pytest.mark.parametrize("change,code", [
    *[({k: None}, EINVAL) for k in ("q", "k", "pos", "inv", "wq", "wk", "yq", "yk")],
    *[({k: A + 8}, EALIGN) for k in ("q", "k", "inv", "wq", "wk", "yq", "yk")], (dict(pos=A + 2), EALIGN),
    (dict(xt=0), EINVAL), (dict(yt=3), EINVAL), (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL),
    (dict(T=-1), ESHAPE), (dict(n_q=0), ESHAPE), (dict(n_k=-1), ESHAPE), (dict(D=60), ESHAPE), (dict(D=264), ESHAPE),
    (dict(rot=68), ESHAPE), (dict(rot=72), ESHAPE), (dict(rot=-8), ESHAPE), (dict(ldq=60), ESHAPE), (dict(hsk=32), ESHAPE),
    (dict(ldq=514), EALIGN), (dict(hsyq=68), EALIGN), (dict(ldyk=132), EALIGN)])
def test_rope_argument_checks(change, code):
    assert call("ht_qk_norm_rope", ROPE, **change) == code


def test_rope_without_rows_launches_nothing():
    assert call("ht_qk_norm_rope", ROPE, T=0, q=None, k=None, yq=None, yk=None) == OK


BACK = dict(dq=A, lddq=256, hsdq=64, dk=A, lddk=128, hsdk=64, yt=BF, q=A, ldq=512, hsq=64, k=A, ldk=512, hsk=64, xt=F32,
            T=300, n_q=4, n_k=2, D=64, rot=64, inter=0, pos=A, inv=A, wq=A, wk=A, eps=1e-6, dxq=A, lddxq=256, hsdxq=64,
            dxk=A, lddxk=128, hsdxk=64, dwq=A, dwk=A, ws=A, ws_bytes=1 << 24, stream=None)


@pytest.mark.parametrize("change,code", [
    *[({k: None}, EINVAL) for k in ("dq", "dk", "q", "k", "pos", "inv", "wq", "wk", "dxq", "dxk", "dwq", "dwk")],
    *[({k: A + 8}, EALIGN) for k in ("dq", "dk", "q", "k", "inv", "wq", "wk", "dxq", "dxk", "dwq", "dwk", "ws")],
    (dict(ws=None), ESMALL), (dict(ws_bytes=16), ESMALL), (dict(xt=1), EINVAL), (dict(yt=7), EINVAL),
    (dict(D=72 + 4), ESHAPE), (dict(rot=128), ESHAPE), (dict(lddq=32), ESHAPE), (dict(hsdxk=66), EALIGN)])
def test_rope_backward_argument_checks(change, code):
    assert call("ht_qk_norm_rope_backward", BACK, **change) == code


def test_rope_workspace():
    assert B.ht_qk_norm_rope_workspace(8192, 32, 8, 128, False) == 0
    assert B.ht_qk_norm_rope_workspace(0, 32, 8, 128, True) == 0
    assert B.ht_qk_norm_rope_workspace(1, 4, 1, 128, True) == 0          # one workgroup: no partial sums
    n = B.ht_qk_norm_rope_workspace(8192, 32, 8, 128, True)
    assert 0 < n <= 1024 * 2 * 128 * 4
    with pytest.raises(B.HTError):
        B.ht_qk_norm_rope_workspace(1, 0, 1, 128, True)


WRITE = dict(k=A, ldk=256, hsk=128, kt=BF, v=A, ldv=1024, hsv=128, vt=F32, T=5, slots=A, cache=None, stream=None)


@pytest.mark.parametrize("change,code", [
    *[({k: None}, EINVAL) for k in ("k", "v", "slots")], *[({k: A + 8}, EALIGN) for k in ("k", "v")],
    (dict(slots=A + 1), EALIGN), (dict(kt=0), EINVAL), (dict(vt=3), EINVAL), (dict(T=-1), ESHAPE),
    (dict(T=(1 << 28) + 1), ESHAPE), (dict(ldk=100), ESHAPE), (dict(hsv=64), ESHAPE), (dict(ldk=260), EALIGN),
    (dict(ldv=1026), EALIGN)])
def test_write_argument_checks(change, code):
    assert call("ht_kv_write", {**WRITE, "cache": cache()}, **change) == code


ATTN = dict(q=A, ldq=1024, hsq=128, T=6, n_q=8, cache=None, table=A, P=2000, ldt=2000, cu=A, kv=A, R=3, max_q=2, max_kv=100000,
            scale=0.1, causal=1, window=0, out=A, ldo=1024, hso=128, ws=A, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("change,code", [
    *[({k: None}, EINVAL) for k in ("q", "table", "cu", "kv", "out")],
    *[({k: A + 8}, EALIGN) for k in ("q", "out", "ws")], *[({k: A + 2}, EALIGN) for k in ("table", "cu", "kv")],
    (dict(T=-1), ESHAPE), (dict(R=0), ESHAPE), (dict(R=1 << 22), ESHAPE), (dict(T=1 << 29), ESHAPE),
    (dict(n_q=0), ESHAPE), (dict(n_q=7), ESHAPE),
    (dict(P=0), ESHAPE), (dict(ldt=7), ESHAPE), (dict(window=-1), ESHAPE), (dict(max_q=-1), ESHAPE), (dict(max_kv=-1), ESHAPE),
    (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL), (dict(ldq=64), ESHAPE),
    (dict(hso=64), ESHAPE), (dict(ldo=1028), EALIGN), (dict(ws=None), ESMALL), (dict(ws_bytes=64), ESMALL)])
def test_attention_argument_checks(change, code):
    assert call("ht_kv_attention", {**ATTN, "cache": cache()}, **change) == code


@pytest.mark.parametrize("bad,code", BAD_CACHES)
def test_cache_checks(bad, code):
    assert call("ht_kv_write", {**WRITE, "cache": cache(**bad)}) == code
    assert call("ht_kv_attention", {**ATTN, "cache": cache(**bad)}) == code
    assert call("ht_kv_write", {**WRITE, "cache": None}) == EINVAL
    assert call("ht_kv_attention", {**ATTN, "cache": None}) == EINVAL


def test_attention_workspace_is_bounded():
    """Partial results only where tokens are split, and never more than a few
    per row of a large batch."""
    d = B.KVCacheDesc(A, A, 1000, 8, 128)
    assert B.ht_kv_attention_workspace(d, 8192, 1, 32, 8192, 8192) == 0
    assert B.ht_kv_attention_workspace(d, 1, 1, 32, 1, 64) == 0
    assert B.ht_kv_attention_workspace(d, 1, 1, 32, 0, 0) == 0           # lengths not known
    # answers beside a prompt of 8192 rows: partial results of the answers' rows, not of the prompt's
    assert 0 < B.ht_kv_attention_workspace(d, 8208, 17, 32, 8192, 131072) <= 64 * 17 * 8 * 32 * 129 * 4 + 256
    assert 0 < B.ht_kv_attention_workspace(d, 1, 1, 32, 1, 100000) <= 64 * 32 * 129 * 4 + 256


# -- the Python layer ---------------------------------------------------------
def t(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


I32 = torch.int32


def test_python_refusals():
    q, k, pos, inv = t(3, 4, 64), t(3, 2, 64), t(3, dtype=I32), t(32, dtype=torch.float64)
    rope = lambda *a, **kw: api.qk_norm_rope(*a, **kw)  # noqa: E731
    for args, kw in (((q.half(), k, pos, inv), {}), ((q, k.bfloat16(), pos, inv), {}), ((q, k[:2], pos, inv), {}),
                     ((q, k, pos.long(), inv), {}), ((q, k, pos[:2], inv), {}), ((q, k, pos, inv.float()), {}),
                     ((q, k, pos, inv), dict(q_weight=t(64))), ((q, k, pos, inv), dict(q_weight=t(64), k_weight=t(63))),
                     ((q, k, pos, inv), dict(out_dtype=torch.float16)), ((q[0], k, pos, inv), {}),
                     ((q, k, pos, inv), dict(out=(t(3, 4, 32), k)))):
        with pytest.raises(ValueError, match="expected|both or neither"):
            rope(*args, **kw)
    codes, scales = api.kv_cache(5, 2, 64, "cpu")
    assert codes.shape == (5, 2, 2, 4096) and scales.shape == (5, 2, 2) and not codes.any()
    for dim in (32, 100, 512):
        with pytest.raises(B.HTError):
            api.kv_cache(5, 2, dim, "cpu")
    slots = t(3, dtype=I32)
    for args in ((k, k, slots.long(), codes, scales), (k, k[:, :1], slots, codes, scales), (k[:2], k, slots, codes, scales),
                 (k, k, slots, codes.float(), scales), (k, k, slots, codes, scales[:4]), (k, k, slots, codes[:, :1], scales),
                 (k.half(), k, slots, codes, scales)):
        with pytest.raises(ValueError, match="expected|both or neither"):
            api.kv_write(*args)
    qb, table, cu, kv = q.bfloat16(), t(1, 4, dtype=I32), t(2, dtype=I32), t(1, dtype=I32)
    for args, kw in (((q, codes, scales, table, cu, kv, 3), {}), ((qb[..., :32], codes, scales, table, cu, kv, 3), {}),
                     ((qb, codes, scales, table[0], cu, kv, 3), {}), ((qb, codes, scales, table, cu[:1], kv, 3), {}),
                     ((qb, codes, scales, table, cu, kv.long(), 3), {}), ((qb, codes, scales, table, cu, kv, 3), dict(out=q)),
                     ((qb, codes, scales, t(1, 8, dtype=I32)[:, ::2], cu, kv, 3), {})):
        with pytest.raises(ValueError, match="expected|both or neither"):
            api.kv_attention(*args, **kw)
    lens, tab, free = t(2, dtype=I32), t(2, 4, dtype=I32), t(9, dtype=I32)
    for args, kw in (((lens.long(), lens, lens, tab, free, free[:1], 2), {}), ((lens, lens[:1], lens, tab, free, free[:1], 2), {}),
                     ((lens, lens, lens, tab[:1], free, free[:1], 2), {}), ((lens, lens, lens, tab, free, free[:2], 2), {}),
                     ((lens, lens, lens, tab, free, free[:1], 2), dict(out=[lens] * 6))):
        with pytest.raises(ValueError, match="expected|both or neither"):
            api.kv_plan(*args, **kw)
    with pytest.raises(ValueError, match="expected|both or neither"):
        api.kv_release(lens, lens, lens, tab, free, free[:1])
    with pytest.raises(ValueError, match="expected|both or neither"):
        api.kv_release(t(2, dtype=torch.bool), lens, lens, tab.t(), free, free[:1])
    # arguments that are right but not on a GPU: host pointers never reach a kernel
    for f, args in ((rope, (q, k, pos, inv)), (api.kv_write, (k, k, slots, codes, scales)),
                    (api.kv_attention, (qb, codes, scales, table, cu, kv, 3)),
                    (api.kv_plan, (lens, lens, lens, tab, free, free[:1], 2)),
                    (api.kv_release, (t(2, dtype=torch.bool), lens, lens, tab, free, free[:1]))):
        with pytest.raises(ValueError, match="must be on the GPU"):
            f(*args)


# -- the host reference -------------------------------------------------------
@pytest.mark.parametrize("D", [64, 128, 192, 256])
def test_block_layout_is_a_permutation_and_the_library_reads_it(D):
    for i, index in enumerate(ref.block_index(D)):
        assert sorted(index.reshape(-1)) == list(range(64 * D))
        codes = torch.zeros(1, 1, 2, 64 * D, dtype=torch.int8)
        want = (np.arange(64)[:, None] * 7 + np.arange(D)[None]) % 251 - 125
        codes[0, 0, i].numpy()[index] = want
        got = api.kv_cache_values(codes, torch.ones(1, 1, 2))[i]
        np.testing.assert_array_equal(got[0, 0].numpy(), want)


def test_reference_write_closed_forms():
    codes, scales = np.zeros((2, 1, 2, 4096), np.int8), np.zeros((2, 1, 2), np.float32)
    k = np.zeros((2, 1, 64), np.float32)
    k[0, 0, :3], k[1, 0, 0] = [1.0, -0.5, 1 / 128], 0.25
    c, s = ref.write(k, 0 * k, [64, 65], codes, scales)
    at = ref.block_index(64)[0]
    assert s[1, 0, 0] == 2.0 ** -6 and s[1, 0, 1] == 2.0 ** -67 and s[0].max() == 0
    assert list(c[1, 0, 0][at[0, :3]]) == [64, -32, 0] and c[1, 0, 0][at[1, 0]] == 16   # 1/128 is half a step: to even
    c2, s2 = ref.write(k[:1] * 4, 0 * k[:1], [66], c, s)
    assert s2[1, 0, 0] == 2.0 ** -4 and list(c2[1, 0, 0][at[0, :2]]) == [16, -8] and c2[1, 0, 0][at[2, 0]] == 64


def test_reference_attention_closed_forms():
    """Equal keys: the mean of the values seen; one token: its value."""
    rng = np.random.default_rng(0)
    codes, scales = ref.random_cache(rng, 2, 1, 64)
    codes[:, :, 0] = 0
    q = rng.normal(size=(3, 1, 64))
    out, _ = ref.attention(q, codes, scales, np.array([[1, 0]]), [0, 3], [70], 0.125)
    v = codes[:, 0, 1][:, ref.block_index(64)[1].reshape(-1)].reshape(2, 64, 64).astype(float)
    v *= scales[:, 0, 1][:, None, None]
    v = np.concatenate([v[1], v[0]])
    np.testing.assert_allclose(out[2, 0], v[:70].mean(0), rtol=1e-12)
    np.testing.assert_allclose(out[0, 0], v[:68].mean(0), rtol=1e-12)
    out, _ = ref.attention(q, codes, scales, np.array([[1, 0]]), [0, 3], [70], 0.125, window=1)
    np.testing.assert_allclose(out[1, 0], v[68], rtol=1e-12)


def test_attention_kernels_of_a_call():
    """Which kernels a call runs, by its sizes: the query's own checks, and one
    call of each kind."""
    d = B.KVCacheDesc(A, A, 1000, 8, 128)
    info = lambda *a, **kw: B.ht_kv_attention_kernels(d, *a, **kw)  # noqa: E731
    assert info(1, 1, 32, 1, 64) == (1, 0, 0) and info(0, 1, 32, 0, 0) == (1, 0, 0)
    assert info(64, 64, 32, 1, 8192)[0] > 1 and info(64, 64, 32, 1, 8192)[1:] == (0, 0)
    assert info(8192, 1, 32, 8192, 8192) == (0, 1, 8)
    assert info(8208, 17, 32, 8192, 8192)[1:] == (1, 8) and info(8208, 17, 32, 8192, 8192)[0] > 1
    assert info(600, 1, 32, 600, 30000)[0] == 0 and info(600, 1, 32, 600, 30000)[1] > 1
    args = dict(cache=ctypes.byref(d), T=4, R=2, n_q=8, max_q=2, max_kv=64, window=0, info=(ctypes.c_int32 * 3)())
    assert call("ht_kv_attention_kernels", args) == OK
    for change, code in ((dict(info=None), EINVAL), (dict(cache=None), EINVAL), (dict(T=-1), ESHAPE), (dict(R=0), ESHAPE),
                         (dict(n_q=7), ESHAPE), (dict(max_q=-1), ESHAPE), (dict(window=-1), ESHAPE)):
        assert call("ht_kv_attention_kernels", args, **change) == code


@pytest.mark.parametrize("window", [2 ** 40, 2 ** 62, 2 ** 63 - 1])
def test_attention_windows_wider_than_any_request(window):
    """A window past every length is no window: the same kernels and workspace,
    up to the largest number the argument holds."""
    d = B.KVCacheDesc(A, A, 1000, 8, 128)
    for T, R, max_q, max_kv in ((1, 1, 1, 100000), (64, 64, 1, 8192), (600, 1, 600, 30000), (8208, 17, 8192, 131072),
                                (5, 1, 2 ** 30, 2 ** 30)):
        sizes = (T, R, 32, max_q, max_kv)
        assert B.ht_kv_attention_kernels(d, *sizes, window) == B.ht_kv_attention_kernels(d, *sizes, 0)
        assert B.ht_kv_attention_workspace(d, *sizes, window) == B.ht_kv_attention_workspace(d, *sizes, 0)


class On:
    """What _on_gpu looks at of a tensor."""

    def __init__(self, device):
        self.device = device
        self.is_cuda = device >= 0

    def get_device(self):
        return self.device


def test_tensors_of_several_devices_are_refused(monkeypatch):
    """The kernels run on the current device and get bare addresses: memory of
    another GPU never reaches them."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    api._on_gpu(On(1), None, On(1))
    api._on_gpu(None)
    for tensors, match in (((On(1), On(0)), "one GPU"), ((On(0), On(1)), "one GPU"), ((On(0), On(0)), "current device"),
                           ((On(1), On(-1)), "must be on the GPU"), ((On(-1), On(1)), "must be on the GPU")):
        with pytest.raises(ValueError, match=match):
            api._on_gpu(*tensors)
    assert torch.empty(1, device="meta").get_device() < 0 and torch.empty(1).get_device() < 0


def test_current_stream_without_torchs_private_lookup(monkeypatch):
    """The current stream's handle comes from a private torch function where
    there is one, and from the public one where there is not."""
    class Stream:
        cuda_stream = 0x1234

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0x5678 + device, raising=False)
    assert B._stream(None) == 0x5678
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    assert B._stream(None) == 0x1234
    assert B._stream(7) == 7 and B._stream(Stream) == 0x1234


def test_roundings_of_an_entry_stay_below_one_scale():
    """Rows appended to a page raise its scale again and again: every entry is
    off by less than one final scale, the halvings alone by more than half."""
    rng = np.random.default_rng(4)
    at = ref.block_index(64)[0]
    most = halved = 0.0
    for trial in range(40):
        codes, scales = np.zeros((1, 1, 2, 4096), np.int8), np.zeros((1, 1, 2), np.float32)
        rows = np.zeros((12, 1, 64), np.float32)
        for t in range(12):
            rows[t, 0] = rng.uniform(-1, 1, 64) * 2.0 ** t
            rows[t, 0, 0] = 2.0 ** (t + rng.integers(0, 2)) * rng.choice([0.5, 0.75, 1 - 2.0 ** -20])
            if t == 0:
                rows[t, 0, 1:4] = [5 / 128, 21 / 128, 1 - 2.0 ** -20]
            codes, scales = ref.write(rows[t:t + 1], rows[t:t + 1], [t], codes, scales)
            if t == 0:
                own = codes[0, 0, 0][at[0]] * float(scales[0, 0, 0])
            off = np.abs(codes[0, 0, 0][at[:t + 1]] * float(scales[0, 0, 0]) - rows[:t + 1, 0]) / scales[0, 0, 0]
            most = max(most, off.max())
            halved = max(halved, (np.abs(codes[0, 0, 0][at[0]] * float(scales[0, 0, 0]) - own) / scales[0, 0, 0]).max())
    assert 0.7 < most < 1 and halved > 0.5, (most, halved)


@pytest.mark.parametrize("D,n_q,H,R,q,kv,prompt", [
    # us measured, prompt kernel against decode kernel
    (64, 32, 4, 4, 300, 300, True), (64, 32, 8, 4, 300, 300, True),       # 17 28; 18 27
    (64, 8, 1, 1, 1500, 1500, False), (64, 32, 4, 1, 100, 1000, False),   # 22 17; 25 15
    (128, 32, 8, 4, 300, 300, True), (128, 32, 8, 4, 200, 200, True),     # 21 37; 18 26
    (128, 32, 8, 4, 512, 512, True), (128, 8, 1, 1, 512, 512, False),     # 29 62; 20 15
    (128, 8, 1, 1, 1500, 1500, False), (128, 32, 8, 1, 100, 1000, False),   # 31 23; 29 15
    (192, 32, 8, 4, 200, 200, True), (192, 32, 4, 4, 100, 100, True),     # 23 56; 19 32
    (192, 8, 1, 1, 1024, 1024, False), (192, 12, 2, 1, 300, 1000, False),   # 38 26; 38 16
    (256, 32, 8, 4, 200, 200, True), (256, 32, 8, 1, 300, 300, True),     # 29 70; 28 34
    (256, 32, 8, 1, 512, 512, True), (256, 8, 1, 1, 1024, 1024, False),   # 37 46; 46 31
    (256, 8, 1, 1, 512, 512, False), (256, 32, 8, 1, 40, 4000, False),    # 36 15; 56 40
    (256, 32, 8, 1, 100, 4000, True), (128, 32, 8, 1, 300, 4000, True)])  # 63 74; 50 70
def test_attention_kernel_of_short_prompts(D, n_q, H, R, q, kv, prompt):
    """The kernel that is faster for the shape."""
    info = B.ht_kv_attention_kernels(B.KVCacheDesc(A, A, 1000, H, D), R * q, R, n_q, q, kv)
    assert (info[1] > 0) == prompt
