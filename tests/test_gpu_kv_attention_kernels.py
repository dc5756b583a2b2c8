"""Every kernel instance and path of ht_kv_attention on the GPU against the
definition in 64 bits: each test first asks the library which kernels its call
runs (ht_kv_attention_kernels), so that another choice of them shows here."""
import numpy as np
import pytest
import torch

import kv_reference as ref
from block_planner_amd import api
from block_planner_amd import binding as B
from test_gpu_kv_attention import bf16, check, dev, gpu, make, run

pytestmark = pytest.mark.gpu

FAR = 10 ** 6   # a hint far above the lengths


def kernels(q, codes, R, max_q, max_kv, window=0):
    d = B.KVCacheDesc(1 << 20, 1 << 20, codes.shape[0], codes.shape[1], codes.shape[3] // 64)
    return B.ht_kv_attention_kernels(d, q.shape[0], R, q.shape[1], max_q, max_kv, window)


HEADS = [(4, 1, 64), (4, 2, 128), (2, 2, 192), (2, 1, 256)]
BATCHES = [([70], [70]), ([130, 33], [200, 500]), ([100, 40, 0, 120], [300, 64, 70, 2100]), ([90, 64], [30, 900])]


@pytest.mark.parametrize("n_q,H,D", HEADS)
@pytest.mark.parametrize("q_len,kv_len", BATCHES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [1, 40, 64, 65, 333, 1500])
def test_prompts_with_a_window(n_q, H, D, q_len, kv_len, causal, window):
    """On the prompt kernel: windows inside a page, over several, wider than the tokens."""
    print(n_q, H, D, q_len, kv_len, causal, window, flush=True)
    args = make(D + window + sum(kv_len), q_len, kv_len, n_q, H, D)[1:]
    hint = dict(max_q=FAR, max_kv=FAR)
    decode, prompt, waves = kernels(args[0], args[1], len(q_len), **hint, window=window)
    assert prompt >= 1 and waves == 4 and (decode == 0) == (len(q_len) == 1)
    check(*args, causal=causal, window=window, **hint)


@pytest.mark.parametrize("n_q,H,D", HEADS)
@pytest.mark.parametrize("window", [0, 65, 700, 2500])
def test_splits_of_prompts(n_q, H, D, window):
    """A prompt whose tokens are split, some of the splits outside the window of
    some tiles, beside a shorter one and answers."""
    args = make(D + window, [100, 1, 50, 3], [3900, 700, 300, 2000], n_q, H, D)[1:]
    hint = dict(max_q=9000, max_kv=9000)
    decode, prompt, waves = kernels(args[0], args[1], 4, **hint, window=window)
    assert decode >= 1 and prompt >= 4 and waves == 4
    check(*args, window=window, **hint)
    args = make(D + window + 1, [150], [2500], n_q, H, D)[1:]
    assert kernels(args[0], args[1], 1, **hint, window=window)[0] == 0
    check(*args, window=window, **hint)


@pytest.mark.parametrize("n_q,H,D", [(16, 1, 64), (16, 1, 128), (16, 1, 192), (16, 1, 256)])
@pytest.mark.parametrize("window", [0, 150])
def test_prompts_of_ordinary_calls(n_q, H, D, window):
    """With the lengths themselves as hints; many rows, checked at some heads."""
    q_len, kv_len = [500, 400], [1400, 400]
    rng, q, codes, scales, table, cu, kv = make(D + window, q_len, kv_len, 4 * n_q, 4, D)
    info = kernels(q, codes, 2, 500, 1400, window)
    assert info[1] >= 1 and info[2] == 4
    got = run(q, codes, scales, table, cu, kv, window=window).double().cpu().numpy()
    heads = [0, 15, 16, 50]
    rows = np.r_[0:3, 120:130, 497:503, 640:645, 898:900]
    for h in heads:
        want, tol = ref.attention(q[:, h:h + 1], codes[:, h // 16:h // 16 + 1], scales[:, h // 16:h // 16 + 1], table, cu,
                                  kv, 1 / np.sqrt(D), True, window)
        assert np.all(np.abs(got[rows, h:h + 1] - want[rows]) <= tol[rows]), h


@pytest.mark.parametrize("n_q,D", [(64, 64), (64, 128), (48, 192), (64, 256)])
def test_tiles_in_turn(n_q, D):
    """max_q below the real length: one workgroup takes all tiles of its head one
    after the other, through the same shared memory."""
    args = make(D, [30, 17], [200, 90], n_q, 1, D)[1:]
    for window in (0, 70):
        info = kernels(args[0], args[1], 2, 1, FAR)
        assert info[1] >= 1
        check(*args, max_q=1, max_kv=FAR)
        check(*args, max_q=1, max_kv=40000)
        if window:
            check(*args, max_q=1, max_kv=FAR, window=window)


# -- the instance of 8 wavefronts: D = 128, rows x heads of 262144 and more -----
def wide(seed, q_len, kv_len, n_q=1024, H=128):
    """Many heads in place of many rows; codes by the library's generator."""
    D, rng = 128, np.random.default_rng(seed)
    n_pages = sum(-(-int(k) // 64) for k in kv_len) + 2
    codes, scales = ref.random_cache(rng, n_pages, H, D)
    table = ref.random_table(rng, kv_len, n_pages, max(-(-int(k) // 64) for k in kv_len))
    q = bf16(rng.standard_normal((sum(q_len), n_q, D), dtype=np.float32))
    cu = np.concatenate([[0], np.cumsum(q_len)]).astype(np.int32)
    return rng, q, codes, scales, table, cu, np.asarray(kv_len, np.int32)


def check_heads(got, q, codes, scales, table, cu, kv, heads, causal=True, window=0):
    group = q.shape[1] // codes.shape[1]
    for h in heads:
        at = slice(h * group, (h + 1) * group)
        want, tol = ref.attention(q[:, at], codes[:, h:h + 1], scales[:, h:h + 1], table, cu, kv, 1 / np.sqrt(128), causal,
                                  window)
        err = np.abs(got[:, at].double().cpu().numpy() - want)
        assert np.all(err <= tol), (h, np.max(err - tol))


@pytest.mark.parametrize("q_len,kv_len,causal,window", [
    ([300], [300], True, 0), ([261], [401], True, 0), ([200, 1, 60, 39], [200, 300, 129, 500], True, 0),
    ([180, 130], [180, 420], False, 0), ([300], [450], True, 100), ([150, 4, 150], [600, 200, 64], True, 65)])
def test_eight_wavefronts(q_len, kv_len, causal, window):
    """Ragged tiles, several requests with answers among them, windows, more rows than tokens."""
    print(q_len, kv_len, causal, window, flush=True)
    rng, q, codes, scales, table, cu, kv = wide(sum(kv_len) + window, q_len, kv_len)
    info = kernels(q, codes, len(q_len), max(q_len), max(kv_len), window)
    assert info[1:] == (1, 8) and (info[0] > 0) == (len(q_len) > 1)
    got = run(q, codes, scales, table, cu, kv, causal=causal, window=window)
    check_heads(got, q, codes, scales, table, cu, kv, (0, 77, 127), causal, window)


def test_eight_wavefronts_hidden_pages_and_nan_rows():
    rng, q, codes, scales, table, cu, kv = wide(1, [260, 40], [300, 129])
    table[0, 1], table[0, 3], table[1, 2] = -1, len(codes), 2 ** 31 - 1
    assert kernels(q, codes, 2, 260, 300)[2] == 8
    clean = run(q, codes, scales, table, cu, kv)
    check_heads(clean, q, codes, scales, table, cu, kv, (0, 64))
    hurt = np.zeros(q.shape[:2], bool)
    for at, x in (((0, 1, 5), np.nan), ((200, 515, 0), np.inf), ((299, 1023, 127), -np.inf)):
        q[at] = x
        hurt[at[:2]] = True
    got = run(q, codes, scales, table, cu, kv)
    assert torch.all(torch.isnan(got[gpu(hurt)])) and torch.equal(got[gpu(~hurt)], clean[gpu(~hurt)])
    assert torch.equal(run(q, codes, scales, table, cu, kv)[gpu(~hurt)], clean[gpu(~hurt)])


def test_eight_wavefronts_tiles_in_turn():
    """Twice as many columns as the hint says: two tiles by each workgroup."""
    rng, q, codes, scales, table, cu, kv = wide(2, [300], [350])
    assert kernels(q, codes, 1, 150, FAR)[1:] == (1, 8)
    got = run(q, codes, scales, table, cu, kv, max_q=150, max_kv=FAR)
    check_heads(got, q, codes, scales, table, cu, kv, (0, 100))


@pytest.mark.parametrize("n_q,H,n_pages,rows,waves", [(16, 8, 34000, 90, 4), (1024, 128, 2200, 280, 8)])
def test_prompts_past_32_bits(n_q, H, n_pages, rows, waves):
    """Blocks of a cache of more than 4 GiB, on the prompt kernel."""
    D = 128
    codes, scales = api.kv_cache(n_pages, H, D, dev())
    assert codes.numel() > 2 ** 32
    rng = np.random.default_rng(13)
    pages = np.array([n_pages - 1, 5, n_pages - 2, n_pages - 7, 1], np.int32)[:-(-rows // 64)]
    slots = (pages[np.arange(rows) // 64] * 64 + np.arange(rows) % 64).astype(np.int32)
    k, v = (rng.standard_normal((rows, H, D), dtype=np.float32) for _ in range(2))
    api.kv_write(gpu(k), gpu(v), gpu(slots), codes, scales)
    at = gpu(pages).long()
    small, small_scales = codes[at].cpu().numpy(), scales[at].cpu().numpy()
    q = bf16(rng.standard_normal((rows, n_q, D), dtype=np.float32))
    cu, kv = np.array([0, rows], np.int32), np.array([rows], np.int32)
    assert kernels(q, codes, 1, rows, FAR)[::2] == (0, waves)
    got = api.kv_attention(gpu(q).to(torch.bfloat16), codes, scales, gpu(pages[None]), gpu(cu), gpu(kv), rows, max_kv=FAR)
    check_heads(got, q, small, small_scales, np.arange(len(pages), dtype=np.int32)[None], cu, kv, (0, H - 1))
