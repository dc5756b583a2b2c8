"""ht_kv_attention on the GPU against the definition in 64 bits, with the
bound that kv_reference.attention derives for every entry."""
import numpy as np
import pytest
import torch

import kv_reference as ref
from block_planner_amd import api
from block_planner_amd import workloads as wl

pytestmark = pytest.mark.gpu


def dev():
    return torch.device("cuda:0")


def bf16(x):
    return wl.bf16_bits_to_f32(wl.to_bf16_bits(x))


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev())


def make(seed, q_len, kv_len, n_q, H, D, spare=3, width=None):
    rng = np.random.default_rng(seed)
    n_pages = sum(-(-int(k) // 64) for k in kv_len) + spare
    codes, scales = ref.random_cache(rng, n_pages, H, D)
    table = ref.random_table(rng, kv_len, n_pages, width)
    q = bf16(rng.normal(size=(sum(q_len), n_q, D)).astype(np.float32))
    cu = np.concatenate([[0], np.cumsum(q_len)]).astype(np.int32)
    return rng, q, codes, scales, table, cu, np.asarray(kv_len, np.int32)


def run(q, codes, scales, table, cu, kv, **kw):
    args = dict(max_q=int(np.max(cu[1:] - cu[:-1])), max_kv=int(kv.max()))
    args.update(kw)
    out = api.kv_attention(gpu(q).to(torch.bfloat16), gpu(codes), gpu(scales), gpu(table), gpu(cu), gpu(kv), **args)
    torch.cuda.synchronize()
    return out


def check(q, codes, scales, table, cu, kv, scale=None, causal=True, window=0, **kw):
    s = 1 / np.sqrt(q.shape[2]) if scale is None else scale
    want, tol = ref.attention(q, codes, scales, table, cu, kv, s, causal, window)
    got = run(q, codes, scales, table, cu, kv, scale=scale, causal=causal, window=window, **kw)
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= tol), f"{np.max(err - tol)} over at {np.unravel_index(np.argmax(err - tol), err.shape)}"
    return got


@pytest.mark.parametrize("n_q,H,D", [(4, 1, 64), (32, 4, 64), (8, 2, 128), (3, 3, 128), (14, 2, 128), (4, 2, 192),
                                     (4, 1, 256), (40, 2, 64)])
@pytest.mark.parametrize("q_len,kv_len", [
    ([1], [1]), ([1], [63]), ([1], [64]), ([1], [65]), ([1, 1, 1], [1, 300, 129]), ([2, 4, 1], [2, 700, 64])])
def test_decode(n_q, H, D, q_len, kv_len):
    print(n_q, H, D, q_len, kv_len, flush=True)
    check(*make(D + n_q + sum(kv_len), q_len, kv_len, n_q, H, D)[1:])


@pytest.mark.parametrize("n_q,H,D", [(4, 1, 64), (4, 2, 128), (2, 2, 192), (2, 1, 256)])
@pytest.mark.parametrize("q_len,kv_len", [([70], [70]), ([130, 1, 33], [130, 200, 500]), ([64, 65], [128, 65])])
def test_prompts(n_q, H, D, q_len, kv_len):
    print(n_q, H, D, q_len, kv_len, flush=True)
    check(*make(D + sum(kv_len), q_len, kv_len, n_q, H, D)[1:])


@pytest.mark.parametrize("n_q,H,D", [(4, 1, 64), (16, 2, 128), (12, 6, 256)])
def test_answers_beside_prompts(n_q, H, D):
    """Requests of both kernels in one batch, long enough that both split
    their tokens; one request with a window over a long cache."""
    check(*make(D, [130, 1, 2, 40, 0, 3], [2200, 5000, 1700, 40, 100, 64], n_q, H, D)[1:])
    check(*make(D + 1, [1, 90], [9000, 3000], n_q, H, D)[1:], window=2500)


@pytest.mark.parametrize("window", [1, 5, 64, 65, 100000])
@pytest.mark.parametrize("q_len,kv_len", [([1, 1], [500, 3]), ([100, 3], [300, 64])])
def test_window(window, q_len, kv_len):
    check(*make(window + sum(kv_len), q_len, kv_len, 4, 2, 64)[1:], window=window)


@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("q_len,kv_len", [([1, 20], [130, 200]), ([90], [90])])
def test_not_causal(window, q_len, kv_len):
    check(*make(sum(kv_len), q_len, kv_len, 4, 2, 128)[1:], causal=False, window=window)


@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_see_nothing(causal):
    """More rows than tokens (the first ones lie before the cache), no tokens
    at all, and requests without rows."""
    rng, q, codes, scales, table, cu, kv = make(5, [5, 3, 0, 1, 40], [2, 0, 70, 10, 30], 4, 2, 64)
    got = check(q, codes, scales, table, cu, kv, causal=causal)
    assert torch.all(got[5:8] == 0)
    if causal:
        assert torch.all(got[:3] == 0) and torch.all(got[9:19] == 0)


def test_pages_outside_the_cache_are_hidden():
    rng, q, codes, scales, table, cu, kv = make(6, [1, 2, 1], [300, 129, 64], 4, 2, 64)
    table[0, 1], table[0, 3] = -1, len(codes)
    table[1, 2] = 2 ** 31 - 1
    table[2, 0] = -2 ** 31
    got = check(q, codes, scales, table, cu, kv)
    assert torch.all(got[3] == 0)


def test_what_lies_past_the_length_does_not_count():
    """Other codes past kv_len and in other pages, and a table wider than the
    lengths with pages of nobody behind it: the same bits."""
    rng, q, codes, scales, table, cu, kv = make(7, [1, 5], [77, 130], 8, 2, 128, width=9)
    first = check(q, codes, scales, table, cu, kv)
    index = ref.block_index(128)
    for r in range(2):
        at = int(kv[r]) % 64
        for i in (0, 1):
            codes[table[r, kv[r] // 64], :, i][:, index[i][at:].reshape(-1)] = -128
        table[r, kv[r] // 64 + 1:] = 0
    free = np.setdiff1d(np.arange(len(codes)), np.concatenate([table[r, :-(-kv[r] // 64)] for r in range(2)]))
    codes[free], scales[free] = 127, np.float32(np.nan)
    assert torch.equal(run(q, codes, scales, table, cu, kv), first)


def test_hints_do_not_change_what_is_computed():
    """max_q and max_kv too small or too large: within the bound all the same."""
    rng, q, codes, scales, table, cu, kv = make(8, [1, 50, 3], [900, 200, 64], 4, 2, 64)
    for max_q, max_kv in ((1, 1), (1, 10 ** 6), (1000, 64), (0, 0), (50, 900), (4, 100000)):
        check(q, codes, scales, table, cu, kv, max_q=max_q, max_kv=max_kv)


def test_values_far_apart():
    """Pages whose values differ by many powers of two, a zero page, large
    scores, zero and huge queries."""
    rng, q, codes, scales, table, cu, kv = make(9, [1, 1, 2, 1], [400, 400, 300, 200], 4, 2, 64)
    scales[:, :, 1] = np.ldexp(1.0, rng.integers(-40, 40, size=scales.shape[:2])).astype(np.float32)
    scales[table[1, 2], :, :] = np.ldexp(1.0, -67)
    codes[table[1, 2]] = 0
    scales[table[2], :, 0] = np.ldexp(1.0, -3)
    q[0, 0] = 0
    q[3] = bf16(q[3] * 1e4)
    q[4] = bf16(q[4] * 1e-30)
    check(q, codes, scales, table, cu, kv)
    check(q, codes, scales, table, cu, kv, scale=-0.2)
    check(q, codes, scales, table, cu, kv, scale=0.0)


def test_heavy_token_over_many_light_ones():
    """One token takes nearly all the weight with a tiny value while thousands
    of light ones carry the result."""
    D, n = 64, 5000
    rng, q, codes, scales, table, cu, kv = make(10, [1], [n], 2, 1, D)
    scales[:, :, 0] = np.ldexp(1.0, -7)
    scales[:, :, 1] = np.ldexp(1.0, 0)
    codes[:, :, 0] = np.clip(codes[:, :, 0], -20, 20)
    index = ref.block_index(D)
    q[:] = 1.0
    codes[table[0, 0], 0, 0][index[0][0]] = 127          # token 0: score 64 * 127/128 / 8 above the rest
    codes[table[0, 0], 0, 1] = 0                          # its page carries nothing
    scales[table[0, 0], 0, 1] = np.ldexp(1.0, -60)
    check(q, codes, scales, table, cu, kv)
    check(q, codes, scales, table, cu, kv, scale=0.35)


def test_infinite_and_nan_queries():
    rng, q, codes, scales, table, cu, kv = make(11, [3, 1], [70, 300], 4, 2, 64)
    clean = check(q, codes, scales, table, cu, kv)
    q[0, 1, 5], q[2, 3, 0], q[3, 0, 63] = np.nan, np.inf, -np.inf
    got = run(q, codes, scales, table, cu, kv)
    hurt = np.zeros(q.shape[:2], bool)
    hurt[0, 1] = hurt[2, 3] = hurt[3, 0] = True
    assert torch.all(torch.isnan(got[gpu(hurt)])) and torch.equal(got[gpu(~hurt)], clean[gpu(~hurt)])


def test_strides_streams_and_repetition():
    """q and out as parts of wider rows, another stream, the same bits again."""
    rng, q, codes, scales, table, cu, kv = make(12, [1, 9], [700, 90], 8, 2, 64, width=20)
    want = check(q, codes, scales, table, cu, kv)
    wide = torch.zeros(10, 20, 64, dtype=torch.bfloat16, device=dev())
    wide[:, 4:12] = gpu(q).to(torch.bfloat16)
    out = torch.full((10, 16, 64), 7.0, dtype=torch.bfloat16, device=dev())
    rest = (gpu(codes), gpu(scales), gpu(np.concatenate([table, table], 1))[:, :20], gpu(cu), gpu(kv))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        api.kv_attention(wide[:, 4:12], *rest, 9, max_kv=700, out=out[:, 2:10])
    side.synchronize()
    assert torch.equal(out[:, 2:10], want)
    assert torch.all(out[:, :2] == 7) and torch.all(out[:, 10:] == 7)


@pytest.mark.parametrize("what", ["decode", "prompt"])
def test_offsets_past_32_bits(what):
    """A cache of more than 4 GiB whose last pages are in use: written and
    read through ht_kv_write and ht_kv_attention."""
    H, D, n_pages = 8, 128, 34000                         # 131 KiB a page and layer
    codes, scales = api.kv_cache(n_pages, H, D, dev())
    assert codes.numel() > 2 ** 32
    rng = np.random.default_rng(13)
    n = 150 if what == "decode" else 90
    rows = 1 if what == "decode" else n
    pages = np.array([n_pages - 1, 5, n_pages - 2], np.int32)
    slots = (pages[np.arange(n) // 64] * 64 + np.arange(n) % 64).astype(np.int32)
    k, v = (rng.normal(size=(n, H, D)).astype(np.float32) for _ in range(2))
    api.kv_write(gpu(k), gpu(v), gpu(slots), codes, scales)
    small = [a.cpu().numpy() for a in (codes[gpu(pages).long()], scales[gpu(pages).long()])]
    q = bf16(rng.normal(size=(rows, 16, D)).astype(np.float32))
    cu, kv = np.array([0, rows], np.int32), np.array([n], np.int32)
    got = api.kv_attention(gpu(q).to(torch.bfloat16), codes, scales, gpu(pages[None]), gpu(cu), gpu(kv), rows)
    want, tol = ref.attention(q, *small, np.arange(3, dtype=np.int32)[None], cu, kv, 1 / np.sqrt(D))
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)


# Short calls go to the decode kernel alone, by the launch hints: a max_kv above
# the lengths sends them to the prompt kernel, whole (10^6) or in splits of
# some tens of pages (40000).
@pytest.mark.parametrize("max_kv", [40000, 10 ** 6])
@pytest.mark.parametrize("n_q,H,D", [(4, 1, 64), (4, 2, 128), (2, 2, 192), (2, 1, 256), (8, 1, 256)])
@pytest.mark.parametrize("q_len,kv_len,causal,window", [
    ([70], [70], True, 0), ([130, 1, 33], [130, 200, 500], True, 0), ([64, 65], [128, 65], False, 0),
    ([100, 3], [300, 64], True, 65), ([90], [90], False, 40), ([100, 40, 0, 120], [60, 0, 70, 4200], True, 0),
    ([130, 1, 2, 40, 0, 3], [2200, 5000, 1700, 40, 100, 64], True, 0), ([1, 90], [5000, 3000], True, 2500)])
def test_short_prompts_in_the_prompt_kernel(n_q, H, D, q_len, kv_len, causal, window, max_kv):
    print(n_q, H, D, q_len, kv_len, causal, window, max_kv, flush=True)
    check(*make(D + sum(kv_len), q_len, kv_len, n_q, H, D)[1:], causal=causal, window=window, max_kv=max_kv)


@pytest.mark.parametrize("n_q,H,D", [(16, 2, 64), (12, 2, 128), (4, 2, 192), (8, 1, 256)])
@pytest.mark.parametrize("q_len,kv_len,window", [
    ([260], [260], 0), ([200, 1, 33], [250, 2000, 500], 0), ([150], [2300], 0), ([90, 17], [3000, 1700], 333),
    ([50, 0, 20], [30, 90, 0], 0)])
def test_short_prompts(n_q, H, D, q_len, kv_len, window):
    """Prompts of many tiles: on the decode kernel, whole and in splits."""
    print(n_q, H, D, q_len, kv_len, window, flush=True)
    check(*make(D + sum(kv_len), q_len, kv_len, n_q, H, D)[1:], window=window)


@pytest.mark.parametrize("max_kv", [300, 10 ** 6])
def test_short_prompts_with_hidden_pages_and_nan_rows(max_kv):
    rng, q, codes, scales, table, cu, kv = make(14, [80, 40, 64], [300, 129, 64], 4, 2, 64)
    table[0, 1], table[0, 3] = -1, len(codes)
    table[1, 2] = 2 ** 31 - 1
    table[2, 0] = -2 ** 31
    clean = check(q, codes, scales, table, cu, kv, max_kv=max_kv)
    assert torch.all(clean[120:] == 0)
    q[0, 1, 5], q[70, 3, 0], q[100, 0, 63] = np.nan, np.inf, -np.inf
    got = run(q, codes, scales, table, cu, kv, max_kv=max_kv)
    hurt = np.zeros(q.shape[:2], bool)
    hurt[0, 1] = hurt[70, 3] = hurt[100, 0] = True
    assert torch.all(torch.isnan(got[gpu(hurt)])) and torch.equal(got[gpu(~hurt)], clean[gpu(~hurt)])
