"""ht_kv_attention at the limits of its arithmetic and of its arguments: scores
of any size, rows of no request, rows of q with one entry far above the rest."""
import numpy as np
import pytest
import torch

import kv_reference as ref
from block_planner_amd import binding as B
from test_gpu_kv_attention import bf16, check, make, run

pytestmark = pytest.mark.gpu


# rows of the requests, launch hint for kv_len: the decode kernel, the prompt kernel whole, and in splits
SIDES = {"decode": ([1, 3], {}), "prompt": ([70, 40], dict(max_kv=10 ** 6)), "splits": ([70, 40], dict(max_kv=40000))}


def assert_side(side, q, codes, q_len, kv, hint):
    d = B.KVCacheDesc(1 << 20, 1 << 20, codes.shape[0], codes.shape[1], codes.shape[3] // 64)
    info = B.ht_kv_attention_kernels(d, len(q), len(q_len), q.shape[1], max(q_len), hint.get("max_kv", int(max(kv))))
    assert (info[1] > 1 if side == "splits" else info[1] > 0) == (side != "decode"), info


@pytest.mark.parametrize("side", SIDES)
@pytest.mark.parametrize("power", [10, 20, 22, 24, 25, 26, 27, 28, 29, 30, 33, 40, 60, 100])
def test_scores_of_any_size(side, power):
    """Scores of about 2^power in log2 units.  From 2^24 on fp32 does not tell
    a whole unit: a row whose two largest scores differ by more than their
    rounding gives the value of its largest (a weight is fp16: 2^-11; the result
    bf16: 2^-8), every row a mean of the values it sees."""
    q_len, hint = SIDES[side]
    rng, q, codes, scales, table, cu, kv = make(power, q_len, [200, 2100], 8, 2, 64)
    assert_side(side, q, codes, q_len, kv, hint)
    D, index = 64, ref.block_index(64)
    scale = 1 / np.sqrt(D)
    vals = []
    for r in range(2):
        pages = table[r, :-(-kv[r] // 64)]
        vals.append([[(codes[pages, h, i][:, index[i].reshape(-1)].astype(np.float64)
                       * scales[pages, h, i].astype(np.float64)[:, None]).reshape(-1, D)[:kv[r]] for i in (0, 1)]
                     for h in range(2)])
    far = max(np.abs(vals[r][h][0] @ q[cu[r]:cu[r + 1]].reshape(-1, D).T).max() for r in range(2) for h in range(2))
    q = bf16(q * np.float32(2.0 ** (power - int(np.floor(np.log2(far * scale * np.log2(np.e)))))))
    got = run(q, codes, scales, table, cu, kv, **hint).double().cpu().numpy()
    assert np.isfinite(got).all()
    sure = 0
    for r in range(2):
        for t in range(cu[r], cu[r + 1]):
            n = kv[r] - (cu[r + 1] - t) + 1
            for a in range(8):
                k, v = vals[r][a // 4][0][:n], vals[r][a // 4][1][:n]
                assert np.all(np.abs(got[t, a]) <= (1 + 2.0 ** -8 + 2.0 ** -11) * np.abs(v).max(0))
                s = k @ q[t, a].astype(np.float64) * scale * np.log2(np.e)
                two = np.sort(s)[-2:]
                if two[1] - two[0] > 64 + 2.0 ** -17 * (np.abs(k) @ np.abs(q[t, a])).max() * scale:
                    sure += 1
                    w = v[np.argmax(s)]
                    assert np.all(np.abs(got[t, a] - w) <= (2.0 ** -8 + 2.0 ** -11) * np.abs(w) + 2.0 ** -30), (t, a)
    assert power < 20 or sure > 0.9 * 8 * len(q)


@pytest.mark.parametrize("n_q,H,D", [(8, 2, 64), (2, 2, 192)])
@pytest.mark.parametrize("q_len,hint", [([1, 2], {}), ([40], dict(max_kv=10 ** 6)), ([40, 1, 30], dict(max_kv=40000)),
                                        ([0, 0], {})])
@pytest.mark.parametrize("before,after", [(0, 5), (3, 0), (2, 700)])
def test_rows_of_no_request_are_zero(n_q, H, D, q_len, hint, before, after):
    """A batch padded to a fixed number of rows (and one that starts late): zeros
    there, in the output's own buffer too, and nothing else of it is touched."""
    rng, q, codes, scales, table, cu, kv = make(3, q_len, [300, 70, 90][:len(q_len)], n_q, H, D)
    clean = run(q, codes, scales, table, cu, kv, **hint)
    n, T = len(q), before + len(q) + after
    wide = bf16(rng.normal(size=(T, n_q, D)).astype(np.float32))
    wide[before:before + n] = q
    wide[0], wide[-1] = (np.nan if before else wide[0]), (np.nan if after else wide[-1])
    buf = torch.full((T + 2, n_q + 3, D + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[1:-1, 2:-1, :D]
    hint = dict(max_q=int(max(q_len)), **hint)
    got = run(wide, codes, scales, table, cu + np.int32(before), kv, out=out, **hint)
    assert got.data_ptr() == out.data_ptr()
    assert torch.equal(out[before:before + n], clean)
    assert torch.all(out[:before] == 0) and torch.all(out[before + n:] == 0)
    out.fill_(7.0)
    assert torch.all(buf == 7)
    assert torch.all(run(wide, codes, scales, table, cu + np.int32(before), kv, **hint)[before + n:] == 0)


def attention_bound(q, codes, scales, table, cu, kv, scale, want):
    """What a result may be off by, [T, n_q, D], with q carried to 2^-22 of its
    row's largest entry: half a bf16 step (2^-8), fp16 weights (2^-11) and fp32
    exponents and sums, the weights' errors carried through the weighted mean
    (a weight off by a factor 1 + e moves the result by e (mean |v| + |out|))."""
    D, H, tol = q.shape[2], codes.shape[1], np.zeros(want.shape)
    index = ref.block_index(D)
    for r in range(len(kv)):
        pages = table[r, :-(-kv[r] // 64)]
        for h in range(H):
            k, v = ((codes[pages, h, i][:, index[i].reshape(-1)].astype(np.float64)
                     * scales[pages, h, i].astype(np.float64)[:, None]).reshape(-1, D)[:kv[r]] for i in (0, 1))
            for t in range(cu[r], cu[r + 1]):
                n = kv[r] - (cu[r + 1] - t) + 1
                for a in range(h * (q.shape[1] // H), (h + 1) * (q.shape[1] // H)):
                    x = q[t, a].astype(np.float64)
                    s = k[:n] @ x * scale
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    off = abs(scale) * 2.0 ** -22 * np.abs(x).max() * np.abs(k[:n]).sum(1).max()
                    off += 2.0 ** -24 * (64 + 4 * np.abs(s).max() + 4 * abs(scale) * (np.abs(k[:n]) @ np.abs(x)).max())
                    size = p @ np.abs(v[:n]) + np.abs(want[t, a])
                    tol[t, a] = 2.0 ** -8 * np.abs(want[t, a]) + (2.0 ** -11 + off) * (1 + 2.0 ** -8) * size + 2.0 ** -126
    return tol


@pytest.mark.parametrize("side", SIDES)
@pytest.mark.parametrize("n_q,H,D", [(8, 2, 64), (4, 2, 128), (2, 2, 192), (4, 1, 256)])
@pytest.mark.parametrize("outlier", [30.0, 200.0, 5000.0])
def test_one_channel_of_q_far_above_the_rest(side, n_q, H, D, outlier):
    """The other channels of q still count with all their bits: the keys of the
    large channel differ little from token to token, so that the rest decides."""
    q_len, hint = SIDES[side]
    rng, q, codes, scales, table, cu, kv = make(int(outlier) + D, q_len, [500, 1100], n_q, H, D)
    assert_side(side, q, codes, q_len, kv, hint)
    index = ref.block_index(D)[0]
    q[:, :, 5] = outlier * np.sign(q[:, :, 5])
    q = bf16(q)
    # every page's keys of that channel: the same small value
    codes[:, :, 0, index[:, 5]] = 4
    scales[:, :, 0] = 2.0 ** -7
    scale = 0.5
    want, _ = ref.attention(q, codes, scales, table, cu, kv, scale)
    tol = attention_bound(q, codes, scales, table, cu, kv, scale, want)
    got = run(q, codes, scales, table, cu, kv, scale=scale, **hint).double().cpu().numpy()
    err = np.abs(got - want)
    assert np.all(err <= tol), f"{np.max(err / tol)} times the bound"


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("side", SIDES)
def test_a_window_past_everything_is_none(side, causal):
    """Up to the largest number, also for requests of more rows than tokens."""
    q_len, hint = SIDES[side]
    args = make(8, q_len, [2, 300], 4, 2, 64)[1:]
    assert_side(side, args[0], args[1], q_len, args[-1], hint)
    want = check(*args, causal=causal, **hint)
    for window in (2 ** 31 - 1, 2 ** 31, 2 ** 62, 2 ** 63 - 1):
        assert torch.equal(run(*args, causal=causal, window=window, **hint), want)


@pytest.mark.parametrize("n_q,H,D", [(8, 2, 64), (4, 2, 128), (2, 2, 192)])
@pytest.mark.parametrize("side", SIDES)
def test_hidden_pages_are_nobodys(side, n_q, H, D):
    """What the cache holds in pages that no request owns, NaN scales among
    them, does not reach a request with hidden pages."""
    q_len, hint = SIDES[side]
    rng, q, codes, scales, table, cu, kv = make(D, q_len, [300, 2100], n_q, H, D)
    assert_side(side, q, codes, q_len, kv, hint)
    table[0, 1], table[1, 3:5], table[1, -1] = -1, len(codes), -7
    want = check(q, codes, scales, table, cu, kv, **hint)
    free = np.setdiff1d(np.arange(len(codes)), table)
    if 0 not in free:   # page 0 and a free one change places
        other = free[0]
        codes[[0, other]], scales[[0, other]] = codes[[other, 0]], scales[[other, 0]]
        table[table == 0] = other
        free = np.setdiff1d(np.arange(len(codes)), table)
    assert 0 in free
    codes[free], scales[free] = -128, np.float32(np.nan)
    assert torch.equal(run(q, codes, scales, table, cu, kv, **hint), want)
