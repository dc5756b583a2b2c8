"""ht_kv_write on the GPU against a plain host version: scaling by powers of
two is exact, so every code and scale has to be equal, those of untouched
pages and tokens too."""
import numpy as np
import pytest
import torch

import kv_reference as ref
from block_planner_amd import api

pytestmark = pytest.mark.gpu
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


def dev():
    return torch.device("cuda:0")


def slots_of(table, kv, q):
    return np.concatenate([table[r, np.arange(a, a + b) // 64] * 64 + np.arange(a, a + b) % 64
                           for r, (a, b) in enumerate(zip(kv, q))]).astype(np.int32)


def run(k, v, slots, codes, scales, kt="fp32", vt="fp32"):
    """Write, check against the host, write again (nothing may change)."""
    kt, vt = torch.from_numpy(k).to(TYPES[kt]), torch.from_numpy(v).to(TYPES[vt])
    cg, sg = torch.from_numpy(codes).to(dev()), torch.from_numpy(scales).to(dev())
    want = ref.write(kt.float().numpy(), vt.float().numpy(), slots, codes, scales)
    sl = torch.from_numpy(slots).to(dev())
    for _ in range(2):
        api.kv_write(kt.to(dev()), vt.to(dev()), sl, cg, sg)
        torch.cuda.synchronize()
        np.testing.assert_array_equal(sg.cpu().numpy(), want[1])
        np.testing.assert_array_equal(cg.cpu().numpy(), want[0])
    return want


@pytest.mark.parametrize("D,H", [(64, 1), (64, 4), (128, 8), (192, 2), (256, 3)])
@pytest.mark.parametrize("kv,q", [
    ([0], [1]), ([63], [1]), ([64], [1]), ([17], [3]), ([0], [64]), ([0], [65]), ([5], [200]),
    ([0, 10, 63, 64, 100], [1, 1, 1, 1, 1]), ([3, 60, 0], [8, 9, 7]), ([0, 1, 0, 30], [130, 1, 64, 70])])
def test_write_matches_host(D, H, kv, q):
    print(D, H, kv, q, flush=True)
    rng = np.random.default_rng(D + len(kv) + sum(q))
    total = [a + b for a, b in zip(kv, q)]
    n_pages = sum(-(-t // 64) for t in total) + 3
    codes, scales = ref.random_cache(rng, n_pages, H, D)
    slots = slots_of(ref.random_table(rng, total, n_pages), kv, q)
    k, v = (rng.normal(size=(sum(q), H, D)) * np.exp(rng.normal(size=(sum(q), H, 1))) for _ in range(2))
    run(k.astype(np.float32), v.astype(np.float32), slots, codes, scales, "bf16" if len(kv) % 2 else "fp32",
        "bf16" if H == 4 else "fp32")


def test_write_many_rows_and_padding():
    """2500 rows (fewer workgroups per window), rows without a slot between
    the requests and slots outside the cache."""
    rng = np.random.default_rng(8)
    kv, q = [0, 7, 64, 33, 0], [900, 1, 700, 1, 800]
    total = [a + b for a, b in zip(kv, q)]
    n_pages = sum(-(-t // 64) for t in total) + 1
    slots = slots_of(ref.random_table(rng, total, n_pages), kv, q)
    cut = [0, 900, 901, 1601, 1602, 2402]
    gap = np.array([-1, -1, n_pages * 64, 2 ** 31 - 1, -2 ** 31], np.int32)
    slots = np.concatenate([p for i in range(5) for p in (slots[cut[i]:cut[i + 1]], gap[:i + 1])] + [gap] * 17)
    codes, scales = ref.random_cache(rng, n_pages, 2, 64)
    k, v = (rng.normal(size=(len(slots), 2, 64)).astype(np.float32) for _ in range(2))
    run(k, v, slots, codes, scales, "bf16", "fp32")


def test_write_odd_values():
    """Zeros, subnormals, the largest and smallest magnitudes, infinities and
    NaN, values at rounding ties and next to a power of two."""
    rng = np.random.default_rng(9)
    n, D = 40, 64
    k = rng.normal(size=(n, 1, D)).astype(np.float32)
    v = k.copy()
    k[:8] = 0
    k[8] = 1e-42
    v[:] = np.float32(3.4e38) * rng.choice([-1, 1, 0.5], size=v.shape).astype(np.float32)
    codes, scales = ref.random_cache(rng, 4, 1, D)
    scales[:] = 0                                       # never written
    run(k[:9], v[:9], np.arange(64, 73, dtype=np.int32), codes, scales)
    x = np.full((n, 1, D), 1.0, np.float32)
    x[0, 0] = np.arange(D) / 128.0 + 1 / 256.0          # ties
    x[1, 0, :4] = [np.inf, -np.inf, np.nan, -0.0]
    x[2, 0] = np.nextafter(np.float32(2), np.float32(0))   # rounds to 128, clamped
    run(x, -x, np.arange(n, dtype=np.int32) + 3, codes, scales)
    bad = np.full((2, 1, D), np.nan, np.float32)
    bad[1] = np.inf
    run(bad, -bad, np.array([0, 1], np.int32), codes, scales)


def test_appending_keeps_entries_within_a_step():
    """Token by token with growing magnitudes: every entry stays within one
    step of the page's final scale (and the codes equal the host's)."""
    rng = np.random.default_rng(10)
    D, n = 128, 64
    k = (rng.normal(size=(n, 2, D)) * np.exp2(np.arange(n) / 8.0)[:, None, None]).astype(np.float32)
    v = rng.normal(size=(n, 2, D)).astype(np.float32)
    codes, scales = ref.random_cache(rng, 2, 2, D)
    cg, sg = torch.from_numpy(codes).to(dev()), torch.from_numpy(scales).to(dev())
    for t in range(n):
        api.kv_write(torch.from_numpy(k[t:t + 1]).to(dev()), torch.from_numpy(v[t:t + 1]).to(dev()),
                     torch.tensor([64 + t], dtype=torch.int32, device=dev()), cg, sg)
        codes, scales = ref.write(k[t:t + 1], v[t:t + 1], [64 + t], codes, scales)
    np.testing.assert_array_equal(cg.cpu().numpy(), codes)
    np.testing.assert_array_equal(sg.cpu().numpy(), scales)
    kk, vv = api.kv_cache_values(cg, sg)
    for got, want, i in ((kk, k, 0), (vv, v, 1)):
        step = scales[1, :, i][None, :, None]
        assert np.all(np.abs(got[1].permute(1, 0, 2).cpu().numpy() - want) <= step)


def test_strides():
    """v as a part of wider rows, k with rows inside heads, a misaligned one."""
    rng = np.random.default_rng(11)
    T, H, D = 70, 2, 64
    codes, scales = ref.random_cache(rng, 3, H, D)
    x = rng.normal(size=(T, 3 * H, D)).astype(np.float32)
    slots = np.arange(64, 64 + T, dtype=np.int32)
    want = ref.write(x[:, :H], x[:, 2 * H:], slots, codes, scales)
    g = torch.from_numpy(x).to(dev())
    for k in (g[:, :H], g[:, :H].transpose(0, 1).contiguous().transpose(0, 1),
              torch.empty(T * H * D + 1, device=dev())[1:].view(T, H, D).copy_(g[:, :H])):
        cg, sg = torch.from_numpy(codes).to(dev()), torch.from_numpy(scales).to(dev())
        api.kv_write(k, g[:, 2 * H:], torch.from_numpy(slots).to(dev()), cg, sg)
        np.testing.assert_array_equal(cg.cpu().numpy(), want[0])
        np.testing.assert_array_equal(sg.cpu().numpy(), want[1])
    api.kv_write(g[:0, :H], g[:0, :H], torch.from_numpy(slots[:0]).to(dev()), cg, sg)
