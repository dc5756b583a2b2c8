"""ht_kv_plan and ht_kv_release on the GPU against a plain host version:
every output equal, table entries of other pages untouched."""
import numpy as np
import pytest
import torch

import kv_reference as ref
from block_planner_amd import api

pytestmark = pytest.mark.gpu


def dev():
    return torch.device("cuda:0")


def ints(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=dev())


def make(rng, R, q, kv, width, spare, n_free=None, pad=0):
    owned = np.asarray([-(-int(k) // 64) for k in kv], np.int32)
    total = int(owned.sum()) + spare
    perm = rng.permutation(total).astype(np.int32)
    table = np.full((R, width + pad), -7, np.int32)
    at = 0
    for r in range(R):
        table[r, :owned[r]] = perm[at:at + owned[r]]
        at += owned[r]
    free = perm[at:] if spare else np.zeros(1, np.int32)
    return owned, table, free, (spare if n_free is None else n_free)


def check(q, kv, owned, table, free, n_free, T, width):
    want = ref.plan(q, kv, owned, table[:, :width], free, n_free, T)
    tg = ints(table)
    got = api.kv_plan(ints(q), ints(kv), ints(owned), tg[:, :width], ints(free), ints([n_free]), T)
    torch.cuda.synchronize()
    for name, g, w in zip(got._fields, got, want):
        np.testing.assert_array_equal(g.cpu().numpy(), w, err_msg=name)
    full = table.copy()
    full[:, :width] = want[6]
    np.testing.assert_array_equal(tg.cpu().numpy(), full, err_msg="table")
    return got


@pytest.mark.parametrize("R,mode", [(1, "decode"), (1, "prompt"), (7, "mixed"), (64, "decode"), (255, "mixed"),
                                    (1024, "decode"), (1025, "mixed"), (3000, "mixed")])
def test_plan_matches_host(R, mode):
    rng = np.random.default_rng(R)
    q = np.ones(R, int)
    if mode == "prompt":
        q[:] = 5000
    if mode == "mixed":
        q = np.where(rng.random(R) < 0.1, rng.integers(0, 700, R), rng.integers(0, 3, R))
    kv = rng.integers(0, 400, R)
    kv[rng.random(R) < 0.2] = 64 * rng.integers(0, 5)      # whole pages, and none
    width = int(max(-(-(a + b) // 64) for a, b in zip(q, kv))) + 1
    owned, table, free, n = make(rng, R, q, kv, width, int(q.sum()) // 64 + R + 5, pad=3)
    check(q, kv, owned, table, free, n, int(q.sum()), width)


def test_plan_refuses_requests_that_do_not_fit():
    """Pages run out in the middle; a request that needs none, and one past a
    request with too short a row, are still served."""
    rng = np.random.default_rng(3)
    q = np.array([64, 1, 300, 64, 1, 2, 640, 1])
    kv = np.array([0, 10, 0, 64, 5, 0, 0, 63])
    owned, table, free, n = make(rng, 8, q, kv, 6, 7)
    got = check(q, kv, owned, table, free, n, int(q.sum()), 6)
    assert int(got.status[1]) >= 2
    for n_free in (0, 1, 6, -5, 99):    # 99: more than the list holds
        check(q, kv, owned, table, free, n_free, int(q.sum()), 6)


def test_plan_empty_and_odd_lengths():
    rng = np.random.default_rng(4)
    q, kv = np.array([0, 0, 0]), np.array([0, 5, 64])
    owned, table, free, n = make(rng, 3, q, kv, 2, 4)
    check(q, kv, owned, table, free, n, 0, 2)
    check(q, kv, owned, table, free, n, 5, 2)            # more rows than the lengths say
    q = np.array([-3, 2, 70])                             # negative counts as zero
    check(q, kv, owned, table, free, n, 72, 4 - 1)
    check(q, kv, owned, table, free, n, 10, 3)            # fewer rows than the lengths say
    # a request that owns more pages than it fills (rewound)
    check(np.array([1, 1, 100]), np.array([0, 5, 20]), owned, table, free, n, 102, 3)


def test_plan_many_refused_pages_do_not_overflow():
    """Requests asking for 2^24 pages each: refused, no wrap of the sums."""
    R = 300
    q, kv = np.full(R, 1), np.full(R, 64 * ((1 << 24) - 2))
    owned = np.zeros(R, np.int32)
    q[0], kv[0] = 3, 0
    table = torch.full((R, 1), -1, dtype=torch.int32, device=dev())
    wide = table.as_strided((R, 1), (1, 1))
    got = api.kv_plan(ints(q), ints(kv), ints(owned), wide, ints([5, 6]), ints([2]), int(q.sum()))
    torch.cuda.synchronize()
    assert got.status.tolist() == [1, R - 1] and got.slots[:4].tolist() == [384, 385, 386, -1]


def test_steps_and_release_cycle():
    """Steps on the outputs of the step before, a release in between, and
    every page accounted for at the end."""
    rng = np.random.default_rng(5)
    R, P, pages = 6, 8, 30
    table = torch.full((R, P), -1, dtype=torch.int32, device=dev())
    free = ints(rng.permutation(pages))
    kv, owned, n_free = ints([0] * R), ints([0] * R), ints([pages])
    h = dict(kv=np.zeros(R, np.int32), own=np.zeros(R, np.int32), tab=table.cpu().numpy(), free=free.cpu().numpy(), n=pages)
    for step in range(12):
        q = rng.integers(0, 90, R)
        T = int(q.sum())
        want = ref.plan(q, h["kv"], h["own"], h["tab"], h["free"], h["n"], T)
        got = api.kv_plan(ints(q), kv, owned, table, free, n_free, T)
        for g, w in zip(got, want):
            np.testing.assert_array_equal(g.cpu().numpy(), w)
        kv, owned, n_free = got.kv_len, got.owned, got.status[:1].clone()
        h.update(kv=want[3].copy(), own=want[4].copy(), tab=want[6], n=int(want[5][0]))
        np.testing.assert_array_equal(table.cpu().numpy(), h["tab"])
        which = rng.random(R) < 0.3
        api.kv_release(torch.tensor(which, device=dev()), kv, owned, table, free, n_free)
        for r in np.flatnonzero(which):
            back = h["tab"][r, :h["own"][r]][::-1]
            h["free"][h["n"]:h["n"] + len(back)] = back
            h["n"] += len(back)
            h["own"][r] = h["kv"][r] = 0
        assert int(n_free) == h["n"]
        np.testing.assert_array_equal(free.cpu().numpy()[:h["n"]], h["free"][:h["n"]])
        np.testing.assert_array_equal(kv.cpu().numpy(), h["kv"])
        held = [p for r in range(R) for p in h["tab"][r, :h["own"][r]]]
        assert sorted(held + list(h["free"][:h["n"]])) == list(range(pages))


def test_release_many_requests():
    rng = np.random.default_rng(6)
    R = 700
    own = rng.integers(0, 4, R).astype(np.int32)
    table = np.arange(R * 4, dtype=np.int32).reshape(R, 4)
    which = (rng.random(R) < 0.5).astype(np.uint8)
    free, n = ints([-1] * 2000), ints([3])
    kv, owned = ints([9] * R), ints(own)
    api.kv_release(torch.tensor(which, device=dev()), kv, owned, ints(table), free, n)
    want = [p for r in np.flatnonzero(which) for p in table[r, :own[r]][::-1]]
    assert int(n) == 3 + len(want) and free[3:3 + len(want)].tolist() == want
    assert owned.tolist() == list(np.where(which, 0, own)) and kv.tolist() == list(np.where(which, 0, 9))
