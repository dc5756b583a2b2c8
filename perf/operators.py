"""Operators between the q|k|v linear and the output linear of a transformer layer, as measured cases.

Four operators share one paged cache of keys and values held in 8 bits:

  plan     page tables, slots and positions of one serving step from the requests' lengths
  rope     norms of q and k per head with the position rotation, forward and backward
  write    keys and values quantised into the cache, one scale per page of 64 tokens, head and K or V
  attend   attention of a batch's query rows over the cache

``run`` computes them with elementary torch operations, or, where ``own`` is
true, by the calls of ``block_planner_amd.api``.  Head layouts are those of
the framework's transformer stacks (32 heads x 64 with 4 KV heads; 32 heads
x 128 with 8 KV heads) or generic.

The cache, as ``include/ht.h`` lays it out: ``codes`` int8 [pages, heads, 2, 64 * D] and ``scales`` fp32
[pages, heads, 2] (index 0: K, 1: V).  A K code of token t = 16 a + r, dim d = 64 c + 16 g + b is at
[a, c, g, r, b] of (4, D/64, 4, 16, 16); a V code of token t = 16 b + 4 g + i, dim d = 16 e + m is at
[e, g, m, b, i] of (D/16, 4, 16, 4, 4).  Codes are whole numbers and the scales powers of two, so every
code is the rounding of an exactly scaled input: ``write`` returns the codes themselves, which have to be
equal, with the scales that give their values.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 64
EPS = 1e-6
MIN_E = -60   # smallest exponent of a page's largest magnitude


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # A serving step of 8 requests that decode one token each: latency only.
        dict(name="plan decode 8", op="plan", requests=8, q_min=1, q_max=1, kv_min=1, kv_max=4096, lens=1),
        # A mixed step: most of 512 requests decode, every eighth brings a chunk of its prompt.
        dict(name="plan mixed 512", op="plan", requests=512, q_min=1, q_max=1, chunk=1024, kv_min=0, kv_max=32768,
             lens=2),
        # One token of a 32 x 128 layer, fp32 as the q|k|v linear gives it.
        dict(name="rope decode 1", op="rope", tokens=1, heads=32, kv_heads=8, dim=128, rot=128, x="fp32", y="bf16",
             norm=True, interleaved=False, backward=False, far=131072),
        # A prompt of a 32 x 64 layer without norms.
        dict(name="rope prefill 8191", op="rope", tokens=8191, heads=32, kv_heads=4, dim=64, rot=64, x="fp32",
             y="bf16", norm=False, interleaved=False, backward=False, far=32768),
        # The backward pass of a training batch of 4 x 2048 tokens.
        dict(name="rope backward 8192", op="rope", tokens=8192, heads=32, kv_heads=8, dim=128, rot=128, x="fp32",
             y="fp32", norm=True, interleaved=False, backward=True, far=2048),
        # 64 requests append one token each.
        dict(name="write decode 64", op="write", requests=64, q_min=1, q_max=1, kv_min=0, kv_max=200, kv_heads=8,
             dim=128, k="bf16", v="fp32", lens=3),
        # Prompts of 4 requests, two of which continue inside a page.
        dict(name="write prefill 4", op="write", requests=4, q_min=2000, q_max=4000, kv_min=0, kv_max=100, kv_heads=8,
             dim=128, k="bf16", v="fp32", lens=4),
        # One request of the 32 x 64 layer early in its answer.
        dict(name="attend decode 1", op="attend", requests=1, q_min=1, q_max=1, kv_min=900, kv_max=1100, heads=32,
             kv_heads=4, dim=64, window=0, lens=5),
        # An ordinary batch of answers of ragged lengths.
        dict(name="attend decode 64", op="attend", requests=64, q_min=1, q_max=1, kv_min=100, kv_max=8192, heads=32,
             kv_heads=8, dim=128, window=0, lens=6),
        # Few requests with long contexts, three drafted tokens each.
        dict(name="attend decode long 3", op="attend", requests=3, q_min=3, q_max=3, kv_min=100000, kv_max=131072,
             heads=32, kv_heads=8, dim=128, window=0, lens=7),
        # One long prompt from the start.
        dict(name="attend prefill 8192", op="attend", requests=1, q_min=8192, q_max=8192, kv_min=8192, kv_max=8192,
             heads=32, kv_heads=8, dim=128, window=0, lens=8),
        # Chunks of prompts over what is in the cache, with a sliding window.
        dict(name="attend chunks 6", op="attend", requests=6, q_min=100, q_max=700, kv_min=1000, kv_max=12000,
             heads=32, kv_heads=4, dim=64, window=4096, lens=9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "rope", "rope", "write", "attend", "attend", "attend"])
    seed = rng.randrange(1 << 30)
    heads, kv_heads = rng.choice([(32, 8), (32, 4), (16, 16), (40, 8), (28, 4), (12, 2), (8, 1)])
    if op == "plan":
        n = _log(rng, 1, 1024)
        return dict(op=op, requests=n, q_min=1, q_max=rng.choice([1, 1, 4]), chunk=rng.choice([0, _log(rng, 2, 1500)]),
                    kv_min=0, kv_max=_log(rng, 64, 32768), lens=seed)
    if op == "rope":
        dim = rng.choice([64, 64, 80, 96, 128, 128, 256])
        return dict(op=op, tokens=_log(rng, 1, 8192), heads=heads, kv_heads=kv_heads, dim=dim,
                    rot=rng.choice([dim, dim, dim // 2]), x=rng.choice(["fp32", "bf16"]), y=rng.choice(["fp32", "bf16"]),
                    norm=rng.random() < 0.7, interleaved=rng.random() < 0.3, backward=rng.random() < 0.4,
                    far=_log(rng, 100, 1000000))
    dim = rng.choice([64, 128, 128, 256])
    if op == "write":
        one = rng.random() < 0.5
        n = _log(rng, 1, 512 if one else 16)
        q = (1, rng.choice([1, 3])) if one else (1, _log(rng, 16, 8192 // n))
        return dict(op=op, requests=n, q_min=q[0], q_max=q[1], kv_min=0, kv_max=_log(rng, 10, 1000), kv_heads=kv_heads,
                    dim=dim, k=rng.choice(["fp32", "bf16"]), v=rng.choice(["fp32", "bf16"]), lens=seed)
    window = rng.choice([0, 0, 0, _log(rng, 64, 8192)])
    if rng.random() < 0.6:   # answers
        n = _log(rng, 1, 128)
        far = _log(rng, 64, min(131072, 2 ** 28 // (n * kv_heads * dim)))
        return dict(op=op, requests=n, q_min=1, q_max=rng.choice([1, 1, 2, 4]), kv_min=rng.choice([4, far]), kv_max=far,
                    heads=heads, kv_heads=kv_heads, dim=dim, window=window, lens=seed)
    n = _log(rng, 1, 8)
    q = _log(rng, 16, 4096 // n)
    return dict(op=op, requests=n, q_min=max(1, q // 4), q_max=q, kv_min=q, kv_max=_log(rng, q, 8192), heads=heads,
                kv_heads=kv_heads, dim=dim, window=window, lens=seed)


def _lengths(case):
    """(q, kv): new rows of each request and, for plan and write, its tokens in the cache before the step; for
    attend with the new ones."""
    r = random.Random("%(op)s %(lens)d" % case)
    n, chunk = case["requests"], case.get("chunk", 0)
    q = [r.randint(case["q_min"], case["q_max"]) for _ in range(n)]
    if chunk:
        q = [r.randint(2, chunk) if i % 8 == 3 else v for i, v in enumerate(q)]
    lo, hi = case["kv_min"], case["kv_max"]
    kv = [int(round(math.exp(r.uniform(math.log(lo + 1), math.log(hi + 1))))) - 1 for _ in range(n)]
    if case["op"] == "attend":
        kv = [max(a, b) for a, b in zip(q, kv)]
    return q, kv


def _ceil(a, b):
    return -(-a // b)


def work(case):
    op = case["op"]
    if op == "plan":
        q, kv = _lengths(case)
        new = sum(max(0, _ceil(a + b, PAGE) - _ceil(b, PAGE)) for a, b in zip(q, kv))
        return {"bytes": 4 * (3 * len(q) + 2 * new + 3 * len(q) + 2 * sum(q)), "flops": 0}
    size = {"fp32": 4, "bf16": 2}
    if op == "rope":
        n = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        x, y = size[case["x"]], size[case["y"]]
        # backward without norms is the rotation of the gradient alone
        per = y + x + (x if case["norm"] else 0) if case["backward"] else x + y
        return {"bytes": n * per + 4 * case["tokens"], "flops": n * (16 if case["backward"] else 8)}
    q, kv = _lengths(case)
    if op == "write":
        n = sum(q) * case["kv_heads"] * case["dim"]
        pages = sum(_ceil(a + b, PAGE) - b // PAGE for a, b in zip(q, kv))
        return {"bytes": n * (size[case["k"]] + size[case["v"]] + 2) + 4 * sum(q) + 8 * pages * case["kv_heads"],
                "flops": 4 * n}
    pairs = tokens = 0
    for a, b in zip(q, kv):
        pos = np.arange(b - a, b)
        first = np.maximum(0, pos + 1 - case["window"]) if case["window"] else np.zeros_like(pos)
        pairs += int((pos + 1 - first).sum())
        tokens += b - int(first[0])
    d, h = case["dim"], case["kv_heads"]
    return {"bytes": 4 * sum(q) * case["heads"] * d + tokens * h * 2 * d + 8 * _ceil(tokens, PAGE) * h,
            "flops": 4 * pairs * case["heads"] * d}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _dtype(name):
    return {"fp32": torch.float32, "bf16": torch.bfloat16}[name]


def _ints(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def _cache(g, pages, heads, dim):
    """Codes and scales of normal keys and values whose pages differ in magnitude."""
    e = torch.randint(1, 4, (pages, heads, 2), generator=g, device="cuda")
    codes = torch.empty(pages, heads, 2, PAGE * dim, dtype=torch.int8, device="cuda")
    step = max(1, (1 << 28) // (heads * 2 * PAGE * dim))
    for i in range(0, pages, step):
        x = torch.randn(codes[i:i + step].shape, generator=g, device="cuda")
        x *= torch.exp2(7.0 - e[i:i + step].float())[..., None]
        codes[i:i + step] = x.round_().clamp_(-127, 127).to(torch.int8)
    return codes, torch.exp2(e.float() - 7.0)


def _table(g, need, width, spare):
    """Random distinct pages for every request, -1 past what it owns, and the pages that are left."""
    free = torch.randperm(sum(need) + spare, generator=g, device="cuda").cpu().numpy().astype(np.int32)
    table, at = np.full((len(need), width), -1, np.int32), 0
    for r, n in enumerate(need):
        table[r, :n] = free[at:at + n]
        at += n
    return table, free[at:]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    s, op = dict(case), case["op"]
    if op == "rope":
        t, h, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        x, y = _dtype(case["x"]), _dtype(case["y"])
        qkv = rand(t, (h + 2 * hk) * d).mul_(1.5).to(x)       # rows of the fused q|k|v linear
        s["q"] = qkv[:, :h * d].view(t, h, d)
        s["k"] = qkv[:, h * d:(h + hk) * d].view(t, hk, d)
        s["positions"] = torch.randint(0, case["far"], (t,), generator=g, device="cuda", dtype=torch.int32)
        i = torch.arange(case["rot"] // 2, dtype=torch.float64, device="cuda")
        s["inv_freq"] = 500000.0 ** (-2.0 * i / case["rot"])
        s["wq"] = 1 + 0.2 * rand(d) if case["norm"] else None
        s["wk"] = 1 + 0.2 * rand(d) if case["norm"] else None
        if case["backward"]:
            s["dq"], s["dk"] = rand(t, h, d).to(y), rand(t, hk, d).to(y)
        return s
    q, kv = _lengths(case)
    n = len(q)
    cu = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
    if op == "plan":
        owned = [_ceil(b, PAGE) for b in kv]
        width = max(_ceil(a + b, PAGE) for a, b in zip(q, kv)) + 2
        new = sum(_ceil(a + b, PAGE) - o for a, b, o in zip(q, kv, owned))
        table, free = _table(g, owned, width, new + 16)
        s.update(q_len=_ints(q), kv_len=_ints(kv), owned=_ints(owned), table=_ints(table), free=_ints(free),
                 n_free=_ints([len(free)]), T=int(cu[-1]))
        s["out"] = tuple(torch.empty(m, dtype=torch.int32, device="cuda") for m in (n + 1, s["T"], s["T"], n, n, 2))
        return s
    s["T"], s["max_q"] = int(cu[-1]), max(q)
    if op == "write":
        need = [_ceil(a + b, PAGE) for a, b in zip(q, kv)]
        table, _ = _table(g, need, max(need), 3)
        pos = np.concatenate([np.arange(b, a + b) for a, b in zip(q, kv)])
        row = np.repeat(np.arange(n), q)
        s["slots"] = _ints(table[row, pos // PAGE] * PAGE + pos % PAGE)
        s["codes"], s["scales"] = _cache(g, sum(need) + 3, case["kv_heads"], case["dim"])
        s["k"] = rand(s["T"], case["kv_heads"], case["dim"]).to(_dtype(case["k"]))
        qkv = rand(s["T"], 3, case["kv_heads"], case["dim"]).to(_dtype(case["v"]))
        s["v"] = qkv[:, 2]                                    # a part of wider rows
        return s
    need = [_ceil(b, PAGE) for b in kv]
    table, _ = _table(g, need, max(need) + 1, 3)
    s["codes"], s["scales"] = _cache(g, sum(need) + 3, case["kv_heads"], case["dim"])
    s["q"] = rand(s["T"], case["heads"], case["dim"]).to(torch.bfloat16)
    s.update(table=_ints(table), cu_q=_ints(cu), kv_len=_ints(kv), max_kv=max(kv))
    s["out"] = torch.empty_like(s["q"])
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["op"]
    if own:
        from block_planner_amd import api

        if op == "plan":
            api.kv_plan(s["q_len"], s["kv_len"], s["owned"], s["table"], s["free"], s["n_free"], s["T"], out=s["out"])
            return (*s["out"], s["table"])
        if op == "rope":
            if s["backward"]:
                return api.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["positions"], s["inv_freq"],
                                                 q_weight=s["wq"], k_weight=s["wk"], eps=EPS,
                                                 interleaved=s["interleaved"])
            return api.qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], q_weight=s["wq"], k_weight=s["wk"],
                                    eps=EPS, interleaved=s["interleaved"], out_dtype=_dtype(s["y"]))
        if op == "write":
            api.kv_write(s["k"], s["v"], s["slots"], s["codes"], s["scales"])
            return s["codes"], s["scales"]
        return api.kv_attention(s["q"], s["codes"], s["scales"], s["table"], s["cu_q"], s["kv_len"], s["max_q"],
                                max_kv=s["max_kv"], window=s["window"], out=s["out"])
    if op == "plan":
        return _plan(s)
    if op == "rope":
        return _rope_backward(s) if s["backward"] else _rope(s)
    return _write(s) if op == "write" else _attend(s)


def _plan(s):
    q, kv, owned, table, free, n_free = (s[k] for k in ("q_len", "kv_len", "owned", "table", "free", "n_free"))
    pages = (kv + q + PAGE - 1) // PAGE
    wide = pages > table.shape[1]
    need = torch.where(wide, 0, (pages - owned).clamp(min=0))
    upto = torch.cumsum(need, 0, dtype=torch.int32)
    served = ~wide & ((need == 0) | (upto <= n_free))
    given = torch.where(served, need, 0)
    i = torch.arange(table.shape[1], device="cuda")[None] - owned[:, None]
    at = n_free - 1 - ((upto - need)[:, None] + i)
    table = torch.where((i >= 0) & (i < given[:, None]), free[at.clamp(0, free.shape[0] - 1)], table)
    cu = torch.nn.functional.pad(torch.cumsum(q, 0, dtype=torch.int32), (1, 0))
    t = torch.arange(s["T"], device="cuda", dtype=torch.int32)
    r = torch.searchsorted(cu[1:], t, right=True)
    pos = kv[r] + t - cu[r]
    slots = torch.where(served[r], table[r, (pos // PAGE).clamp(max=table.shape[1] - 1)] * PAGE + pos % PAGE, -1)
    status = torch.stack([n_free[0] - given.sum(dtype=torch.int32), (~served).sum(dtype=torch.int32)])
    return cu, slots, pos, torch.where(served, kv + q, kv), owned + given, status, table


def _angles(s):
    a = s["positions"].double()[:, None] * s["inv_freq"][None]
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _turn(x, cos, sin, interleaved):
    """The first 2 * cos.shape[-1] dims rotated by pairs: (i, i + half), or (2i, 2i + 1) where interleaved."""
    half = cos.shape[-1]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1 if interleaved else -2).flatten(-2)
    return torch.cat([y, x[..., 2 * half:]], -1)


def _rope(s):
    cos, sin = _angles(s)

    def one(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
        return _turn(x, cos, sin, s["interleaved"]).to(_dtype(s["y"]))

    return one(s["q"], s["wq"]), one(s["k"], s["wk"])


def _rope_backward(s):
    cos, sin = _angles(s)

    def one(dy, x, w):
        g = _turn(dy.float(), cos, -sin, s["interleaved"])
        if w is None:
            return g.to(x.dtype), None
        x, t = x.float(), x.dtype
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        n = x * r
        dw = (g * n).sum((0, 1), dtype=torch.float64).float()
        g = g * w
        return (r * (g - n * (g * n).mean(-1, keepdim=True))).to(t), dw

    (dq, dwq), (dk, dwk) = one(s["dq"], s["q"], s["wq"]), one(s["dk"], s["k"], s["wk"])
    return dq, dk, dwq, dwk


def _write(s):
    slots = s["slots"].long()
    page, at = slots // PAGE, slots % PAGE
    codes, scales = s["codes"], s["scales"]
    pages, heads = codes.shape[:2]
    dim = s["dim"]
    x = torch.stack([s["k"].float(), s["v"].float()], 2)                              # [T, heads, 2, D]
    top = torch.where(x.isfinite(), x.abs(), 0.0).amax(-1)
    index = page[:, None, None].expand(-1, heads, 2)
    top = torch.zeros(pages, heads, 2, device="cuda").scatter_reduce_(0, index, top, "amax")
    first = torch.full((pages,), PAGE, device="cuda").scatter_reduce_(0, page, at, "amin")[:, None, None]
    e_new = torch.where(top > 0, torch.frexp(top)[1], MIN_E).clamp(min=MIN_E)
    e_old = torch.frexp(scales)[1] + 6
    e = torch.where(first >= PAGE, e_old, torch.where(first == 0, e_new, torch.maximum(e_old, e_new)))
    down = torch.where((first > 0) & (first < PAGE), e_old - e, 0)
    codes.copy_((codes.float() * torch.exp2(down.float())[..., None]).round())
    x = torch.ldexp(x, (7 - e)[page][..., None]).nan_to_num(nan=0.0, posinf=127.0, neginf=-127.0)
    x = x.round().clamp(-127, 127).to(torch.int8)
    k = codes[:, :, 0].view(pages, heads, 4, dim // 64, 4, 16, 16).permute(0, 2, 5, 1, 3, 4, 6)
    k[page, at // 16, at % 16] = x[:, :, 0].view(-1, heads, dim // 64, 4, 16)
    v = codes[:, :, 1].view(pages, heads, dim // 16, 4, 16, 4, 4).permute(0, 5, 3, 6, 1, 2, 4)
    v[page, at // 16, at % 16 // 4, at % 4] = x[:, :, 1].view(-1, heads, dim // 16, 16)
    scales.copy_(torch.exp2((e - 7).float()))
    return codes, scales


def _attend(s):
    d, heads, hk = s["dim"], s["heads"], s["kv_heads"]
    group, pages = heads // hk, (s["max_kv"] + PAGE - 1) // PAGE
    table, cu, kv = s["table"][:, :pages].clamp(min=0).long(), s["cu_q"], s["kv_len"]
    n = table.shape[0]
    scales = s["scales"][table][..., None, None]                                      # [R, P, heads, 2, 1, 1]
    k = s["codes"][:, :, 0][table].view(n, pages, hk, 4, d // 64, 4, 16, 16).permute(0, 2, 1, 3, 6, 4, 5, 7)
    k = k.reshape(n, hk, pages, PAGE, d).float() * scales[:, :, :, 0].transpose(1, 2)
    v = s["codes"][:, :, 1][table].view(n, pages, hk, d // 16, 4, 16, 4, 4).permute(0, 2, 1, 6, 4, 7, 3, 5)
    v = v.reshape(n, hk, pages, PAGE, d).float() * scales[:, :, :, 1].transpose(1, 2)
    k, v = k.view(n * hk, -1, d), v.view(n * hk, -1, d)
    # rows of every request, padded to the longest
    i = torch.arange(s["max_q"], device="cuda")[None]
    count = (cu[1:] - cu[:-1])[:, None]
    row = torch.where(i < count, cu[:-1, None] + i, s["T"])                           # [R, max_q]
    q = torch.cat([s["q"], s["q"].new_zeros(1, heads, d)])[row].float() / math.sqrt(d)
    q = q.view(n, -1, hk, group, d).transpose(1, 2).reshape(n * hk, -1, d)
    p = torch.bmm(q, k.transpose(1, 2)).view(n, hk, s["max_q"], group, -1)
    pos = (kv[:, None] - count + i)[:, :, None]
    j = torch.arange(pages * PAGE, device="cuda")[None, None]
    seen = (j <= pos) & (j < kv[:, None, None])
    if s["window"]:
        seen &= j > pos - s["window"]
    seen = seen[:, None, :, None]
    p = p.masked_fill_(~seen, -math.inf)
    top = p.amax(-1, keepdim=True).clamp(min=-3e38)
    p = p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.bmm(p.view(n * hk, s["max_q"] * group, -1), v).view(n, hk, -1, group, d) / total.clamp(min=1e-30)
    o = o.transpose(1, 2).reshape(-1, heads, d)
    out = torch.empty(s["T"] + 1, heads, d, device="cuda")
    out[row.view(-1)] = o
    return out[:-1].to(torch.bfloat16)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    return {"plan": _exact_plan, "rope": _exact_rope, "write": _exact_write, "attend": _exact_attend}[op](s)


def _exact_plan(s):
    q, kv, owned, table, free = (s[k].cpu().numpy().astype(np.int64) for k in ("q_len", "kv_len", "owned", "table", "free"))
    left, refused, asked = int(s["n_free"]), 0, 0
    stack, slots, places = list(free[:left]), [], []
    kv2, owned2 = kv.copy(), owned.copy()
    for r in range(len(q)):
        pages = -(-(kv[r] + q[r]) // PAGE)
        need = max(0, pages - owned[r]) if pages <= table.shape[1] else 0
        asked += need
        ok = pages <= table.shape[1] and (need == 0 or asked <= left)
        for c in range(need if ok else 0):
            table[r, owned[r] + c] = stack.pop()
        refused += not ok
        kv2[r] += q[r] if ok else 0
        owned2[r] += need if ok else 0
        for p in range(kv[r], kv[r] + q[r]):
            places.append(p)
            slots.append(table[r, p // PAGE] * PAGE + p % PAGE if ok else -1)
    cu = np.concatenate([[0], np.cumsum(q)])
    return [np.asarray(a, np.int32) for a in (cu, slots, places, kv2, owned2, [len(stack), refused], table)]


def _exact_rope(s):
    """Rotation as multiplication by exp(i angle) of the pairs taken as complex numbers, everything in float64."""
    half = s["rot"] // 2
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       torch.outer(s["positions"].double(), s["inv_freq"]))[:, None]

    def rotate(x, by):
        first = x[..., :2 * half].unflatten(-1, (half, 2) if s["interleaved"] else (2, half))
        first = first if s["interleaved"] else first.transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(first.contiguous()) * by)
        return torch.cat([(z if s["interleaved"] else z.transpose(-1, -2)).flatten(-2), x[..., 2 * half:]], -1)

    def inverse_norm(x):
        return 1 / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS)

    out, dws = [], []
    for name in ("q", "k"):
        x, w = s[name].double(), s["w" + name]
        if not s["backward"]:
            out.append(rotate(x if w is None else x * inverse_norm(x) * w.double(), turn))
            continue
        g = rotate(s["d" + name].double(), turn.conj())
        if w is None:
            out.append(g)
            dws.append(None)
            continue
        r = inverse_norm(x)
        dws.append((g * x * r).sum((0, 1)))
        g = g * w.double()
        out.append(r * g - x * r ** 3 * (g * x).sum(-1, keepdim=True) / x.shape[-1])
    return tuple(out + dws)


def _exact_write(s):
    """Page by page on the host: codes are whole numbers, scales powers of two."""
    codes, scales, slots = s["codes"].cpu().numpy(), s["scales"].double().cpu().numpy(), s["slots"].cpu().numpy()
    dim = s["dim"]
    t, d = np.meshgrid(np.arange(PAGE), np.arange(dim), indexing="ij")
    where = [(((t // 16 * (dim // 64) + d // 64) * 4 + d % 64 // 16) * 16 + t % 16) * 16 + d % 16,
             (((d // 16 * 4 + t % 16 // 4) * 16 + d % 16) * 4 + t // 16) * 4 + t % 4]
    for page in np.unique(slots // PAGE):
        rows = np.flatnonzero(slots // PAGE == page)
        at = slots[rows] % PAGE
        for kind, name in enumerate(("k", "v")):
            x = s[name][torch.from_numpy(rows).cuda()].double().cpu().numpy()         # [n, heads, D]
            for h in range(codes.shape[1]):
                top = np.abs(x[:, h]).max()
                e = max(MIN_E, math.frexp(top)[1]) if top else MIN_E
                if at[0]:
                    old = int(round(math.log2(scales[page, h, kind]))) + 7
                    e = max(e, old)
                    codes[page, h, kind] = np.rint(np.ldexp(codes[page, h, kind].astype(np.float64), old - e))
                codes[page, h, kind][where[kind][at]] = np.clip(np.rint(np.ldexp(x[:, h], 7 - e)), -127, 127)
                scales[page, h, kind] = math.ldexp(1.0, e - 7)
    return codes, scales


def _exact_attend(s):
    d, group = s["dim"], s["heads"] // s["kv_heads"]
    cu, kv, table = s["cu_q"].tolist(), s["kv_len"].tolist(), s["table"].long()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    t, c = torch.meshgrid(torch.arange(PAGE, device="cuda"), torch.arange(d, device="cuda"), indexing="ij")
    place = [(((t // 16 * (d // 64) + c // 64) * 4 + c % 64 // 16) * 16 + t % 16) * 16 + c % 16,
             (((c // 16 * 4 + t % 16 // 4) * 16 + c % 16) * 4 + t // 16) * 4 + t % 4]
    for r in range(len(kv)):
        pages = table[r, :_ceil(kv[r], PAGE)]
        pos = torch.arange(kv[r] - cu[r + 1] + cu[r], kv[r], device="cuda")
        j = torch.arange(kv[r], device="cuda")
        bad = j[None] > pos[:, None]
        if s["window"]:
            bad |= pos[:, None] - j[None] >= s["window"]
        for h in range(s["kv_heads"]):
            kh, vh = ((s["codes"][pages, h, i][:, place[i].view(-1)].double() * s["scales"][pages, h, i, None].double())
                      .view(-1, d)[:kv[r]] for i in (0, 1))
            for a in range(h * group, (h + 1) * group):
                x = s["q"][cu[r]:cu[r + 1], a].double() @ kh.t() / math.sqrt(d)
                x = torch.where(bad, -math.inf, x)
                out[cu[r]:cu[r + 1], a] = torch.softmax(x, -1) @ vh
    return out
