"""Plain implementations, in 64 bits and on the host, of the cache operators:
page plan, norm and rotation of q and k, the 8-bit cache and attention over it.
Loops over requests, pages and rows; nothing shared with the library."""
import math

import numpy as np

PAGE, MIN_E = 64, -60


def plan(q_len, kv_len, owned, table, free, n_free, T):
    """The outputs of ht_kv_plan, and the table after it."""
    table = table.copy()
    R, P = table.shape
    q = [max(0, int(v)) for v in q_len]
    left, asked, at, refused = min(max(int(n_free), 0), len(free)), 0, 0, 0
    start = left
    cu, slots, pos, kv2, own2 = [0], [], [], [], []
    for r in range(R):
        kv, own = max(0, int(kv_len[r])), max(0, int(owned[r]))
        want = -(-(kv + q[r]) // PAGE)
        need = max(0, want - own) if want <= P else 0
        asked += need
        ok = want <= P and (need == 0 or asked <= start)
        if ok:
            for c in range(need):
                table[r, own + c] = free[start - 1 - at]
                at += 1
        refused += not ok
        kv2.append(kv + q[r] if ok else kv)
        own2.append(own + need if ok else own)
        for p in range(kv, kv + q[r]):
            pos.append(p)
            slots.append(int(table[r, p // PAGE]) * PAGE + p % PAGE if ok and table[r, p // PAGE] >= 0 else -1)
        cu.append(cu[-1] + q[r])
    slots = (slots + [-1] * T)[:T]
    pos = (pos + [0] * T)[:T]
    i32 = lambda a: np.asarray(a, np.int32)  # noqa: E731
    return i32(cu), i32(slots), i32(pos), i32(kv2), i32(own2), i32([start - at, refused]), table


def rotate(x, positions, inv_freq, interleaved, sign=1.0):
    """x [T, H, D] fp64, pairs rotated by sign * position * inv_freq."""
    half = len(inv_freq)
    y = x.copy()
    a = sign * positions.astype(np.float64)[:, None] * inv_freq[None]
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    i = np.arange(half)
    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    y[..., lo] = x[..., lo] * c - x[..., hi] * s
    y[..., hi] = x[..., hi] * c + x[..., lo] * s
    return y


def norm_rope(x, w, positions, inv_freq, eps, interleaved):
    x = x.astype(np.float64)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w.astype(np.float64)
    return rotate(x, positions, inv_freq, interleaved)


def norm_rope_backward(dy, x, w, positions, inv_freq, eps, interleaved):
    """(dx, dw)."""
    g = rotate(dy.astype(np.float64), positions, inv_freq, interleaved, -1.0)
    if w is None:
        return g, None
    x, w = x.astype(np.float64), w.astype(np.float64)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dw = (g * x * r).sum((0, 1))
    wg = g * w
    return r * wg - x * r ** 3 * (wg * x).sum(-1, keepdims=True) / x.shape[-1], dw


def block_index(D):
    """(K, V): byte of token t, dim d in a block, [64, D] each."""
    k, v = np.zeros((PAGE, D), int), np.zeros((PAGE, D), int)
    for t in range(PAGE):
        for d in range(D):
            k[t, d] = np.ravel_multi_index((t // 16, d // 64, d % 64 // 16, t % 16, d % 16), (4, D // 64, 4, 16, 16))
            v[t, d] = np.ravel_multi_index((d // 16, t % 16 // 4, d % 16, t // 16, t % 4), (D // 16, 4, 16, 4, 4))
    return k, v


def write(k, v, slots, codes, scales):
    """New (codes, scales) after ht_kv_write."""
    codes, scales = codes.copy(), scales.copy()
    index = block_index(k.shape[2])
    n_pages = codes.shape[0]
    pages = {}
    for t, s in enumerate(slots):
        if 0 <= s < n_pages * PAGE:
            pages.setdefault(int(s) // PAGE, []).append((t, int(s) % PAGE))
    for page, rows in pages.items():
        ts, at = [t for t, _ in rows], [o for _, o in rows]
        for kind, src in enumerate((k, v)):
            for h in range(codes.shape[1]):
                x = src[ts, h].astype(np.float64)
                top = np.abs(x[np.isfinite(x)]).max(initial=0.0)
                e = max(MIN_E, math.frexp(top)[1]) if top > 0 else MIN_E
                blk = codes[page, h, kind]
                if at[0] > 0:
                    m, old = math.frexp(float(scales[page, h, kind]))
                    old = max(MIN_E, old + 6) if m else MIN_E
                    e = max(e, old)
                    blk[:] = np.rint(np.ldexp(blk.astype(np.float64), old - e)).astype(np.int8)
                c = np.rint(np.ldexp(np.nan_to_num(x, nan=0.0, posinf=1e300, neginf=-1e300), 7 - e))
                blk[index[kind][at]] = np.clip(c, -127, 127).astype(np.int8)
                scales[page, h, kind] = math.ldexp(1.0, e - 7)
    return codes, scales


def attention(q, codes, scales, table, cu_q, kv_len, scale, causal=True, window=0):
    """(out, bound): the definition in 64 bits, [T, n_q, D], and what a result
    may be off by: half a bf16 step of the result, fp16 weights (half a step),
    q's 15-bit planes (2^-15 of the row's largest entry against sum |k|) and
    fp32 exponents and sums, each carried through the weighted mean."""
    T, n_q, D = q.shape
    n_pages, H = codes.shape[:2]
    group = n_q // H
    index = block_index(D)
    out, tol = np.zeros((T, n_q, D)), np.zeros((T, n_q, D))
    for r in range(len(kv_len)):
        kv = min(max(int(kv_len[r]), 0), table.shape[1] * PAGE)
        rows = range(max(int(cu_q[r]), 0), min(int(cu_q[r + 1]), T))
        pages = table[r, :-(-kv // PAGE)].astype(np.int64)
        there = np.repeat((pages >= 0) & (pages < n_pages), PAGE)[:kv]
        pages = np.where((pages >= 0) & (pages < n_pages), pages, 0)
        for h in range(H):
            k, v = ((codes[pages, h, i][:, index[i].reshape(-1)].astype(np.float64)
                     * scales[pages, h, i].astype(np.float64)[:, None]).reshape(-1, D)[:kv] for i in (0, 1))
            j = np.arange(kv)
            for i, t in enumerate(rows):
                pos = kv - len(rows) + i
                seen = there.copy()
                if causal:
                    seen &= j <= pos
                if window:
                    seen &= j > pos - window
                if not seen.any():
                    continue
                ks, vs = k[seen], v[seen]
                for a in range(h * group, (h + 1) * group):
                    x = q[t, a].astype(np.float64)
                    s = ks @ x * scale
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    out[t, a] = p @ vs
                    mean = p @ np.abs(vs)
                    off = abs(scale) * 2.0 ** -15 * np.abs(x).max() * np.abs(ks).sum(1).max()
                    off += 2.0 ** -24 * (64 + 4 * np.abs(s).max() + 4 * abs(scale) * (np.abs(ks) @ np.abs(x)).max())
                    tol[t, a] = 2.0 ** -8 * np.abs(out[t, a]) + (2.0 ** -11 + 2 * off) * (mean + np.abs(out[t, a])) + 2.0 ** -126
    return out, tol


def random_cache(rng, n_pages, H, D):
    """Codes and scales with pages of different magnitudes."""
    e = rng.integers(-2, 5, size=(n_pages, H, 2))
    codes = np.clip(np.rint(rng.normal(size=(n_pages, H, 2, PAGE * D)) * 32), -127, 127).astype(np.int8)
    return codes, np.ldexp(1.0, e - 7).astype(np.float32)


def random_table(rng, kv_len, n_pages, width=None):
    """Distinct pages per request, -1 past its last."""
    need = [-(-int(n) // PAGE) for n in kv_len]
    perm = rng.permutation(n_pages)[:sum(need)]
    table = np.full((len(need), width or max(1, max(need))), -1, np.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = perm[at:at + n]
        at += n
    return table
