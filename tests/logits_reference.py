"""Plain implementations, in 64 bits and on the host, of the norm with the
residual's addition, the 8-bit rows, token log probabilities and distillation
from a teacher's top logits.  Loops over rows; nothing shared with the library."""
import math

import numpy as np
import torch

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
HALF = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8}     # half a step, relative


def rounded(a, dtype):
    """fp64 -> the nearest values of the type, as fp64 (through fp32 for bf16:
    sums of two such values are exact in fp64, so one rounding is meant)."""
    if dtype == "fp32":
        return a.astype(np.float32).astype(np.float64)
    b = np.ascontiguousarray(a, np.float64)
    m, e = np.frexp(b)
    return np.ldexp(np.rint(m * 256.0), e - 8)


def norm(h, w, eps):
    return h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * w


def norm_backward(dy, h, w, dh, eps):
    """(d, dw)."""
    r = 1 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    g = dy * w
    d = r * g - h * r ** 3 * (g * h).sum(-1, keepdims=True) / h.shape[-1]
    return d + (0 if dh is None else dh), (dy * h * r).sum(0)


def q8_index(M, K):
    """Byte of row m, column k in the codes; the scale's place."""
    m, k = np.meshgrid(np.arange(M), np.arange(K), indexing="ij")
    kb, e = k // 64, k % 64
    codes = ((m // 16 * (K // 64) + kb) * 64 + m % 16 + 16 * (e // 16)) * 16 + e % 16
    return codes, kb * (16 * -(-M // 16)) + m


def q8_encode(y):
    """(codes [M, K], scales [M, K / 64]) of fp64 or fp32 values."""
    M, K = y.shape
    codes, scales = np.zeros((M, K)), np.ones((M, K // 64))
    for m in range(M):
        for b in range(K // 64):
            v = y[m, 64 * b:64 * b + 64].astype(np.float64)
            if not np.all(np.isfinite(v)):
                scales[m, b] = np.nan
                continue
            top = np.abs(v).max()
            if top == 0:
                continue
            e = max(math.frexp(top)[1], -119)
            scales[m, b] = 2.0 ** (e - 7)
            codes[m, 64 * b:64 * b + 64] = np.clip(np.rint(v / 2.0 ** (e - 7)), -127, 127)
    return codes, scales


# -- rows of logits -----------------------------------------------------------
def row_logp(x, temperature):
    """log softmax of one row (fp64); None: nothing is allowed."""
    z = x / temperature
    top = z.max()
    if top == -np.inf:
        return None
    with np.errstate(over="ignore"):
        d = z - top
    return d - np.log(np.exp(d).sum())


def top_of(x, k):
    """Indices of the k largest, equal ones in order."""
    return np.argsort(-(x + 0.0), kind="stable")[:k]


def mean_far(x, logp, temperature):
    """Mean over the row's distribution of how far entries lie under the
    largest: what the rounding of a difference and its scaling weighs."""
    if logp is None:
        return 0.0
    p = np.exp(logp)
    far = np.where(p > 0, (x.max() - np.where(p > 0, x, 0.0)) / temperature, 0.0)
    return float((p * far).sum())


def token_logprobs(x, tokens, k, temperature):
    """(logp [M, n], entropy, top logp, top tokens, bounds of the first three in
    units of 2^-24) of rows x (fp64 of what the kernel reads).

    A difference is off by half a step, its product with log2(e) / T by three
    more: 4 |d|; the sum, of at most 60 additions deep (16 a step, 32 steps, 6
    lanes, 4 wavefronts) of exponentials good to 2, by 62 and 4 E|d|; logarithms
    and the last products by 8 of what they give.  An entropy sums d 2^d: the same
    of E|d| and E[d^2]."""
    M = len(x)
    n = tokens.shape[1]
    logp, ent, top, ids = np.zeros((M, n)), np.zeros(M), np.zeros((M, k)), np.zeros((M, k), int)
    b1, b2, b3 = np.zeros((M, n)), np.zeros(M), np.zeros((M, k))
    for m in range(M):
        lp = row_logp(x[m], temperature)
        ids[m] = top_of(x[m], k)
        row = np.full(x.shape[1], -np.inf) if lp is None else lp
        far = mean_far(x[m], lp, temperature)
        p = np.exp(row)
        ent[m] = -(p * np.where(p > 0, row, 0.0)).sum()
        most = x[m].max() if lp is not None else 0.0
        z = (most - np.where(p > 0, x[m], most)) / temperature
        b2[m] = 100 + 100 * far + 8 * (p * z * z).sum() + 8 * ent[m]
        bound = lambda v: 8 * np.where(np.isfinite(row[v]), z[v] + np.abs(row[v]), 0) + 8 * far + 100  # noqa: E731
        in_v = (tokens[m] >= 0) & (tokens[m] < x.shape[1])
        v = np.where(in_v, tokens[m], 0)
        logp[m] = np.where(in_v, row[v], 0.0)
        b1[m] = bound(v)
        top[m], b3[m] = row[ids[m]], bound(ids[m])
    return logp, ent, top, ids, b1, b2, b3


def gradient(x, temperature, tokens, g, e):
    """(dx, bound in units of 2^-24): gradient of sum g logp + e H."""
    dx, tol = np.zeros_like(x), np.zeros_like(x)
    for m in range(len(x)):
        lp = row_logp(x[m], temperature)
        if lp is None:
            continue
        p = np.exp(lp)
        lz = np.where(p > 0, lp, 0.0)
        H = -(p * lz).sum()
        one, size, G = np.zeros(x.shape[1]), np.zeros(x.shape[1]), 0.0
        for j, v in enumerate(tokens[m]):
            if 0 <= v < x.shape[1]:
                one[v] += g[m, j]
                size[v] += abs(g[m, j])
                G += g[m, j]
        dx[m] = (one - p * G - e[m] * p * (lz + H)) / temperature
        far = np.where(p > 0, (x[m].max() - np.where(p > 0, x[m], 0.0)) / temperature, 0.0)
        rel = 16 * far + 8 * mean_far(x[m], lp, temperature) + 200
        ent = 100 + 100 * mean_far(x[m], lp, temperature) + 8 * (p * far * far).sum()
        # the entropy's own error and the roundings of log p
        weight = np.abs(g[m]).sum() + abs(e[m]) * (np.abs(lz) + H)
        tol[m] = (p * (weight * rel + abs(e[m]) * (ent + rel)) + size * (len(tokens[m]) + 4)) / temperature
    return dx, tol


def teacher_p(ids, t, V, temperature):
    """(p, log p) of one row's entries, zeros where they are not kept."""
    keep = (ids >= 0) & (ids < V) & (t > -np.inf)
    if not keep.any():
        return np.zeros(len(ids)), np.zeros(len(ids))
    z = np.where(keep, t, 0.0) / temperature
    z = z - z[keep].max()
    e = np.where(keep, np.exp(np.where(keep, z, 0.0)), 0.0)
    p = e / e.sum()
    return p, np.where(keep, z - np.log(e.sum()), 0.0)


def distill(x, ids, t, temperature, w):
    """(loss, dx, bounds of both in units of 2^-24); dx of sum w loss, rows of
    weight 0 left out."""
    M, V = x.shape
    loss, dx, bl, bx = np.zeros(M), np.zeros_like(x), np.zeros(M), np.zeros_like(x)
    for m in range(M):
        if w[m] == 0:
            continue
        p, lt = teacher_p(ids[m], t[m], V, temperature)
        if not p.any():
            continue
        lp = row_logp(x[m], temperature)
        if lp is None:
            loss[m] = np.inf
            continue
        far = mean_far(x[m], lp, temperature)
        z = (x[m].max() - np.where(np.isfinite(x[m]), x[m], x[m].max())) / temperature
        # p of an entry: its exponent's 4 |d| and the sum over k entries, 10 deep
        rp = 8 * np.abs(np.where(p > 0, lt, 0)).max() + 40
        for j in np.flatnonzero(p):
            v = ids[m, j]
            gap = lt[j] - lp[v]
            loss[m] += p[j] * gap
            if np.isfinite(gap):
                bl[m] += p[j] * (abs(gap) * (rp + 20) + 8 * z[v] + 8 * far + 100 + 8 * abs(lp[v]) + rp)
            dx[m, v] -= p[j]
            bx[m, v] += p[j] * (rp + len(ids[m]) + 4)
        q = np.exp(lp)
        dx[m] = (dx[m] + q) * w[m] / temperature
        bx[m] = (bx[m] + q * (16 * z + 8 * far + 200)) * abs(w[m]) / temperature
    return loss, dx, bl, bx
