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
            e = math.frexp(top)[1]
            scales[m, b] = 2.0 ** (e - 7)
            codes[m, 64 * b:64 * b + 64] = np.clip(np.rint(v / 2.0 ** (e - 7)), -127, 127)
    return codes, scales
