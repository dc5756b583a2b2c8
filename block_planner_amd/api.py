"""Convenience layer over the C ABI: allocates device buffers with torch and
calls the ``ht_*`` entry points.  No arithmetic of the method happens here.

    fmt = plan(W)                      # uint8 [N, K/64] on the GPU
    pw  = pack(W, fmt)                 # PackedLinear (owns its buffer)
    y   = linear(pw, x_bf16)           # fp32 [M, N]
    y   = mlp([pw0, pw1, ...], x_bf16) # Linear + ReLU per layer

and, between the q|k|v and the output linear of a transformer layer, over a
paged cache of keys and values in 8 bits (formats and formulas in ht.h):

    codes, scales = kv_cache(n_pages, n_kv_heads, head_dim, device)
    step = kv_plan(q_len, kv_len, owned, table, free_pages, n_free, T)
    q, k = qk_norm_rope(q, k, step.positions, inv_freq, q_weight=..., k_weight=...)
    kv_write(k, v, step.slots, codes, scales)
    o    = kv_attention(q, codes, scales, table, step.cu_q, step.kv_len, max_q)

between two layers and around the last linear (formulas in ht.h):

    y, h = add_rms_norm(x, weight, residual)               # y bf16 for the next linear
    rows, h = add_rms_norm_q8(x, weight, residual)         # or 8-bit rows: linear(pw, rows)
    r = token_logprobs(logits, tokens, top=20)             # r.logprobs, r.entropy, r.top_logprobs, r.top_tokens
    loss, dlogits = distill_step(logits, r.top_tokens, r.top_logprobs, weight)   # of another model's top ones
"""
from __future__ import annotations

import math
from dataclasses import dataclass
from typing import NamedTuple

import torch

from . import binding as B


@dataclass
class PackedLinear:
    buf: torch.Tensor            # uint8 device buffer (owned)
    desc: B.PackedWeight
    counts: list

    @property
    def N(self) -> int:
        return int(self.desc.N)

    @property
    def K(self) -> int:
        return int(self.desc.K)

    @property
    def nbytes(self) -> int:
        return int(self.desc.bytes)


def plan_params(eps_int4=0.08, eps_int8=0.01, eps_bf16=0.0, eps_fp16=0.0, prefer_bf16=True,
                force_format=-1) -> B.PlanParams:
    p = B.PlanParams()
    p.eps_int4, p.eps_int8, p.eps_bf16, p.eps_fp16 = eps_int4, eps_int8, eps_bf16, eps_fp16
    p.prefer_bf16 = 1 if prefer_bf16 else 0
    p.force_format = force_format
    return p


def plan(W: torch.Tensor, stream=None, **params) -> torch.Tensor:
    N, K = W.shape
    fmt = torch.empty((N, K // 64), dtype=torch.uint8, device=W.device)
    B.ht_plan(W, fmt, plan_params(**params), stream=stream)
    return fmt


def counts(fmt: torch.Tensor, stream=None) -> list:
    c = torch.empty(5, dtype=torch.int64, device=fmt.device)
    B.ht_plan_counts(fmt, c, stream=stream)
    return [int(v) for v in c.cpu()]


def _aligned_empty(nbytes: int, device, align: int = 256) -> torch.Tensor:
    raw = torch.empty(nbytes + align, dtype=torch.uint8, device=device)
    off = (-raw.data_ptr()) % align
    return raw[off:off + nbytes]


def pack(W: torch.Tensor, fmt: torch.Tensor, row_tile: int = 16, stream=None, cnt=None) -> PackedLinear:
    N, K = W.shape
    cnt = counts(fmt, stream=stream) if cnt is None else cnt
    nbytes = B.ht_pack_bytes(N, K, row_tile, cnt)
    buf = _aligned_empty(nbytes, W.device)
    desc = B.ht_pack(W, fmt, row_tile, cnt, buf, stream=stream)
    return PackedLinear(buf=buf, desc=desc, counts=cnt)


@dataclass
class RefreshState:
    """Buffers of ht_refresh for one weight shape, allocated once: the packed
    buffer at its upper bound, the format map, the device counts and the
    initialised workspace."""
    N: int
    K: int
    row_tile: int
    buf: torch.Tensor
    fmt: torch.Tensor
    counts: torch.Tensor
    ws: torch.Tensor


def refresh_state(N: int, K: int, row_tile: int, device, stream=None) -> RefreshState:
    buf_bytes, ws_bytes = B.ht_refresh_bytes(N, K, row_tile)
    ws = _aligned_empty(ws_bytes, device)
    B.ht_workspace_init(ws, stream=stream)
    return RefreshState(N, K, row_tile, _aligned_empty(buf_bytes, device),
                        torch.empty((N, K // 64), dtype=torch.uint8, device=device),
                        torch.empty(5, dtype=torch.int64, device=device), ws)


def refresh(W: torch.Tensor, st: RefreshState, stream=None, **params) -> PackedLinear:
    """Re-plan and re-pack W into st.buf in one pass (ht_refresh), then
    build the descriptor from the counts (one 40-byte copy to the host).
    The previous packed weight of st is overwritten."""
    B.ht_refresh(W, st.fmt, st.buf, st.counts, st.ws, plan_params(**params), row_tile=st.row_tile, stream=stream)
    cnt = [int(v) for v in st.counts.cpu()]
    if int(st.ws[8:12].view(torch.int32).item()) != 0:
        raise RuntimeError("ht_refresh: a wait between workgroups expired (not all workgroups were resident); "
                           "the refreshed buffer is invalid")
    desc = B.ht_refresh_desc(st.N, st.K, st.row_tile, cnt, st.buf)
    return PackedLinear(buf=st.buf[:int(desc.bytes)], desc=desc, counts=cnt)


def workspace(nbytes: int, device) -> torch.Tensor | None:
    if nbytes == 0:
        return None
    return _aligned_empty(nbytes, device)


def linear(pw: PackedLinear, x, act: int = B.HT_ACT_NONE, out: torch.Tensor | None = None,
           ws: torch.Tensor | None = None, path: int = B.HT_PATH_AUTO, stream=None) -> torch.Tensor:
    """x: bf16 [M, K], or Q8Rows (ht_linear_forward_q8, which takes no path)."""
    if isinstance(x, Q8Rows):
        return _linear_q8(pw, x, act, out, ws, path, stream)
    M = x.shape[0]
    y = torch.empty((M, pw.N), dtype=torch.float32, device=x.device) if out is None else out
    if ws is None:
        ws = workspace(B.ht_linear_workspace(pw.desc, M, path), x.device)
    B.ht_linear_forward(pw.desc, x, y, act=act, path=path, ws=ws, stream=stream)
    return y


def linear_backward_data(pw: PackedLinear, dy: torch.Tensor, out: torch.Tensor | None = None,
                         ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """dX = dY . W_hat (fp32 dY [M, N] -> fp32 dX [M, K])."""
    M = dy.shape[0]
    dx = torch.empty((M, pw.K), dtype=torch.float32, device=dy.device) if out is None else out
    if ws is None:
        ws = workspace(B.ht_linear_backward_workspace(pw.desc, M), dy.device)
    B.ht_linear_backward_data(pw.desc, dy, dx, ws=ws, stream=stream)
    return dx


def linear_backward_weight(dy: torch.Tensor, x_bf16: torch.Tensor, out: torch.Tensor | None = None,
                           accumulate: bool = False, stream=None) -> torch.Tensor:
    """dW = dY^T . x (STE gradient of the fp32 master; fp32 [N, K]); with
    accumulate the product is added to `out`."""
    M, N = dy.shape
    K = x_bf16.shape[1]
    dw = torch.empty((N, K), dtype=torch.float32, device=dy.device) if out is None else out
    B.ht_linear_backward_weight(dy, x_bf16, dw, accumulate=accumulate, stream=stream)
    return dw


def mlp_workspace(layers: list, M: int, device, stream=None) -> torch.Tensor:
    """An initialised workspace for mlp() over these layers at batch M."""
    ws = workspace(B.ht_mlp_workspace([pw.desc for pw in layers], M), device)
    B.ht_workspace_init(ws, stream=stream)
    return ws


def mlp(layers: list, x: torch.Tensor, dump: bool = False, out: torch.Tensor | None = None,
        ws: torch.Tensor | None = None, path: int = B.HT_PATH_AUTO, stream=None):
    M = x.shape[0]
    descs = [pw.desc for pw in layers]
    y = torch.empty((M, layers[-1].N), dtype=torch.float32, device=x.device) if out is None else out
    if ws is None:
        ws = mlp_workspace(layers, M, x.device, stream=stream)
    act_dump = None
    if dump:
        tot = sum(M * pw.N for pw in layers[:-1])
        act_dump = torch.empty(max(tot, 8), dtype=torch.bfloat16, device=x.device)
    B.ht_mlp_forward(descs, x, y, act_dump=act_dump, path=path, ws=ws, stream=stream)
    if dump:
        slabs, off = [], 0
        for pw in layers[:-1]:
            slabs.append(act_dump[off:off + M * pw.N].view(M, pw.N))
            off += M * pw.N
        return y, slabs
    return y


# -----------------------------------------------------------------------------
# Attention beside the linears
# -----------------------------------------------------------------------------
def _need(t: torch.Tensor, name: str, dtype, shape: tuple) -> None:
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")


def _ints(*specs) -> None:
    """Every (tensor, name, n): int32 [n], dense."""
    i32 = torch.int32
    for t, name, n in specs:
        shape = t.shape
        if t.dtype is not i32 or len(shape) != 1 or shape[0] != n or not t.is_contiguous():
            _need(t, name, i32, (n,))


def _on_gpu(*tensors) -> None:
    """The kernels run on the current device and get bare addresses: host
    memory and other devices' never reach them."""
    on = None
    for t in tensors:
        if t is not None and t.get_device() != on:
            if t.get_device() < 0:
                raise ValueError("every tensor must be on the GPU")
            if on is not None:
                raise ValueError(f"every tensor must be on one GPU, got cuda:{on} and cuda:{t.get_device()}")
            on = t.get_device()
    if on is not None and on != torch.cuda.current_device():
        raise ValueError(f"the tensors are on cuda:{on}, the current device is cuda:{torch.cuda.current_device()}")


def _using(stream):
    """Context in which a call given a stream allocates, copies and launches:
    temporaries belong to that stream then."""
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


def _table(t: torch.Tensor, R: int) -> None:
    if t.dim() != 2 or t.dtype != torch.int32 or t.shape[0] != R or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"table: expected int32 [{R}, pages] with dense rows, got {t.dtype} {tuple(t.shape)}")


def _rows(t: torch.Tensor, name: str) -> torch.Tensor:
    """[T, heads, D] fp32 or bf16 as the kernels read it: the last dim dense,
    pointer and strides in whole 16-byte pieces (a copy where they are not)."""
    shape, dt = t.shape, t.dtype
    if len(shape) != 3 or (dt is not torch.float32 and dt is not torch.bfloat16):
        raise ValueError(f"{name}: expected fp32 or bf16 [rows, heads, dim], got {dt} {tuple(shape)}")
    rs, hs, ds = t.stride()
    D, piece = shape[2], 3 if dt is torch.float32 else 7      # strides in 16-byte pieces
    if ds == 1 and rs >= D and not rs & piece and (shape[1] == 1 or (hs >= D and not hs & piece)) and not t.data_ptr() & 15:
        return t
    return t.clone(memory_format=torch.contiguous_format)


def _out_rows(t: torch.Tensor, name: str, shape, dtype) -> torch.Tensor:
    if t.dtype is not dtype or t.shape != shape or t.stride(2) != 1:
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)} with a dense last dim, got {t.dtype} {tuple(t.shape)}")
    return t


def _scratch(nbytes: int, device) -> torch.Tensor | None:
    """Workspace of a call that needs 16-byte alignment (torch's allocator
    gives 512)."""
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def kv_cache(n_pages: int, n_kv_heads: int, head_dim: int, device) -> tuple:
    """(codes int8 [n_pages, n_kv_heads, 2, 64 * head_dim], scales fp32
    [n_pages, n_kv_heads, 2]) of one layer's cache, zeroed."""
    B.ht_kv_cache_bytes(n_pages, n_kv_heads, head_dim)   # refuses what the kernels do not take
    return (torch.zeros(n_pages, n_kv_heads, 2, B.HT_KV_PAGE * head_dim, dtype=torch.int8, device=device),
            torch.zeros(n_pages, n_kv_heads, 2, dtype=torch.float32, device=device))


def _cache_desc(codes: torch.Tensor, scales: torch.Tensor) -> B.KVCacheDesc:
    shape = codes.shape
    if len(shape) != 4 or codes.dtype is not torch.int8 or shape[2] != 2 or shape[3] % B.HT_KV_PAGE:
        raise ValueError(f"codes: expected int8 [pages, heads, 2, 64 * dim], got {codes.dtype} {tuple(shape)}")
    if not codes.is_contiguous():
        raise ValueError("codes: expected a contiguous tensor")
    _need(scales, "scales", torch.float32, shape[:3])
    return B.KVCacheDesc(codes.data_ptr(), scales.data_ptr(), shape[0], shape[1], shape[3] // B.HT_KV_PAGE)


def kv_cache_values(codes: torch.Tensor, scales: torch.Tensor) -> tuple:
    """The keys and values a cache (or a selection of its pages) stands for:
    two fp32 tensors [pages, heads, 64, dim].  Plain indexing, for inspection
    and for moving a prefix to another format."""
    n, h, _, b = codes.shape
    d = b // B.HT_KV_PAGE
    k = codes[:, :, 0].reshape(n, h, 4, d // 64, 4, 16, 16).permute(0, 1, 2, 5, 3, 4, 6).reshape(n, h, 64, d)
    v = codes[:, :, 1].reshape(n, h, d // 16, 4, 16, 4, 4).permute(0, 1, 5, 3, 6, 2, 4).reshape(n, h, 64, d)
    return k.float() * scales[:, :, 0, None, None], v.float() * scales[:, :, 1, None, None]


class KVStep(NamedTuple):
    """What kv_plan gives for one step (all int32, on the device)."""
    cu_q: torch.Tensor        # [R + 1] first row of each request
    slots: torch.Tensor       # [T] 64 * page + offset, -1: not stored
    positions: torch.Tensor   # [T]
    kv_len: torch.Tensor      # [R] tokens in the cache after the step
    owned: torch.Tensor       # [R] pages owned after the step
    status: torch.Tensor      # [2] pages left free, requests refused


def kv_step(R: int, T: int, device) -> KVStep:
    """Buffers for kv_plan's outputs.  A step's lengths are inputs of the next
    plan, which must not write over them (HT_EINVAL): two sets, used in turn,
    serve any number of steps."""
    return KVStep(*(torch.empty(n, dtype=torch.int32, device=device) for n in (R + 1, T, T, R, R, 2)))


def kv_plan(q_len: torch.Tensor, kv_len: torch.Tensor, owned: torch.Tensor, table: torch.Tensor,
            free_pages: torch.Tensor, n_free: torch.Tensor, T: int, out=None, stream=None) -> KVStep:
    """Page tables, slots and positions of one step (ht_kv_plan).  q_len,
    kv_len, owned int32 [R]; table int32 [R, pages] gets the new pages in
    place; free_pages int32 [n] with its first n_free[0] entries free; T the
    sum of q_len.  Nothing else changes: the next step takes step.kv_len,
    step.owned and step.status[:1] as kv_len, owned and n_free."""
    if stream is not None:
        with _using(stream):
            return kv_plan(q_len, kv_len, owned, table, free_pages, n_free, T, out)
    R = q_len.shape[0]
    _ints((q_len, "q_len", R), (kv_len, "kv_len", R), (owned, "owned", R), (n_free, "n_free", 1),
          (free_pages, "free_pages", free_pages.numel()))
    _table(table, R)
    if out is None:
        out = kv_step(R, T, q_len.device)
    else:
        _ints(*zip(out, KVStep._fields, (R + 1, T, T, R, R, 2)))
        if not isinstance(out, KVStep):
            out = KVStep(*out)
    _on_gpu(q_len, kv_len, owned, table, free_pages, n_free, *out)
    B.ht_kv_plan(q_len, kv_len, owned, table, free_pages, n_free, T, *out)
    return out


def kv_release(which: torch.Tensor, kv_len: torch.Tensor, owned: torch.Tensor, table: torch.Tensor,
               free_pages: torch.Tensor, n_free: torch.Tensor, stream=None) -> None:
    """Give back the pages of the requests with which[r] (bool or uint8 [R]);
    kv_len, owned, free_pages and n_free change in place (ht_kv_release)."""
    R = which.shape[0]
    if which.dtype not in (torch.bool, torch.uint8) or which.dim() != 1 or not which.is_contiguous():
        raise ValueError(f"which: expected contiguous bool or uint8 [requests], got {which.dtype} {tuple(which.shape)}")
    _ints((kv_len, "kv_len", R), (owned, "owned", R), (n_free, "n_free", 1),
          (free_pages, "free_pages", free_pages.numel()))
    _table(table, R)
    _on_gpu(which, kv_len, owned, table, free_pages, n_free)
    B.ht_kv_release(which, kv_len, owned, table, free_pages, n_free, stream=stream)


def rope_inv_freq(rot: int, base: float = 10000.0, device=None) -> torch.Tensor:
    """fp64 [rot / 2]: base^(-2 i / rot), the angle per position of each pair."""
    i = torch.arange(rot // 2, dtype=torch.float64, device=device)
    return base ** (-2.0 * i / rot)


def _rope_args(q, k, positions, inv_freq, q_weight, k_weight):
    T, _, D = q.shape
    if k is not None and (k.dtype != q.dtype or k.shape[0] != T or k.shape[2] != D):
        raise ValueError(f"k: expected {q.dtype} [{T}, heads, {D}], got {k.dtype} {tuple(k.shape)}")
    _need(positions, "positions", torch.int32, (T,))
    _need(inv_freq, "inv_freq", torch.float64, (inv_freq.numel(),))
    if (q_weight is None) != (k_weight is None):
        raise ValueError("q_weight and k_weight: both or neither")
    if q_weight is not None:
        _need(q_weight, "q_weight", torch.float32, (D,))
        _need(k_weight, "k_weight", torch.float32, (D,))


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor, inv_freq: torch.Tensor,
                 q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                 interleaved: bool = False, out_dtype=None, out=None, stream=None) -> tuple:
    """Norm of every head (with weights given) and rotation by position of q
    [T, n_q, D] and k [T, n_k, D] (or None) in one pass (ht_qk_norm_rope).
    fp32 or bf16, any row and head strides; positions int32 [T]; inv_freq
    fp64 [rot / 2].  Returns (q, k) in out_dtype (q's own by default)."""
    if stream is not None:
        with _using(stream):
            return qk_norm_rope(q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, out_dtype, out)
    q = _rows(q, "q")
    k = _rows(k, "k") if k is not None else None
    _rope_args(q, k, positions, inv_freq, q_weight, k_weight)
    dt = q.dtype if out_dtype is None else out_dtype
    if dt not in (torch.float32, torch.bfloat16):
        raise ValueError(f"out_dtype: expected fp32 or bf16, got {dt}")
    if out is None:
        # dense, whatever the strides of q and k
        yq = torch.empty_like(q, dtype=dt, memory_format=torch.contiguous_format)
        yk = torch.empty_like(k, dtype=dt, memory_format=torch.contiguous_format) if k is not None else None
    else:
        yq = _out_rows(out[0], "out[0]", q.shape, dt)
        yk = _out_rows(out[1], "out[1]", k.shape, dt) if k is not None else None
    _on_gpu(q, k, positions, inv_freq, q_weight, k_weight, yq, yk)
    B.ht_qk_norm_rope(q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, yq, yk)
    return yq, yk


def qk_norm_rope_backward(dq: torch.Tensor, dk: torch.Tensor | None, q: torch.Tensor, k: torch.Tensor | None,
                          positions: torch.Tensor, inv_freq: torch.Tensor, q_weight: torch.Tensor | None = None,
                          k_weight: torch.Tensor | None = None, eps: float = 1e-6, interleaved: bool = False,
                          out=None, ws: torch.Tensor | None = None, stream=None) -> tuple:
    """Gradients of qk_norm_rope: (dq, dk) of its inputs, in their type, and
    fp32 (dq_weight, dk_weight) (None without weights)."""
    if stream is not None:
        with _using(stream):
            return qk_norm_rope_backward(dq, dk, q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, out, ws)
    q, dq = _rows(q, "q"), _rows(dq, "dq")
    k, dk = (_rows(k, "k"), _rows(dk, "dk")) if k is not None else (None, None)
    _rope_args(q, k, positions, inv_freq, q_weight, k_weight)
    if dq.shape != q.shape or (k is not None and (dk.shape != k.shape or dk.dtype != dq.dtype)):
        raise ValueError("dq, dk: expected the shapes of q and k, one type")
    _on_gpu(dq, dk, q, k, positions, inv_freq, q_weight, k_weight, ws)
    if out is None:
        xq = torch.empty_like(q, memory_format=torch.contiguous_format)
        xk = torch.empty_like(k, memory_format=torch.contiguous_format) if k is not None else None
    else:
        xq = _out_rows(out[0], "out[0]", q.shape, q.dtype)
        xk = _out_rows(out[1], "out[1]", k.shape, k.dtype) if k is not None else None
        _on_gpu(xq, xk)
    dwq = dwk = None
    if q_weight is not None:
        dwq, dwk = torch.empty_like(q_weight), torch.empty_like(k_weight)
        if ws is None:
            n_k = k.shape[1] if k is not None else 0
            ws = _scratch(B.ht_qk_norm_rope_workspace(q.shape[0], q.shape[1], n_k, q.shape[2], True), q.device)
    B.ht_qk_norm_rope_backward(dq, dk, q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, xq, xk, dwq,
                               dwk, ws=ws)
    return xq, xk, dwq, dwk


def kv_write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
             stream=None) -> None:
    """Quantise keys and values [T, heads, D] (fp32 or bf16, each its own
    type) into the cache at slots int32 [T] (ht_kv_write), in place."""
    if stream is not None:
        with _using(stream):
            return kv_write(k, v, slots, codes, scales)
    desc = _cache_desc(codes, scales)
    k, v = _rows(k, "k"), _rows(v, "v")
    shape = (slots.shape[0], codes.shape[1], codes.shape[3] // B.HT_KV_PAGE)
    if tuple(k.shape) != shape or tuple(v.shape) != shape:
        raise ValueError(f"k, v: expected {shape}, got {tuple(k.shape)} and {tuple(v.shape)}")
    _need(slots, "slots", torch.int32, shape[:1])
    _on_gpu(k, v, slots, codes, scales)
    B.ht_kv_write(k, v, slots, desc)


def kv_attention(q: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, table: torch.Tensor, cu_q: torch.Tensor,
                 kv_len: torch.Tensor, max_q: int, max_kv: int | None = None, scale: float | None = None,
                 causal: bool = True, window: int = 0, out: torch.Tensor | None = None,
                 ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of the rows q bf16 [T, n_q, D] over the cache
    (ht_kv_attention): bf16 [T, n_q, D].  max_q and max_kv (default: what the
    table can hold) are the largest lengths the caller knows of; scale is
    1 / sqrt(D) by default; window > 0 keeps each row to its last `window`
    tokens.  Rows of no request (from cu_q[R] on) give zeros."""
    if stream is not None:
        with _using(stream):
            return kv_attention(q, codes, scales, table, cu_q, kv_len, max_q, max_kv, scale, causal, window, out, ws)
    desc = _cache_desc(codes, scales)
    if q.dtype != torch.bfloat16:
        raise ValueError(f"q: expected bf16 [rows, heads, dim], got {q.dtype}")
    q = _rows(q, "q")
    T, n_q, D = q.shape
    if D != codes.shape[3] // B.HT_KV_PAGE:
        raise ValueError(f"q: expected head dim {codes.shape[3] // B.HT_KV_PAGE}, got {D}")
    R = kv_len.shape[0]
    _table(table, R)
    _ints((cu_q, "cu_q", R + 1), (kv_len, "kv_len", R))
    if out is not None:
        _out_rows(out, "out", q.shape, q.dtype)
    _on_gpu(q, codes, scales, table, cu_q, kv_len, out, ws)
    if max_kv is None:
        max_kv = table.shape[1] * B.HT_KV_PAGE
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    if ws is None:
        ws = _scratch(B.ht_kv_attention_workspace(desc, T, R, n_q, max_q, max_kv, window), q.device)
    B.ht_kv_attention(q, desc, table, cu_q, kv_len, max_q, max_kv, 1.0 / math.sqrt(D) if scale is None else scale,
                      causal, window, out, ws=ws)
    return out


# -----------------------------------------------------------------------------
# Between two layers, and around the last linear
# -----------------------------------------------------------------------------
class Q8Rows(NamedTuple):
    """Rows in 8 bits with a scale per 64 columns, as the W8A8 linear takes
    them (ht_q8_rows)."""
    codes: torch.Tensor       # int8 [ceil(M / 16), K / 64, 64, 16]
    scales: torch.Tensor      # fp32 [K / 64, 16 * ceil(M / 16)]
    M: int


def q8_rows(M: int, K: int, device) -> Q8Rows:
    """Buffers for 8-bit rows [M, K]."""
    B.ht_q8_bytes(M, K)       # refuses what the kernels do not take
    return _new_q8(M, K, device)


def _new_q8(M: int, K: int, device) -> Q8Rows:
    G = -(-M // 16)
    return Q8Rows(torch.empty(G, K // 64, 64, 16, dtype=torch.int8, device=device),
                  torch.empty(K // 64, 16 * G, dtype=torch.float32, device=device), int(M))


def _q8_desc(q: Q8Rows) -> B.Q8Desc:
    codes, scales, M = q
    G, KB = -(-M // 16), codes.shape[1] if codes.dim() == 4 else -1
    _need(codes, "codes", torch.int8, (G, KB, 64, 16))
    _need(scales, "scales", torch.float32, (KB, 16 * G))
    return B.Q8Desc(codes.data_ptr(), scales.data_ptr(), M, 64 * KB)


def q8_values(q: Q8Rows, dtype=torch.bfloat16, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values of 8-bit rows, [M, K] bf16 (where they are exact) or fp32
    (ht_q8_values)."""
    if stream is not None:
        with _using(stream):
            return q8_values(q, dtype, out)
    desc = _q8_desc(q)
    if dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"dtype: expected fp32 or bf16, got {dtype}")
    if out is None:
        out = torch.empty(desc.M, desc.K, dtype=dtype, device=q.codes.device)
    else:
        _out_matrix(out, "out", (desc.M, desc.K), dtype)
    _on_gpu(q.codes, q.scales, out)
    B.ht_q8_values(desc, out)
    return out


def _linear_q8(pw: PackedLinear, x: Q8Rows, act, out, ws, path, stream) -> torch.Tensor:
    if stream is not None:
        with _using(stream):
            return _linear_q8(pw, x, act, out, ws, path, None)
    if path != B.HT_PATH_AUTO:
        raise ValueError("8-bit rows take no path")
    desc = _q8_desc(x)
    if out is None:
        out = torch.empty(desc.M, pw.N, dtype=torch.float32, device=x.codes.device)
    else:
        _out_matrix(out, "out", (desc.M, pw.N), torch.float32)
    _on_gpu(pw.buf, x.codes, x.scales, out, ws)
    if desc.M == 0:
        return out
    if ws is None:
        ws = workspace(B.ht_linear_q8_workspace(pw.desc, desc.M), out.device)
    B.ht_linear_forward_q8(pw.desc, desc, out, act=act, ws=ws)
    return out


def _matrix(t: torch.Tensor, name: str, shape=None) -> torch.Tensor:
    """[M, K] fp32 or bf16 as the kernels read it: dense rows, pointer and
    stride in whole 16-byte pieces (a copy where they are not)."""
    s, dt = t.shape, t.dtype
    if len(s) != 2 or (dt is not torch.float32 and dt is not torch.bfloat16):
        raise ValueError(f"{name}: expected fp32 or bf16 [rows, columns], got {dt} {tuple(s)}")
    if shape is not None and s != shape:
        raise ValueError(f"{name}: expected {tuple(shape)}, got {tuple(s)}")
    ld, cs = t.stride()
    if cs == 1 and (s[0] == 1 or (ld >= s[1] and not ld & (3 if dt is torch.float32 else 7))) and not t.data_ptr() & 15:
        return t
    return t.clone(memory_format=torch.contiguous_format)


def _out_matrix(t: torch.Tensor, name: str, shape, dtype) -> torch.Tensor:
    if t.dtype is not dtype or t.shape != shape or (t.stride(1) != 1 and t.shape[1] != 1):
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)} with dense rows, got {t.dtype} {tuple(t.shape)}")
    return t


def _norm_args(x, weight, residual):
    x = _matrix(x, "x")
    if residual is not None:
        residual = _matrix(residual, "residual", x.shape)
    _need(weight, "weight", torch.float32, x.shape[1:])
    return x, residual


def add_rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6,
                 out_dtype=None, out=None, stream=None) -> tuple:
    """(y, h): h = x + residual in residual's type (None without one) and the
    norm y of it times weight fp32 [K], in out_dtype (bf16 by default, what
    the next linear takes), in one pass (ht_add_rms_norm).  x and residual
    [M, K] fp32 or bf16, each its own type; out: (y, h), which may be x and
    residual themselves."""
    if stream is not None:
        with _using(stream):
            return add_rms_norm(x, weight, residual, eps, out_dtype, out)
    x, residual = _norm_args(x, weight, residual)
    dt = torch.bfloat16 if out_dtype is None else out_dtype
    if dt not in (torch.float32, torch.bfloat16):
        raise ValueError(f"out_dtype: expected fp32 or bf16, got {dt}")
    if out is None:
        y = torch.empty_like(x, dtype=dt, memory_format=torch.contiguous_format)
        h = torch.empty_like(residual, memory_format=torch.contiguous_format) if residual is not None else None
    else:
        y = _out_matrix(out[0], "out[0]", x.shape, dt)
        h = _out_matrix(out[1], "out[1]", x.shape, residual.dtype) if residual is not None else None
    _on_gpu(x, residual, weight, y, h)
    B.ht_add_rms_norm(x, residual, weight, eps, h, y)
    return y, h


def add_rms_norm_q8(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6,
                    out=None, stream=None) -> tuple:
    """(rows, h) as add_rms_norm, the norm as Q8Rows for linear(); K % 64 == 0.
    out: (q8_rows(M, K), h)."""
    if stream is not None:
        with _using(stream):
            return add_rms_norm_q8(x, weight, residual, eps, out)
    x, residual = _norm_args(x, weight, residual)
    if out is None:
        q = _new_q8(*x.shape, x.device)
        h = torch.empty_like(residual, memory_format=torch.contiguous_format) if residual is not None else None
    else:
        q, h = out[0], _out_matrix(out[1], "out[1]", x.shape, residual.dtype) if residual is not None else None
    desc = _q8_desc(q)
    _on_gpu(x, residual, weight, q.codes, q.scales, h)
    B.ht_add_rms_norm(x, residual, weight, eps, h, None, desc)
    return q, h


def add_rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, dh: torch.Tensor | None = None,
                          eps: float = 1e-6, x_dtype=None, out: torch.Tensor | None = None,
                          ws: torch.Tensor | None = None, stream=None) -> tuple:
    """(dx, dresidual, dweight) of add_rms_norm: dy the gradient of y, h what
    the norm saw (x where there was no residual), dh the gradient h has from
    elsewhere, in h's type.  dx in x_dtype (h's by default) is dresidual itself
    where the types agree; dweight fp32 [K].  out: dresidual's buffer."""
    if stream is not None:
        with _using(stream):
            return add_rms_norm_backward(dy, h, weight, dh, eps, x_dtype, out, ws)
    h, _ = _norm_args(h, weight, None)
    dy = _matrix(dy, "dy", h.shape)
    if dh is not None:
        if dh.dtype != h.dtype:
            raise ValueError(f"dh: expected h's type {h.dtype}, got {dh.dtype}")
        dh = _matrix(dh, "dh", h.shape)
    dt = h.dtype if x_dtype is None else x_dtype
    if dt not in (torch.float32, torch.bfloat16):
        raise ValueError(f"x_dtype: expected fp32 or bf16, got {dt}")
    if out is None:
        dres = torch.empty(h.shape, dtype=h.dtype, device=h.device)
    else:
        dres = _out_matrix(out, "out", h.shape, h.dtype)
    dx = None if dt is h.dtype else torch.empty(h.shape, dtype=dt, device=h.device)
    dw = torch.empty_like(weight)
    _on_gpu(dy, h, dh, weight, dres, ws)
    if ws is None:
        ws = _scratch(B.ht_add_rms_norm_workspace(*h.shape), h.device)
    B.ht_add_rms_norm_backward(dy, h, dh, weight, eps, dres, dx, dw, ws=ws)
    return dres if dx is None else dx, dres, dw


def _logits(t: torch.Tensor) -> torch.Tensor:
    """[M, V] fp32 or bf16 with dense rows (a copy where they are not)."""
    s, dt = t.shape, t.dtype
    if len(s) != 2 or (dt is not torch.float32 and dt is not torch.bfloat16):
        raise ValueError(f"logits: expected fp32 or bf16 [rows, vocabulary], got {dt} {tuple(s)}")
    ld, cs = t.stride()
    if (cs == 1 or s[1] == 1) and (s[0] == 1 or ld >= s[1]):
        return t
    return t.clone(memory_format=torch.contiguous_format)


def _tokens(t: torch.Tensor, M: int) -> None:
    if t.dtype is not torch.int32 or t.dim() not in (1, 2) or t.shape[0] != M or not t.is_contiguous():
        raise ValueError(f"tokens: expected contiguous int32 [{M}] or [{M}, n], got {t.dtype} {tuple(t.shape)}")


def _dlogits(logits: torch.Tensor, out: torch.Tensor | None) -> torch.Tensor:
    if out is None:
        return torch.empty_like(logits, memory_format=torch.contiguous_format)
    return _out_matrix(out, "out", logits.shape, logits.dtype)


class TokenLogprobs(NamedTuple):
    """What token_logprobs gives (all fp32 but top_tokens, int32)."""
    logprobs: torch.Tensor | None   # of the given tokens, in their shape
    entropy: torch.Tensor           # [M]
    top_logprobs: torch.Tensor      # [M, top]
    top_tokens: torch.Tensor        # [M, top]
    stats: torch.Tensor             # [M, 2], for token_logprobs_backward


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor | None = None, top: int = 0, temperature: float = 1.0,
                   ws: torch.Tensor | None = None, stream=None) -> TokenLogprobs:
    """Log probabilities of given tokens, entropy and the `top` most likely
    tokens of rows of logits [M, V], fp32 or bf16, any row stride, in one pass
    (ht_token_logprobs).  tokens int32 [M] or [M, n]; one outside [0, V) is not
    scored (0).  -Inf logits are not allowed ones."""
    if stream is not None:
        with _using(stream):
            return token_logprobs(logits, tokens, top, temperature, ws)
    logits = _logits(logits)
    M, V = logits.shape
    if tokens is not None:
        _tokens(tokens, M)
    if not 0 <= top <= min(64, V):
        raise ValueError(f"top: expected 0 to {min(64, V)}, got {top}")
    _on_gpu(logits, tokens, ws)
    # one allocation for the fp32 results
    n = B._count(tokens) * M
    buf = torch.empty(n + (3 + top) * M, dtype=torch.float32, device=logits.device)
    r = TokenLogprobs(None if tokens is None else buf.as_strided(tokens.shape, tokens.stride()),
                      buf.as_strided((M,), (1,), n), buf.as_strided((M, top), (top, 1), n + 3 * M),
                      torch.empty((M, top), dtype=torch.int32, device=logits.device),
                      buf.as_strided((M, 2), (2, 1), n + M))
    if ws is None:
        ws = _scratch(B.ht_token_logprobs_workspace(M, V, top), logits.device)
    B.ht_token_logprobs(logits, tokens, temperature, *r, ws=ws)
    return r


def token_logprobs_backward(d_logprobs: torch.Tensor | None, d_entropy: torch.Tensor | None, logits: torch.Tensor,
                            tokens: torch.Tensor | None, stats: torch.Tensor, entropy: torch.Tensor | None = None,
                            temperature: float = 1.0, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient of the logits, in their type, from those of the given tokens'
    log probabilities and of the entropy (either may be None); stats and
    entropy of the forward call.  out may be the logits themselves."""
    if stream is not None:
        with _using(stream):
            return token_logprobs_backward(d_logprobs, d_entropy, logits, tokens, stats, entropy, temperature, out)
    x = _logits(logits)
    M = x.shape[0]
    if (tokens is None) != (d_logprobs is None):
        raise ValueError("tokens and d_logprobs: both or neither")
    if tokens is not None:
        _tokens(tokens, M)
        _need(d_logprobs, "d_logprobs", torch.float32, tokens.shape)
    _need(stats, "stats", torch.float32, (M, 2))
    if d_entropy is not None:
        _need(d_entropy, "d_entropy", torch.float32, (M,))
        if entropy is None:
            raise ValueError("d_entropy needs the entropy of the forward call: both or neither")
        _need(entropy, "entropy", torch.float32, (M,))
    out = _dlogits(x, out)
    _on_gpu(d_logprobs, d_entropy, x, tokens, stats, entropy, out)
    B.ht_token_logprobs_backward(d_logprobs, d_entropy, x, tokens, stats, entropy, temperature, out)
    return out


def _teacher(logits: torch.Tensor, ids: torch.Tensor, teacher: torch.Tensor) -> None:
    M = logits.shape[0]
    if ids.dim() != 2 or not 1 <= ids.shape[1] <= 1024:
        raise ValueError(f"ids: expected int32 [{M}, 1 to 1024], got {ids.dtype} {tuple(ids.shape)}")
    _need(ids, "ids", torch.int32, (M, ids.shape[1]))
    _need(teacher, "teacher", torch.float32, ids.shape)


def distill_loss(logits: torch.Tensor, ids: torch.Tensor, teacher: torch.Tensor, temperature: float = 1.0,
                 stream=None) -> tuple:
    """(loss, stats) of a student's logits [M, V] against a teacher's top
    entries: ids int32 [M, k] (outside [0, V): not kept), teacher fp32 [M, k]
    its logits or log probabilities there (ht_distill_loss).  loss fp32 [M] is
    the divergence of the softmax over the kept entries from the student's
    over all, both at the temperature."""
    if stream is not None:
        with _using(stream):
            return distill_loss(logits, ids, teacher, temperature)
    logits = _logits(logits)
    _teacher(logits, ids, teacher)
    M = logits.shape[0]
    loss, stats = (torch.empty(s, dtype=torch.float32, device=logits.device) for s in ((M,), (M, 2)))
    _on_gpu(logits, ids, teacher)
    B.ht_distill_loss(logits, ids, teacher, temperature, loss, stats)
    return loss, stats


def distill_backward(d_loss: torch.Tensor, logits: torch.Tensor, ids: torch.Tensor, teacher: torch.Tensor,
                     stats: torch.Tensor, temperature: float = 1.0, out: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """Gradient of the student's logits, in their type, from the loss's, fp32
    [M] (ht_distill_backward).  out may be the logits themselves."""
    if stream is not None:
        with _using(stream):
            return distill_backward(d_loss, logits, ids, teacher, stats, temperature, out)
    x = _logits(logits)
    _teacher(x, ids, teacher)
    _need(d_loss, "d_loss", torch.float32, x.shape[:1])
    _need(stats, "stats", torch.float32, (x.shape[0], 2))
    out = _dlogits(x, out)
    _on_gpu(d_loss, x, ids, teacher, stats, out)
    B.ht_distill_backward(d_loss, x, ids, teacher, stats, temperature, out)
    return out


def distill_step(logits: torch.Tensor, ids: torch.Tensor, teacher: torch.Tensor, weight: torch.Tensor | None = None,
                 temperature: float = 1.0, out: torch.Tensor | None = None, stats: torch.Tensor | None = None,
                 stream=None) -> tuple:
    """(loss, dlogits): distill_loss and, in the same pass, the gradient of
    sum(weight * loss), weight fp32 [M] (1 without; rows of weight 0 are not
    read, their loss is 0) (ht_distill_step).  out may be the logits
    themselves; stats fp32 [M, 2] gets what distill_backward starts from."""
    if stream is not None:
        with _using(stream):
            return distill_step(logits, ids, teacher, weight, temperature, out, stats)
    x = _logits(logits)
    _teacher(x, ids, teacher)
    M = x.shape[0]
    if weight is not None:
        _need(weight, "weight", torch.float32, (M,))
    if stats is not None:
        _need(stats, "stats", torch.float32, (M, 2))
    out = _dlogits(x, out)
    loss = torch.empty(M, dtype=torch.float32, device=x.device)
    _on_gpu(x, ids, teacher, weight, out, stats)
    B.ht_distill_step(x, ids, teacher, weight, temperature, loss, stats, out)
    return loss, out


def scale_rows(x: torch.Tensor, factor: torch.Tensor, stream=None) -> None:
    """x [M, V] (fp32 or bf16, dense rows) times factor fp32 [1] in place;
    nothing moves where it is 1 (ht_scale_rows)."""
    if stream is not None:
        with _using(stream):
            return scale_rows(x, factor)
    if x.dim() != 2:
        raise ValueError(f"x: expected [rows, columns], got {tuple(x.shape)}")
    _out_matrix(x, "x", x.shape, x.dtype)
    _need(factor, "factor", torch.float32, (1,))
    _on_gpu(x, factor)
    B.ht_scale_rows(x, factor)
