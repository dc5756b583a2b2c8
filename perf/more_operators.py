"""Operators around the last linear of a transformer, as measured cases.

Three operators, forward and backward:

  norm      residual addition and root-mean-square norm, its output in fp32, bf16 or 8 bits; its gradients
  logprobs  log probabilities of given tokens, entropy and top alternatives from rows of logits; the logits' gradient
  distill   loss of a student's logits against a teacher's top logits, alone or with the logits' gradient (a step)

``run`` computes them with elementary torch operations, or, where ``own`` is true, by the calls of
``block_planner_amd.api``.  Widths are those of the framework's linear stacks or generic, vocabularies generic.

An 8-bit output has, per row and 64 columns, 2^(E-1) <= max |y| < 2^E, codes clamp(rne(y 2^(7-E)), -127, 127) and the
scale 2^(E-7); it is returned as the values it stands for (exact in bf16).
"""
import math
import random

import torch

own = False

EPS = 1e-6
BLOCK = 64


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # One token between two layers: latency only.
        dict(name="norm decode 1", op="norm", rows=1, width=4096, x="fp32", r="fp32", y="bf16"),
        # A prompt's rows between two layers, fp32 from the linear, bf16 for the next one.
        dict(name="norm prompt 8192", op="norm", rows=8192, width=4096, x="fp32", r="fp32", y="bf16"),
        # A prompt's rows for a linear with 8-bit inputs over a bf16 residual stream, read back.
        dict(name="norm 8 bits 3001", op="norm", rows=3001, width=2048, x="fp32", r="bf16", y="q8"),
        # Training: 4 x 2048 tokens, the residual's own gradient added.
        dict(name="norm backward 8192", op="norm_backward", rows=8192, width=2048, x="fp32", r="fp32", y="fp32"),
        # One answer's token with its alternatives: latency.
        dict(name="logprobs answer 1", op="logprobs", rows=1, vocab=128000, pad=0, x="fp32", tokens=1, top=5,
             temperature=1.0, masked=False),
        # A serving step under a grammar that bans a part of the vocabulary.
        dict(name="logprobs answers 64", op="logprobs", rows=64, vocab=32000, pad=0, x="fp32", tokens=1, top=20,
             temperature=0.7, masked=True),
        # Scoring a long prompt; it is also how a teacher's top logits are kept for distillation.
        dict(name="logprobs prompt 4096", op="logprobs", rows=4096, vocab=128000, pad=0, x="bf16", tokens=1, top=32,
             temperature=1.0, masked=False),
        # A policy's update: log probabilities weighted by advantages, an entropy bonus; an odd vocabulary.
        dict(name="logprobs backward 2000", op="logprobs_backward", rows=2000, vocab=50001, pad=0, x="fp32", tokens=1,
             temperature=1.0, masked=False),
        # Evaluating a quantised student against its teacher.
        dict(name="distill loss 2048", op="distill", rows=2048, vocab=32000, pad=0, x="fp32", top=64, temperature=2.0),
        # Small training batches of a short vocabulary.
        dict(name="distill step 33", op="distill_step", rows=33, vocab=1003, pad=0, x="bf16", top=8, temperature=1.0),
        # An ordinary training batch, fp32 logits as the linear gives them.
        dict(name="distill step 4096", op="distill_step", rows=4096, vocab=32000, pad=0, x="fp32", top=32,
             temperature=2.0),
        # The largest vocabulary in bf16.
        dict(name="distill step large", op="distill_step", rows=4096, vocab=128000, pad=0, x="bf16", top=20,
             temperature=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "logprobs", "logprobs", "logprobs_backward", "distill",
                     "distill_step", "distill_step"])
    if op.startswith("norm"):
        y = rng.choice(["fp32", "bf16"] if op == "norm_backward" else ["fp32", "bf16", "bf16", "q8"])
        width = 64 * _log(rng, 1, 128) if y == "q8" or rng.random() < 0.5 else 8 * _log(rng, 8, 1024)
        return dict(op=op, rows=_log(rng, 1, min(16384, (1 << 25) // width)), width=width,
                    x=rng.choice(["fp32", "fp32", "bf16"]), r=rng.choice(["fp32", "bf16", "none"]), y=y)
    vocab = _log(rng, 500, 160000)
    case = dict(op=op, rows=_log(rng, 1, min(8192, (1 << 28) // vocab)), vocab=vocab,
                pad=rng.choice([0, 0, 0, 1, _log(rng, 2, 128)]), x=rng.choice(["fp32", "bf16"]))
    if op.startswith("logprobs"):
        case["tokens"] = rng.choice([1, 1, 1, 4])
        if op == "logprobs":
            case["top"] = rng.choice([0, 1, 5, 20, 32, 64])
        case["temperature"] = rng.choice([1.0, 1.0, 0.7, 1.3])
        case["masked"] = rng.random() < 0.3
    else:
        case["top"] = _log(rng, 1, 128)
        case["temperature"] = rng.choice([1.0, 2.0, 4.0])
    return case


SIZE = {"fp32": 4, "bf16": 2, "none": 0}


def work(case):
    op, n = case["op"], case["rows"]
    x = SIZE[case["x"]]
    if op == "norm":
        k, r = case["width"], SIZE[case["r"]]
        # 8 bits: the codes written, read back and their values written
        y = 1 + 1 + 2 + 8 / BLOCK if case["y"] == "q8" else SIZE[case["y"]]
        return {"bytes": n * k * (x + 2 * r + y) + 4 * k, "flops": 6 * n * k}
    if op == "norm_backward":
        k, r = case["width"], SIZE[case["r"]]
        h = r or x
        grads = h if x == h else h + x   # one tensor serves both where the types agree
        return {"bytes": n * k * (SIZE[case["y"]] + h + r + grads) + 8 * k, "flops": 12 * n * k}
    v = case["vocab"]
    if op == "logprobs":
        return {"bytes": n * (v * x + 8 * case["tokens"] + 4 + 8 * case["top"]), "flops": 8 * n * v}
    if op == "logprobs_backward":
        return {"bytes": n * (2 * v * x + 8 * case["tokens"] + 16), "flops": 8 * n * v}
    if op == "distill":
        return {"bytes": n * (v * x + 8 * case["top"] + 4), "flops": 5 * n * v}
    live = n - _idle(n)
    return {"bytes": live * (2 * v * x + 8 * case["top"]) + _idle(n) * v * x + 8 * n, "flops": 8 * live * v}


def _idle(rows):
    """Rows of a training batch that carry no weight (padding, prompts)."""
    return rows // 8


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _dtype(name):
    return {"fp32": torch.float32, "bf16": torch.bfloat16}[name]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    s, op, n = dict(case), case["op"], case["rows"]
    if op.startswith("norm"):
        k = case["width"]
        s["w"] = 1 + 0.2 * rand(k)
        loud = 1 + 2.0 * (torch.rand(k, generator=g, device="cuda") < 0.01)     # a few channels carry more
        if op == "norm":
            s["xs"] = (rand(n, k) * 0.5).to(_dtype(case["x"]))
            s["res"] = None if case["r"] == "none" else (rand(n, k) * 1.5 * loud).to(_dtype(case["r"]))
            return s
        s["h"] = (rand(n, k) * 1.5 * loud).to(_dtype(case["x"] if case["r"] == "none" else case["r"]))
        s["dy"] = (rand(n, k) * 0.1).to(_dtype(case["y"]))
        s["dh"] = None if case["r"] == "none" else (rand(n, k) * 0.1).to(s["h"].dtype)
        return s
    v = case["vocab"]
    x = torch.empty(n, v + case["pad"], device="cuda", dtype=_dtype(case["x"]))
    step = max(1, (1 << 27) // (v + case["pad"]))
    for i in range(0, n, step):
        x[i:i + step] = rand(*x[i:i + step].shape).mul_(2.2)
    x = x[:, :v]
    likely = torch.randint(0, v, (n, 6), generator=g, device="cuda")            # what the model is sure of
    x.scatter_(1, likely, (9 + 2.5 * rand(n, 6)).to(x.dtype))
    s["logits"] = x
    if op.startswith("logprobs"):
        if case["masked"]:
            x[:, torch.rand(v, generator=g, device="cuda") < 0.4] = -math.inf
            if n > 1:
                x[n // 2] = -math.inf                                           # nothing is allowed there
        other = torch.randint(0, v, (n, case["tokens"]), generator=g, device="cuda")
        some = torch.rand(n, case["tokens"], generator=g, device="cuda") < 0.7
        s["ids"] = torch.where(some, likely[:, :case["tokens"]], other).to(torch.int32)
        if n > 8:
            s["ids"][::7] = -1                                                  # rows that are not scored
        if case["tokens"] == 1:
            s["ids"] = s["ids"][:, 0].contiguous()
        if op == "logprobs_backward":
            s["dlogp"] = rand(*s["ids"].shape)
            s["dent"] = 0.01 * torch.rand(n, generator=g, device="cuda")
            s["stats"], s["entropy"] = _stats(x, 1 / case["temperature"])
        return s
    # the teacher's top entries among the student's likely tokens and others
    k = case["top"]
    ids = torch.empty(n, k, device="cuda", dtype=torch.int32)
    for i in range(0, n, step):
        noise = x[i:i + step].float()
        noise += rand(*noise.shape)
        ids[i:i + step] = noise.topk(k, -1).indices
    s["teacher"] = torch.gather(x, 1, ids.long()).float() + rand(n, k)
    if n > 4 and k > 2:
        ids[::5, k - k // 3:] = -1                                              # a teacher that kept fewer
    s["ids"] = ids
    if op == "distill_step":
        s["weight"] = torch.full((n,), 1.0 / (n - _idle(n)), device="cuda")
        s["weight"][torch.randperm(n, generator=g, device="cuda")[:_idle(n)]] = 0
    return s


def _stats(x, scale):
    """What the forward pass keeps of each row for the backward pass: fp32 (a, b), the largest logit (-Inf: the row allows
    nothing) and log2 sum exp((x - a) scale), and the entropy."""
    a = x.amax(-1, keepdim=True)
    some = a > -math.inf
    d = (x.double() - torch.where(some, a, 0.0)) * (scale / math.log(2))
    p = torch.exp2(d)
    total = torch.where(some, p.sum(-1, keepdim=True), 1.0)
    b = total.log2()
    entropy = (b - (p * d.clamp(min=-2000.0)).sum(-1, keepdim=True) / total) * math.log(2)
    return torch.cat([a, b], 1).float(), entropy[:, 0].float()


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["op"]
    if own:
        from block_planner_amd import api

        if op == "norm":
            if s["y"] == "q8":
                q, h = api.add_rms_norm_q8(s["xs"], s["w"], s["res"], eps=EPS)
                return api.q8_values(q), h
            return api.add_rms_norm(s["xs"], s["w"], s["res"], eps=EPS, out_dtype=_dtype(s["y"]))
        if op == "norm_backward":
            return api.add_rms_norm_backward(s["dy"], s["h"], s["w"], s["dh"], eps=EPS, x_dtype=_dtype(s["x"]))
        if op == "logprobs":
            r = api.token_logprobs(s["logits"], s["ids"], top=s["top"], temperature=s["temperature"])
            return r.logprobs, r.entropy, r.top_logprobs, r.top_tokens
        if op == "logprobs_backward":
            return api.token_logprobs_backward(s["dlogp"], s["dent"], s["logits"], s["ids"], s["stats"], s["entropy"],
                                               temperature=s["temperature"])
        if op == "distill":
            return api.distill_loss(s["logits"], s["ids"], s["teacher"], temperature=s["temperature"])[0]
        return api.distill_step(s["logits"], s["ids"], s["teacher"], s["weight"], temperature=s["temperature"])
    return {"norm": _norm, "norm_backward": _norm_backward, "logprobs": _logprobs,
            "logprobs_backward": _logprobs_backward, "distill": _distill, "distill_step": _distill_step}[op](s)


def _norm(s):
    h = None if s["res"] is None else (s["xs"].float() + s["res"].float()).to(s["res"].dtype)
    x = (s["xs"] if h is None else h).float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["w"]
    if s["y"] != "q8":
        return y.to(_dtype(s["y"])), h
    b = y.view(y.shape[0], -1, BLOCK)
    e = torch.frexp(b.abs().amax(-1, keepdim=True))[1]
    codes = torch.ldexp(b, 7 - e).round().clamp(-127, 127)
    return torch.ldexp(codes, e - 7).view_as(y).to(torch.bfloat16), h


def _norm_backward(s):
    h, dy = s["h"].float(), s["dy"].float()
    n = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    dw = (dy * n).sum(0, dtype=torch.float64).float()
    g = dy * s["w"]
    d = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * (g - n * (g * n).mean(-1, keepdim=True))
    if s["dh"] is not None:
        d = d + s["dh"].float()
    return d.to(_dtype(s["x"])), d.to(s["h"].dtype), dw


def _order(x):
    """Whole numbers in the order of the floats x (no NaN), a lower index before a higher one among equals."""
    bits = (x + 0.0).view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    return (key << 32) - torch.arange(x.shape[1], device=x.device)


def _logprobs(s):
    x = s["logits"].float()
    top = x.amax(-1, keepdim=True)
    some = top > -math.inf
    d = (x - torch.where(some, top, 0.0)).div_(s["temperature"])
    p = d.exp()
    total = p.sum(-1, keepdim=True)
    log_total = total.log()
    entropy = torch.where(some, log_total - d.clamp_(min=-1e4).mul_(p).sum(-1, keepdim=True) / total, 0.0)[:, 0]

    def logp(at):
        z = (torch.gather(x, 1, at) - torch.where(some, top, 0.0)) / s["temperature"]
        return torch.where(some, z - log_total, -math.inf)

    ids = s["ids"].long().view(x.shape[0], -1)
    given = torch.where(ids >= 0, logp(ids.clamp(min=0)), 0.0).view(s["ids"].shape)
    best = _order(x).topk(s["top"], -1).indices
    return given, entropy, logp(best), best.to(torch.int32)


def _logprobs_backward(s):
    x, t = s["logits"], s["temperature"]
    a, b = s["stats"][:, :1], s["stats"][:, 1:]
    some = a > -math.inf
    logp = ((x.double() - torch.where(some, a, 0.0)) / t - b.double() * math.log(2)).float()
    ids = s["ids"].long().view(x.shape[0], -1)
    g = torch.where(ids >= 0, s["dlogp"].view(x.shape[0], -1), 0.0)
    d = logp.clamp(min=-1e4).add_(s["entropy"][:, None]).mul_(s["dent"][:, None]).add_(g.sum(-1, keepdim=True))
    d = d.mul_(logp.exp_()).neg_()
    d.scatter_add_(1, ids.clamp(min=0), g)
    return (torch.where(some, d, 0.0) / t).to(x.dtype)


def _teacher(s):
    """(p, log p, places) of the entries that count: softmax over a row's kept ones."""
    ids = s["ids"].long()
    z = torch.where(ids >= 0, s["teacher"].float() / s["temperature"], -math.inf)
    z = z - z.amax(-1, keepdim=True)
    p = z.exp()
    total = p.sum(-1, keepdim=True)
    return p / total, z - total.log(), ids.clamp(min=0)


def _student(s):
    x, t = s["logits"].float(), s["temperature"]
    z = (x - x.amax(-1, keepdim=True)).div_(t)
    return z.sub_(z.exp().sum(-1, keepdim=True).log())


def _loss(s, logq):
    p, logp, ids = _teacher(s)
    return torch.where(p > 0, p * (logp - torch.gather(logq, 1, ids)), 0.0).sum(-1)


def _distill(s):
    return _loss(s, _student(s))


def _distill_step(s):
    logq, w = _student(s), s["weight"]
    loss = torch.where(w != 0, _loss(s, logq), 0.0)
    p, _, ids = _teacher(s)
    d = logq.exp_().scatter_add_(1, ids, -p)
    return loss, d.mul_((w / s["temperature"])[:, None]).to(s["logits"].dtype)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op.startswith("norm"):
        return _exact_norm(s) if op == "norm" else _exact_norm_backward(s)
    part = max(1, (1 << 26) // case["vocab"])
    by_row = [k for k, v in s.items() if isinstance(v, torch.Tensor)]
    rows = [_EXACT[op]({k: v[i:i + part] if k in by_row else v for k, v in s.items()})
            for i in range(0, case["rows"], part)]
    joined = tuple(torch.cat(r) for r in zip(*rows))
    return joined if len(joined) > 1 else joined[0]


def _exact_norm(s):
    h = None if s["res"] is None else s["xs"].double() + s["res"].double()
    x = s["xs"].double() if h is None else h.to(s["res"].dtype).double()
    y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * s["w"].double()
    if s["y"] == "q8":
        b = y.unflatten(-1, (-1, BLOCK))
        step = torch.exp2(torch.floor(torch.log2(b.abs().amax(-1, keepdim=True))) - 6)
        y = ((b / step).round().clamp(-127, 127) * step).flatten(-2)
    return y, h


def _exact_norm_backward(s):
    h, g, w = s["h"].double(), s["dy"].double(), s["w"].double()
    k = h.shape[-1]
    r = 1 / torch.sqrt((h * h).sum(-1, keepdim=True) / k + EPS)
    dw = (g * h * r).sum(0)
    g = g * w
    d = r * g - r ** 3 * h * (g * h).sum(-1, keepdim=True) / k
    if s["dh"] is not None:
        d += s["dh"].double()
    return d, d, dw


def _exact_rows(s):
    """(log softmax, rows that allow something)"""
    z = s["logits"].double() / s["temperature"]
    some = (z > -math.inf).any(-1, keepdim=True)
    return torch.where(some, torch.log_softmax(torch.where(some, z, 0.0), -1), -math.inf), some


def _exact_logprobs(s):
    logp, some = _exact_rows(s)
    p = logp.exp()
    entropy = -torch.where(p > 0, p * logp, 0.0).sum(-1)
    ids = s["ids"].long()
    given = torch.gather(logp, 1, ids.clamp(min=0).view(len(ids), -1)).view(ids.shape)
    given = torch.where(ids < 0, 0.0, given)
    best = torch.sort(s["logits"].float(), dim=-1, descending=True, stable=True).indices[:, :s["top"]]
    return given, entropy, torch.gather(logp, 1, best), best.int()


def _exact_logprobs_backward(s):
    logp, some = _exact_rows(s)
    p = logp.exp()
    plogp = torch.where(p > 0, p * logp, 0.0)
    entropy = -plogp.sum(-1, keepdim=True)
    ids = s["ids"].long().view(len(p), -1)
    g = (s["dlogp"].double().view(ids.shape) * (ids >= 0))
    one = torch.zeros_like(p).scatter_add_(1, ids.clamp(min=0), g)
    d = one - p * g.sum(-1, keepdim=True) - s["dent"].double()[:, None] * (plogp + p * entropy)
    return (torch.where(some, d, 0.0) / s["temperature"],)


def _exact_teacher(s):
    """The teacher's distribution, laid out over the vocabulary."""
    keep = s["ids"] >= 0
    p = torch.softmax(torch.where(keep, s["teacher"].double() / s["temperature"], -math.inf), -1)
    return torch.zeros(s["logits"].shape, dtype=torch.float64, device="cuda").scatter_add_(
        1, s["ids"].long().clamp(min=0), p)


def _exact_distill(s):
    logq, _ = _exact_rows(s)
    p = _exact_teacher(s)
    return (torch.where(p > 0, p * (p.log() - logq), 0.0).sum(-1),)


def _exact_distill_step(s):
    logq, _ = _exact_rows(s)
    w = s["weight"].double()
    loss = _exact_distill(s)[0]
    return torch.where(w != 0, loss, 0.0), (logq.exp() - _exact_teacher(s)) * (w / s["temperature"])[:, None]


_EXACT = {"logprobs": _exact_logprobs, "logprobs_backward": _exact_logprobs_backward, "distill": _exact_distill,
          "distill_step": _exact_distill_step}
