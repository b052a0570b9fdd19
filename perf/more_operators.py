"""Operators of the draft's head in 8 bits and of its training, and what they cost.

Three operators: the residual's addition with the root-mean-square norm and an
output of 8-bit codes with a scale for each 128 entries (rmsnorm_fp8), the
product of such rows with weights of 8-bit codes and a scale for each block of
128 x 128 (linear_fp8: an LM head, a draft layer's projections), and the loss
that trains a draft on its target's top logits with its gradient
(distill_loss).

``run`` computes them in elementary torch operations in 32 bits, or, with
``own``, through the package's entry points. ``exact`` is the definition in 64
bits, written separately. Run from the repository's root.
"""
import math
import random

import numpy as np
import torch

own = False
DEV = "cuda"
BLOCK = 128  # entries (of a row), or rows and entries (of a weight), that share a scale
FP8_MAX = 448.0  # largest e4m3 value
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------- cases ---

def listed():
    return [
        # the frontier rows of one sequence's draft step, before the LM head: latency
        {"name": "norm 8B b1", "op": "rmsnorm_fp8", "rows": 10, "dim": 4096, "dtype": "bf16", "residual": True},
        # every slot of a batch's draft trees, before a projection or the target's head
        {"name": "norm trees 13B b64", "op": "rmsnorm_fp8", "rows": 3904, "dim": 5120, "dtype": "bf16", "residual": True},
        # a prompt's tokens in 32 bits, no residual
        {"name": "norm prompt 70B fp32", "op": "rmsnorm_fp8", "rows": 8001, "dim": 8192, "dtype": "fp32", "residual": False},
        # a projection of a draft layer for a single token: latency and the weight's bytes
        {"name": "projection one token", "op": "linear_fp8", "rows": 1, "out": 6144, "in": 4096, "dtype": "bf16"},
        # the draft's LM head at batch 1: ten frontier rows against the whole vocabulary
        {"name": "head 8B b1", "op": "linear_fp8", "rows": 10, "out": 128256, "in": 4096, "dtype": "bf16"},
        # the draft's LM head for the frontier rows of 64 sequences
        {"name": "head 8B b64", "op": "linear_fp8", "rows": 640, "out": 128256, "in": 4096, "dtype": "bf16"},
        # the target's LM head for the trees of eight sequences, logits in 32 bits
        {"name": "head trees 70B b8", "op": "linear_fp8", "rows": 520, "out": 128256, "in": 8192, "dtype": "fp32"},
        # a draft layer's wide projection for the tokens of a training batch or of prompts (a ragged number)
        {"name": "projection prompts", "op": "linear_fp8", "rows": 4001, "out": 14336, "in": 4096, "dtype": "bf16"},
        # the frontier rows of one draft step, the target's top 16 logits beside them, the rest as one bucket: latency
        {"name": "distill 8B b1", "op": "distill_loss", "rows": 10, "vocab": 128256, "dtype": "bf16", "top": 16,
         "rest": True, "temperature": 1.0},
        # a batch's draft rows
        {"name": "distill 8B b64", "op": "distill_loss", "rows": 640, "vocab": 128256, "dtype": "bf16", "top": 16,
         "rest": True, "temperature": 1.0},
        # a training batch of whole sequences, logits in 32 bits, a longer list taken for the whole distribution
        {"name": "distill 13B sequences", "op": "distill_loss", "rows": 4096, "vocab": 32000, "dtype": "fp32", "top": 64,
         "rest": False, "temperature": 2.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rmsnorm_fp8", "linear_fp8", "linear_fp8", "distill_loss"])
    dtype = rng.choice(["bf16", "fp32"])
    if op == "rmsnorm_fp8":
        dim = 16 * _log(rng, 1, 1024)
        rows = min(_log(rng, 1, 16384), 8001 * 8192 // dim)
        return {"op": op, "rows": rows, "dim": dim, "dtype": dtype, "residual": rng.random() < 0.6}
    if op == "linear_fp8":
        out, inner = _log(rng, 8, 128256), 16 * _log(rng, 2, 1024)
        inner = min(inner, 128256 * 8192 // out // 16 * 16)
        rows = max(1, min(_log(rng, 1, 4096), 520 * 128256 * 8192 // (out * inner)))
        return {"op": op, "rows": rows, "out": out, "in": inner, "dtype": dtype}
    vocab = rng.choice([32000, 128256, 8 * _log(rng, 16, 16000)])
    rows = min(_log(rng, 1, 4096), 4096 * 32000 * 4 // (vocab * (2 if dtype == "bf16" else 4)))
    return {"op": op, "rows": rows, "vocab": vocab, "dtype": dtype, "top": _log(rng, 1, 128), "rest": rng.random() < 0.5,
            "temperature": rng.choice([1.0, round(rng.uniform(0.5, 4.0), 2)])}


# ------------------------------------------------------------------ inputs ---

def _blocks(n):
    return -(-n // BLOCK)


def _stride(n):
    """Scales of a row: one for each 128 entries, rows padded to a multiple of four."""
    return -(-_blocks(n) // 4) * 4


def _normal_codes(n, g):
    """Codes of normal entries whose blocks' largest are near the type's largest value."""
    codes = torch.empty(n, dtype=torch.uint8, device=DEV)
    step = 1 << 28
    for at in range(0, n, step):
        m = min(step, n - at)
        x = torch.randn(m, device=DEV, generator=g) * 100
        codes[at:at + m] = x.clamp_(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": c}
    n = c["rows"]
    dt = DTYPES[c["dtype"]]
    if c["op"] == "rmsnorm_fp8":
        D = c["dim"]
        spread = torch.exp(torch.randn(D, device=DEV, generator=g))  # some channels are far larger than others
        s["x"] = (torch.randn(n, D, device=DEV, generator=g) * spread).to(dt)
        if c["residual"]:
            s["residual"] = (torch.randn(n, D, device=DEV, generator=g) * 4 * spread).to(dt)
            s["sum"] = torch.empty_like(s["x"])
        s["weight"] = (1 + 0.2 * torch.randn(D, device=DEV, generator=g)).to(dt)
        s["codes"] = torch.empty(n, D, dtype=torch.uint8, device=DEV)
        s["scales"] = torch.empty(n, _stride(D), dtype=torch.uint8, device=DEV)
    elif c["op"] == "linear_fp8":
        N, K = c["out"], c["in"]
        s["x"], s["w"] = _normal_codes(n * K, g).view(n, K), _normal_codes(N * K, g).view(N, K)
        s["xs"] = torch.randint(127 - 8, 127 - 3, (n, _stride(K)), device=DEV, generator=g).to(torch.uint8)
        s["ws"] = torch.randint(127 - 15, 127 - 12, (_blocks(N), _stride(K)), device=DEV, generator=g).to(torch.uint8)
        s["out"] = torch.empty(n, N, dtype=dt, device=DEV)
    else:
        V, top = c["vocab"], min(c["top"], c["vocab"])
        s["logits"] = torch.empty(n, V, dtype=dt, device=DEV)
        s["ids"] = torch.empty(n, top, dtype=torch.int32, device=DEV)
        s["teacher"] = torch.empty(n, top, device=DEV)
        lse = torch.empty(n, device=DEV)
        step = max(1, (1 << 28) // V)
        for at in range(0, n, step):  # the target's rows: the draft's, off by some noise; one row in eight has no weight
            m = min(step, n - at)
            x = 2.5 * torch.randn(m, V, device=DEV, generator=g)
            s["logits"][at:at + m] = x
            x += 1.2 * torch.randn(m, V, device=DEV, generator=g)
            vals, ids = torch.topk(x, top, dim=1)
            s["ids"][at:at + m], s["teacher"][at:at + m] = ids, vals
            lse[at:at + m] = torch.logsumexp(x / c["temperature"], 1)
            del x
        if c["rest"]:
            s["lse"] = lse
        on = torch.rand(n, device=DEV, generator=g) < 0.875
        s["weight"] = torch.where(on, (0.5 + torch.rand(n, device=DEV, generator=g)) / n, 0.0)
        s["loss"] = torch.empty(n, device=DEV)
        s["grad"] = torch.empty_like(s["logits"])
    if own:  # the workspace that a program keeps beside its buffers: faults found on the device go to its status word
        from speculative_decoding_dynamic_gb300 import eagle as E
        s["E"] = E
        s["cfg"] = E.TreeCfg(1, c.get("vocab", 1024), 1, 1, 1, 0.0, E.EAGLE_BF16 if c["dtype"] == "bf16" else E.EAGLE_F32)
        s["wsp"] = E.alloc_workspace(E.eagle_workspace_bytes(s["cfg"]))
    return s


# -------------------------------------------------------------------- runs ---

def run(s):
    return (_run_own if own else _run_plain)(s)


def _norm_outputs(s):
    """Codes and scales as what they stand for: e4m3 values and powers of two."""
    out = {"codes": s["codes"].view(torch.float8_e4m3fn),
           "scales": s["scales"][:, :_blocks(s["case"]["dim"])].view(torch.float8_e8m0fnu)}
    if "sum" in s:
        out["sum"] = s["sum"]
    return out


def _run_own(s):
    E, c = s["E"], s["case"]
    dt = E.EAGLE_BF16 if c["dtype"] == "bf16" else E.EAGLE_F32
    if c["op"] == "rmsnorm_fp8":
        E.eagle_rmsnorm_fp8(c["rows"], c["dim"], dt, s["x"], c["dim"], s.get("residual"), s.get("sum"), s["weight"], 1e-5,
                            s["codes"], s["scales"], s["wsp"])
        return _norm_outputs(s)
    if c["op"] == "linear_fp8":
        E.eagle_linear_fp8(c["rows"], c["out"], c["in"], s["x"], s["xs"], s["w"], s["ws"], dt, s["out"], s["wsp"])
        return s["out"]
    E.eagle_distill_loss(s["cfg"], s["wsp"], c["rows"], s["ids"].shape[1], s["logits"], s["ids"], s["teacher"], s.get("lse"),
                         c["temperature"], s["weight"], s["loss"], s["grad"])
    return {"loss": s["loss"], "grad": s["grad"]}


def _run_plain(s):
    return {"rmsnorm_fp8": _plain_norm, "linear_fp8": _plain_linear, "distill_loss": _plain_distill}[s["case"]["op"]](s)


def _plain_norm(s):
    c = s["case"]
    n, D = c["rows"], c["dim"]
    x = s["x"].float()
    if c["residual"]:
        s["sum"].copy_(x + s["residual"].float())
        x = s["sum"].float()
    rstd = 1.0 / torch.sqrt(x.double().square().mean(1, keepdim=True) + 1e-5)  # scales turn on it: 64 bits
    y = x * rstd.float() * s["weight"].float()
    y = torch.nn.functional.pad(y, (0, -D % BLOCK)).view(n, -1, BLOCK)
    # the smallest power of two (at least 2^-126) with amax <= 448 of it
    m, e = torch.frexp(y.abs().amax(2))
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(m > 0, e, -126).clamp(min=-126)
    s["scales"].zero_()
    s["scales"][:, :_blocks(D)] = (e + 127).to(torch.uint8)
    q = (y * torch.exp2(-e.double()).float()[..., None]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    s["codes"].copy_(q.view(torch.uint8).view(n, -1)[:, :D])
    return _norm_outputs(s)


def _plain_linear(s):
    c = s["case"]
    N, K = c["out"], c["in"]
    scale = lambda b: torch.exp2(b.float() - 127).repeat_interleave(BLOCK, 1)[:, :K]  # noqa: E731
    x = s["x"].view(torch.float8_e4m3fn).float() * scale(s["xs"])
    w = s["w"].view(torch.float8_e4m3fn).float() * scale(s["ws"]).repeat_interleave(BLOCK, 0)[:N]
    s["out"].copy_(x @ w.t())
    return s["out"]


def _plain_distill(s):
    c = s["case"]
    tau, ids, w = c["temperature"], s["ids"].long(), s["weight"]
    z = s["logits"].float() / tau
    t = s["teacher"] / tau
    t = t - (s["lse"][:, None] if c["rest"] else t.amax(1, keepdim=True))
    p = torch.exp(t)
    if not c["rest"]:
        t = t - torch.log(p.sum(1, keepdim=True))
        p = torch.exp(t)
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    lse = top + torch.log(total)
    loss = (p * (t - (z.gather(1, ids) - lse))).sum(1)
    q = e / total
    if c["rest"]:
        others = e.scatter(1, ids, 0.0)
        left = others.sum(1, keepdim=True)
        r = (1.0 - p.double().sum(1, keepdim=True)).clamp(min=0).float()
        on = (r > 0) & (left > 0)
        loss = loss + torch.where(on, r * (torch.log(r) - torch.log(left / total)), 0.0)[:, 0]
        grad = (p.sum(1, keepdim=True) + r) * q - torch.where(on, r / left, 0.0) * others
    else:
        grad = q
    grad = grad.scatter_add(1, ids, -p)
    s["loss"].copy_(torch.where(w != 0, w * loss, 0.0))
    s["grad"].copy_(torch.where(w[:, None] != 0, grad * (w / tau)[:, None], 0.0))
    return {"loss": s["loss"], "grad": s["grad"]}


# -------------------------------------------------------------------- work ---

def work(c):
    n, es = c["rows"], 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "rmsnorm_fp8":
        D = c["dim"]
        return {"bytes": n * D * (es * (3 if c["residual"] else 1) + 1) + n * _blocks(D) + D * es, "flops": 6 * n * D}
    if c["op"] == "linear_fp8":
        N, K = c["out"], c["in"]
        return {"bytes": N * K + n * K + _blocks(K) * (n + _blocks(N)) + n * N * es, "flops": 2 * n * N * K}
    # a row without weight is written but not read
    return {"bytes": int(n * c["vocab"] * es * 1.875) + n * (8 * c["top"] + 12), "flops": 8 * n * c["vocab"]}


# ------------------------------------------------------------------- exact ---

def exact(case, seed):
    s = prepare(case, seed)
    return {"rmsnorm_fp8": _exact_norm, "linear_fp8": _exact_linear, "distill_loss": _exact_distill}[case["op"]](s, case)


def _decode64(codes):
    """e4m3 codes as doubles: sign, 4 exponent bits (bias 7), 3 fraction bits."""
    c = codes.long()
    e, f = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e > 0, (1 + f / 8) * torch.exp2((e - 7).double()), f / 8 * 2.0 ** -6)
    return torch.where((c & 128) > 0, -mag, mag)


def _round64(x):
    """Doubles rounded to the nearest e4m3 value, ties to even, saturating."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -40))).clamp(min=-6.0)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-FP8_MAX, FP8_MAX)


def _exact_norm(s, c):
    n, D = c["rows"], c["dim"]
    codes = torch.empty(n, D, device=DEV)
    scales = torch.empty(n, _blocks(D), dtype=torch.float64, device=DEV)
    total = torch.empty(n, D, dtype=torch.float64, device=DEV) if c["residual"] else None
    for at in range(0, n, 1024):
        x = s["x"][at:at + 1024].double()
        if c["residual"]:
            x = x + s["residual"][at:at + 1024].double()
            total[at:at + 1024] = x
            x = x.to(s["x"].dtype).double()  # the norm is of the sum as it is stored
        y = x * (x.pow(2).sum(1, keepdim=True) / D + 1e-5).pow(-0.5) * s["weight"].double()
        for b in range(_blocks(D)):
            part = y[:, b * BLOCK:(b + 1) * BLOCK]
            amax = part.abs().max(1, keepdim=True).values
            k = torch.ceil(torch.log2((amax / FP8_MAX).clamp(min=2.0 ** -126)))
            k = torch.where(FP8_MAX * torch.exp2(k - 1) >= amax, k - 1, k)
            k = torch.where(FP8_MAX * torch.exp2(k) < amax, k + 1, k).clamp(min=-126.0)
            scales[at:at + 1024, b] = torch.exp2(k)[:, 0]
            codes[at:at + 1024, b * BLOCK:(b + 1) * BLOCK] = _round64(part / torch.exp2(k)).float()
    out = {"codes": codes, "scales": scales}
    if total is not None:
        out["sum"] = total
    return out


def _exact_linear(s, c):
    N, K = c["out"], c["in"]
    out = torch.empty(c["rows"], N, dtype=torch.float64, device=DEV)
    each = torch.arange(K, device=DEV) // BLOCK
    x = _decode64(s["x"]) * 2.0 ** (s["xs"][:, each].double() - 127)
    for at in range(0, N, 8192):
        rows = torch.arange(at, min(N, at + 8192), device=DEV)
        w = _decode64(s["w"][rows]) * 2.0 ** (s["ws"][rows // BLOCK][:, each].double() - 127)
        out[:, at:at + 8192] = x @ w.t()
    return out


def _exact_distill(s, c):
    n, tau = c["rows"], c["temperature"]
    loss = torch.zeros(n, dtype=torch.float64, device=DEV)
    grad = torch.zeros(n, c["vocab"], dtype=torch.float64, device=DEV)
    for at in range(0, n, 256):
        pick = torch.nonzero(s["weight"][at:at + 256])[:, 0] + at
        if not len(pick):
            continue
        logq = torch.log_softmax(s["logits"][pick].double() / tau, 1)
        ids, w = s["ids"][pick].long(), s["weight"][pick].double()
        t = s["teacher"][pick].double() / tau
        logp = t - s["lse"][pick].double()[:, None] if c["rest"] else torch.log_softmax(t, 1)
        p = logp.exp()
        value = (p * (logp - logq.gather(1, ids))).sum(1)
        slope = torch.zeros_like(logq).scatter_(1, ids, -p)
        if c["rest"]:
            r = (1 - p.sum(1)).clamp(min=0)
            logo = logq.scatter(1, ids, -math.inf)
            logR = torch.logsumexp(logo, 1)
            has = (r > 0) & torch.isfinite(logR)
            value += torch.where(has, r * (r.log() - logR), 0.0)
            slope -= torch.where(has, r, 0.0)[:, None] * torch.where(has[:, None], (logo - logR[:, None]).exp(), 0.0)
            slope += (p.sum(1) + r)[:, None] * logq.exp()
        else:
            slope += logq.exp()
        loss[pick] = w * value
        grad[pick] = slope * (w / tau)[:, None]
    return {"loss": loss, "grad": grad}
