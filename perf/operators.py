"""Operators of a draft-verify cycle on compressed storage, and what they cost.

Five operators: writing K/V into a cache of 8-bit codes with a scale per block
of positions and head (kvq_store), tree-masked attention that reads it
(kvq_attention), the accepted path's move inside it (kvq_compact), an LM head
with 4-bit weights and group scales (lmhead_quant), and the log-probabilities
of given tokens with rank, entropy and top alternatives (token_logprobs).

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
HEADS = {"llama8b": (32, 8), "vicuna13b": (40, 40), "llama70b": (64, 8)}  # query heads, KV heads; head_dim 128
D = 128
FP8_MAX = 448.0  # largest e4m3 value


# ------------------------------------------------------------------- cases ---

def listed():
    return [
        # the tree's keys and values of one layer, written before its attention; ragged prefixes, partial blocks
        {"name": "store tree 8B b64", "op": "kvq_store", "model": "llama8b", "batch": 64, "T": 61, "lo": 256, "hi": 2048,
         "block": 32, "packed": False},
        # prompts of different lengths packed one after the other, written after their projections (MHA)
        {"name": "store prompts 13B", "op": "kvq_store", "model": "vicuna13b", "batch": 5, "T": 4001, "lo": 0, "hi": 0,
         "block": 64, "packed": True},
        # the accepted path of one sequence over a whole model's layers: latency
        {"name": "compact 8B b1", "op": "kvq_compact", "model": "llama8b", "batch": 1, "layers": 32, "T": 61, "lo": 300,
         "hi": 300, "block": 32, "depth": 6},
        # the same for a batch of short chats
        {"name": "compact 8B b64", "op": "kvq_compact", "model": "llama8b", "batch": 64, "layers": 32, "T": 61, "lo": 64,
         "hi": 250, "block": 32, "depth": 6},
        # one new token per sequence (no draft tree), ragged lengths: reading the cache is all there is
        {"name": "decode 8B b64", "op": "kvq_attention", "model": "llama8b", "batch": 64, "T": 1, "lo": 256, "hi": 2048,
         "block": 64},
        # a draft tree of one sequence
        {"name": "tree 8B b1", "op": "kvq_attention", "model": "llama8b", "batch": 1, "T": 61, "lo": 2048, "hi": 2048,
         "block": 64},
        # draft trees of a batch, ragged lengths
        {"name": "tree 8B b64", "op": "kvq_attention", "model": "llama8b", "batch": 64, "T": 61, "lo": 256, "hi": 2048,
         "block": 32},
        # draft trees over long contexts
        {"name": "tree 70B b8 32K", "op": "kvq_attention", "model": "llama70b", "batch": 8, "T": 65, "lo": 32768,
         "hi": 32768, "block": 128},
        # what a server answers with: the accepted tokens of a verified batch, rows picked by the accepted slots
        {"name": "logprobs accepted 8B b64", "op": "token_logprobs", "vocab": 128256, "dtype": "bf16", "seqs": 64,
         "per_seq": 7, "rows": 61, "n_alt": 5, "temperature": 1.0, "slots": True},
        # scoring a prompt: every position of one sequence
        {"name": "logprobs prompt 13B", "op": "token_logprobs", "vocab": 32000, "dtype": "fp32", "seqs": 1,
         "per_seq": 4096, "rows": 4096, "n_alt": 10, "temperature": 0.8, "slots": False},
        # the draft's LM head at batch 1: ten frontier rows against the whole vocabulary
        {"name": "lmhead 8B b1", "op": "lmhead_quant", "vocab": 128256, "hidden": 4096, "rows": 10, "group": 128,
         "dtype": "bf16"},
        # eight frontier rows, the widest hidden state
        {"name": "lmhead 70B b1", "op": "lmhead_quant", "vocab": 128256, "hidden": 8192, "rows": 8, "group": 128,
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["kvq_store", "kvq_compact", "kvq_attention", "kvq_attention", "token_logprobs", "lmhead_quant"])
    model = rng.choice(list(HEADS))
    hkv = HEADS[model][1]
    block = rng.choice([16, 32, 64, 128])
    if op == "kvq_store":
        packed = rng.random() < 0.5
        B = _log(rng, 1, 64)
        most = 20000 * 40 // (B * hkv)  # tokens of a sequence at the largest listed case's cost
        T = min(_log(rng, 1, 4000), max(1, min(most, 20000 // B)))
        lo = 0 if packed else rng.randint(0, 500)
        hi = lo + (0 if packed else rng.randint(0, 1500))
        return {"op": op, "model": model, "batch": B, "T": T, "lo": lo, "hi": hi, "block": block, "packed": packed}
    if op == "kvq_compact":
        B = _log(rng, 1, 64)
        layers = max(1, min(rng.randint(1, 40), 16384 // (B * hkv)))
        lo = rng.randint(0, 100)
        return {"op": op, "model": model, "batch": B, "layers": layers, "T": rng.randint(9, 65), "lo": lo,
                "hi": lo + rng.randint(0, 150), "block": block, "depth": rng.randint(1, 8)}
    if op == "kvq_attention":
        T = rng.choice([1, rng.randint(2, 16), rng.randint(17, 65), rng.randint(66, 200)])
        B = _log(rng, 1, 64)
        hi = _log(rng, 16, 32768)
        cost = 8 * 64 * 65 * 32768 // 4  # query rows x keys, against the largest listed case's
        hi = max(16, min(hi, cost // (B * HEADS[model][0] * T), 2_000_000 // (B * hkv)))
        return {"op": op, "model": model, "batch": B, "T": T, "lo": rng.randint(0, hi), "hi": hi, "block": block}
    if op == "token_logprobs":
        vocab = rng.choice([32000, 128256, 8 * rng.randint(125, 16000)])
        dtype = rng.choice(["bf16", "fp32"])
        slots = rng.random() < 0.5
        seqs = _log(rng, 1, 64) if slots else rng.randint(1, 3)
        per = rng.randint(1, 9) if slots else _log(rng, 1, 1000)
        rows = rng.randint(max(per, 9), 30) if slots else per
        return {"op": op, "vocab": vocab, "dtype": dtype, "seqs": seqs, "per_seq": per, "rows": rows,
                "n_alt": rng.randint(0, 16), "temperature": rng.choice([1.0, round(rng.uniform(0.3, 1.7), 2)]),
                "slots": slots}
    group = rng.choice([32, 64, 128])
    hidden = 128 * rng.randint(2, 64)
    vocab = 8 * rng.randint(500, 128256 // 8)
    return {"op": op, "vocab": vocab, "hidden": hidden, "rows": rng.randint(1, 24), "group": group,
            "dtype": rng.choice(["bf16", "fp32"])}


# ------------------------------------------------------------------ inputs ---

def _spread(lo, hi, n, rng):
    """n lengths spread evenly over [lo, hi], in an order of the seed."""
    return rng.permutation(np.linspace(lo, hi, n).round().astype(np.int64))


def _geometry(c):
    """(B, layers, positions, KV heads, blocks) of the cache of a case."""
    B, layers = c["batch"], c.get("layers", 1)
    most = -(-(c["hi"] + c["T"]) // 64) * 64
    return B, layers, most, HEADS[c["model"]][1], -(-most // c["block"])


def _cache(c, g):
    """A cache in use: every position holds the codes of some normal K/V row, scales of that size."""
    B, layers, most, H, nb = _geometry(c)
    n = B * layers * 2 * most * H * D
    codes = torch.empty(n, dtype=torch.uint8, device=DEV)
    step = 1 << 28
    for at in range(0, n, step):
        m = min(step, n - at)
        x = torch.randn(m, device=DEV, generator=g, dtype=torch.float32)
        codes[at:at + m] = (x * 100).clamp_(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        del x
    scales = torch.exp2(torch.randint(-8, -5, (B, layers, 2, nb, H), device=DEV, generator=g).float())
    return codes.view(B, layers, 2, most, H, D), scales


def _tree(B, T, rng):
    """Random trees of T slots (parents first): [B, T, T] visibility and the packed mask words."""
    see = np.zeros((B, T, T), bool)
    for i in range(T):
        see[:, i, i] = True
        if i:
            p = rng.randint(max(0, i - 12), i, B)
            see[:, i, :] |= see[np.arange(B), p, :]
    W = -(-T // 32)
    bits = np.zeros((B, T, W * 32), np.uint64)
    bits[:, :, :T] = see
    words = (bits.reshape(B, T, W, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
    return see, words.view(np.int32)


def _int(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a).astype(np.int32))).to(DEV)


def _paths(B, n, depth, rng):
    """Accepted slots of each sequence, root first, -1 padding: lengths 0, 1, .., depth in turn, ascending slots."""
    acc = np.arange(B) % (depth + 1)
    slots = np.full((B, depth + 1), -1, np.int64)
    slots[:, 0] = 0
    for b in range(B):
        a = acc[b] = min(acc[b] if B > 1 else depth, n - 1)
        slots[b, 1:a + 1] = np.sort(rng.permutation(n - 1)[:a]) + 1
    return acc, slots


def prepare(case, seed):
    c = dict(case)
    rng = np.random.RandomState(seed % (1 << 31))
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": c}
    op = c["op"]
    if op.startswith("kvq"):
        B, layers, most, H, nb = _geometry(c)
        s["start"] = _int(_spread(c["lo"], c["hi"], B, rng))
        s["codes"], s["scales"] = _cache(c, g)
    if op == "kvq_store":
        count = _spread(max(1, c["T"] // 2), c["T"], B, rng) if c["packed"] else np.full(B, c["T"])
        rows = int(count.sum()) if c["packed"] else B * c["T"]
        first = np.cumsum(count) - count if c["packed"] else np.arange(B) * c["T"]
        s["count"], s["first"] = _int(count), _int(first)
        s["k"], s["v"] = (torch.randn(rows, H, D, device=DEV, generator=g).to(torch.bfloat16) for _ in range(2))
    elif op == "kvq_compact":
        acc, slots = _paths(B, c["T"], c["depth"], rng)
        s["accept"], s["slots"] = _int(acc), _int(slots)
        s["new_len"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    elif op == "kvq_attention":
        Hq, T = HEADS[c["model"]][0], c["T"]
        s["q"] = torch.randn(B, T, Hq, D, device=DEV, generator=g).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        if T > 1:
            see, words = _tree(B, T, rng)
            s["see"], s["mask"], s["n_tree"] = torch.from_numpy(see).to(DEV), _int(words), _int(np.full(B, T))
    elif op == "token_logprobs":
        n, per, rows, V = c["seqs"], c["per_seq"], c["rows"], c["vocab"]
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        s["logits"] = torch.empty(n, rows, V, dtype=dt, device=DEV)
        for b in range(n):
            s["logits"][b] = 2.5 * torch.randn(rows, V, device=DEV, generator=g)
        slots = np.tile(np.arange(per), (n, 1))
        if c["slots"]:
            _, slots = _paths(n, rows, per - 1, rng)
            s["slots"] = _int(slots)
        # half of the tokens are likely ones: the argmax of 64 random candidates
        row = torch.from_numpy(np.maximum(slots, 0)).to(DEV)
        cand = torch.randint(0, V, (n, per, 64), device=DEV, generator=g)
        x = s["logits"].gather(1, row[..., None].expand(n, per, V).long()) if n * per < 600 else s["logits"][:, :per]
        best = cand.gather(2, x.gather(2, cand).float().argmax(2, keepdim=True))[..., 0]
        tokens = torch.where(torch.rand(n, per, device=DEV, generator=g) < 0.5, best, cand[..., 0])
        s["tokens"] = torch.where(torch.from_numpy(slots).to(DEV) >= 0, tokens, -1).to(torch.int32)
        f = dict(dtype=torch.float32, device=DEV)
        i = dict(dtype=torch.int32, device=DEV)
        s["logprob"], s["entropy"], s["rank"] = (torch.empty(n, per, **f), torch.empty(n, per, **f),
                                                 torch.empty(n, per, **i))
        s["alt_ids"], s["alt_logprobs"] = torch.empty(n, per, c["n_alt"], **i), torch.empty(n, per, c["n_alt"], **f)
    else:
        V, H, G, M = c["vocab"], c["hidden"], c["group"], c["rows"]
        s["hidden"] = torch.randn(M, H, device=DEV, generator=g).to(torch.bfloat16)
        s["codes"] = torch.empty(V, H // 2, dtype=torch.uint8, device=DEV)
        for at in range(0, V, 16384):
            m = min(16384, V - at)
            w = (torch.randn(m, H, device=DEV, generator=g) * 2.6).round_().clamp_(-7, 7).to(torch.uint8) + 8
            w &= 15
            s["codes"][at:at + m] = w[:, ::2] | (w[:, 1::2] << 4)
        s["scales"] = (0.0077 * (0.7 + 0.6 * torch.rand(V, H // G, device=DEV, generator=g))).to(torch.bfloat16)
        s["logits"] = torch.empty(M, V, dtype=torch.bfloat16 if c["dtype"] == "bf16" else torch.float32, device=DEV)
    if own:  # the configuration and workspace that a program keeps beside its buffers
        _handles(s)
    return s


def _handles(s):
    from speculative_decoding_dynamic_gb300 import eagle as E
    c = s["case"]
    s["E"] = E
    if c["op"].startswith("kvq"):
        B, layers, most, H, nb = _geometry(c)
        s["kv"] = E.kvq_contiguous(B, HEADS[c["model"]][0], H, D, layers, most, c["block"])
        if c["op"] == "kvq_attention":
            s["ws"] = E.alloc_workspace(E.eagle_kvq_attention_workspace_bytes(s["kv"], c["T"]))
        return
    dt = E.EAGLE_BF16 if c["dtype"] == "bf16" else E.EAGLE_F32
    if c["op"] == "token_logprobs":
        s["cfg"] = E.TreeCfg(1, c["vocab"], 1, 1, 1, 0.0, dt)
    else:
        k = next(k for k in range(16, 0, -1) if c["rows"] % k == 0)
        s["cfg"] = E.TreeCfg(c["rows"] // k, c["vocab"], k, 1, 1, 0.0, dt)
    s["ws"] = E.alloc_workspace(E.eagle_workspace_bytes(s["cfg"]))


# -------------------------------------------------------------------- runs ---

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    E, c = s["E"], s["case"]
    op = c["op"]
    if op == "kvq_store":
        E.eagle_kvq_store(s["kv"], 0, c["T"], s["k"], s["v"], s["k"].stride(0), s["first"], s["start"], s["count"],
                          s["codes"], s["scales"])
        return {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"]}
    if op == "kvq_compact":
        E.eagle_kvq_compact(s["kv"], s["codes"], s["scales"], s["start"], s["accept"], s["slots"], s["slots"].shape[1],
                            s["new_len"])
        return {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"], "new_len": s["new_len"]}
    if op == "kvq_attention":
        E.eagle_kvq_tree_attention(s["kv"], c["T"], s["q"], s["codes"], s["scales"], 0, s["start"], s.get("mask"),
                                   s.get("n_tree"), s["out"], s["ws"])
        return s["out"]
    if op == "token_logprobs":
        E.eagle_token_logprobs(s["cfg"], s["ws"], c["seqs"], c["per_seq"], c["rows"], s["logits"], c["temperature"],
                               s.get("slots"), s["tokens"], c["n_alt"], s["logprob"], s["rank"], s["entropy"],
                               s["alt_ids"], s["alt_logprobs"])
        return {k: s[k] for k in ("logprob", "rank", "entropy", "alt_ids", "alt_logprobs")}
    E.eagle_lmhead_quant(s["cfg"], s["ws"], c["hidden"], c["group"], s["hidden"], s["codes"], s["scales"], s["logits"])
    return s["logits"]


def _run_plain(s):
    return {"kvq_store": _plain_store, "kvq_compact": _plain_compact, "kvq_attention": _plain_attention,
            "token_logprobs": _plain_logprobs, "lmhead_quant": _plain_lmhead}[s["case"]["op"]](s)


def _block_scale(amax):
    """The smallest power of two s (at least 2^-126) with amax <= 448 s."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.exp2(torch.where(amax > 0, e, -126).clamp(min=-126).double()).float()


def _to_codes(x):
    return x.clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _values(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _plain_store(s):
    c = s["case"]
    B, _, most, H, nb = _geometry(c)
    blk = c["block"]
    start, count = s["start"].long(), s["count"].long()
    pos = torch.arange(nb * blk, device=DEV)[None]
    new = (pos >= start[:, None]) & (pos < (start + count)[:, None])  # [B, positions]
    old = (pos >= start[:, None] // blk * blk) & (pos < start[:, None])
    at = (s["first"].long()[:, None] + pos - start[:, None]).clamp(0, s["k"].shape[0] - 1)
    fresh = torch.stack([s["k"], s["v"]])[:, at].float().transpose(0, 1)  # [B, 2, positions, H, D]
    fresh = fresh * new[:, None, :, None, None]
    blocks = lambda x: x.view(B, -1, nb, blk, *x.shape[3:])  # noqa: E731
    need = _block_scale(blocks(fresh).abs().amax((3, 5)))  # [B, 2, nb, H]
    had = s["scales"][:, 0]
    kept = old.view(B, nb, blk).any(2)[:, None, :, None]
    touched = new.view(B, nb, blk).any(2)[:, None, :, None]
    scale = torch.where(kept, torch.maximum(had, need), need)
    scale = torch.where(touched, scale, had)
    each = scale.repeat_interleave(blk, 2)[..., None]
    ratio = (had / scale).repeat_interleave(blk, 2)[:, :, :most, :, None]
    codes = s["codes"][:, 0]
    grown = _to_codes(_values(codes) * ratio)
    pick = lambda m: m[:, None, :most, None, None]  # noqa: E731
    moved = pick(old) & touched.repeat_interleave(blk, 2)[:, :, :most, :, None]
    codes = torch.where(moved, grown, codes)
    codes = torch.where(pick(new), _to_codes(fresh / each)[:, :, :most], codes)
    s["codes"][:, 0] = codes
    s["scales"][:, 0] = scale
    return {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"]}


def _plain_compact(s):
    c = s["case"]
    B, layers, most, H, nb = _geometry(c)
    blk, n = c["block"], s["slots"].shape[1]
    start, slots = s["start"].long(), s["slots"].long()
    j = torch.arange(n, device=DEV)[None]
    moves = (j > 0) & (j <= s["accept"].long()[:, None]) & (slots > j)  # [B, n]
    src = (start[:, None] + slots).clamp(0, most - 1)
    dst = (start[:, None] + j).clamp(0, most - 1)
    b = torch.arange(B, device=DEV)[:, None]
    rows = s["codes"].transpose(1, 3).transpose(2, 3)  # [B, positions, 2, layers, H, D] view: (b, pos) first
    sc = s["scales"].transpose(1, 3).transpose(2, 3)   # [B, blocks, 2, layers, H] view
    take = rows[b, src]                                 # [B, n, 2, layers, H, D]
    s_src = sc[b, src // blk]                           # [B, n, 2, layers, H]
    # the scale of a destination block: its own, or the largest of a row that moves into it
    into = (torch.arange(nb, device=DEV)[None, :, None] == (dst // blk)[:, None]) & moves[:, None]  # [B, nb, n]
    lift = torch.where(into[..., None, None, None], s_src[:, None], 0.0).amax(2)
    new = torch.maximum(sc, lift)
    grown = new > sc
    pos = torch.arange(most, device=DEV)
    in_reach = pos[None] < (start + s["accept"].long() + 1)[:, None]
    lifted = grown[:, pos // blk] & in_reach[:, :, None, None, None]
    ratio = (sc / new)[:, pos // blk][..., None]
    rows.copy_(torch.where(lifted[..., None], _to_codes(_values(rows.contiguous()) * ratio), rows))
    put = _to_codes(_values(take) * (s_src / new[b, dst // blk])[..., None])
    bb, jj = torch.nonzero(moves, as_tuple=True)
    rows[bb, dst[bb, jj]] = put[bb, jj]
    sc.copy_(new)
    s["new_len"].copy_(start + s["accept"].long() + 1)
    return {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"], "new_len": s["new_len"]}


def _plain_attention(s):
    c = s["case"]
    B, _, most, H, nb = _geometry(c)
    T, Hq = c["T"], HEADS[c["model"]][0]
    L = c["hi"] + T  # no sequence has more keys
    each = s["scales"][:, 0].repeat_interleave(c["block"], 2)[:, :, :L, :, None]
    kv = _values(s["codes"][:, 0, :, :L].contiguous()) * each  # [B, 2, L, H, D]
    k, v = kv[:, 0].transpose(1, 2), kv[:, 1].transpose(1, 2)  # [B, H, L, D]
    q = s["q"].float().view(B, T, H, Hq // H, D).permute(0, 2, 1, 3, 4).reshape(B, H, -1, D)
    pos, start = torch.arange(L, device=DEV), s["start"].long()
    slot = pos[None] - start[:, None]  # [B, L]
    see = (slot < 0)[:, None].expand(B, T, L)
    if T == 1:
        see = see | (slot == 0)[:, None]
    else:
        inside = ((slot >= 0) & (slot < T))[:, None]
        see = see | (inside & s["see"].gather(2, slot.clamp(0, T - 1)[:, None].expand(B, T, L)))
    x = (q @ k.transpose(2, 3)) / math.sqrt(D)  # [B, H, T*G, L]
    x = x.view(B, H, T, -1, L).masked_fill(~see[:, None, :, None], -math.inf).view(B, H, -1, L)
    p = torch.exp(x - x.amax(3, keepdim=True))
    o = (p @ v) / p.sum(3, keepdim=True)
    s["out"].copy_(o.view(B, H, T, Hq // H, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D))
    return s["out"]


def _plain_logprobs(s):
    c = s["case"]
    n, per, V = c["seqs"], c["per_seq"], c["vocab"]
    tok = s["tokens"].long()
    slot = s["slots"].long() if c["slots"] else torch.arange(per, device=DEV)[None].expand(n, per)
    live = (tok >= 0) & (slot >= 0)
    b = torch.arange(n, device=DEV)[:, None]
    x = s["logits"][b, slot.clamp(min=0)].float().view(n * per, V)
    t = tok.clamp(min=0).view(-1, 1)
    z = (x - x.amax(1, keepdim=True)) / c["temperature"]
    e = torch.exp(z)
    total = e.sum(1, keepdim=True)
    lse = torch.log(total)
    ent = lse[:, 0] - (e * z).sum(1) / total[:, 0]
    xt = x.gather(1, t)
    rank = ((x > xt) | ((x == xt) & (torch.arange(V, device=DEV) < t))).sum(1)
    vals, ids = torch.sort(x, dim=1, descending=True, stable=True)
    ids, k = ids[:, :c["n_alt"]], c["n_alt"]
    nan = torch.full((), math.nan, device=DEV)
    dead = ~live
    s["logprob"].copy_(torch.where(dead, nan, (z.gather(1, t) - lse).view(n, per)))
    s["entropy"].copy_(torch.where(dead, nan, ent.view(n, per)))
    s["rank"].copy_(torch.where(dead, -1, rank.view(n, per)))
    s["alt_ids"].copy_(torch.where(dead[..., None], -1, ids.view(n, per, k)))
    s["alt_logprobs"].copy_(torch.where(dead[..., None], nan, (z.gather(1, ids) - lse).view(n, per, k)))
    return {k: s[k] for k in ("logprob", "rank", "entropy", "alt_ids", "alt_logprobs")}


def _plain_lmhead(s):
    c = s["case"]
    w = torch.stack([s["codes"] & 15, s["codes"] >> 4], 2).view(c["vocab"], -1, c["group"])
    w = (w.float() - 8.0) * s["scales"].float()[..., None]
    s["logits"].copy_(s["hidden"].float() @ w.view(c["vocab"], -1).t())
    return s["logits"]


# -------------------------------------------------------------------- work ---

def work(c):
    op = c["op"]
    if op == "lmhead_quant":
        V, H, M = c["vocab"], c["hidden"], c["rows"]
        out = 2 if c["dtype"] == "bf16" else 4
        return {"bytes": V * H // 2 + V * H // c["group"] * 2 + M * H * 2 + M * V * out, "flops": 2 * M * V * H}
    if op == "token_logprobs":
        n = c["seqs"] * c["per_seq"]
        if c["slots"]:
            n = sum(1 + min(b % c["per_seq"] if c["seqs"] > 1 else c["per_seq"] - 1, c["rows"] - 1) for b in range(c["seqs"]))
        return {"bytes": n * c["vocab"] * (2 if c["dtype"] == "bf16" else 4) + c["seqs"] * c["per_seq"] * (16 + 8 * c["n_alt"]),
                "flops": 6 * n * c["vocab"]}
    B, layers, most, H, nb = _geometry(c)
    row = H * D
    if op == "kvq_store":
        tokens = sum(np.linspace(max(1, c["T"] // 2), c["T"], B).round()) if c["packed"] else B * c["T"]
        return {"bytes": int(tokens) * 2 * row * 3, "flops": int(tokens) * 2 * row * 3}
    if op == "kvq_compact":
        moved = sum(min(b % (c["depth"] + 1) if B > 1 else c["depth"], c["T"] - 1) for b in range(B))
        return {"bytes": max(1, moved) * layers * 2 * (2 * row + 8 * H), "flops": 0}
    Hq, T = HEADS[c["model"]][0], c["T"]
    lens = np.linspace(c["lo"], c["hi"], B).round()
    keys = int(lens.sum()) + B * T
    pairs = int(lens.sum()) * T + B * T * (T + 1) // 2
    return {"bytes": keys * 2 * (row + H * 4 // c["block"]) + 2 * B * T * Hq * D * 2, "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------- exact ---

def exact(case, seed):
    s = prepare(case, seed)
    return {"kvq_store": _exact_store, "kvq_compact": _exact_compact, "kvq_attention": _exact_attention,
            "token_logprobs": _exact_logprobs, "lmhead_quant": _exact_lmhead}[case["op"]](s, case)


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


def _scale64(amax):
    k = torch.ceil(torch.log2((amax / FP8_MAX).clamp(min=2.0 ** -126)))
    k = torch.where(FP8_MAX * torch.exp2(k - 1) >= amax, k - 1, k)
    k = torch.where(FP8_MAX * torch.exp2(k) < amax, k + 1, k)
    return torch.exp2(k.clamp(min=-126.0))


def _exact_store(s, c):
    blk = c["block"]
    codes = s["codes"].view(torch.float8_e4m3fn).float()
    scales = s["scales"].clone()
    for b, (p, n, at) in enumerate(zip(s["start"].tolist(), s["count"].tolist(), s["first"].tolist())):
        for w, x in enumerate((s["k"], s["v"])):
            x = x[at:at + n].double()  # [n, H, D]
            lo = p // blk * blk
            pad = -(p + n) % blk
            whole = torch.nn.functional.pad(x, (0, 0, 0, 0, p - lo, pad)).view(-1, blk, *x.shape[1:])
            need = _scale64(whole.abs().amax((1, 3)))  # [blocks, H]
            had = scales[b, 0, w, lo // blk:lo // blk + len(need)].double()
            if p > lo:
                need[0] = torch.maximum(need[0], had[0])
                back = _decode64(s["codes"][b, 0, w, lo:p]) * had[0][None, :, None]
                codes[b, 0, w, lo:p] = _round64(back / need[0][None, :, None]).float()
            scales[b, 0, w, lo // blk:lo // blk + len(need)] = need.float()
            q = _round64(whole / need[:, None, :, None])
            codes[b, 0, w, p:p + n] = q.reshape(-1, *x.shape[1:])[p - lo:p - lo + n].float()
    return {"codes": codes, "scales": scales}


def _exact_compact(s, c):
    blk = c["block"]
    codes, scales = s["codes"].view(torch.float8_e4m3fn).float(), s["scales"].double()
    was = scales.clone()
    for b, (p, a) in enumerate(zip(s["start"].tolist(), s["accept"].tolist())):
        path = s["slots"][b].tolist()
        pairs = [(p + path[j], p + j) for j in range(1, a + 1) if path[j] > j]
        for src, dst in pairs:
            scales[b, :, :, dst // blk] = torch.maximum(scales[b, :, :, dst // blk], was[b, :, :, src // blk])
        for blkno in {d // blk for _, d in pairs}:
            lo, hi = blkno * blk, min((blkno + 1) * blk, p + a + 1)
            back = _decode64(s["codes"][b, :, :, lo:hi]) * was[b, :, :, blkno, None, :, None]
            codes[b, :, :, lo:hi] = _round64(back / scales[b, :, :, blkno, None, :, None]).float()
        for src, dst in pairs:
            back = _decode64(s["codes"][b, :, :, src]) * was[b, :, :, src // blk, :, None]
            codes[b, :, :, dst] = _round64(back / scales[b, :, :, dst // blk, :, None]).float()
    return {"codes": codes, "scales": scales.float(), "new_len": None}


def _exact_attention(s, c):
    T, blk = c["T"], c["block"]
    B, H = c["batch"], HEADS[c["model"]][1]
    G = HEADS[c["model"]][0] // H
    out = torch.empty(B, T, H * G, D, dtype=torch.float64, device=DEV)
    for b, L in enumerate(s["start"].tolist()):
        n = L + T
        sc = s["scales"][b, 0].double()
        see = torch.ones(T, n, dtype=torch.bool, device=DEV)
        if T > 1:
            see[:, L:] = s["see"][b]
        for h in range(H):
            per = sc[:, torch.arange(n, device=DEV) // blk, h]  # [2, n]
            k, v = (_decode64(s["codes"][b, 0, w, :n, h]) * per[w][:, None] for w in (0, 1))
            for g in range(G):
                x = s["q"][b, :, h * G + g].double() @ k.t() * D ** -0.5
                x = torch.where(see, x, torch.tensor(-math.inf, device=DEV, dtype=torch.float64))
                out[b, :, h * G + g] = torch.softmax(x, 1) @ v
    return out


def _exact_logprobs(s, c):
    n, per = c["seqs"], c["per_seq"]
    full = dict(fill_value=math.nan, dtype=torch.float64, device=DEV)
    lp, ent = torch.full((n, per), **full), torch.full((n, per), **full)
    alt = torch.full((n, per, c["n_alt"]), **full)
    tok = s["tokens"].tolist()
    for b in range(n):
        slot = s["slots"][b].tolist() if c["slots"] else list(range(per))
        keep = [j for j in range(per) if slot[j] >= 0 and tok[b][j] >= 0]
        for at in range(0, len(keep), 256):
            j = torch.tensor(keep[at:at + 256], device=DEV)
            x = s["logits"][b, torch.tensor([slot[i] for i in keep[at:at + 256]], device=DEV)].double()
            y = torch.log_softmax(x / c["temperature"], 1)
            lp[b, j] = y.gather(1, s["tokens"][b, j].long()[:, None])[:, 0]
            ent[b, j] = -(y.exp() * y).sum(1)
            if c["n_alt"]:
                alt[b, j] = torch.topk(y, c["n_alt"], dim=1).values
    return {"logprob": lp, "rank": None, "entropy": ent, "alt_ids": None, "alt_logprobs": alt}


def _exact_lmhead(s, c):
    out = torch.empty(c["rows"], c["vocab"], dtype=torch.float64, device=DEV)
    h = s["hidden"].double()
    for at in range(0, c["vocab"], 8192):
        b = s["codes"][at:at + 8192].long()
        w = torch.empty(b.shape[0], c["hidden"], dtype=torch.float64, device=DEV)
        w[:, 0::2] = (b % 16 - 8).double()
        w[:, 1::2] = (b // 16 - 8).double()
        w *= s["scales"][at:at + 8192].double().repeat_interleave(c["group"], 1)
        out[:, at:at + 8192] = h @ w.t()
    return out
