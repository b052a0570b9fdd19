"""Plain numpy forms, in 64 bits, of the 8-bit KV cache's operators, the 4-bit
LM head and the token log-probabilities, written from their definitions in
include/eagle.h. Nothing here calls the library."""
from __future__ import annotations

import numpy as np

D = 128
# ------------------------------------------------------------------ e4m3 ---
_c = np.arange(256)
_e, _f = (_c >> 3) & 15, _c & 7
E4M3 = np.where(_e > 0, (1 + _f / 8.0) * 2.0 ** (_e - 7.0), _f / 8.0 * 2.0 ** -6)
E4M3 = np.where(_c & 128, -E4M3, E4M3)
E4M3[0x7F] = E4M3[0xFF] = np.nan
_POS = E4M3[:0x7F]  # ascending: 0 .. 448


def encode(x):
    """Nearest e4m3 code (ties to even, saturating) of finite doubles."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(_POS, a), 1, len(_POS) - 1)
    lo = hi - 1
    dl, dh = a - _POS[lo], _POS[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def block_scale(amax):
    """Smallest power of two s >= 2^-126 with amax <= 448 s."""
    k = np.ceil(np.log2(np.maximum(amax, 2.0 ** -200) / 448.0))
    k = np.where(448.0 * 2.0 ** (k - 1) >= amax, k - 1, k)
    k = np.where(448.0 * 2.0 ** k < amax, k + 1, k)
    return 2.0 ** np.maximum(k, -126)


def bf16_round(x):
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) >> 16
    return (u.astype(np.uint32) << 16).view(np.float32)


# ----------------------------------------------------------------- cache ---

def views(kv, codes, scales):
    """[B, layers, 2, max_len, H, D] and [B, layers, 2, blocks, H] views of flat arrays."""
    st = np.lib.stride_tricks.as_strided
    return (st(codes, (kv.batch, kv.layers, 2, kv.max_len, kv.n_kv_heads, D),
               (kv.seq_stride, kv.layer_stride, kv.kv_stride, kv.pos_stride, D, 1)),
            st(scales, (kv.batch, kv.layers, 2, kv.n_blocks, kv.n_kv_heads),
               tuple(4 * s for s in (kv.scale_seq_stride, kv.scale_layer_stride, kv.scale_kv_stride,
                                     kv.scale_block_stride, 1))))


def _moved(codes, old, new):
    """Codes from scale `old` to `new` (fp32 ratio, as the definition's product rounds it)."""
    r = (np.float32(old) / np.float32(new)).astype(np.float64)
    return encode(E4M3[codes] * r)


def store(kv, layer, T, k, v, row_start, start, count, codes, scales):
    """k, v: [rows, H, D] float32 holding bf16 values; codes / scales: the views, updated in place."""
    blk = kv.block
    for b in range(kv.batch):
        p, n = int(start[b]), T if count is None else int(count[b])
        r0 = b * T if row_start is None else int(row_start[b])
        if n < 0 or n > T or p < 0 or p + n > kv.max_len or r0 < 0:
            continue
        for w, x in enumerate((k, v)):
            for blkno in range(p // blk, -(-(p + n) // blk) if n else 0):
                lo, hi = max(p, blkno * blk), min(p + n, (blkno + 1) * blk)
                rows = x[r0 + lo - p:r0 + hi - p].astype(np.float64)  # [t, H, D]
                s = block_scale(np.abs(rows).max((0, 2))).astype(np.float32)
                if blkno * blk < p:
                    had = scales[b, layer, w, blkno].copy()
                    s = np.maximum(s, had)
                    for h in range(kv.n_kv_heads):
                        if s[h] > had[h]:
                            old = codes[b, layer, w, blkno * blk:p, h]
                            old[...] = _moved(old, had[h], s[h])
                scales[b, layer, w, blkno] = s
                q = rows.astype(np.float32) / s[None, :, None]
                codes[b, layer, w, lo:hi] = encode(q)


def compact(kv, codes, scales, L, accept, slots):
    """codes / scales: the views, updated in place; returns new_len (None where a sequence is refused)."""
    blk, out = kv.block, []
    for b in range(kv.batch):
        p, a = int(L[b]), int(accept[b])
        path = slots[b]
        if a < 0 or a > 16 or a >= len(path) or p < 0 or p + a >= kv.max_len or \
                any(int(path[j]) < j or p + int(path[j]) >= kv.max_len for j in range(1, a + 1)):
            out.append(None)
            continue
        out.append(p + a + 1)
        pairs = [(p + int(path[j]), p + j) for j in range(1, a + 1) if int(path[j]) > j]
        was_c, was_s = codes[b].copy(), scales[b].copy()
        for src, dst in pairs:
            scales[b][:, :, dst // blk] = np.maximum(scales[b][:, :, dst // blk], was_s[:, :, src // blk])
        moved = {dst for _, dst in pairs}
        for blkno in {d // blk for d in moved}:
            for pos in range(blkno * blk, min((blkno + 1) * blk, p + a + 1)):
                if pos not in moved:
                    grown = scales[b][:, :, blkno] > was_s[:, :, blkno]
                    new = _moved(was_c[:, :, pos], was_s[:, :, blkno][..., None], scales[b][:, :, blkno][..., None])
                    codes[b][:, :, pos] = np.where(grown[..., None], new, was_c[:, :, pos])
        for src, dst in pairs:
            codes[b][:, :, dst] = _moved(was_c[:, :, src], was_s[:, :, src // blk][..., None],
                                         scales[b][:, :, dst // blk][..., None])
    return out


def attention(kv, T, q, codes, scales, layer, L, see, n_tree):
    """q [B, T, Hq, D] (float32 of bf16 values); see [B, T, T] bool or None (chain). Returns (out, tolerance),
    both [B, T, Hq, D]; the tolerance bounds the kernels' documented roundings:
      - the output's own, half a bf16 step: 2^-8 |out|
      - fp16 softmax weights, 2^-11 each, and below fp16's normal range 2^-25 of the largest weight each
      - scores: q within 2^-17 of its row's largest element, fp32 sums of 128 products (2^-23 each,
        truncating), the scaling to the log2 domain and the exponential (2^-20 in all)."""
    Hq, H = kv.n_q_heads, kv.n_kv_heads
    G = Hq // H
    out = np.zeros((kv.batch, T, Hq, D))
    tol = np.zeros_like(out)
    for b in range(kv.batch):
        p, n = int(L[b]), T if n_tree is None else int(n_tree[b])
        if p < 0 or p + T > kv.max_len or n < 1 or n > T:
            continue
        nk = p + n
        blk = np.arange(nk) // kv.block
        vis = np.ones((n, nk), bool)
        vis[:, p:] = np.tril(np.ones((n, n), bool)) if see is None else see[b, :n, :n]
        for h in range(H):
            K, V = (E4M3[codes[b, layer, w, :nk, h]] * scales[b, layer, w, blk, h][:, None].astype(np.float64)
                    for w in (0, 1))
            top = 448.0 * scales[b, layer, 1, blk, h].max()
            for g in range(G):
                x = q[b, :n, h * G + g].astype(np.float64)
                s = np.where(vis, x @ K.T / np.sqrt(D), -np.inf)
                ds = (2.0 ** -17 * np.abs(x).max(1, keepdims=True) * np.abs(K).sum(1)[None] +
                      128 * 2.0 ** -23 * (np.abs(x) @ np.abs(K).T)) / np.sqrt(D) + 2.0 ** -20 * (1 + np.abs(np.where(vis, s, 0)))
                m = s.max(1, keepdims=True)
                live = m[:, 0] > -np.inf
                w = np.exp(s - np.where(live[:, None], m, 0))
                l = w.sum(1, keepdims=True)
                w = np.divide(w, l, out=np.zeros_like(w), where=l > 0)
                o = w @ V
                out[b, :n, h * G + g] = o
                ds = np.where(vis, ds, 0)
                tol[b, :n, h * G + g] = 2.0 ** -8 * np.abs(o) + (w * (2.0 ** -11 + 2 * ds + 2 * (w * ds).sum(1, keepdims=True))) @ np.abs(V) \
                    + nk * 2.0 ** -25 * top + 1e-30
    return out, tol


# --------------------------------------------------------------- LM head ---

def unpack_w4(codes, scales, group):
    """[V, H] doubles of codes [V, H/2] and scales [V, H/group]."""
    w = np.empty((codes.shape[0], 2 * codes.shape[1]))
    w[:, 0::2] = (codes & 15) - 8.0
    w[:, 1::2] = (codes >> 4) - 8.0
    return w * np.repeat(scales.astype(np.float64), group, 1)


def pack_w4(weight, group):
    """weight [V, H] float32 of bf16 values -> (codes, scales float32 of bf16 values)."""
    V, H = weight.shape
    x = weight.reshape(V, H // group, group)
    s = bf16_round(np.abs(x).max(2) / np.float32(7))
    q = np.divide(x, s[..., None], out=np.zeros_like(x), where=s[..., None] > 0)
    c = (8 + np.clip(np.rint(q), -7, 7)).astype(np.uint8).reshape(V, H)
    return c[:, 0::2] | (c[:, 1::2] << 4), s


# ------------------------------------------------------------- log-probs ---

def logprobs(x, tok, temperature, k):
    """One row of doubles -> (logprob, rank, entropy, ids, logprobs of the ids)."""
    x = np.asarray(x, np.float64)
    z = (x - x.max()) / temperature
    e = np.exp(z)
    lse = np.log(e.sum())
    y = z - lse
    p = e / e.sum()
    ent = -(p * np.where(p > 0, y, 0.0)).sum()
    ids = np.lexsort((np.arange(len(x)), -x))
    return y[tok], int(np.nonzero(ids == tok)[0][0]), ent, ids[:k], y[ids[:k]]
