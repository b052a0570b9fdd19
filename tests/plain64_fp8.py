"""Plain numpy forms, in 64 bits, of the 8-bit rows and products and of the
distillation loss, written from their definitions in include/eagle.h. Nothing
here calls the library."""
from __future__ import annotations

import numpy as np
from plain64 import E4M3, block_scale

BLOCK = 128


def stride(dim):
    return (dim + 511) // 512 * 4


def norm_rows(x, residual, weight, eps, rounded):
    """(s, y): the row or its sum with the residual as stored (`rounded`: to the rows' type), and what is coded."""
    s = np.asarray(x, np.float64)
    if residual is not None:
        s = rounded(s + np.asarray(residual, np.float64)).astype(np.float64)
    if weight is None:
        return s, s
    return s, s / np.sqrt((s * s).mean(1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def scale_bytes(amax):
    return (np.log2(block_scale(amax)) + 127).astype(np.int64)


def blocks(y):
    """[rows, blocks, 128] of a row matrix, the last block filled with zeros."""
    pad = -y.shape[1] % BLOCK
    return np.pad(y, ((0, 0), (0, pad))).reshape(y.shape[0], -1, BLOCK)


def half_step(v):
    """Half of e4m3's step at the values v (of the binade that holds them)."""
    e = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -9)))
    return 2.0 ** (np.maximum(e, -6) - 4)


def dequant_rows(codes, scales):
    each = np.repeat(scales.astype(np.float64), BLOCK, 1)[:, :codes.shape[1]]
    return E4M3[codes] * 2.0 ** (each - 127)


def dequant_weight(codes, scales):
    each = np.repeat(scales, BLOCK, 0)[:codes.shape[0]]
    return dequant_rows(codes, each)


def distill(z, ids, t, lse, temperature, weight):
    """(loss [n], gradient [n, V], and the quantities that the tests' tolerances are made of)."""
    n, V = z.shape
    loss, grad, size, gsize = np.zeros(n), np.zeros((n, V)), np.zeros(n), np.zeros((n, V))
    for i in range(n):
        w = 1.0 if weight is None else float(weight[i])
        pick = np.nonzero(ids[i] >= 0)[0]
        if w == 0.0 or (lse is None and len(pick) == 0):
            continue
        y = z[i].astype(np.float64) / temperature
        top = y.max()
        e = np.exp(y - top)
        q, lnq = e / e.sum(), y - top - np.log(e.sum())
        at = ids[i][pick]
        lt = t[i][pick].astype(np.float64) / temperature
        if lse is None:
            lnp = lt - lt.max() - np.log(np.exp(lt - lt.max()).sum())
            r = 0.0
        else:
            lnp = lt - float(lse[i])
            r = max(0.0, 1.0 - np.exp(lnp).sum())
        p = np.exp(lnp)
        live = p > 0
        others = np.ones(V, bool)
        others[at] = False
        with np.errstate(invalid="ignore", divide="ignore"):
            loss[i] = (p[live] * (lnp[live] - lnq[at][live])).sum()
            size[i] = (p[live] * (np.abs(lnp[live]) + np.abs(lnq[at][live]))).sum()
            qr = q[others].sum()
            g = (p.sum() + r) * q
            mag = g * (1 + np.abs(np.where(q > 0, lnq, 0)))
            if r > 0 and qr > 0:
                loss[i] += r * (np.log(r) - np.log(qr))
                size[i] += np.abs(np.log(r)) + np.abs(np.log(qr)) + 2
                g[others] -= r * q[others] / qr
                mag[others] += (r + 1) * q[others] / qr * (1 + np.abs(np.where(q > 0, lnq, 0))[others])
        g[at] -= p
        mag[at] += p
        loss[i] *= w
        size[i] = abs(w) * (1 + size[i])
        grad[i], gsize[i] = w / temperature * g, abs(w) / temperature * mag
    return loss, grad, size, gsize
