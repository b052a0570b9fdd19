"""The distillation loss where the draft's probability of the rest is far below
the smallest 32-bit number, and what its rows are refused for.

Tolerances, with d = 2^-24 (V / 1024 + 64) for a sum over the row. The rest is
taken relative to its own largest logit, so with s_j = q_j / q_R an entry of it
is w / T (mass q_j - r s_j): an exponential's argument is rounded three times
(2^-24 of it each) and its result is within 2^-22, r within 2^-21, so each term
is within (d + 2^-19) (1 + |its logarithm|) of itself (r's: of (r + 1) s_j). The
loss is within 2 (d + 2^-20) of the sum of its terms' magnitudes, the logarithms
of r and q_R counted whole for r's error. What is below 2^-126 before the weight
is flushed. A bf16 gradient is rounded once more (2^-8 of the value)."""
import numpy as np
import pytest
import torch
from test_gpu_distill import _case, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E():
    from speculative_decoding_dynamic_gb300 import eagle
    return eagle


def _lse(y):
    m = y.max()
    return m + np.log(np.exp(y - m).sum())


def _far(z, ids, t, lse, T, weight):
    """(loss, gradient, the loss's and the gradient's magnitudes) in 64 bits, probabilities by their logarithms."""
    n, V = z.shape
    loss, size = np.zeros(n), np.zeros(n)
    grad, gsize = np.zeros((n, V)), np.zeros((n, V))
    for i in range(n):
        y = z[i] / T
        lnq = y - _lse(y)
        at = ids[i].astype(np.int64)
        lnp = t[i].astype(np.float64) / T - float(lse[i])
        p = np.exp(lnp)
        r = 1.0 - p.sum()
        others = np.ones(V, bool)
        others[at] = False
        lnqr = _lse(lnq[others])
        assert r > 0
        loss[i] = (p * (lnp - lnq[at])).sum() + r * (np.log(r) - lnqr)
        size[i] = 1 + (p * (np.abs(lnp) + np.abs(lnq[at]))).sum() + abs(np.log(r)) + abs(lnqr) + 2
        mass, q = p.sum() + r, np.exp(lnq)
        lns = lnq - lnqr
        s = np.where(others, np.exp(np.minimum(lns, 0)), 0)
        grad[i] = mass * q - r * s
        grad[i][at] -= p
        gsize[i] = mass * q * (1 + np.abs(lnq)) + (r + 1) * s * (1 + np.abs(lns))
        gsize[i][at] += p * (1 + np.abs(lnp))
    w = np.ones(n) if weight is None else weight.astype(np.float64)
    return w * loss, (w / T)[:, None] * grad, np.abs(w) * size, np.abs(w / T)[:, None] * gsize


def _check(loss, grad, want, V, dt, scale):
    wl, wg, size, gsize = want
    d = 2.0 ** -24 * (V / 1024 + 64)
    assert np.isfinite(loss).all() and np.isfinite(grad).all()
    tol = size * 2 * (d + 2.0 ** -20)
    assert np.all(np.abs(loss - wl) <= tol), (np.abs(loss - wl) / tol).max()
    gt = gsize * (d + 2.0 ** -19) + 2.0 ** -124 * np.maximum(1.0, scale)[:, None]
    gt = gt + (2.0 ** -8 if dt == "bf16" else 2.0 ** -24) * (np.abs(wg) + gt)
    assert np.all(np.abs(grad - wg) <= gt), (np.abs(grad - wg) / gt).max()


# gaps of the logits between the listed ids and the rest in units of the temperature, about: 60 .. 5000
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,V,top,T,gaps,weight", [
    (8, 4096, 8, 1.0, (60, 80, 85, 86, 87, 90, 95, 100), None),
    (4, 4096, 8, 1.0, (300, 1000, 70, 88), 1024.0),
    (6, 65536, 16, 1.0, (75, 80, 84, 86, 100, 1000), 1024.0),
    (6, 4096, 3, 0.2, (13, 15, 16, 17, 20, 60), 3.0),
    (4, 32000, 20, 0.1, (5, 7, 9, 11), 0.25),
    (170, 8192, 8, 0.5, tuple(range(30, 60)), -2.0),
    (3, 4096, 4, 1e5, (10, 8e6, 6e7), None),
    (2, 128256, 1, 2.0, (150, 10000), None)])
def test_rest_far_below_the_list(E, dt, rows, V, top, T, gaps, weight):
    rng, T = np.random.default_rng(rows * 31 + V + top), float(np.float32(T))
    z, ids, t, lse = _case(rng, rows, V, top, "fp32", T, True)
    lse = (lse.astype(np.float64) + 0.5).astype(np.float32)  # the list leaves some 0.4 or more
    zl = z.double().numpy()
    for i in range(rows):
        zl[i, ids[i]] += gaps[i % len(gaps)]
    z = torch.from_numpy(zl).to(torch.bfloat16 if dt == "bf16" else torch.float32)
    w = None if weight is None else np.full(rows, weight, np.float32)
    loss, grad, status = _run(E, z, ids, t, lse, T, w)
    assert status == 0
    _check(loss, grad, _far(z.double().numpy(), ids, t, lse, T, w), V, dt, np.full(rows, abs(weight or 1.0) / T))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,V", [(5, 4096), (3, 65536)])
def test_list_far_below_the_rest(E, dt, rows, V):
    """The other side: the draft rules the listed ids nearly out."""
    rng = np.random.default_rng(V)
    z, ids, t, lse = _case(rng, rows, V, 8, "fp32", 1.0, True)
    zl = z.double().numpy()
    for i in range(rows):
        zl[i, ids[i]] -= (60, 86, 95, 300, 2000)[i]
    z = torch.from_numpy(zl).to(torch.bfloat16 if dt == "bf16" else torch.float32)
    loss, grad, status = _run(E, z, ids, t, lse, 1.0, None)
    assert status == 0
    _check(loss, grad, _far(z.double().numpy(), ids, t, lse, 1.0, None), V, dt, np.ones(rows))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,V", [(4, 4096), (2, 65536)])
def test_rest_ruled_out(E, dt, rows, V):
    """A rest masked with the type's lowest value is one masked with -inf, the same bits; up to 2^20 max(1, T) below the row's
    largest logit it is the draft's own."""
    tt = torch.bfloat16 if dt == "bf16" else torch.float32
    z, ids, t, lse = _case(np.random.default_rng(V + 1), rows, V, 8, dt, 1.0, True)
    lse = lse + np.float32(0.5)
    others = torch.ones(rows, V, dtype=torch.bool).scatter_(1, torch.from_numpy(ids.astype(np.int64)), False)
    out = []
    for mask in (-float("inf"), torch.finfo(tt).min, -1e30, -1.2e6):
        loss, grad, status = _run(E, z.masked_fill(others, mask), ids, t, lse, 1.0, None)
        assert status == 0 and np.isfinite(loss).all() and not grad[others.numpy()].any()
        out.append((loss, grad))
    for loss, grad in out[1:]:
        assert np.array_equal(loss, out[0][0]) and np.array_equal(grad, out[0][1])
    near = z.masked_fill(others, -9e5)
    loss, grad, status = _run(E, near, ids, t, lse, 1.0, None)
    assert status == 0
    _check(loss, grad, _far(near.double().numpy(), ids, t, lse, 1.0, None), V, dt, np.ones(rows))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_rest_far_below_at_the_lowest_temperatures(E, dt):
    """Ordinary logits at T = 1e-6 are millions of temperatures apart. (The target's logits are near 0, so that an lse
    in 32 bits says what its list leaves.)"""
    rows, V, top, T = 4, 8192, 8, float(np.float32(1e-6))
    rng = np.random.default_rng(21)
    z, ids, _, _ = _case(rng, rows, V, top, "fp32", 1.0, True)
    zl = z.double().numpy()
    for i in range(rows):
        zl[i, ids[i]] += (0, 1, 9, 30)[i]
    z = torch.from_numpy(zl).to(torch.bfloat16 if dt == "bf16" else torch.float32)
    t = (-T * 3 * rng.random((rows, top))).astype(np.float32)
    y = t.astype(np.float64) / T
    lse = np.array([_lse(v) + 0.5 for v in y], np.float32)
    w = np.full(rows, 1e-3, np.float32)
    loss, grad, status = _run(E, z, ids, t, lse, T, w)
    assert status == 0
    _check(loss, grad, _far(z.double().numpy(), ids, t, lse, T, w), V, dt, np.full(rows, 1e-3 / T))
