"""The distillation loss and its gradient against the plain 64-bit form.

Tolerances. An exponential's argument is rounded twice (2^-23 of it) and its
result is within 2^-22; the row's sum adds V / 1024 + 64 roundings of 2^-24 at
most (a thread's sums, then a tree); so with d = 2^-24 (V / 1024 + 64) the lse is
within d + 2^-20, each ln q and q with it (q also by 2^-20 |ln q|), and r within
2^-21. `size` and `gsize` of the plain form collect the terms that these
multiply. A bf16 gradient is rounded once more (2^-8 of the value)."""
import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))
import plain64_fp8 as F  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def E():
    from speculative_decoding_dynamic_gb300 import eagle
    return eagle


def _cfg(E, V, dt):
    return E.TreeCfg(1, V, 1, 1, 1, 0.0, E.EAGLE_BF16 if dt == "bf16" else E.EAGLE_F32)


def _case(rng, rows, V, top, dt, temperature, rest):
    z = (2.5 * rng.standard_normal((rows, V))).astype(np.float32)
    z = torch.from_numpy(z).to(DT[dt])
    target = z.float().numpy() + 1.2 * rng.standard_normal((rows, V)).astype(np.float32)
    ids = np.argsort(-target, axis=1)[:, :top].astype(np.int32)
    t = np.take_along_axis(target, ids.astype(np.int64), 1).astype(np.float32)
    y = target.astype(np.float64) / temperature
    lse = (y.max(1) + np.log(np.exp(y - y.max(1, keepdims=True)).sum(1))).astype(np.float32) if rest else None
    return z, ids, t, lse


def _run(E, z, ids, t, lse, temperature, weight, grad=True, in_place=False):
    rows, V = z.shape
    dt = "bf16" if z.dtype == torch.bfloat16 else "fp32"
    cfg = _cfg(E, V, dt)
    ws = E.alloc_workspace(E.eagle_workspace_bytes(cfg))
    dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    logits = z.cuda().clone()
    loss = torch.full((rows,), 7.0, device="cuda")
    d = logits if in_place else torch.full_like(logits, 7.0) if grad else None
    E.eagle_distill_loss(cfg, ws, rows, ids.shape[1], logits, dev(ids), dev(t), dev(lse), temperature, dev(weight), loss, d)
    status = E.eagle_status_fetch(ws)
    return loss.cpu().double().numpy(), None if d is None else d.cpu().double().numpy(), status


def _check(loss, grad, want, V, dt):
    wl, wg, size, gsize = want
    d = 2.0 ** -24 * (V / 1024 + 64)
    tol = size * 2 * (d + 2.0 ** -20)
    assert np.all(np.abs(loss - wl) <= tol), (np.abs(loss - wl) / np.maximum(tol, 1e-300)).max()
    if grad is None:
        return
    gt = gsize * (d + 2.0 ** -19)
    gt = gt + (2.0 ** -8 if dt == "bf16" else 2.0 ** -24) * (np.abs(wg) + gt) + 1e-37
    assert np.all(np.abs(grad - wg) <= gt), (np.abs(grad - wg) / gt).max()


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("rest", [True, False])
@pytest.mark.parametrize("rows,V,top,temperature", [
    (1, 8, 1, 1.0), (3, 8, 8, 1.0), (5, 136, 16, 2.0), (4, 1024, 256, 0.5), (2, 8192, 3, 4.0), (9, 32000, 16, 1.0),
    (700, 1000, 7, 1.3), (2, 65536, 64, 1.0), (3, 128256, 16, 1.0), (200, 32000, 20, 1.0)])
def test_loss_and_gradient(E, dt, rest, rows, V, top, temperature):
    rng = np.random.default_rng(rows * 7919 + V + top)
    z, ids, t, lse = _case(rng, rows, V, top, dt, temperature, rest)
    weight = (rng.random(rows) * 2 - 0.5).astype(np.float32)
    weight[rng.random(rows) < 0.2] = 0
    loss, grad, status = _run(E, z, ids, t, lse, temperature, weight)
    assert status == 0
    _check(loss, grad, F.distill(z.double().numpy(), ids, t, lse, temperature, weight), V, dt)


@pytest.mark.parametrize("dt,V", [("bf16", 262144), ("fp32", 131072)])
def test_longest_rows(E, dt, V):
    rng = np.random.default_rng(V)
    z, ids, t, lse = _case(rng, 2, V, 32, dt, 1.0, True)
    loss, grad, status = _run(E, z, ids, t, lse, 1.0, None)
    assert status == 0
    _check(loss, grad, F.distill(z.double().numpy(), ids, t, lse, 1.0, None), V, dt)


@pytest.mark.parametrize("rows,V", [(3, 128256), (400, 32000)])
def test_in_place_and_loss_alone(E, rows, V):
    rng = np.random.default_rng(rows)
    z, ids, t, lse = _case(rng, rows, V, 16, "bf16", 1.0, True)
    loss, grad, _ = _run(E, z, ids, t, lse, 1.0, None)
    again, over, _ = _run(E, z, ids, t, lse, 1.0, None, in_place=True)
    alone, none, _ = _run(E, z, ids, t, lse, 1.0, None, grad=False)
    assert none is None and np.array_equal(loss, again) and np.array_equal(loss, alone) and np.array_equal(grad, over)


def test_padding_masks_and_certain_rows(E):
    """Lists with padding, rows without a list, masked logits (-inf, the type's lowest), a draft that is sure of the
    listed ids, one that rules one of them out, a target that is sure."""
    rng = np.random.default_rng(11)
    V, top = 4096, 8
    z, ids, t, lse = _case(rng, 10, V, top, "fp32", 1.0, True)
    z = z.clone()
    ids[0, 2:] = -1
    ids[1, :] = -5
    keep = torch.zeros(V, dtype=torch.bool)
    keep[torch.from_numpy(ids[2].astype(np.int64))] = True
    keep[:100] = True
    z[2, ~keep] = -float("inf")
    z[3, ~keep] = torch.finfo(torch.float32).min
    z[4, torch.from_numpy(ids[4].astype(np.int64))] += 60.0
    z[5, int(ids[5, 1])] = -float("inf")
    t[6, 1:] = -float("inf")
    lse[6] = t[6, 0]
    z[7] = -1e30
    z[7, int(ids[7, 0])] = -1e30 * (1 - 1e-6)
    t[8] = -200.0
    lse[8] = 0.0
    others = torch.ones(V, dtype=torch.bool)
    others[torch.from_numpy(ids[9].astype(np.int64))] = False
    z[9, others] = -float("inf")  # nothing is left outside the list
    for use in (lse, None):
        loss, grad, status = _run(E, z, ids, t, use, 1.0, None)
        assert status == (0 if use is not None else 0)
        with np.errstate(invalid="ignore", over="ignore"):
            want = F.distill(z.double().numpy(), ids, t, use, 1.0, None)
        # the logits of row 7 are 1e24 apart from one another; its exact loss is finite and huge
        fine = [i for i in range(10) if i not in (5, 7)]
        _check(loss[fine], grad[fine], [a[fine] for a in want], V, "fp32")
        assert loss[5] == np.inf and want[0][5] == np.inf
        _check(np.zeros(1), grad[5:6], [np.zeros(1), want[1][5:6], np.zeros(1), want[3][5:6]], V, "fp32")
        assert np.isclose(loss[7], want[0][7], rtol=1e-5) and np.isfinite(grad[7]).all()
        if use is None:
            assert loss[1] == 0 and not grad[1].any()


def test_faults_stay_in_their_rows(E):
    rng = np.random.default_rng(12)
    V, top = 40000, 6
    z, ids, t, lse = _case(rng, 12, V, top, "bf16", 1.0, True)
    clean_loss, clean_grad, _ = _run(E, z, ids, t, lse, 1.0, None)
    bad = {0: "nan", 1: "inf", 2: "none", 3: "list nan", 4: "list inf", 5: "lse", 6: "twice", 7: "far id", 8: "weight"}
    z, weight = z.clone(), np.ones(12, np.float32)
    z[0, 5] = float("nan")
    z[1, 39999] = float("inf")
    z[2] = -float("inf")
    t[3, 2] = np.nan
    t[4, 1] = np.inf
    lse[5] = np.inf
    ids[6, 4] = ids[6, 1]
    ids[7, 0] = V
    weight[8] = np.nan
    for row in bad:
        only = slice(row, row + 1)
        _, _, status = _run(E, z[only], ids[only], t[only], lse[only], 1.0, weight[only])
        assert status == (3 if row in (6, 7) else 1), bad[row]
    loss, grad, status = _run(E, z, ids, t, lse, 1.0, weight)
    assert status in (1, 3)
    assert np.isnan(loss[:9]).all() and not grad[:9].any()
    assert np.array_equal(loss[9:], clean_loss[9:]) and np.array_equal(grad[9:], clean_grad[9:])
    # a row of weight 0 is not looked at
    loss, grad, status = _run(E, z, ids, t, lse, 1.0, np.zeros(12, np.float32))
    assert status == 0 and not loss.any() and not grad.any()


def test_gradient_is_the_difference_of_the_loss(E):
    """Central differences at h = 2^-4: off by h^2 / 6 of the third derivative (below 1 at weight and temperature 1)
    and by two losses' error over 2 h."""
    rng = np.random.default_rng(13)
    V, h = 64, 2.0 ** -4
    z, ids, t, lse = _case(rng, 1, V, 5, "fp32", 1.0, True)
    _, grad, _ = _run(E, z, ids, t, lse, 1.0, None)
    both = z.repeat(2 * V, 1)
    both[torch.arange(V), torch.arange(V)] += h
    both[torch.arange(V) + V, torch.arange(V)] -= h
    rep = lambda a: np.repeat(a, 2 * V, 0)  # noqa: E731
    loss, _, _ = _run(E, both, rep(ids), rep(t), rep(lse), 1.0, None, grad=False)
    size = F.distill(z.double().numpy(), ids, t, lse, 1.0, None)[2]
    tol = h * h / 6 + 2 * size * 2.1 * 2.0 ** -17 / (2 * h)
    assert np.all(np.abs((loss[:V] - loss[V:]) / (2 * h) - grad[0]) <= tol)


def test_captured(E):
    """A graph of the loss and its gradient replayed on other inputs."""
    rng = np.random.default_rng(14)
    V, rows = 32000, 40
    cfg = _cfg(E, V, "bf16")
    ws = E.alloc_workspace(E.eagle_workspace_bytes(cfg))
    z, ids, t, lse = _case(rng, rows, V, 16, "bf16", 1.0, True)
    z2, ids2, t2, lse2 = _case(rng, rows, V, 16, "bf16", 1.0, True)
    dev = [z.cuda(), *(torch.from_numpy(a).cuda() for a in (ids, t, lse))]
    loss, d = torch.empty(rows, device="cuda"), torch.empty_like(dev[0])
    call = lambda: E.eagle_distill_loss(cfg, ws, rows, 16, *dev, 1.0, None, loss, d)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for a, b in zip(dev, (z2, *(torch.from_numpy(a) for a in (ids2, t2, lse2)))):
        a.copy_(b)
    g.replay()
    torch.cuda.synchronize()
    _check(loss.cpu().double().numpy(), d.cpu().double().numpy(), F.distill(z2.double().numpy(), ids2, t2, lse2, 1.0, None), V, "bf16")


def test_list_from_the_target_head(E):
    """A training step's head: the target's list from its fused head (ids, logits, lse), the draft's logits from the
    8-bit head, the loss and the gradient."""
    rng = np.random.default_rng(15)
    rows, V, H, k = 24, 4096, 512, 8
    cfg = E.TreeCfg(3, V, k, 1, 1, 0.0, E.EAGLE_F32)
    ws = E.alloc_workspace(E.eagle_workspace_bytes(cfg))
    weight = (torch.from_numpy(rng.standard_normal((V, H))) * 0.15).bfloat16().cuda()
    hidden = torch.from_numpy(rng.standard_normal((rows, H))).bfloat16().cuda()
    drafted = (hidden.float() + 0.5 * torch.randn(rows, H, device="cuda", generator=torch.Generator("cuda").manual_seed(1))).bfloat16()
    scratch = E.alloc_workspace(E.eagle_lmhead_topk_scratch_bytes(cfg))
    lse, ids, t = torch.empty(rows, device="cuda"), torch.empty(rows, k, dtype=torch.int32, device="cuda"), torch.empty(rows, k, device="cuda")
    E.eagle_lmhead_topk(cfg, ws, H, hidden, weight, scratch, lse, ids, t)
    wc, xc = E.alloc_fp8(V, H, V // 128), E.alloc_fp8(rows, H)
    logits, loss = torch.empty(rows, V, device="cuda"), torch.empty(rows, device="cuda")
    d = torch.empty_like(logits)
    E.eagle_linear_fp8_pack(V, H, weight, *wc)
    E.eagle_rmsnorm_fp8(rows, H, E.EAGLE_BF16, drafted, H, None, None, None, 0.0, *xc, ws)
    E.eagle_linear_fp8(rows, V, H, *xc, *wc, E.EAGLE_F32, logits, ws)
    E.eagle_distill_loss(cfg, ws, rows, k, logits, ids, t, lse, 1.0, None, loss, d)
    assert E.eagle_status_fetch(ws) == 0
    want = F.distill(logits.double().cpu().numpy(), ids.cpu().numpy(), t.cpu().numpy(), lse.cpu().numpy(), 1.0, None)
    _check(loss.cpu().double().numpy(), d.cpu().double().numpy(), want, V, "fp32")
