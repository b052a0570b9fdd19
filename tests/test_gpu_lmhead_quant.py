"""The LM head with 4-bit weights on the GPU against 64-bit sums of the exact
weights, and the packer bit for bit.

The products of bf16 hidden entries and integer codes are exact; a group's sum
and the groups' scaled sums are fp32 (tensor-core additions may truncate), so
an entry lies within H * 2^-23 * sum |hidden * weight| of the exact sum, plus
half a bf16 step (2^-8) when the output is bf16."""
import numpy as np
import pytest

import plain64 as P

pytestmark = pytest.mark.gpu


def _E():
    from speculative_decoding_dynamic_gb300 import eagle as E
    return E


def _head(E, h, codes, scales, group, out_dtype, extra=0):
    import torch
    M, H = h.shape
    V = codes.shape[0]
    k = next(k for k in range(16, 0, -1) if M % k == 0)
    cfg = E.TreeCfg(M // k, V, k, 1, 1, 0.0, E.EAGLE_BF16 if out_dtype == torch.bfloat16 else E.EAGLE_F32)
    ws = E.alloc_workspace(E.eagle_workspace_bytes(cfg))
    out = torch.full((M + extra, V), 7.0, dtype=out_dtype, device="cuda")
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    E.eagle_lmhead_quant(cfg, ws, H, group, dev(h).to(torch.bfloat16), dev(codes), dev(scales).to(torch.bfloat16), out)
    torch.cuda.synchronize()
    assert E.eagle_status_fetch(ws) == 0
    return out.double().cpu().numpy()


@pytest.mark.parametrize("M,V,H,group", [
    (1, 64, 128, 128),           # one slice, four warps without work and more
    (8, 1000, 256, 64),          # a vocabulary that ends inside 16 rows
    (10, 2440, 4096, 128),       # two n-tiles, tiles of fewer rows at the end
    (9, 8 * 1217, 1152, 32),     # nine slices: uneven over the warps
    (16, 5000, 5120, 128),       # the widest pass of sixteen rows
    (24, 3000, 2048, 64),        # two passes
    (8, 4096, 8192, 128),        # the widest hidden state
    (17, 1024, 8192, 32),        # three passes of eight rows or fewer
])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_logits_within_the_fp32_bound(M, V, H, group, out):
    import torch
    E = _E()
    rng = np.random.default_rng(M * V + H)
    h = P.bf16_round(rng.standard_normal((M, H)) * 2.0 ** rng.integers(-4, 5, (M, 1)))
    codes = rng.integers(0, 256, (V, H // 2)).astype(np.uint8)  # every code, 0 (-8) among them
    scales = P.bf16_round(rng.uniform(1e-3, 5e-2, (V, H // group)) * np.where(rng.random((V, H // group)) < 0.1, -1, 1))
    scales[:, 0] = 0.0
    w = P.unpack_w4(codes, scales, group)
    want = h.astype(np.float64) @ w.T
    tol = H * 2.0 ** -23 * (np.abs(h).astype(np.float64) @ np.abs(w).T)
    if out == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    got = _head(E, h, codes, scales, group, torch.bfloat16 if out == "bf16" else torch.float32, extra=1)
    bad = np.abs(got[:M] - want) > tol + 1e-30
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5])
    assert (got[M] == 7.0).all()  # the row after the last is untouched


@pytest.mark.parametrize("group", [32, 64, 128])
def test_one_hot_hidden_rows_return_weight_columns(group):
    """Exact: every column of the weight, entry by entry, so no entry or scale is misplaced."""
    import torch
    E = _E()
    rng = np.random.default_rng(group)
    V, H = 264, 256
    codes = rng.integers(0, 256, (V, H // 2)).astype(np.uint8)
    scales = P.bf16_round(rng.uniform(0.01, 1.0, (V, H // group)))
    w = P.unpack_w4(codes, scales, group)
    for at in range(0, H, 16):
        h = np.zeros((16, H), np.float32)
        h[np.arange(16), at + np.arange(16)] = 2.0 ** np.arange(-8, 8)
        got = _head(E, h, codes, scales, group, torch.float32)
        assert (got == (w[:, at:at + 16] * 2.0 ** np.arange(-8, 8)).T.astype(np.float32)).all()


@pytest.mark.parametrize("V,H,group", [(8, 32, 32), (100, 192, 64), (4001, 512, 128), (16, 96, 32)])
def test_pack_is_the_definition_and_near_the_weight(V, H, group):
    import torch
    E = _E()
    rng = np.random.default_rng(V)
    w = P.bf16_round(rng.standard_normal((V, H)) * 0.02)
    w[V // 2, :group] = 0.0
    w[0, :8] = [7, -7, 3.5, -3.5, 2.5, 0.5, -0.5, 1.5]  # ties: scale 1 where the rest is small
    w[0, 8:group] = 0.0
    codes = torch.full((V + 1, H // 2), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((V + 1, H // group), 9.0, dtype=torch.bfloat16, device="cuda")
    E.eagle_lmhead_quant_pack(V, H, group, torch.from_numpy(w).cuda().to(torch.bfloat16), codes, scales)
    wc, ws = P.pack_w4(w, group)
    assert (codes[:V].cpu().numpy() == wc).all() and (codes[V] == 0x55).all()
    assert (scales[:V].float().cpu().numpy() == ws).all() and (scales[V] == 9.0).all()
    # half a step of the scale, and the largest entry's share of the scale's own rounding (2^-8 of 7 steps)
    back = P.unpack_w4(wc, ws, group)
    step = np.repeat(ws, group, 1)
    assert (np.abs(back - w) <= (0.5 + 7 * 2.0 ** -8) * step).all()


def test_draft_step_on_the_packed_head():
    """Pack, head and expansion in a row (what a draft step calls), in a captured graph."""
    import torch
    E = _E()
    rng = np.random.default_rng(3)
    B, k, V, H = 2, 4, 2048, 512
    cfg = E.TreeCfg(B, V, k, 2, 8, 0.0, E.EAGLE_F32)
    ws = E.alloc_workspace(E.eagle_workspace_bytes(cfg))
    w = torch.from_numpy(P.bf16_round(rng.standard_normal((V, H)) * 0.05)).cuda().to(torch.bfloat16)
    h = P.bf16_round(rng.standard_normal((B * k, H)))
    codes = torch.empty(V, H // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(V, H // 64, dtype=torch.bfloat16, device="cuda")
    logits = torch.zeros(B * k, V, device="cuda")
    lse = torch.empty(B, 2, k, device="cuda")
    ftok = torch.empty(B, k, dtype=torch.int32, device="cuda")
    fcount = torch.empty(B, dtype=torch.int32, device="cuda")
    dh = torch.from_numpy(h).cuda().to(torch.bfloat16)

    def step():
        E.eagle_lmhead_quant_pack(V, H, 64, w, codes, scales)
        E.eagle_tree_init(cfg, ws)
        E.eagle_lmhead_quant(cfg, ws, H, 64, dh, codes, scales, logits)
        E.eagle_expand(cfg, ws, 0, logits, None, lse, ftok, fcount)

    step()
    torch.cuda.synchronize()
    logits.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    g.replay()
    torch.cuda.synchronize()
    assert E.eagle_status_fetch(ws) == 0
    x = logits.view(B, k, V)[:, 0].cpu().numpy()
    assert (fcount.cpu().numpy() == k).all()
    for b in range(B):
        assert (ftok[b].cpu().numpy() == np.lexsort((np.arange(V), -x[b]))[:k]).all()


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_a_non_finite_row_is_nan_and_the_others_unharmed(value):
    import torch
    E = _E()
    rng = np.random.default_rng(21)
    M, V, H, group = 10, 640, 512, 64
    h = P.bf16_round(rng.standard_normal((M, H)))
    h[1] *= 2.0 ** 100
    h[2] *= 2.0 ** -120
    h[3, ::2] *= 2.0 ** -20  # entries far below their row's largest stay exact
    h[4] = 0.0
    h[5, 17] = value
    codes = rng.integers(0, 256, (V, H // 2)).astype(np.uint8)
    scales = P.bf16_round(rng.uniform(0.01, 1.0, (V, H // group)))
    w = P.unpack_w4(codes, scales, group)
    got = _head(E, h, codes, scales, group, torch.float32)
    assert np.isnan(got[5]).all()
    keep = [m for m in range(M) if m != 5]
    x = h[keep].astype(np.float64)
    tol = H * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)
    assert (np.abs(got[keep] - x @ w.T) <= tol).all()
    assert (got[4] == 0).all()


def test_rows_whose_plain_sums_overflow():
    """Entries near the largest bf16 number and scales as small: the logits are ordinary, a group's sum of entries is not."""
    import torch
    E = _E()
    rng = np.random.default_rng(22)
    M, V, H, group = 3, 128, 256, 64
    h = P.bf16_round(np.full((M, H), 2.0 ** 127) * rng.choice([1.0, 1.5, -1.0], (M, H), p=[0.6, 0.3, 0.1]))
    codes = rng.integers(0, 256, (V, H // 2)).astype(np.uint8)
    scales = P.bf16_round(2.0 ** -125 * rng.uniform(1.0, 2.0, (V, H // group)))
    w = P.unpack_w4(codes, scales, group)
    got = _head(E, h, codes, scales, group, torch.float32)
    x = h.astype(np.float64)
    assert (np.abs(got - x @ w.T) <= H * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)).all()


@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_tiny_rows_under_huge_scales_and_the_reverse(out):
    """Ordinary logits from hidden entries and scales far from 1, in either direction: nothing on the way overflows."""
    import torch
    E = _E()
    rng = np.random.default_rng(23)
    M, V, H, group = 5, 256, 512, 64
    for e in (-110, -90, -60, 60, 90, 110):
        h = P.bf16_round(rng.standard_normal((M, H)) * 2.0 ** e)
        codes = rng.integers(0, 256, (V, H // 2)).astype(np.uint8)
        scales = P.bf16_round(rng.uniform(1.0, 2.0, (V, H // group)) * 2.0 ** -e)
        w = P.unpack_w4(codes, scales, group)
        got = _head(E, h, codes, scales, group, torch.bfloat16 if out == "bf16" else torch.float32)
        x = h.astype(np.float64)
        tol = H * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)
        if out == "bf16":
            tol = tol + 2.0 ** -8 * (np.abs(x @ w.T) + tol)
        assert (np.abs(got - x @ w.T) <= tol).all(), e


@pytest.mark.parametrize("group", [32, 64, 128])
def test_weights_of_zero_within_the_documented_bound(group):
    """Codes of 8 (weight 0) and next to it under scales that are not 0. A group's products are summed as codes from
    -8 times the sum of its hidden entries on, so the bound counts |c - 8| + 8: every one of the H products and of
    the group's 4 + group / 16 other additions rounds a sum of at most sum |h| (|c - 8| + 8) scale by 2^-23."""
    import torch
    E = _E()
    rng = np.random.default_rng(24)
    M, V, H = 10, 256, 1024
    h = P.bf16_round(rng.standard_normal((M, H)) * 3)
    codes = np.full((V, H // 2), 0x88, np.uint8)
    codes[V // 2:] = rng.choice([0x88, 0x89, 0x78, 0x98], (V - V // 2, H // 2))
    scales = P.bf16_round(rng.uniform(0.01, 1.0, (V, H // group)))
    w = P.unpack_w4(codes, scales, group)
    got = _head(E, h, codes, scales, group, torch.float32)
    x = h.astype(np.float64)
    tol = H * 2.0 ** -23 * (np.abs(x) @ (np.abs(w) + 8 * np.repeat(scales.astype(np.float64), group, 1)).T)
    assert (np.abs(got - x @ w.T) <= tol).all()


@pytest.mark.parametrize("M,H,group", [(16, 5504, 128), (16, 5248, 32), (16, 5376, 64), (16, 5632, 128), (12, 7296, 128),
                                       (9, 8192, 64), (17, 5504, 128)])
def test_passes_at_the_limits_of_shared_memory(M, H, group):
    """The widest hidden states of a pass of nine to sixteen rows, and those beyond it."""
    import torch
    E = _E()
    rng = np.random.default_rng(M + H)
    V = 152 * 16 + 40
    h = P.bf16_round(rng.standard_normal((M, H)))
    codes = rng.integers(0, 256, (V, H // 2)).astype(np.uint8)
    scales = P.bf16_round(rng.uniform(1e-3, 5e-2, (V, H // group)))
    w = P.unpack_w4(codes, scales, group)
    got = _head(E, h, codes, scales, group, torch.float32, extra=1)
    x = h.astype(np.float64)
    tol = H * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)
    assert (np.abs(got[:M] - x @ w.T) <= tol).all() and (got[M] == 7.0).all()
