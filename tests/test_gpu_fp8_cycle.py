"""DeviceCycle with the 8-bit head: whole cycles, eager and as one captured graph replayed on another stream, the
head's logits and the tree against 64-bit forms and the oracle; and training on such a cycle's rows."""
import os
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.dirname(__file__))
import oracle  # noqa: E402
import plain64 as P  # noqa: E402
import plain64_fp8 as F  # noqa: E402

pytestmark = pytest.mark.gpu
D = 128


def _bits(x):
    return (np.asarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def _dev(a, dt=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dt is None else t.to(dt)


@pytest.mark.parametrize("B,k,depth,budget,hid,normed", [(1, 4, 3, 12, 256, True), (2, 8, 4, 40, 400, False), (12, 8, 2, 20, 512, True)])
def test_cycles_with_the_8_bit_head(B, k, depth, budget, hid, normed):
    import torch
    from speculative_decoding_dynamic_gb300 import cycle as C, eagle as E
    rng = np.random.default_rng(B + budget)
    V, H = 2000, 2
    cfg = E.TreeCfg(B, V, k, depth, budget, 0.0, E.EAGLE_BF16)
    T = cfg.T
    row = H * D
    kv = E.KvCfg(B, 4, H, D, 1, 200, E.EAGLE_BF16, 2 * 200 * row, 2 * 200 * row, 200 * row, row)
    dc = C.DeviceCycle(cfg, kv, fp8_head=hid)
    weight = P.bf16_round(rng.standard_normal((V, hid)) * 0.1)
    norm = P.bf16_round(1 + 0.2 * rng.standard_normal(hid)) if normed else None
    codes, scales = E.alloc_fp8(V, hid, -(-V // 128))
    E.eagle_linear_fp8_pack(V, hid, _dev(weight, torch.bfloat16), codes, scales)
    head = C.Fp8Head(codes, scales, None if norm is None else _dev(norm, torch.bfloat16), 1e-6)
    w64 = F.dequant_weight(codes.cpu().numpy(), scales.cpu().numpy())
    hidden = torch.empty(depth, B * k, hid, dtype=torch.bfloat16, device="cuda")
    draft = torch.empty(depth, B, k, V, dtype=torch.bfloat16, device="cuda")
    target = torch.empty(B, T, V, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(B, T, 4, D, dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros(B * 2 * 200 * row, dtype=torch.bfloat16, device="cuda")
    L, root = rng.integers(1, 100, B).astype(np.int32), rng.integers(0, V, B).astype(np.int32)
    d_L, d_root = _dev(L), _dev(root)

    def run():
        dc.run(draft, d_L, d_root, q, cache, 0, target, 5, 0, E.GREEDY, 1.0, head=(head, hidden))

    graph, side = None, torch.cuda.Stream()
    for step in range(3):
        x_h = P.bf16_round(rng.standard_normal((depth, B * k, hid)) * 3)
        hidden.copy_(_dev(x_h, torch.bfloat16))
        x_t = P.bf16_round(rng.standard_normal((B, T, V)) * 2)
        target.copy_(_dev(x_t, torch.bfloat16))
        if step == 0:
            run()
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    run()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                graph.replay()
            torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert dc.status() == 0
        for s in range(depth):
            # the rows as the exact norm gives them, coded: a code within half a step (2^-4 of its value, or 2^-17 of
            # its block's largest), the sums' bound and half a bf16 step
            _, y = F.norm_rows(x_h[s], None, norm, float(np.float32(1e-6)), None)
            dy = (2.0 ** -4 + 2.0 ** -18) * np.abs(y) + np.repeat(np.abs(F.blocks(y)).max(2), 128, 1)[:, :hid] * 2.0 ** -17
            want = y @ w64.T
            tol = (dy + hid * 2.0 ** -22 * np.abs(y)) @ np.abs(w64).T
            tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
            assert (np.abs(draft[s].float().cpu().numpy().reshape(B * k, V) - want) <= tol + 1e-30).all(), (step, s)
        t = oracle.Tree(oracle.TreeCfg(B, V, k, depth, budget, 0.0))
        lse = dc.row_lse.cpu().numpy()
        for s in range(depth):
            t.expand(s, _bits(draft[s].float().cpu().numpy()), np.ascontiguousarray(lse[:, s, :]))
        t.rerank()
        tr = t.build_tree(L, root)
        for key in ("tokens", "parent", "depth", "pos", "n_tree"):
            assert (getattr(dc, key).cpu().numpy() == tr[key]).all(), (step, key)
        a, slots, toks, _ = oracle.verify_greedy(_bits(x_t), tr["tokens"], tr["parent"], tr["n_tree"], depth)
        assert (dc.accept_len.cpu().numpy() == a).all() and (dc.out_tokens.cpu().numpy() == toks).all()
    # the last step's rows against a target's lists (its top 8 logits and lse): what the draft is trained on
    rows = B * k
    cfg1 = E.TreeCfg(B, V, k, 1, 1, 0.0, E.EAGLE_BF16)
    ws = E.alloc_workspace(E.eagle_workspace_bytes(cfg1))
    z = draft[-1].float().cpu().numpy().reshape(rows, V).astype(np.float64)
    tgt = (z + rng.standard_normal((rows, V))).astype(np.float32)
    ids = np.argsort(-tgt, axis=1)[:, :8].astype(np.int32)
    tt = np.take_along_axis(tgt, ids.astype(np.int64), 1)
    lse = np.log(np.exp(tgt.astype(np.float64)).sum(1)).astype(np.float32)
    loss, grad = torch.empty(rows, device="cuda"), torch.empty(rows, V, dtype=torch.bfloat16, device="cuda")
    E.eagle_distill_loss(cfg1, ws, rows, 8, draft[-1], _dev(ids), _dev(tt), _dev(lse), 1.0, None, loss, grad)
    assert E.eagle_status_fetch(ws) == 0
    wl, wg, size, gsize = F.distill(z, ids, tt, lse, 1.0, None)
    d = 2.0 ** -24 * (V / 1024 + 64)
    assert np.all(np.abs(loss.cpu().double().numpy() - wl) <= size * 2 * (d + 2.0 ** -20))
    gt = gsize * (d + 2.0 ** -19)
    assert np.all(np.abs(grad.cpu().double().numpy() - wg) <= gt + 2.0 ** -8 * (np.abs(wg) + gt))


def test_the_8_bit_head_is_refused_where_it_has_no_buffers():
    import torch
    from speculative_decoding_dynamic_gb300 import cycle as C, eagle as E
    cfg = E.TreeCfg(1, 128, 2, 1, 2, 0.0, E.EAGLE_BF16)
    kv = E.kvq_contiguous(1, 2, 2, D, 1, 16, 16)
    z = torch.zeros(1, 2, 256, dtype=torch.bfloat16, device="cuda")
    head = C.Fp8Head(*E.alloc_fp8(128, 256, 1))
    for dc in (C.DeviceCycle(cfg, kv), C.DeviceCycle(cfg, kv, fp8_head=512)):
        with pytest.raises(ValueError, match="8-bit rows"):
            dc.draft(None, head=(head, z))
    with pytest.raises(ValueError, match="8-bit head"):
        C.DeviceCycle(cfg, kv, fused_head=True, fp8_head=256).draft(None, head=(head, z))
