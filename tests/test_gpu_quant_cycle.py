"""The 8-bit cache, the 4-bit head and the log-probabilities together, as
DeviceCycle issues them: whole cycles, eager and as one captured graph replayed
on another stream, every stage against the oracle or the plain 64-bit forms."""
import numpy as np
import pytest

import oracle
import plain64 as P

pytestmark = pytest.mark.gpu
D = 128


def _bf16_bits(x):
    return (np.asarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def _dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _dev_bf16(a):
    import torch
    return _dev(np.asarray(a, np.float32)).to(torch.bfloat16)


def _logits(t):
    return t.float().cpu().numpy()


def _see(mask, B, T):
    words = mask.cpu().numpy().view(np.uint32).reshape(B, T, -1)
    return ((words[:, :, np.arange(T) // 32] >> (np.arange(T) % 32)) & 1).astype(bool)


@pytest.mark.parametrize("B,Hq,H,k,depth,budget,block,group,n_alt", [
    (1, 8, 2, 4, 3, 12, 16, 64, 4),     # more than 16 query rows per KV head
    (3, 4, 4, 3, 2, 6, 64, 32, 0),      # seven: the path for few rows; no alternatives
    (2, 32, 8, 8, 5, 60, 32, 128, 16),  # 8B's heads and tree
])
def test_cycles_with_the_quantised_parts(B, Hq, H, k, depth, budget, block, group, n_alt):
    import torch
    from speculative_decoding_dynamic_gb300 import cycle as C, eagle as E
    rng = np.random.default_rng(100 * B + budget)
    V, hid = 2000, 256
    cfg = E.TreeCfg(B, V, k, depth, budget, 0.0, E.EAGLE_BF16)
    T = cfg.T
    kv = E.kvq_contiguous(B, Hq, H, D, 1, 200, block)
    dc = C.DeviceCycle(cfg, kv, n_alt=n_alt)
    codes, scales = E.alloc_kvq(kv)
    L = rng.integers(1, 200 - T - 3 * (depth + 1), B).astype(np.int32)
    root = rng.integers(0, V, B).astype(np.int32)

    # the prompt's K and V, and the head's weight packed on the device
    prompt = [P.bf16_round(rng.standard_normal((int(L.sum()), H, D))) for _ in range(2)]
    first = (np.cumsum(L) - L).astype(np.int32)
    zero = np.zeros(B, np.int32)
    E.eagle_kvq_store(kv, 0, int(L.max()), _dev_bf16(prompt[0]), _dev_bf16(prompt[1]), H * D, _dev(first), _dev(zero),
                      _dev(L), codes, scales, dc.ws)
    weight = P.bf16_round(rng.standard_normal((V, hid)) * 0.1)
    w_codes = torch.empty(V, hid // 2, dtype=torch.uint8, device="cuda")
    w_scales = torch.empty(V, hid // group, dtype=torch.bfloat16, device="cuda")
    E.eagle_lmhead_quant_pack(V, hid, group, _dev_bf16(weight), w_codes, w_scales)
    head = (w_codes, w_scales, group)
    w64 = P.unpack_w4(*P.pack_w4(weight, group), group)

    h_codes, h_scales = np.zeros(codes.numel(), np.uint8), np.zeros(scales.numel(), np.float32)
    vc, vs = P.views(kv, h_codes, h_scales)
    P.store(kv, 0, int(L.max()), *prompt, first, zero, L, vc, vs)

    hidden = torch.empty(depth, B * k, hid, dtype=torch.bfloat16, device="cuda")
    new_k, new_v = (torch.empty(B, T, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.empty(B, T, Hq, D, dtype=torch.bfloat16, device="cuda")
    target = torch.empty(B, T, V, dtype=torch.bfloat16, device="cuda")
    draft = torch.empty(depth, B, k, V, dtype=torch.bfloat16, device="cuda")
    d_L, d_root = _dev(L), _dev(root)

    def run():
        dc.run(draft, d_L, d_root, q, (codes, scales), 0, target, 5, 0, E.GREEDY, 1.0, head=(head, hidden),
               new_kv=(new_k, new_v))

    graph, side = None, torch.cuda.Stream()
    for step in range(3):
        x_h = P.bf16_round(rng.standard_normal((depth, B * k, hid)))
        x_k, x_v = (P.bf16_round(rng.standard_normal((B, T, H, D))) for _ in range(2))
        x_q = P.bf16_round(rng.standard_normal((B, T, Hq, D)) * 2)
        for dst, src in ((hidden, x_h), (new_k, x_k), (new_v, x_v), (q, x_q)):
            dst.copy_(_dev_bf16(src))
        d_L.copy_(_dev(L)), d_root.copy_(_dev(root))
        # a target that likes each slot's first child: paths of some length are accepted
        dc.draft(draft, head=(head, hidden))
        dc.build(d_L, d_root)
        tokens, parent, n = (x.cpu().numpy() for x in (dc.tokens, dc.parent, dc.n_tree))
        x_t = rng.standard_normal((B, T, V)) * 2
        for b in range(B):
            for j in range(int(n[b]) - 1, 0, -1):
                if j % 3:
                    x_t[b, parent[b, j], tokens[b, j]] = 12
        target.copy_(_dev_bf16(P.bf16_round(x_t)))
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

        # the head: the fp32 bound of the exact sums, and half a bf16 step
        for s in range(depth):
            want = x_h[s].astype(np.float64) @ w64.T
            tol = hid * 2.0 ** -23 * (np.abs(x_h[s]).astype(np.float64) @ np.abs(w64).T)
            tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
            assert (np.abs(_logits(draft[s]).reshape(B * k, V) - want) <= tol + 1e-30).all(), (step, s)
        # the tree and the accepted path: the oracle's from the same rows
        t = oracle.Tree(oracle.TreeCfg(B, V, k, depth, budget, 0.0))
        lse = dc.row_lse.cpu().numpy()
        for s in range(depth):
            t.expand(s, _bf16_bits(_logits(draft[s])), np.ascontiguousarray(lse[:, s, :]))
        t.rerank()
        tr = t.build_tree(L, root)
        for key in ("tokens", "parent", "depth", "pos", "n_tree"):
            assert (getattr(dc, key).cpu().numpy() == tr[key]).all(), (step, key)
        x_t = _logits(target)
        a, slots, toks, _ = oracle.verify_greedy(_bf16_bits(x_t), tr["tokens"], tr["parent"], tr["n_tree"], depth)
        assert (dc.accept_len.cpu().numpy() == a).all() and (dc.out_tokens.cpu().numpy() == toks).all()
        assert (dc.slots.cpu().numpy() == slots).all()
        # the cache and the attention over it
        n = tr["n_tree"]
        P.store(kv, 0, T, x_k.reshape(B * T, H, D), x_v.reshape(B * T, H, D), None, L, n, vc, vs)
        want, tol = P.attention(kv, T, x_q, vc, vs, 0, L, _see(dc.mask, B, T), n)
        assert (np.abs(_logits(dc.attn_out) - want) <= tol).all(), step
        # what the server reports of the accepted tokens
        for b in range(B):
            for j in range(depth + 1):
                got = dc.logprob[b, j].item(), dc.rank[b, j].item(), dc.entropy[b, j].item()
                if j > a[b]:
                    assert np.isnan(got[0]) and got[1] == -1 and np.isnan(got[2])
                    continue
                lp, rank, ent, ids, alts = P.logprobs(x_t[b, slots[b, j]], toks[b, j], 1.0, n_alt)
                assert abs(got[0] - lp) <= 2.0 ** -17 + 2.0 ** -22 * abs(lp) and got[1] == rank == 0
                assert abs(got[2] - ent) <= 2.0 ** -16 * (1 + ent)
                assert (dc.alt_ids[b, j].cpu().numpy() == ids).all()
                assert (np.abs(dc.alt_logprobs[b, j].cpu().numpy() - alts) <= 2.0 ** -17 + 2.0 ** -22 * np.abs(alts)).all()
        L = np.array(P.compact(kv, vc, vs, L, a, slots), np.int32)
        assert (dc.new_len.cpu().numpy() == L).all()
        assert (codes.cpu().numpy().ravel() == h_codes).all() and (scales.cpu().numpy().ravel() == h_scales).all(), step
        root = toks[np.arange(B), a].astype(np.int32)


def test_the_fused_head_refuses_the_4_bit_weight():
    import torch
    from speculative_decoding_dynamic_gb300 import cycle as C, eagle as E
    cfg = E.TreeCfg(1, 128, 2, 1, 2, 0.0, E.EAGLE_BF16)
    dc = C.DeviceCycle(cfg, E.kvq_contiguous(1, 2, 2, D, 1, 16, 16), fused_head=True)
    z = torch.zeros(8, device="cuda")
    with pytest.raises(ValueError, match="4-bit head"):
        dc.draft(None, head=((z, z, 32), z))


def test_store_refuses_the_16_bit_cache():
    import torch
    from speculative_decoding_dynamic_gb300 import cycle as C, eagle as E
    cfg = E.TreeCfg(1, 128, 2, 1, 2, 0.0, E.EAGLE_BF16)
    row = 2 * D
    dc = C.DeviceCycle(cfg, E.KvCfg(1, 2, 2, D, 1, 16, E.EAGLE_BF16, 2 * 16 * row, 2 * 16 * row, 16 * row, row))
    z = torch.zeros(8, device="cuda")
    with pytest.raises(ValueError, match="8-bit cache"):
        dc.store(z, z, z, 0, z)
