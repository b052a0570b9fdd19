"""One draft-verify cycle on device buffers, in C-ABI call order.

Allocation of the caller-owned workspaces and outputs, then the sequence
tree_init -> expand x D -> rerank -> build_tree -> tree_attention -> verify ->
kv_compact. With a KvqCfg the cache is the 8-bit one (the tree's K and V are
stored, attended to and compacted in it), a head given as (codes, scales, group)
is the 4-bit one, and with n_alt the accepted tokens come with their
log-probabilities. Every step runs in libeagle's kernels; this module only
holds buffers and passes pointers.
"""
from __future__ import annotations

import torch

from . import eagle as E


def torch_dtype(code: int) -> torch.dtype:
    return torch.float32 if code == E.EAGLE_F32 else torch.bfloat16


class DeviceCycle:
    """Buffers for one cycle of a (TreeCfg, KvCfg or KvqCfg) problem on one device.

    n_alt: None, or how many alternatives `logprobs` reports per accepted token (0..16)."""

    def __init__(self, cfg: E.TreeCfg, kv: E.KvCfg | E.KvqCfg, device="cuda", fused_head: bool = False,
                 n_alt: int | None = None):
        if n_alt is not None and not 0 <= n_alt <= E.MAX_TOPK:
            raise ValueError(f"DeviceCycle: n_alt {n_alt} is not 0..{E.MAX_TOPK}")
        self.cfg, self.kv = cfg, kv
        self.fused_head = fused_head
        self.quant_kv = isinstance(kv, E.KvqCfg)
        self.n_alt = n_alt
        dev = torch.device(device)
        B, D, k, T, W = cfg.batch, cfg.depth, cfg.top_k, cfg.T, cfg.W
        i32 = dict(dtype=torch.int32, device=dev)
        self.ws = E.alloc_workspace(E.eagle_workspace_bytes(cfg), dev)
        attn_bytes = E.eagle_kvq_attention_workspace_bytes if self.quant_kv else E.eagle_attention_workspace_bytes
        self.attn_ws = E.alloc_workspace(attn_bytes(kv, T), dev)
        self.row_lse = torch.empty(B, D, k, dtype=torch.float32, device=dev)
        self.ftok = torch.empty(B, k, **i32)
        self.fcount = torch.empty(B, **i32)
        self.tokens = torch.empty(B, T, **i32)
        self.parent = torch.empty(B, T, **i32)
        self.depth = torch.empty(B, T, **i32)
        self.pos = torch.empty(B, T, **i32)
        self.mask = torch.empty(B, T, W, **i32)  # uint32 bit rows
        self.n_tree = torch.empty(B, **i32)
        self.attn_out = torch.empty(B, T, kv.n_q_heads, kv.head_dim, dtype=torch_dtype(kv.dtype), device=dev)
        self.accept_len = torch.empty(B, **i32)
        self.slots = torch.empty(B, D + 1, **i32)
        self.out_tokens = torch.empty(B, D + 1, **i32)
        self.new_len = torch.empty(B, **i32)
        if fused_head:  # stage 1 in the LM head's epilogue: per-CTA partials and the merged top-k
            self.lm_scratch = E.alloc_workspace(E.eagle_lmhead_topk_scratch_bytes(cfg), dev)
            self.lm_lse = torch.empty(B * k, dtype=torch.float32, device=dev)
            self.lm_ids = torch.empty(B * k, k, **i32)
            self.lm_vals = torch.empty(B * k, k, dtype=torch.float32, device=dev)
        if n_alt is not None:
            f32 = dict(dtype=torch.float32, device=dev)
            self.logprob = torch.empty(B, D + 1, **f32)
            self.rank = torch.empty(B, D + 1, **i32)
            self.entropy = torch.empty(B, D + 1, **f32)
            self.alt_ids = torch.empty(B, D + 1, n_alt, **i32)
            self.alt_logprobs = torch.empty(B, D + 1, n_alt, **f32)

    # ---- stages -----------------------------------------------------------
    def draft(self, draft_logits: torch.Tensor, stream=None, steps=None, lse_in=None, head=None):
        """Stages 1-3. draft_logits: [D, B, k, V] (one contiguous block per step);
        lse_in: optional [D, B, k] row log-sum-exp supplied from upstream.
        head: optional (weight [V, H], hidden [D, B*k, H]), both bf16: each
        step's rows are then first written into draft_logits[s] by the LM head,
        or, with fused_head, reduced to their lse and top-k in the LM head's
        epilogue and expanded from those (draft_logits unused). A weight given
        as (codes, scales, group) is the 4-bit head of eagle_lmhead_quant: for
        up to 32 rows (24 at H = 8192); past them the 16-bit head takes less time."""
        cfg = self.cfg
        if self.fused_head and head is not None and isinstance(head[0], tuple):
            raise ValueError("DeviceCycle.draft: the 4-bit head has no form with stage 1 in its epilogue (fused_head)")
        E.eagle_tree_init(cfg, self.ws, stream)
        for s in range(cfg.depth if steps is None else steps):
            if head is not None and self.fused_head:
                weight, hidden = head
                self.head_topk(weight, hidden[s], stream)
                E.eagle_expand_topk(cfg, self.ws, s, self.lm_ids, self.lm_vals, self.lm_lse, self.row_lse, self.ftok,
                                    self.fcount, stream)
                continue
            if head is not None:
                weight, hidden = head
                if isinstance(weight, tuple):
                    codes, scales, group = weight
                    E.eagle_lmhead_quant(cfg, self.ws, hidden.shape[-1], group, hidden[s], codes, scales,
                                         draft_logits[s], stream)
                else:
                    E.eagle_lmhead(cfg, self.ws, hidden.shape[-1], hidden[s], weight, draft_logits[s], stream)
            E.eagle_expand(cfg, self.ws, s, draft_logits[s], None if lse_in is None else lse_in[s], self.row_lse,
                           self.ftok, self.fcount, stream)
        if steps is None:
            E.eagle_rerank(cfg, self.ws, stream)

    def head_topk(self, weight, hidden_s, stream=None):
        """LM head of one step with stage 1 in its epilogue (fused_head)."""
        E.eagle_lmhead_topk(self.cfg, self.ws, hidden_s.shape[-1], hidden_s, weight, self.lm_scratch, self.lm_lse,
                            self.lm_ids, self.lm_vals, stream)

    def build(self, prefix_len, root_token, stream=None):
        E.eagle_build_tree(self.cfg, self.ws, prefix_len, root_token, self.tokens, self.parent, self.depth, self.pos,
                           self.mask, self.n_tree, stream)

    def _need_quant_kv(self):
        if not self.quant_kv:
            raise ValueError("DeviceCycle.store: only the 8-bit cache (a KvqCfg) is written here")

    def store(self, k, v, cache, layer, prefix_len, stream=None):
        """The tree's K and V of a layer into the 8-bit cache: k, v [B, T, Hkv, 128] bf16, tree slot j
        of a sequence at position prefix_len + j (slots past n_tree are not written)."""
        kv = self.kv
        self._need_quant_kv()
        E.eagle_kvq_store(kv, layer, self.cfg.T, k, v, kv.n_kv_heads * kv.head_dim, None, prefix_len, self.n_tree,
                          *cache, ws=self.ws, stream=stream)

    def attention(self, q, cache, layer, prefix_len, stream=None):
        """cache: the 16-bit cache's tensor, or the 8-bit cache's (codes, scales)."""
        if self.quant_kv:
            codes, scales = cache
            E.eagle_kvq_tree_attention(self.kv, self.cfg.T, q, codes, scales, layer, prefix_len, self.mask,
                                       self.n_tree, self.attn_out, self.attn_ws, stream)
            return
        E.eagle_tree_attention(self.kv, self.cfg.T, q, cache, layer, prefix_len, self.mask, self.n_tree,
                               self.attn_out, self.attn_ws, stream)

    def verify(self, mode, temperature, target, seed, cycle, stream=None):
        """Stage 6; lossless uniforms are Philox words of (seed, cycle) drawn on the device."""
        E.eagle_verify(self.cfg, self.ws, mode, temperature, seed, cycle, target, self.tokens, self.parent,
                       self.n_tree, self.accept_len, self.slots, self.out_tokens, stream=stream)

    def logprobs(self, target, temperature=1.0, stream=None):
        """Log-probability, rank, entropy and n_alt alternatives of the accepted tokens and the bonus (after verify)."""
        if self.n_alt is None:
            raise ValueError("DeviceCycle.logprobs: the cycle was made without log-probabilities (n_alt)")
        cfg = self.cfg
        E.eagle_token_logprobs(cfg, self.ws, cfg.batch, cfg.depth + 1, cfg.T, target, temperature, self.slots,
                               self.out_tokens, self.n_alt, self.logprob, self.rank, self.entropy,
                               self.alt_ids if self.n_alt else None, self.alt_logprobs if self.n_alt else None, stream)

    def compact(self, cache, prefix_len, stream=None):
        if self.quant_kv:
            codes, scales = cache
            E.eagle_kvq_compact(self.kv, codes, scales, prefix_len, self.accept_len, self.slots, self.cfg.depth + 1,
                                self.new_len, self.ws, stream)
            return
        E.eagle_kv_compact(self.kv, cache, prefix_len, self.accept_len, self.slots, self.cfg.depth + 1, self.new_len,
                           self.ws, stream)

    def run(self, draft_logits, prefix_len, root_token, q, cache, layer, target, seed, cycle, mode, temperature=1.0,
            compact=True, stream=None, head=None, new_kv=None):
        """The whole cycle (all stages) enqueued on `stream`. new_kv: optional (k, v) of the tree's
        slots, stored in the 8-bit cache first. Log-probabilities are at the verification's temperature (greedy: 1)."""
        if new_kv is not None:
            self._need_quant_kv()  # before the first launch
        self.draft(draft_logits, stream, head=head)
        self.build(prefix_len, root_token, stream)
        if new_kv is not None:
            self.store(*new_kv, cache, layer, prefix_len, stream)
        self.attention(q, cache, layer, prefix_len, stream)
        self.verify(mode, temperature, target, seed, cycle, stream)
        if self.n_alt is not None:
            self.logprobs(target, 1.0 if mode == E.GREEDY else temperature, stream)
        if compact:
            self.compact(cache, prefix_len, stream)

    def status(self, stream=None) -> int:
        a = E.eagle_status_fetch(self.ws, stream)
        b = E.eagle_status_fetch(self.attn_ws, stream)
        return a or b

