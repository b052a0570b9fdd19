"""Python binding of libeagle (ctypes). Argument marshalling only.

Every function has the name of the C entry point it calls (see
include/eagle.h for the contract). Tensors are torch CUDA tensors; their data
pointers and the current CUDA stream are passed through. Importing this module
fails loudly if the CUDA library has not been built: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# EAGLE_DEBUG=1: the checked library (each launching call waits and returns
# its own kernels' device status; internal indices range-checked)
DEBUG = os.environ.get("EAGLE_DEBUG", "0") not in ("", "0")
LIB_PATH = os.path.join(_HERE, "libeagle_debug.so" if DEBUG else "libeagle.so")
if not os.path.exists(LIB_PATH):
    raise ImportError(f"{os.path.basename(LIB_PATH)} is missing ({LIB_PATH}); build it with "
                      "`python -m speculative_decoding_dynamic_gb300.build" + (" --debug" if DEBUG else "") +
                      "` (nvcc, sm_103a)")
_lib = ctypes.CDLL(LIB_PATH)

EAGLE_OK = 0
EAGLE_F32, EAGLE_BF16 = 0, 1
GREEDY, LOSSLESS, DRAFT = 0, 1, 2
MAX_TOPK, MAX_DEPTH, MAX_SLOTS, MAX_CANDIDATES = 16, 16, 256, 1024


class EagleError(RuntimeError):
    def __init__(self, fn: str, code: int):
        msg = _lib.eagle_status_string(code).decode()
        if code == -3:  # EAGLE_ERR_LAUNCH: add the CUDA error
            cmsg = ctypes.c_char_p()
            cerr = _lib.eagle_last_cuda_error(ctypes.byref(cmsg))
            msg += f"; CUDA error {cerr}: {cmsg.value.decode() if cmsg.value else ''}"
        super().__init__(f"{fn} -> {code} ({msg})")
        self.code = code


class TreeCfg(ctypes.Structure):
    """eagle_tree_cfg."""
    _fields_ = [("batch", ctypes.c_int), ("vocab", ctypes.c_int), ("top_k", ctypes.c_int), ("depth", ctypes.c_int),
                ("node_budget", ctypes.c_int), ("threshold", ctypes.c_float), ("logit_dtype", ctypes.c_int),
                ("policy", ctypes.c_int)]

    @property
    def T(self) -> int:
        return self.node_budget + 1

    @property
    def W(self) -> int:
        return (self.T + 31) // 32

    @property
    def C(self) -> int:
        return self.top_k + (self.depth - 1) * self.top_k * self.top_k


class KvCfg(ctypes.Structure):
    """eagle_kv_cfg (strides in elements)."""
    _fields_ = [("batch", ctypes.c_int), ("n_q_heads", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("layers", ctypes.c_int), ("max_len", ctypes.c_int),
                ("dtype", ctypes.c_int), ("seq_stride", ctypes.c_int64), ("layer_stride", ctypes.c_int64),
                ("kv_stride", ctypes.c_int64), ("pos_stride", ctypes.c_int64)]


class KvqCfg(ctypes.Structure):
    """eagle_kvq_cfg (strides of codes in bytes, of scales in elements)."""
    _fields_ = [("batch", ctypes.c_int), ("n_q_heads", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("layers", ctypes.c_int), ("max_len", ctypes.c_int),
                ("block", ctypes.c_int), ("dtype", ctypes.c_int), ("seq_stride", ctypes.c_int64),
                ("layer_stride", ctypes.c_int64), ("kv_stride", ctypes.c_int64), ("pos_stride", ctypes.c_int64),
                ("scale_seq_stride", ctypes.c_int64), ("scale_layer_stride", ctypes.c_int64),
                ("scale_kv_stride", ctypes.c_int64), ("scale_block_stride", ctypes.c_int64)]

    @property
    def n_blocks(self) -> int:
        return -(-self.max_len // (self.block or 1))  # a block of 0 is the library's to refuse

    def extent(self, layers: int) -> tuple[int, int]:
        """Bytes of codes and elements of scales that `layers` layers of the cache span."""
        heads, max_len, b, k = self.n_kv_heads, self.max_len, self.batch - 1, layers - 1
        return (b * self.seq_stride + k * self.layer_stride + self.kv_stride + (max_len - 1) * self.pos_stride +
                heads * self.head_dim,
                b * self.scale_seq_stride + k * self.scale_layer_stride + self.scale_kv_stride +
                (-(-max_len // (self.block or 1)) - 1) * self.scale_block_stride + heads)


_p = ctypes.c_void_p
_i = ctypes.c_int
_sz = ctypes.c_size_t
_TP = ctypes.POINTER(TreeCfg)
_KP = ctypes.POINTER(KvCfg)
_QP = ctypes.POINTER(KvqCfg)

_lib.eagle_workspace_bytes.argtypes = [_TP]
_lib.eagle_workspace_bytes.restype = _sz
_lib.eagle_tree_init.argtypes = [_TP, _p, _sz, _p]
_lib.eagle_expand.argtypes = [_TP, _p, _sz, _i, _p, _p, _p, _p, _p, _p]
_lib.eagle_expand_sampled.argtypes = [_TP, _p, _sz, _i, _p, _p, ctypes.c_uint64, ctypes.c_uint64, _p, _p, _p, _p]
_lib.eagle_test_expand_starved.argtypes = [_TP, _p, _sz, _i, _p, _p, _p, _p, _p]
_lib.eagle_lmhead.argtypes = [_TP, _p, _sz, _i, _p, _p, _p, _p]
_lib.eagle_lmhead_topk_scratch_bytes.argtypes = [_TP]
_lib.eagle_lmhead_topk_scratch_bytes.restype = _sz
_lib.eagle_lmhead_topk.argtypes = [_TP, _p, _sz, _i, _p, _p, _p, _sz, _p, _p, _p, _p]
_lib.eagle_rerank.argtypes = [_TP, _p, _sz, _p]
_lib.eagle_tree_value.argtypes = [_TP, _p, _sz, _p, _p]
_lib.eagle_build_tree.argtypes = [_TP, _p, _sz, _p, _p, _p, _p, _p, _p, _p, _p, _p]
_lib.eagle_attention_workspace_bytes.argtypes = [_KP, _i]
_lib.eagle_attention_workspace_bytes.restype = _sz
_lib.eagle_tree_attention.argtypes = [_KP, _i, _p, _p, _i, _p, _p, _p, _p, _p, _sz, _p]
_u64 = ctypes.c_uint64
_lib.eagle_verify.argtypes = [_TP, _p, _sz, _i, ctypes.c_float, _u64, _u64, _p, _p, _p, _p, _p, _p, _p, _p, _p]
_lib.eagle_shard_partials.argtypes = [_TP, _p, _sz, _i, _i, _i, _p, _p, _p, _p]
_lib.eagle_shard_merge.argtypes = [_TP, _p, _sz, _i, _i, _p, _p, _p, _p, _p, _p, _p]
_lib.eagle_expand_topk.argtypes = [_TP, _p, _sz, _i, _p, _p, _p, _p, _p, _p, _p]
_lib.eagle_verify_argmax.argtypes = [_TP, _p, _sz, _p, _p, _p, _p, _p, _p, _p, _p]
_lib.eagle_kv_compact.argtypes = [_KP, _p, _p, _p, _p, _i, _p, _p, _p]
_lib.eagle_verify_static.argtypes = [_TP, _i, ctypes.c_float, _u64, _u64, _p, _p, _p, _p, _p, _p, _p, _p]
_lib.eagle_status_fetch.argtypes = [_p, ctypes.POINTER(ctypes.c_int), _p]
_lib.eagle_tree_export.argtypes = [_TP, _p, _sz, _p, _p, _p, _p, _p, _p, _p, _p]
_lib.eagle_verify_export.argtypes = [_TP, _p, _sz, _p, _p, _p, _p]
_lib.eagle_test_sampling.argtypes = [_p, _p, _i, _p, _p, _p]
_i64 = ctypes.c_int64
_lib.eagle_kvq_store.argtypes = [_QP, _i, _i, _p, _p, _i64, _p, _p, _p, _p, _p, _p, _p]
_lib.eagle_kvq_compact.argtypes = [_QP, _p, _p, _p, _p, _p, _i, _p, _p, _p]
_lib.eagle_kvq_attention_workspace_bytes.argtypes = [_QP, _i]
_lib.eagle_kvq_attention_workspace_bytes.restype = _sz
_lib.eagle_kvq_tree_attention.argtypes = [_QP, _i, _p, _p, _p, _i, _p, _p, _p, _p, _p, _sz, _p]
_lib.eagle_lmhead_quant.argtypes = [_TP, _p, _sz, _i, _i, _p, _p, _p, _p, _p]
_lib.eagle_lmhead_quant_pack.argtypes = [_i, _i, _i, _p, _p, _p, _p]
_lib.eagle_token_logprobs.argtypes = [_TP, _p, _sz, _i, _i, _i, _p, ctypes.c_float, _p, _p, _i, _p, _p, _p, _p, _p, _p]
_lib.eagle_fp8_scale_stride.argtypes = [_i]
_lib.eagle_rmsnorm_fp8.argtypes = [_i, _i, _i, _p, _i64, _p, _p, _p, ctypes.c_float, _p, _p, _p, _p]
_lib.eagle_linear_fp8.argtypes = [_i, _i, _i, _p, _p, _p, _p, _i, _p, _p, _p]
_lib.eagle_linear_fp8_pack.argtypes = [_i, _i, _p, _p, _p, _p]
_lib.eagle_distill_loss.argtypes = [_TP, _p, _sz, _i, _i, _p, _p, _p, _p, ctypes.c_float, _p, _p, _p, _p]
_lib.eagle_kernel_launches.restype = ctypes.c_uint64
_lib.eagle_last_cuda_error.argtypes = [ctypes.POINTER(ctypes.c_char_p)]
_lib.eagle_last_cuda_error.restype = _i
_lib.eagle_status_string.argtypes = [_i]
_lib.eagle_status_string.restype = ctypes.c_char_p


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, rc: int) -> None:
    if rc != EAGLE_OK:
        raise EagleError(fn, rc)


def _ws(ws) -> tuple[int, int]:
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _need(fn: str, name: str, t, dtypes, n: int, dev: int) -> int | None:
    """The address of a tensor argument of `fn`: contiguous, on device `dev` (the current one), of one of `dtypes`, with
    at least n elements (None and raw addresses pass: the library checks what it can of those)."""
    if t is None or type(t) is int:
        return t
    if t.dtype in dtypes and t.get_device() == dev and t.is_contiguous() and t.numel() >= n:
        return t.data_ptr()
    if t.dtype not in dtypes:
        raise ValueError(f"{fn}: {name} is {t.dtype}, not {' or '.join(map(str, dtypes))}")
    if t.get_device() != dev:
        raise ValueError(f"{fn}: {name} is on {t.device}, not on the current CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{fn}: {name} is not contiguous")
    raise ValueError(f"{fn}: {name} has {t.numel()} elements, needs {n}")


def _ws_on(fn: str, ws, dev: int) -> tuple[int | None, int]:
    """Address and bytes of a workspace argument of `fn`, checked like its other tensors (kernels write its status
    word); None and a raw address, as a call that needs the status word alone takes it, have no bytes."""
    if isinstance(ws, torch.Tensor):
        size = ws.element_size()
        return _need(fn, "ws", ws, (ws.dtype,), -(-4 // size), dev), ws.numel() * size
    return (ws, 0) if ws is None or isinstance(ws, int) else _ws(ws)


_get_device = getattr(torch._C, "_cuda_getDevice", None)


def _device() -> int:
    """The current device's index; -2 (no tensor's) before CUDA is initialised."""
    if not torch.cuda.is_initialized():
        return -2
    return _get_device() if _get_device is not None else torch.cuda.current_device()


# the current stream's handle without a stream object around it: a third of a small call's time on the host
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_on(stream, dev: int) -> int | None:
    if stream is None and _raw_stream is not None:
        return _raw_stream(dev)
    return _stream(stream)


_I32 = (torch.int32,)
_W32 = (torch.int32, torch.uint32)
_F32 = (torch.float32,)
_BF16 = (torch.bfloat16,)
_U8 = (torch.uint8,)
_CODES = (torch.uint8, torch.float8_e4m3fn)


def eagle_workspace_bytes(cfg: TreeCfg) -> int:
    return int(_lib.eagle_workspace_bytes(ctypes.byref(cfg)))


def eagle_attention_workspace_bytes(kv: KvCfg, T: int) -> int:
    return int(_lib.eagle_attention_workspace_bytes(ctypes.byref(kv), T))


def alloc_workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """A 256-byte aligned uint8 device tensor (torch allocations are 512-byte aligned)."""
    if nbytes <= 0:
        raise ValueError("invalid configuration (workspace size 0)")
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def eagle_tree_init(cfg, ws, stream=None):
    _check("eagle_tree_init", _lib.eagle_tree_init(ctypes.byref(cfg), *_ws(ws), _stream(stream)))


def eagle_expand(cfg, ws, step, draft_logits, row_lse_in, row_lse, frontier_tokens, frontier_count, stream=None):
    _check("eagle_expand", _lib.eagle_expand(ctypes.byref(cfg), *_ws(ws), step, _ptr(draft_logits),
                                             _ptr(row_lse_in), _ptr(row_lse), _ptr(frontier_tokens),
                                             _ptr(frontier_count), _stream(stream)))


def eagle_expand_sampled(cfg, ws, step, draft_logits, row_lse_in, seed, cycle, row_lse, frontier_tokens,
                         frontier_count, stream=None):
    """Stages 1+2 with the children drawn from each row's softmax without replacement (Gumbel-top-k)."""
    _check("eagle_expand_sampled", _lib.eagle_expand_sampled(ctypes.byref(cfg), *_ws(ws), step, _ptr(draft_logits),
                                                             _ptr(row_lse_in), int(seed), int(cycle), _ptr(row_lse),
                                                             _ptr(frontier_tokens), _ptr(frontier_count),
                                                             _stream(stream)))


def eagle_test_expand_starved(cfg, ws, step, draft_logits, row_lse, frontier_tokens, frontier_count, stream=None):
    """Failure-path test hook: expansion whose row ring receives no copies (status 2 expected)."""
    _check("eagle_test_expand_starved", _lib.eagle_test_expand_starved(ctypes.byref(cfg), *_ws(ws), step,
                                                                       _ptr(draft_logits), _ptr(row_lse),
                                                                       _ptr(frontier_tokens), _ptr(frontier_count),
                                                                       _stream(stream)))


def eagle_lmhead(cfg, ws, hidden_dim, hidden, weight, draft_logits, stream=None):
    _check("eagle_lmhead", _lib.eagle_lmhead(ctypes.byref(cfg), *_ws(ws), hidden_dim, _ptr(hidden), _ptr(weight),
                                             _ptr(draft_logits), _stream(stream)))


def eagle_lmhead_topk_scratch_bytes(cfg: TreeCfg) -> int:
    return int(_lib.eagle_lmhead_topk_scratch_bytes(ctypes.byref(cfg)))


def eagle_lmhead_topk(cfg, ws, hidden_dim, hidden, weight, scratch, row_lse, topk_ids, topk_logits, stream=None):
    _check("eagle_lmhead_topk", _lib.eagle_lmhead_topk(ctypes.byref(cfg), *_ws(ws), hidden_dim, _ptr(hidden),
                                                       _ptr(weight), *_ws(scratch), _ptr(row_lse), _ptr(topk_ids),
                                                       _ptr(topk_logits), _stream(stream)))


def eagle_rerank(cfg, ws, stream=None):
    _check("eagle_rerank", _lib.eagle_rerank(ctypes.byref(cfg), *_ws(ws), _stream(stream)))


def eagle_tree_value(cfg, ws, value_sum, stream=None):
    _check("eagle_tree_value", _lib.eagle_tree_value(ctypes.byref(cfg), *_ws(ws), _ptr(value_sum), _stream(stream)))


def eagle_build_tree(cfg, ws, prefix_len, root_token, tokens, parent, depth, pos_ids, mask, n_tree, stream=None):
    _check("eagle_build_tree", _lib.eagle_build_tree(ctypes.byref(cfg), *_ws(ws), _ptr(prefix_len), _ptr(root_token),
                                                     _ptr(tokens), _ptr(parent), _ptr(depth), _ptr(pos_ids),
                                                     _ptr(mask), _ptr(n_tree), _stream(stream)))


def eagle_tree_attention(kv, T, q, kv_cache, layer, prefix_len, mask, n_tree, out, ws, stream=None):
    _check("eagle_tree_attention", _lib.eagle_tree_attention(ctypes.byref(kv), T, _ptr(q), _ptr(kv_cache), layer,
                                                             _ptr(prefix_len), _ptr(mask), _ptr(n_tree), _ptr(out),
                                                             *_ws(ws), _stream(stream)))


def eagle_verify(cfg, ws, mode, temperature, seed, cycle, target_logits, tokens, parent, n_tree, accept_len,
                 accepted_slots, out_tokens, draft_logits=None, stream=None):
    _check("eagle_verify", _lib.eagle_verify(ctypes.byref(cfg), *_ws(ws), mode, float(temperature), int(seed),
                                             int(cycle), _ptr(target_logits), _ptr(draft_logits), _ptr(tokens),
                                             _ptr(parent), _ptr(n_tree), _ptr(accept_len), _ptr(accepted_slots),
                                             _ptr(out_tokens), _stream(stream)))


def eagle_verify_static(cfg, mode, temperature, seed, cycle, target_logits, tokens, parent, n_tree, accept_len,
                        accepted_slots, out_tokens, stream=None):
    """eagle_verify for callers that may not allocate: scratch lives in a fixed device array of the library."""
    _check("eagle_verify_static", _lib.eagle_verify_static(ctypes.byref(cfg), mode, float(temperature), int(seed),
                                                           int(cycle), _ptr(target_logits), _ptr(tokens),
                                                           _ptr(parent), _ptr(n_tree), _ptr(accept_len),
                                                           _ptr(accepted_slots), _ptr(out_tokens), _stream(stream)))


def eagle_shard_partials(cfg, ws, rows, shard_vocab, vocab_offset, logits, part_max_sum, part_keys, stream=None):
    _check("eagle_shard_partials", _lib.eagle_shard_partials(ctypes.byref(cfg), *_ws(ws), rows, shard_vocab,
                                                             vocab_offset, _ptr(logits), _ptr(part_max_sum),
                                                             _ptr(part_keys), _stream(stream)))


def eagle_shard_merge(cfg, ws, n_shards, rows, part_max_sum, part_keys, row_lse, topk_ids, topk_logits, row_argmax,
                      stream=None):
    _check("eagle_shard_merge", _lib.eagle_shard_merge(ctypes.byref(cfg), *_ws(ws), n_shards, rows,
                                                       _ptr(part_max_sum), _ptr(part_keys), _ptr(row_lse),
                                                       _ptr(topk_ids), _ptr(topk_logits), _ptr(row_argmax),
                                                       _stream(stream)))


def eagle_expand_topk(cfg, ws, step, topk_ids, topk_logits, row_lse_in, row_lse, frontier_tokens, frontier_count,
                      stream=None):
    _check("eagle_expand_topk", _lib.eagle_expand_topk(ctypes.byref(cfg), *_ws(ws), step, _ptr(topk_ids),
                                                       _ptr(topk_logits), _ptr(row_lse_in), _ptr(row_lse),
                                                       _ptr(frontier_tokens), _ptr(frontier_count), _stream(stream)))


def eagle_verify_argmax(cfg, ws, row_argmax, tokens, parent, n_tree, accept_len, accepted_slots, out_tokens,
                        stream=None):
    _check("eagle_verify_argmax", _lib.eagle_verify_argmax(ctypes.byref(cfg), *_ws(ws), _ptr(row_argmax),
                                                           _ptr(tokens), _ptr(parent), _ptr(n_tree),
                                                           _ptr(accept_len), _ptr(accepted_slots), _ptr(out_tokens),
                                                           _stream(stream)))


def eagle_kv_compact(kv, kv_cache, prefix_len, accept_len, accepted_slots, slots_stride, new_len, ws=None,
                     stream=None):
    _check("eagle_kv_compact", _lib.eagle_kv_compact(ctypes.byref(kv), _ptr(kv_cache), _ptr(prefix_len),
                                                     _ptr(accept_len), _ptr(accepted_slots), slots_stride,
                                                     _ptr(new_len), _ptr(ws), _stream(stream)))


def kvq_contiguous(batch, n_q_heads, n_kv_heads, head_dim, layers, max_len, block) -> KvqCfg:
    """The 8-bit cache with codes [batch, layers, 2, max_len, n_kv_heads, head_dim] and scales
    [batch, layers, 2, ceil(max_len / block), n_kv_heads], both contiguous."""
    row, nb = n_kv_heads * head_dim, -(-max_len // max(1, block))
    return KvqCfg(batch, n_q_heads, n_kv_heads, head_dim, layers, max_len, block, EAGLE_BF16,
                  layers * 2 * max_len * row, 2 * max_len * row, max_len * row, row,
                  layers * 2 * nb * n_kv_heads, 2 * nb * n_kv_heads, nb * n_kv_heads, n_kv_heads)


def alloc_kvq(kv: KvqCfg, device="cuda") -> tuple[torch.Tensor, torch.Tensor]:
    """Zeroed codes and scales of a contiguous 8-bit cache."""
    shape = (kv.batch, kv.layers, 2)
    return (torch.zeros(*shape, kv.max_len, kv.n_kv_heads, kv.head_dim, dtype=torch.uint8, device=device),
            torch.zeros(*shape, kv.n_blocks, kv.n_kv_heads, dtype=torch.float32, device=device))


def _behind(t):
    """A slice of fused rows as all that lies behind its start in its storage."""
    if not isinstance(t, torch.Tensor) or t.is_contiguous():
        return t
    return t.as_strided((t.untyped_storage().nbytes() // t.element_size() - t.storage_offset(),), (1,))


def _apart(fn, name, t, row_stride, dim):
    """_behind, of rows of at least `dim` entries that lie row_stride apart."""
    if not isinstance(t, torch.Tensor) or t.is_contiguous():
        return t
    inner, rows = 1, 0  # entries of a row and, past its end, rows so far
    for size, stride in zip(reversed(t.shape), reversed(t.stride())):
        if size == 1:
            continue
        if inner >= dim and stride == row_stride * max(rows, 1):
            rows = max(rows, 1) * size
        elif rows == 0 and stride == inner:
            inner *= size
        else:
            raise ValueError(f"{fn}: {name}'s strides {tuple(t.stride())} are not those of rows of {dim} with row_stride {row_stride}")
    return _behind(t)


def eagle_kvq_store(kv, layer, T, k, v, row_stride, row_start, start, count, codes, scales, ws=None, stream=None):
    fn, dev, B = "eagle_kvq_store", _device(), kv.batch
    # dense rows: the last one reaches its heads' end (packed rows: the caller's row_start says how far)
    rows = 0 if row_start is not None else (B * T - 1) * row_stride + kv.n_kv_heads * kv.head_dim
    n_codes, n_scales = kv.extent(layer + 1)
    _check(fn, _lib.eagle_kvq_store(ctypes.byref(kv), layer, T, _need(fn, "k", _behind(k), _BF16, rows, dev),
                                    _need(fn, "v", _behind(v), _BF16, rows, dev), row_stride,
                                    _need(fn, "row_start", row_start, _I32, B, dev),
                                    _need(fn, "start", start, _I32, B, dev), _need(fn, "count", count, _I32, B, dev),
                                    _need(fn, "codes", codes, _CODES, n_codes, dev),
                                    _need(fn, "scales", scales, _F32, n_scales, dev),
                                    None if ws is None else _ws_on(fn, ws, dev)[0], _stream_on(stream, dev)))


def eagle_kvq_compact(kv, codes, scales, prefix_len, accept_len, accepted_slots, slots_stride, new_len, ws=None,
                      stream=None):
    fn, dev, B = "eagle_kvq_compact", _device(), kv.batch
    n_codes, n_scales = kv.extent(kv.layers) if kv.layers > 0 else (0, 0)
    _check(fn, _lib.eagle_kvq_compact(ctypes.byref(kv), _need(fn, "codes", codes, _CODES, n_codes, dev),
                                      _need(fn, "scales", scales, _F32, n_scales, dev),
                                      _need(fn, "prefix_len", prefix_len, _I32, B, dev),
                                      _need(fn, "accept_len", accept_len, _I32, B, dev),
                                      _need(fn, "accepted_slots", accepted_slots, _I32, B * slots_stride, dev),
                                      slots_stride, _need(fn, "new_len", new_len, _I32, B, dev),
                                      None if ws is None else _ws_on(fn, ws, dev)[0], _stream_on(stream, dev)))


def eagle_kvq_attention_workspace_bytes(kv: KvqCfg, T: int) -> int:
    return int(_lib.eagle_kvq_attention_workspace_bytes(ctypes.byref(kv), T))


def eagle_kvq_tree_attention(kv, T, q, codes, scales, layer, prefix_len, mask, n_tree, out, ws, stream=None):
    """Tree attention over the 8-bit cache; mask None: slot i sees slots 0..i (T = 1: a decode step)."""
    fn, dev, B = "eagle_kvq_tree_attention", _device(), kv.batch
    n = B * T * kv.n_q_heads * kv.head_dim
    n_codes, n_scales = kv.extent(layer + 1)
    _check(fn, _lib.eagle_kvq_tree_attention(ctypes.byref(kv), T, _need(fn, "q", q, _BF16, n, dev),
                                             _need(fn, "codes", codes, _CODES, n_codes, dev),
                                             _need(fn, "scales", scales, _F32, n_scales, dev), layer,
                                             _need(fn, "prefix_len", prefix_len, _I32, B, dev),
                                             _need(fn, "mask", mask, _W32, B * T * ((T + 31) // 32), dev),
                                             _need(fn, "n_tree", n_tree, _I32, B, dev),
                                             _need(fn, "out", out, _BF16, n, dev), *_ws_on(fn, ws, dev),
                                             _stream_on(stream, dev)))


def _logit_dtypes(cfg):
    return _BF16 if cfg.logit_dtype == EAGLE_BF16 else _F32


def eagle_lmhead_quant(cfg, ws, hidden_dim, group, hidden, codes, scales, draft_logits, stream=None):
    """LM-head logits from 4-bit weights with group scales (eagle_lmhead_quant_pack)."""
    fn, dev, M = "eagle_lmhead_quant", _device(), cfg.batch * cfg.top_k
    n = cfg.vocab * hidden_dim
    _check(fn, _lib.eagle_lmhead_quant(ctypes.byref(cfg), *_ws_on(fn, ws, dev), hidden_dim, group,
                                       _need(fn, "hidden", hidden, _BF16, M * hidden_dim, dev),
                                       _need(fn, "codes", codes, _U8, n // 2, dev),
                                       _need(fn, "scales", scales, _BF16, n // max(1, group), dev),
                                       _need(fn, "draft_logits", draft_logits, _logit_dtypes(cfg), M * cfg.vocab, dev),
                                       _stream_on(stream, dev)))


def eagle_lmhead_quant_pack(vocab, hidden_dim, group, weight, codes, scales, stream=None):
    fn, dev, n = "eagle_lmhead_quant_pack", _device(), vocab * hidden_dim
    _check(fn, _lib.eagle_lmhead_quant_pack(vocab, hidden_dim, group, _need(fn, "weight", weight, _BF16, n, dev),
                                            _need(fn, "codes", codes, _U8, n // 2, dev),
                                            _need(fn, "scales", scales, _BF16, n // max(1, group), dev),
                                            _stream_on(stream, dev)))


def eagle_token_logprobs(cfg, ws, n_seq, per_seq, rows_per_seq, logits, temperature, slots, tokens, n_alt, logprob,
                         rank=None, entropy=None, alt_ids=None, alt_logprobs=None, stream=None):
    """Log-probability, rank, entropy and top alternatives of given tokens (slots None: entry j reads row j)."""
    fn, dev, n = "eagle_token_logprobs", _device(), n_seq * per_seq
    rows = n_seq * rows_per_seq * cfg.vocab
    _check(fn, _lib.eagle_token_logprobs(ctypes.byref(cfg), *_ws_on(fn, ws, dev), n_seq, per_seq, rows_per_seq,
                                         _need(fn, "logits", logits, _logit_dtypes(cfg), rows, dev), float(temperature),
                                         _need(fn, "slots", slots, _I32, n, dev), _need(fn, "tokens", tokens, _I32, n, dev),
                                         n_alt, _need(fn, "logprob", logprob, _F32, n, dev),
                                         _need(fn, "rank", rank, _I32, n, dev), _need(fn, "entropy", entropy, _F32, n, dev),
                                         _need(fn, "alt_ids", alt_ids, _I32, n * n_alt, dev),
                                         _need(fn, "alt_logprobs", alt_logprobs, _F32, n * n_alt, dev),
                                         _stream_on(stream, dev)))


def eagle_fp8_scale_stride(dim: int) -> int:
    return int(_lib.eagle_fp8_scale_stride(dim))


def _scale_stride(dim):  # the same without a call into the library
    return (dim + 511) // 512 * 4


def _dtypes(code):
    return _BF16 if code == EAGLE_BF16 else _F32


_EXP = tuple(t for t in (torch.uint8, getattr(torch, "float8_e8m0fnu", None)) if t is not None)


def alloc_fp8(rows: int, dim: int, scale_rows: int | None = None, device="cuda") -> tuple[torch.Tensor, torch.Tensor]:
    """Codes [rows, dim] and scale bytes of 8-bit rows (a weight's, one scale row for 128 rows: scale_rows)."""
    n = rows if scale_rows is None else scale_rows
    return (torch.zeros(rows, dim, dtype=torch.uint8, device=device),
            torch.zeros(n, eagle_fp8_scale_stride(dim), dtype=torch.uint8, device=device))


def eagle_rmsnorm_fp8(rows, dim, dtype, x, row_stride, residual, sum, weight, eps, codes, scales, ws=None, stream=None):
    """Residual, root-mean-square norm and 8-bit codes with a scale for each 128 entries (weight None: no norm)."""
    fn, dev, dt = "eagle_rmsnorm_fp8", _device(), _dtypes(dtype)
    n = (rows - 1) * row_stride + dim
    if row_stride != dim:  # rows inside wider ones
        x, residual, sum = (_apart(fn, name, t, row_stride, dim)
                            for name, t in (("x", x), ("residual", residual), ("sum", sum)))
    _check(fn, _lib.eagle_rmsnorm_fp8(rows, dim, dtype, _need(fn, "x", x, dt, n, dev), row_stride,
                                      _need(fn, "residual", residual, dt, n, dev),
                                      _need(fn, "sum", sum, dt, n, dev), _need(fn, "weight", weight, dt, dim, dev),
                                      float(eps), _need(fn, "codes", codes, _CODES, rows * dim, dev),
                                      _need(fn, "scales", scales, _EXP, rows * _scale_stride(dim), dev),
                                      None if ws is None else _ws_on(fn, ws, dev)[0], _stream_on(stream, dev)))


def eagle_linear_fp8(rows, out_dim, in_dim, x_codes, x_scales, w_codes, w_scales, out_dtype, out, ws=None, stream=None):
    """out [rows, out_dim] = x w^T on 8-bit codes with power-of-two scales."""
    fn, dev, stride = "eagle_linear_fp8", _device(), _scale_stride(in_dim)
    _check(fn, _lib.eagle_linear_fp8(rows, out_dim, in_dim, _need(fn, "x_codes", x_codes, _CODES, rows * in_dim, dev),
                                     _need(fn, "x_scales", x_scales, _EXP, rows * stride, dev),
                                     _need(fn, "w_codes", w_codes, _CODES, out_dim * in_dim, dev),
                                     _need(fn, "w_scales", w_scales, _EXP, -(-out_dim // 128) * stride, dev), out_dtype,
                                     _need(fn, "out", out, _dtypes(out_dtype), rows * out_dim, dev),
                                     None if ws is None else _ws_on(fn, ws, dev)[0], _stream_on(stream, dev)))


def eagle_linear_fp8_pack(out_dim, in_dim, weight, codes, scales, stream=None):
    fn, dev, n = "eagle_linear_fp8_pack", _device(), out_dim * in_dim
    _check(fn, _lib.eagle_linear_fp8_pack(out_dim, in_dim, _need(fn, "weight", weight, _BF16, n, dev),
                                          _need(fn, "codes", codes, _CODES, n, dev),
                                          _need(fn, "scales", scales, _EXP,
                                                -(-out_dim // 128) * eagle_fp8_scale_stride(in_dim), dev),
                                          _stream_on(stream, dev)))


def eagle_distill_loss(cfg, ws, rows, n_top, logits, teacher_ids, teacher_logits, teacher_lse, temperature, row_weight,
                       loss, dlogits=None, stream=None):
    """Loss of a draft's rows against its target's top logits, and (dlogits) its gradient."""
    fn, dev, n, dt = "eagle_distill_loss", _device(), rows * n_top, _logit_dtypes(cfg)
    _check(fn, _lib.eagle_distill_loss(ctypes.byref(cfg), *_ws_on(fn, ws, dev), rows, n_top,
                                       _need(fn, "logits", logits, dt, rows * cfg.vocab, dev),
                                       _need(fn, "teacher_ids", teacher_ids, _I32, n, dev),
                                       _need(fn, "teacher_logits", teacher_logits, _F32, n, dev),
                                       _need(fn, "teacher_lse", teacher_lse, _F32, rows, dev), float(temperature),
                                       _need(fn, "row_weight", row_weight, _F32, rows, dev),
                                       _need(fn, "loss", loss, _F32, rows, dev),
                                       _need(fn, "dlogits", dlogits, dt, rows * cfg.vocab, dev), _stream_on(stream, dev)))


def eagle_status_fetch(ws, stream=None) -> int:
    """Synchronises the stream; returns the device status code (0 = no fault) and clears it."""
    st = ctypes.c_int(0)
    _lib.eagle_status_fetch(_ptr(ws), ctypes.byref(st), _stream(stream))
    return int(st.value)


def eagle_tree_export(cfg, ws, cand_token=None, cand_parent=None, cand_depth=None, cand_logv=None, cand_valid=None,
                      kept=None, n_kept=None, stream=None):
    _check("eagle_tree_export", _lib.eagle_tree_export(ctypes.byref(cfg), *_ws(ws), _ptr(cand_token),
                                                       _ptr(cand_parent), _ptr(cand_depth), _ptr(cand_logv),
                                                       _ptr(cand_valid), _ptr(kept), _ptr(n_kept), _stream(stream)))


def eagle_verify_export(cfg, ws, row_max=None, row_argmax=None, row_mass=None, stream=None):
    _check("eagle_verify_export", _lib.eagle_verify_export(ctypes.byref(cfg), *_ws(ws), _ptr(row_max),
                                                           _ptr(row_argmax), _ptr(row_mass), _stream(stream)))


def eagle_test_sampling(words, ys, n, gumbel_out, log_out, stream=None):
    _check("eagle_test_sampling", _lib.eagle_test_sampling(_ptr(words), _ptr(ys), n, _ptr(gumbel_out), _ptr(log_out),
                                                           _stream(stream)))


def eagle_kernel_launches() -> int:
    return int(_lib.eagle_kernel_launches())


def raw_call(name: str, *args) -> int:
    """Call an entry point with raw ctypes arguments and return its status (host-side checks in tests)."""
    return int(getattr(_lib, name)(*args))
