"""Host-side checks of the 8-bit cache, the 4-bit LM head and the token
log-probabilities: every refusal happens before any CUDA call, so none of
these needs a GPU (pointers are fake addresses that a refused call never
follows)."""
import ctypes
import os
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.dirname(__file__))
import plain64 as P  # noqa: E402

PTR = 1 << 20  # an aligned fake address


@pytest.fixture(scope="module")
def E():
    from speculative_decoding_dynamic_gb300 import build
    build.build()
    from speculative_decoding_dynamic_gb300 import eagle
    return eagle


def _kv(E, **kw):
    kv = E.kvq_contiguous(2, 8, 2, 128, 3, 256, 32)
    for k, v in kw.items():
        setattr(kv, k, v)
    return kv


BAD_CFG = [
    (dict(batch=0), -1), (dict(n_q_heads=7), -1), (dict(n_kv_heads=0), -1), (dict(max_len=0), -1), (dict(layers=-1), -1),
    (dict(block=0), -1), (dict(block=24), -1), (dict(block=256), -1), (dict(dtype=5), -1), (dict(seq_stride=-16), -1),
    (dict(pos_stride=240), -1), (dict(scale_block_stride=1), -1), (dict(scale_kv_stride=-1), -1),
    (dict(head_dim=64), -2), (dict(dtype=0), -2), (dict(pos_stride=264), -2), (dict(layer_stride=8), -2),
    (dict(batch=70000), -2), (dict(seq_stride=1 << 40), -2),
]


@pytest.mark.parametrize("kw,code", BAD_CFG)
def test_every_call_refuses_a_bad_cache_description(E, kw, code):
    kv = ctypes.byref(_kv(E, **kw))
    assert E.raw_call("eagle_kvq_store", kv, 0, 4, PTR, PTR, 256, None, PTR, None, PTR, PTR, None, None) == code
    assert E.raw_call("eagle_kvq_compact", kv, PTR, PTR, PTR, PTR, PTR, 7, PTR, None, None) == code
    assert E.raw_call("eagle_kvq_tree_attention", kv, 4, PTR, PTR, PTR, 0, PTR, None, None, PTR, PTR, 1 << 40, None) == code
    assert E.eagle_kvq_attention_workspace_bytes(_kv(E, **kw), 4) == 0


def test_store_refusals(E):
    kv = ctypes.byref(_kv(E))
    good = [kv, 0, 4, PTR, PTR, 256, None, PTR, None, PTR, PTR, None, None]
    for at, value, code in ((1, -1, -1), (2, 0, -1), (3, None, -1), (4, None, -1), (5, 248, -1), (7, None, -1), (9, None, -1),
                            (10, None, -1), (5, 260, -2), (3, PTR + 8, -2), (4, PTR + 2, -2), (9, PTR + 4, -2)):
        args = list(good)
        args[at] = value
        assert E.raw_call("eagle_kvq_store", *args) == code, (at, value)


def test_compact_refusals(E):
    good = [ctypes.byref(_kv(E)), PTR, PTR, PTR, PTR, PTR, 7, PTR, None, None]
    for at, value, code in [(i, None, -1) for i in (1, 2, 3, 4, 5, 7)] + [(6, 0, -1), (1, PTR + 4, -2)]:
        args = list(good)
        args[at] = value
        assert E.raw_call("eagle_kvq_compact", *args) == code, (at, value)
    assert E.raw_call("eagle_kvq_compact", ctypes.byref(_kv(E, layers=0)), *good[1:]) == 0  # nothing to move
    assert E.raw_call("eagle_kvq_compact", ctypes.byref(_kv(E, layers=40000)), *good[1:]) == -2


def test_attention_refusals(E):
    kv = _kv(E)
    need = E.eagle_kvq_attention_workspace_bytes(kv, 61)
    assert need > 0
    assert E.eagle_kvq_attention_workspace_bytes(kv, 0) == 0 and E.eagle_kvq_attention_workspace_bytes(kv, 257) == 0
    good = [ctypes.byref(kv), 61, PTR, PTR, PTR, 0, PTR, PTR, PTR, PTR, PTR, need, None]
    for at, value, code in ((1, 0, -1), (1, 257, -1), (5, -1, -1), (2, None, -1), (3, None, -1), (4, None, -1), (6, None, -1),
                            (9, None, -1), (2, PTR + 2, -2), (3, PTR + 8, -2), (9, PTR + 8, -2), (10, None, -4),
                            (10, PTR + 16, -4), (11, need - 1, -4)):
        args = list(good)
        args[at] = value
        assert E.raw_call("eagle_kvq_tree_attention", *args) == code, (at, value)


def _cfg(E, **kw):
    base = dict(batch=2, vocab=1024, top_k=4, depth=1, node_budget=1, threshold=0.0, logit_dtype=E.EAGLE_BF16)
    base.update(kw)
    return E.TreeCfg(**base)


def test_lmhead_quant_refusals(E):
    cfg = _cfg(E)
    n = E.eagle_workspace_bytes(cfg)
    good = [ctypes.byref(cfg), PTR, n, 256, 128, PTR, PTR, PTR, PTR, None]
    for at, value, code in [(i, None, -1) for i in (5, 6, 7, 8)] + [(i, PTR + 8, -2) for i in (5, 6, 7, 8)] + [
            (0, None, -1), (1, None, -4), (2, n - 1, -4), (3, 0, -1), (3, 192, -2), (3, 8320, -2), (4, 16, -1), (4, 96, -1)]:
        args = list(good)
        args[at] = value
        assert E.raw_call("eagle_lmhead_quant", *args) == code, (at, value)
    odd = _cfg(E, vocab=1028, logit_dtype=E.EAGLE_F32)
    assert E.raw_call("eagle_lmhead_quant", ctypes.byref(odd), PTR, E.eagle_workspace_bytes(odd), *good[3:]) == -2
    good = [64, 256, 32, PTR, PTR, PTR, None]
    for at, value, code in [(0, 0, -1), (1, 0, -1), (1, 272, -2), (2, 48, -1), (3, None, -1), (4, None, -1), (5, None, -1),
                            (3, PTR + 2, -2)]:
        args = list(good)
        args[at] = value
        assert E.raw_call("eagle_lmhead_quant_pack", *args) == code, (at, value)


def test_token_logprobs_refusals(E):
    cfg = _cfg(E)
    n = E.eagle_workspace_bytes(cfg)
    f = ctypes.c_float
    good = [ctypes.byref(cfg), PTR, n, 3, 7, 61, PTR, f(1.0), PTR, PTR, 5, PTR, PTR, PTR, PTR, PTR, None]
    for at, value, code in [(0, None, -1), (1, None, -4), (2, n - 1, -4), (3, 0, -1), (4, 0, -1), (5, 0, -1), (6, None, -1),
                            (6, PTR + 2, -2), (7, f(0.0), -1), (7, f(-1.0), -1), (7, f(float("nan")), -1),
                            (7, f(float("inf")), -1), (9, None, -1), (10, -1, -1), (10, 17, -1), (11, None, -1),
                            (14, None, -1), (15, None, -1), (3, 1 << 23, -2)]:
        args = list(good)
        args[at] = value
        assert E.raw_call("eagle_token_logprobs", *args) == code, (at, value)
    args = list(good)
    args[8], args[4] = None, 62  # without slots, entry j reads row j: no more entries than rows
    assert E.raw_call("eagle_token_logprobs", *args) == -1


def test_token_logprobs_refuses_a_temperature_whose_reverse_overflows(E):
    cfg = _cfg(E)
    for t in (1e-39, 2.0 ** -127):
        args = [ctypes.byref(cfg), PTR, E.eagle_workspace_bytes(cfg), 3, 7, 61, PTR, ctypes.c_float(t), PTR, PTR, 5, PTR, PTR,
                PTR, PTR, PTR, None]
        assert E.raw_call("eagle_token_logprobs", *args) == -1, t


def test_binding_refuses_tensors_that_do_not_fit(E):
    import torch
    kv = E.kvq_contiguous(1, 2, 2, 128, 1, 64, 32)
    codes, scales = E.alloc_kvq(kv, "cpu")
    rows = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    start = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="float32"):
        E.eagle_kvq_store(kv, 0, 4, rows.float(), rows, 256, None, start, None, codes, scales)
    with pytest.raises(ValueError, match="current CUDA device"):
        E.eagle_kvq_store(kv, 0, 4, rows, rows, 256, None, start, None, codes, scales)


def test_cache_extent_of_the_contiguous_form(E):
    kv = E.kvq_contiguous(3, 8, 2, 128, 5, 100, 32)
    assert kv.n_blocks == 4
    assert kv.extent(5) == (3 * 5 * 2 * 100 * 2 * 128, 3 * 5 * 2 * 4 * 2)


def test_plain_e4m3_rounding():
    """The tests' own encoder: every code's value encodes to itself, midpoints go to the even code."""
    fin = np.isfinite(P.E4M3)
    assert (P.encode(P.E4M3[fin]) == np.arange(256)[fin]).all()
    mid = (P._POS[:-1] + P._POS[1:]) / 2
    c = P.encode(mid)
    assert (c % 2 == 0).all() and (P.encode(-mid) == (c | 128)).all()
    assert P.encode(1e9) == 0x7E and P.encode(-1e9) == 0xFE
    for e in (-126, -50, 0, 100):
        assert P.block_scale(448.0 * 2.0 ** e) == 2.0 ** e
        assert P.block_scale(np.nextafter(448.0, 500) * 2.0 ** e) == 2.0 ** (e + 1)
    assert P.block_scale(0.0) == 2.0 ** -126


@pytest.mark.parametrize("kw,code", BAD_CFG)
def test_binding_leaves_a_bad_cache_description_to_the_library(E, kw, code):
    kv = _kv(E, **kw)

    class Ws:  # a workspace's address and size
        def data_ptr(self): return PTR
        def numel(self): return 1 << 40
        def element_size(self): return 1

    for call in (lambda: E.eagle_kvq_store(kv, 0, 4, PTR, PTR, 256, None, PTR, None, PTR, PTR, None, 0),
                 lambda: E.eagle_kvq_compact(kv, PTR, PTR, PTR, PTR, PTR, 7, PTR, None, 0),
                 lambda: E.eagle_kvq_tree_attention(kv, 4, PTR, PTR, PTR, 0, PTR, None, None, PTR, Ws(), 0)):
        with pytest.raises(E.EagleError) as e:
            call()
        assert e.value.code == code
    empty = E.kvq_contiguous(2, 8, 2, 128, 3, 256, 0)
    assert E.eagle_kvq_attention_workspace_bytes(empty, 4) == 0


def test_binding_refuses_a_workspace_that_is_not_on_the_current_device(E):
    """Kernels write the status word: a workspace in host memory (or on another GPU) is refused like any other tensor."""
    import torch
    kv, cfg = _kv(E), _cfg(E)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    for call in (lambda: E.eagle_kvq_store(kv, 0, 4, PTR, PTR, 256, None, PTR, None, PTR, PTR, ws, 0),
                 lambda: E.eagle_kvq_compact(kv, PTR, PTR, PTR, PTR, PTR, 7, PTR, ws, 0),
                 lambda: E.eagle_kvq_tree_attention(kv, 4, PTR, PTR, PTR, 0, PTR, None, None, PTR, ws, 0),
                 lambda: E.eagle_lmhead_quant(cfg, ws, 256, 128, PTR, PTR, PTR, PTR, 0),
                 lambda: E.eagle_token_logprobs(cfg, ws, 3, 7, 61, PTR, 1.0, PTR, PTR, 0, PTR, stream=0)):
        with pytest.raises(ValueError, match="ws is on cpu"):
            call()
    with pytest.raises(E.EagleError) as e:
        E.eagle_lmhead_quant(cfg, None, 256, 128, PTR, PTR, PTR, PTR, 0)
    assert e.value.code == -4


def test_cycle_refuses_log_probabilities_it_has_no_buffers_for(E):
    from speculative_decoding_dynamic_gb300 import cycle as C
    cfg, kv = _cfg(E), E.kvq_contiguous(2, 2, 2, 128, 1, 16, 16)
    with pytest.raises(ValueError, match="n_alt"):
        C.DeviceCycle(cfg, kv, device="cpu").logprobs(None)
    for n_alt in (-1, 17):
        with pytest.raises(ValueError, match="n_alt"):
            C.DeviceCycle(cfg, kv, device="cpu", n_alt=n_alt)
    assert C.DeviceCycle(cfg, kv, device="cpu", n_alt=16).alt_ids.shape == (2, 2, 16)


def test_cycle_refuses_new_rows_for_the_16_bit_cache_before_its_first_launch(E):
    from speculative_decoding_dynamic_gb300 import cycle as C
    row = 2 * 128
    kv = E.KvCfg(2, 2, 2, 128, 1, 16, E.EAGLE_BF16, 2 * 16 * row, 2 * 16 * row, 16 * row, row)
    dc = C.DeviceCycle(_cfg(E), kv, device="cpu")
    n = E.eagle_kernel_launches()
    with pytest.raises(ValueError, match="8-bit cache"):
        dc.run(PTR, PTR, PTR, PTR, PTR, 0, PTR, 0, 0, E.GREEDY, stream=0, new_kv=(PTR, PTR))
    assert E.eagle_kernel_launches() == n
