"""The 8-bit KV cache on the GPU against plain 64-bit forms (plain64.py):
writing (eagle_kvq_store) and moving the accepted path (eagle_kvq_compact) bit
for bit over the whole buffers, attention (eagle_kvq_tree_attention) within
the bound that its roundings give element by element."""
import numpy as np
import pytest

import plain64 as P

pytestmark = pytest.mark.gpu
D = 128


def _E():
    from speculative_decoding_dynamic_gb300 import eagle as E
    return E


def _bf16(rng, shape, scale=1.0):
    return P.bf16_round(rng.standard_normal(shape) * scale)


def _dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _dev_bf16(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(torch.bfloat16)


def _layout(E, B, Hq, H, layers, max_len, block, odd):
    """A contiguous cache, or one with other orders and gaps: positions outside the layers, padded rows."""
    if not odd:
        return E.kvq_contiguous(B, Hq, H, D, layers, max_len, block)
    row = H * D + 48
    nb = -(-max_len // block)
    # [kv][position][layer][sequence]: a row of every sequence and layer side by side
    return E.KvqCfg(B, Hq, H, D, layers, max_len, block, E.EAGLE_BF16, row, B * row, max_len * layers * B * row,
                    layers * B * row, 3 + H * nb, B * (3 + H * nb), layers * B * (3 + H * nb), H)


def _buffers(kv, rng, layers=None, lo=-9, hi=-4):
    c, s = kv.extent(kv.layers)
    codes = rng.integers(0, 256, c + 64).astype(np.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x11
    scales = (2.0 ** rng.integers(lo, hi, s + 16)).astype(np.float32)
    return codes, scales


# ----------------------------------------------------------------- store ---

STORE = [
    # block, H, T, starts, counts (None: T each), packed, odd layout, value scale
    (16, 8, 1, [0, 15, 16, 100], None, False, False, 1.0),
    (32, 8, 61, [0, 31, 32, 77], None, False, False, 1.0),
    (32, 3, 61, [5, 64], [61, 0], False, True, 30.0),
    (64, 40, 33, [63, 1, 64], [1, 33, 2], True, False, 1.0),
    (128, 2, 300, [0, 127, 1], [300, 257, 299], True, True, 1e-3),
    (128, 5, 7, [250], [6], False, False, 1.0),
    (16, 1, 130, [126], None, False, True, 1e4),
]


@pytest.mark.parametrize("block,H,T,starts,counts,packed,odd,scale", STORE)
def test_store_is_the_definition_bit_for_bit(block, H, T, starts, counts, packed, odd, scale):
    import torch
    E = _E()
    rng = np.random.default_rng(block * 1000 + T)
    B = len(starts)
    n = np.array(counts if counts is not None else [T] * B)
    max_len = int(max(s + c for s, c in zip(starts, n)))  # the last token takes the last position
    kv = _layout(E, B, H, H, 2, max_len, block, odd)
    codes, scales = _buffers(kv, rng)
    first = (np.cumsum(n) - n + 3) if packed else None
    rows = int(n.sum()) + 3 if packed else B * T
    stride = H * D + (8 if odd else 0)
    # rows of very different size, zeros and negative zeros among them
    k, v = (_bf16(rng, (rows, stride), scale) * 2.0 ** rng.integers(-6, 7, (rows, 1)) for _ in range(2))
    k[::5] = 0.0
    v[::3, ::7] = -0.0
    k, v = P.bf16_round(k), P.bf16_round(v)
    want_c, want_s = codes.copy(), scales.copy()
    P.store(kv, 1, T, k[:, :H * D].reshape(rows, H, D), v[:, :H * D].reshape(rows, H, D), first, starts, counts,
            *P.views(kv, want_c, want_s))
    dc, ds = _dev(codes), _dev(scales)
    i32 = lambda a: None if a is None else _dev(np.asarray(a, np.int32))  # noqa: E731
    ws = E.alloc_workspace(256)
    E.eagle_kvq_store(kv, 1, T, _dev_bf16(k), _dev_bf16(v), stride, i32(first), i32(starts), i32(counts), dc, ds, ws)
    torch.cuda.synchronize()
    assert E.eagle_status_fetch(ws) == 0
    assert (ds.cpu().numpy() == want_s).all()
    assert (dc.cpu().numpy() == want_c).all()


def test_store_token_by_token_grows_the_block_scale():
    """Forty decode steps, the values growing: each step moves the block's earlier codes to its new scale."""
    import torch
    E = _E()
    rng = np.random.default_rng(5)
    kv = E.kvq_contiguous(2, 4, 2, D, 1, 96, 32)
    codes, scales = _buffers(kv, rng)
    vc, vs = P.views(kv, codes, scales)
    dc, ds = _dev(codes), _dev(scales)
    start = np.array([7, 30])
    for step in range(40):
        k, v = (_bf16(rng, (2, 2, D), 1.2 ** step) for _ in range(2))
        P.store(kv, 0, 1, k, v, None, start + step, None, vc, vs)
        E.eagle_kvq_store(kv, 0, 1, _dev_bf16(k), _dev_bf16(v), 2 * D, None, _dev((start + step).astype(np.int32)), None,
                          dc, ds)
    torch.cuda.synchronize()
    assert (ds.cpu().numpy() == scales).all()
    assert (dc.cpu().numpy() == codes).all()


def test_store_extreme_values_and_scales_from_elsewhere():
    """bf16's largest and smallest values; an old scale that is no power of two."""
    import torch
    E = _E()
    rng = np.random.default_rng(6)
    kv = E.kvq_contiguous(3, 2, 2, D, 1, 64, 16)
    codes, scales = _buffers(kv, rng)
    scales *= np.float32(1.37)
    k, v = _bf16(rng, (3 * 20, 2, D)), _bf16(rng, (3 * 20, 2, D))
    k[0, 0, 0] = 3.3895313892515355e38
    k[20:40] = P.bf16_round(k[20:40] * 1e-39)  # subnormal values
    v[20:40] = 0.0
    start = [5, 3, 9]
    want_c, want_s = codes.copy(), scales.copy()
    P.store(kv, 0, 20, k, v, None, start, None, *P.views(kv, want_c, want_s))
    dc, ds = _dev(codes), _dev(scales)
    E.eagle_kvq_store(kv, 0, 20, _dev_bf16(k), _dev_bf16(v), 2 * D, None, _dev(np.array(start, np.int32)), None, dc, ds)
    torch.cuda.synchronize()
    assert (ds.cpu().numpy() == want_s).all()
    assert (dc.cpu().numpy() == want_c).all()


def test_store_leaves_sequences_with_bad_lengths_alone():
    import torch
    E = _E()
    rng = np.random.default_rng(8)
    for bad in (dict(count=[4, 9]), dict(count=[4, -1]), dict(start=[0, -1]), dict(start=[0, 61]), dict(first=[0, -2])):
        kv = E.kvq_contiguous(2, 2, 2, D, 1, 64, 16)
        codes, scales = _buffers(kv, rng)
        k = _bf16(rng, (16, 2, D))
        first, start, count = bad.get("first", [0, 8]), bad.get("start", [0, 8]), bad.get("count", [4, 4])
        want_c, want_s = codes.copy(), scales.copy()
        P.store(kv, 0, 8, k, k, first, start, count, *P.views(kv, want_c, want_s))
        dc, ds = _dev(codes), _dev(scales)
        ws = E.alloc_workspace(256)
        i32 = lambda a: _dev(np.asarray(a, np.int32))  # noqa: E731
        E.eagle_kvq_store(kv, 0, 8, _dev_bf16(k), _dev_bf16(k), 2 * D, i32(first), i32(start), i32(count), dc, ds, ws)
        torch.cuda.synchronize()
        assert E.eagle_status_fetch(ws) == 3
        assert (ds.cpu().numpy() == want_s).all() and (dc.cpu().numpy() == want_c).all(), bad


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_store_reports_non_finite_values(value):
    import torch
    E = _E()
    kv = E.kvq_contiguous(1, 2, 2, D, 1, 64, 16)
    dc, ds = E.alloc_kvq(kv)
    ws = E.alloc_workspace(256)
    k = torch.ones(4, 2, D, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    v[2, 1, 77] = value
    E.eagle_kvq_store(kv, 0, 4, k, v, 2 * D, None, _dev(np.zeros(1, np.int32)), None, dc, ds, ws)
    assert E.eagle_status_fetch(ws) == 1


# --------------------------------------------------------------- compact ---

@pytest.mark.parametrize("block", [16, 32, 128])
@pytest.mark.parametrize("odd", [False, True])
def test_compact_is_the_definition_bit_for_bit(block, odd):
    import torch
    E = _E()
    rng = np.random.default_rng(block + odd)
    H, layers, T, Dp = 5, 3, 61, 16
    L = np.array([0, 1, block - 2, block - 1, 200, 100, 77, 256 - 17])
    B = len(L)
    kv = _layout(E, B, H, H, layers, 256, block, odd)
    codes, scales = _buffers(kv, rng)
    accept = np.array([3, 0, 16, 5, 7, 1, 16, 16])
    slots = np.full((B, Dp + 1), -1)
    for b in range(B):
        a = accept[b]
        top = min(T, 256 - L[b])
        slots[b, :a + 1] = np.concatenate([[0], 1 + np.sort(rng.permutation(top - 1)[:a])])
    slots[4, :8] = np.arange(8)  # already in place
    want_c, want_s = codes.copy(), scales.copy()
    new_len = P.compact(kv, *P.views(kv, want_c, want_s), L, accept, slots)
    dc, ds, ws = _dev(codes), _dev(scales), E.alloc_workspace(256)
    got_len = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    i32 = lambda a: _dev(np.asarray(a, np.int32))  # noqa: E731
    E.eagle_kvq_compact(kv, dc, ds, i32(L), i32(accept), i32(slots), Dp + 1, got_len, ws)
    torch.cuda.synchronize()
    assert E.eagle_status_fetch(ws) == 0
    assert got_len.tolist() == new_len
    assert (ds.cpu().numpy() == want_s).all()
    assert (dc.cpu().numpy() == want_c).all()


def test_compact_refuses_bad_paths():
    import torch
    E = _E()
    rng = np.random.default_rng(1)
    for L, a, path in ((10, 2, [0, 2, 1]), (10, 17, [0] * 4), (10, 4, [0, 1, 2, 3]), (60, 2, [0, 1, 4]), (62, 2, [0, 1, 2]),
                       (-1, 1, [0, 1]), (10, -1, [0, 1])):
        kv = E.kvq_contiguous(2, 2, 2, D, 1, 64, 16)
        codes, scales = _buffers(kv, rng)
        slots = np.full((2, 4), -1)
        slots[0, :min(4, len(path))] = path[:4]
        slots[1] = [0, 2, 3, 9]
        want_c, want_s = codes.copy(), scales.copy()
        new_len = P.compact(kv, *P.views(kv, want_c, want_s), [L, 5], [a, 3], slots)
        assert new_len == [None, 9]
        dc, ds, ws = _dev(codes), _dev(scales), E.alloc_workspace(256)
        got = torch.full((2,), -7, dtype=torch.int32, device="cuda")
        i32 = lambda x: _dev(np.asarray(x, np.int32))  # noqa: E731
        E.eagle_kvq_compact(kv, dc, ds, i32([L, 5]), i32([a, 3]), i32(slots), 4, got, ws)
        torch.cuda.synchronize()
        assert E.eagle_status_fetch(ws) == 3 and got.tolist() == [-7, 9]
        assert (ds.cpu().numpy() == want_s).all() and (dc.cpu().numpy() == want_c).all()


# ------------------------------------------------------------- attention ---

def _tree(rng, B, T, n):
    see = np.zeros((B, T, T), bool)
    for b in range(B):
        for i in range(n[b]):
            see[b, i, i] = True
            if i:
                see[b, i] |= see[b, rng.integers(0, i)]
    return see


def _pack_mask(see):
    B, T, _ = see.shape
    W = -(-T // 32)
    bits = np.zeros((B, T, W * 32), np.uint64)
    bits[:, :, :T] = see
    return (bits.reshape(B, T, W, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32).view(np.int32)


def _attend(E, kv, T, L, n_tree, see, codes, scales, q, layer, ws=None):
    import torch
    ws = ws if ws is not None else E.alloc_workspace(E.eagle_kvq_attention_workspace_bytes(kv, T))
    out = torch.full((kv.batch, T, kv.n_q_heads, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    i32 = lambda a: None if a is None else _dev(np.asarray(a, np.int32))  # noqa: E731
    E.eagle_kvq_tree_attention(kv, T, _dev_bf16(q), _dev(codes), _dev(scales), layer, i32(L),
                               None if see is None else _dev(_pack_mask(see)), i32(n_tree), out, ws)
    torch.cuda.synchronize()
    return out.float().cpu().numpy(), E.eagle_status_fetch(ws)


ATTN = [
    # Hq, H, T, lengths, block, tree (else a chain), n_tree ragged, odd layout
    (4, 4, 1, [0, 1, 14, 15, 16], 16, False, False, False),         # decode, shortest lengths
    (32, 8, 1, [31, 32, 33, 700, 2047], 64, False, False, False),
    (64, 8, 1, [5000], 128, False, False, True),
    (16, 1, 1, [63, 64, 300], 32, False, False, False),              # all sixteen rows
    (12, 4, 5, [0, 40, 333], 16, True, True, False),                 # 15 rows
    (8, 8, 16, [100, 0, 31], 32, True, True, True),
    (8, 4, 8, [500], 32, False, False, False),
    (40, 40, 61, [0, 200], 64, True, False, False),                  # tensor-core path, MHA
    (32, 8, 61, [0, 1, 63, 64, 700], 32, True, True, False),
    (32, 8, 61, [2048], 64, True, False, False),                     # cut into many pieces
    (64, 8, 65, [900, 3], 128, True, True, True),
    (24, 2, 9, [130], 16, True, False, False),                       # 108 rows, G = 12
    (20, 4, 40, [77, 190], 16, False, True, False),                  # G = 5: rows of a slot straddle row blocks
    (8, 8, 200, [10, 129], 64, True, True, False),                   # seven mask words
    (4, 2, 256, [300], 32, False, False, False),
    (34, 2, 1, [257, 5], 32, False, False, False),                   # 17 rows of one slot
]


@pytest.mark.parametrize("Hq,H,T,L,block,tree,ragged,odd", ATTN)
def test_attention_within_the_bound_of_its_roundings(Hq, H, T, L, block, tree, ragged, odd):
    E = _E()
    rng = np.random.default_rng(Hq * 100 + T + len(L))
    B = len(L)
    max_len = max(L) + T + 3
    kv = _layout(E, B, Hq, H, 2, max_len, block, odd)
    codes, scales = _buffers(kv, rng)
    n = np.full(B, T)
    if ragged:
        n = rng.integers(1, T + 1, B)
        n[0] = T
    vc, vs = P.views(kv, codes, scales)
    for b in range(B):  # positions that no row may see: NaN codes, and NaN scales where a whole block is unused
        vc[b, :, :, L[b] + n[b]:] = 0x7F
        vs[b, :, :, -(-(L[b] + int(n[b])) // block):] = np.nan
    q = _bf16(rng, (B, T, Hq, D), 2.0)
    see = _tree(rng, B, T, n) if tree else None
    want, tol = P.attention(kv, T, q, vc, vs, 1, L, see, n if ragged else None)
    got, status = _attend(E, kv, T, L, n if ragged else None, see, codes, scales, q, 1)
    assert status == 0
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], float(np.nanmax(np.abs(got - want) - tol)))


@pytest.mark.parametrize("T", [1, 61])
def test_attention_with_scales_far_apart_and_masked_rows(T):
    """Blocks whose scales differ by 2^40 and are no powers of two, rows of q far apart in size, and tree
    slots whose mask row is empty (with no prefix: a row that sees nothing is zero)."""
    E = _E()
    rng = np.random.default_rng(T)
    B, Hq, H = 3, 8, 2
    L = [0, 150, 700]
    kv = E.kvq_contiguous(B, Hq, H, D, 2, 800, 16)
    codes, scales = _buffers(kv, rng, lo=-30, hi=11)
    vc, vs = P.views(kv, codes, scales)
    vs[:, :, 0] = 2.0 ** rng.integers(-11, -7, vs[:, :, 0].shape)  # K: scores stay moderate
    vs *= rng.uniform(1.0, 1.9, vs.shape).astype(np.float32)
    q = P.bf16_round(_bf16(rng, (B, T, Hq, D)) * 2.0 ** rng.integers(-8, 3, (B, T, Hq, 1)))
    see = _tree(rng, B, T, [T] * B)
    see[0, T // 2] = False
    see[1, 0] = False
    want, tol = P.attention(kv, T, q, vc, vs, 0, L, see, None)
    got, status = _attend(E, kv, T, L, None, see, codes, scales, q, 0)
    assert status == 0
    assert (got[0, T // 2] == 0).all()
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4])


@pytest.mark.parametrize("T", [1, 33])
def test_attention_peaked_rows(T):
    """One key takes almost all of the weight and thousands share the rest: small weights must not vanish."""
    E = _E()
    rng = np.random.default_rng(3)
    Hq, H, L = 4, 1, 3000
    kv = E.kvq_contiguous(1, Hq, H, D, 1, L + T, 64)
    codes, scales = _buffers(kv, rng)
    vc, vs = P.views(kv, codes, scales)
    vs[:] = 2.0 ** -8
    q = np.zeros((1, T, Hq, D), np.float32)
    q[..., 0] = 4.0
    vc[:, :, 0, :, :, 0] = P.encode(0.0)
    vc[0, 0, 0, 5, 0, 0] = P.encode(448.0)  # score 4 * 448 / 256 / sqrt(128) above the rest
    vs[0, 0, 0, 0] = 2.0 ** -4              # sixteen times that: the others weigh e^-9.9 each
    vc[0, 0, 1] &= 0x7F                     # V positive: the small weights add up
    want, tol = P.attention(kv, T, q, vc, vs, 0, [L], None, None)
    got, status = _attend(E, kv, T, [L], None, None, codes, scales, q, 0)
    assert status == 0 and (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("T", [1, 61])
def test_attention_bad_lengths_give_zero_rows_and_status(T):
    E = _E()
    rng = np.random.default_rng(4)
    kv = E.kvq_contiguous(4, 8, 2, D, 1, 128, 32)
    codes, scales = _buffers(kv, rng)
    q = _bf16(rng, (4, T, 8, D))
    L = [20, -1, 128 - T + 1, 128 - T]
    want, tol = P.attention(kv, T, q, *P.views(kv, codes, scales), 0, L, None, None)
    got, status = _attend(E, kv, T, L, None, None, codes, scales, q, 0)
    assert status == 3
    assert (got[1] == 0).all() and (got[2] == 0).all() and (np.abs(got - want) <= tol).all()


def test_attention_many_sequences():
    """More sequences than a warp finds in one step, lengths from 0 on, some out of range."""
    E = _E()
    rng = np.random.default_rng(9)
    B, T = 150, 3
    kv = E.kvq_contiguous(B, 4, 2, D, 1, 160, 16)
    codes, scales = _buffers(kv, rng)
    L = rng.integers(0, 150, B)
    L[::11] = 400
    q = _bf16(rng, (B, T, 4, D))
    want, tol = P.attention(kv, T, q, *P.views(kv, codes, scales), 0, L, None, None)
    got, status = _attend(E, kv, T, L, None, None, codes, scales, q, 0)
    assert status == 3 and (np.abs(got - want) <= tol).all()


def test_attention_long_cache_offsets_beyond_32_bits():
    """Positions past 2^32 bytes into the cache: one sequence and layer of a cache of 2^22 positions."""
    import torch
    E = _E()
    rng = np.random.default_rng(10)
    H, max_len, T = 8, (1 << 22) + 128, 4
    kv = E.kvq_contiguous(1, 8, H, D, 1, max_len, 128)
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    codes, scales = E.alloc_kvq(kv)
    n = 700
    L = max_len - T
    # all but the last positions are zero codes with a tiny K scale: score 0, V 0
    k, v = (_bf16(rng, (n, H, D)) for _ in range(2))
    E.eagle_kvq_store(kv, 0, n, _dev_bf16(k), _dev_bf16(v), H * D, None, _dev(np.array([max_len - n], np.int32)), None,
                      codes, scales)
    scales[scales == 0] = 1.0
    q = _bf16(rng, (1, T, 8, D), 6.0)
    out = torch.empty(1, T, 8, D, dtype=torch.bfloat16, device="cuda")
    ws = E.alloc_workspace(E.eagle_kvq_attention_workspace_bytes(kv, T))
    E.eagle_kvq_tree_attention(kv, T, _dev_bf16(q), codes, scales, 0, _dev(np.array([L], np.int32)), None, None, out, ws)
    tail = codes[0, 0, :, -n:].cpu().numpy()
    blk = np.arange(max_len - n, max_len) // 128
    sc = scales[0, 0].cpu().numpy()
    want = np.zeros((T, 8, D))
    for h in range(H):
        K, V = (P.E4M3[tail[w, :, h]] * sc[w, blk, h][:, None] for w in (0, 1))
        for i in range(T):
            s = (K @ q[0, i, h].astype(np.float64) / np.sqrt(D))[:n - T + 1 + i]
            m = max(s.max(), 0.0)
            w = np.exp(s - m)
            want[i, h] = w @ V[:len(s)] / (w.sum() + (max_len - n) * np.exp(-m))
    assert E.eagle_status_fetch(ws) == 0
    got = out[0].float().cpu().numpy()
    # bf16 output, fp16 weights, and fp32 running sums of up to 2^22 / (152 * 8 * 4) weights per lane
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * np.abs(want).max()).all()


# ------------------------------------------------------- used together ---

def test_cycles_over_the_cache_captured_and_replayed():
    """Prompt, then three cycles of store, attention and compaction in one captured graph replayed on
    another stream, against the plain forms run in the same order."""
    import torch
    E = _E()
    rng = np.random.default_rng(12)
    B, Hq, H, T, layers, dep = 3, 8, 2, 17, 2, 4
    kv = E.kvq_contiguous(B, Hq, H, D, layers, 256, 32)
    codes, scales = _buffers(kv, rng)
    vc, vs = P.views(kv, codes, scales)
    dc, ds = _dev(codes), _dev(scales)
    L = np.array([33, 1, 90])
    i32 = lambda a: _dev(np.asarray(a, np.int32))  # noqa: E731
    prompt = [_bf16(rng, (int(L.sum()), H, D)) for _ in range(2 * layers)]
    first = np.cumsum(L) - L
    ws = E.alloc_workspace(E.eagle_kvq_attention_workspace_bytes(kv, T))
    for l in range(layers):
        P.store(kv, l, int(L.max()), prompt[2 * l], prompt[2 * l + 1], first, [0] * B, L, vc, vs)
        E.eagle_kvq_store(kv, l, int(L.max()), _dev_bf16(prompt[2 * l]), _dev_bf16(prompt[2 * l + 1]), H * D, i32(first),
                          i32([0] * B), i32(L), dc, ds, ws)
    k = torch.empty(layers, 2, B * T, H, D, dtype=torch.bfloat16, device="cuda")
    q = torch.empty(B, T, Hq, D, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(layers, B, T, Hq, D, dtype=torch.bfloat16, device="cuda")
    mask = torch.empty(B, T, 1, dtype=torch.int32, device="cuda")
    d_L, d_n, d_acc = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(3))
    d_slots = torch.empty(B, dep + 1, dtype=torch.int32, device="cuda")
    new_len = torch.empty(B, dtype=torch.int32, device="cuda")

    def cycle():
        for l in range(layers):
            E.eagle_kvq_store(kv, l, T, k[l, 0], k[l, 1], H * D, None, d_L, d_n, dc, ds, ws)
            E.eagle_kvq_tree_attention(kv, T, q, dc, ds, l, d_L, mask, d_n, out[l], ws)
        E.eagle_kvq_compact(kv, dc, ds, d_L, d_acc, d_slots, dep + 1, new_len, ws)

    graph = None
    side = torch.cuda.Stream()
    for c in range(3):
        n = rng.integers(dep + 1, T + 1, B)
        see = _tree(rng, B, T, n)
        acc = rng.integers(0, dep + 1, B)
        slots = np.full((B, dep + 1), -1)
        for b in range(B):
            slots[b, :acc[b] + 1] = np.concatenate([[0], 1 + np.sort(rng.permutation(n[b] - 1)[:acc[b]])])
        hk, hq = _bf16(rng, (layers, 2, B * T, H, D), 1.5), _bf16(rng, (B, T, Hq, D), 1.5)
        for dst, src in ((k, _dev_bf16(hk)), (q, _dev_bf16(hq)), (mask, _dev(_pack_mask(see))), (d_L, i32(L)),
                         (d_n, i32(n)), (d_acc, i32(acc)), (d_slots, i32(slots))):
            dst.copy_(src)
        if graph is None:
            keep = dc.clone(), ds.clone()
            cycle()  # first calls set kernel attributes
            torch.cuda.synchronize()
            dc.copy_(keep[0]), ds.copy_(keep[1])
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                cycle()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.current_stream().wait_stream(side)
        want = []
        for l in range(layers):
            P.store(kv, l, T, hk[l, 0], hk[l, 1], None, L, n, vc, vs)
            want.append(P.attention(kv, T, hq, vc, vs, l, L, see, n))
        L = np.array(P.compact(kv, vc, vs, L, acc, slots))
        torch.cuda.synchronize()
        assert E.eagle_status_fetch(ws) == 0
        for l in range(layers):
            assert (np.abs(out[l].float().cpu().numpy() - want[l][0]) <= want[l][1]).all(), (c, l)
        assert (new_len.cpu().numpy() == L).all()
        assert (ds.cpu().numpy() == scales).all() and (dc.cpu().numpy() == codes).all(), c


def test_two_calls_at_once_on_their_own_workspaces():
    import torch
    E = _E()
    rng = np.random.default_rng(14)
    cases = []
    for s, (T, L) in enumerate(((1, [900, 40]), (61, [300, 1200]))):
        kv = E.kvq_contiguous(2, 32, 8, D, 1, 1400, 64)
        codes, scales = _buffers(kv, rng)
        q = _bf16(rng, (2, T, 32, D))
        want, tol = P.attention(kv, T, q, *P.views(kv, codes, scales), 0, L, None, None)
        ws = E.alloc_workspace(E.eagle_kvq_attention_workspace_bytes(kv, T))
        out = torch.empty(2, T, 32, D, dtype=torch.bfloat16, device="cuda")
        cases.append((torch.cuda.Stream(), kv, T, _dev_bf16(q), _dev(codes), _dev(scales), _dev(np.array(L, np.int32)), out, ws,
                      want, tol))
    torch.cuda.synchronize()
    for _ in range(20):
        for st, kv, T, q, codes, scales, L, out, ws, _, _ in cases:
            E.eagle_kvq_tree_attention(kv, T, q, codes, scales, 0, L, None, None, out, ws, stream=st)
    torch.cuda.synchronize()
    for *_, out, ws, want, tol in cases:
        assert E.eagle_status_fetch(ws) == 0
        assert (np.abs(out.float().cpu().numpy() - want) <= tol).all()


def test_row_blocks_without_rows_between_items_of_a_worker():
    """320 query rows per KV head: the second pair of row blocks has one block without rows, and workers pass from
    such items to full ones. Scales far apart, so that another tile's would show; repeated, bit for bit."""
    import torch
    E = _E()
    rng = np.random.default_rng(31)
    B, Hq, H, T = 24, 64, 8, 40
    kv = E.kvq_contiguous(B, Hq, H, D, 1, 1600, 16)
    codes, scales = _buffers(kv, rng, lo=-9, hi=-3)
    L = rng.integers(900, 1500, B)
    q = _bf16(rng, (B, T, Hq, D), 0.2)
    ws = E.alloc_workspace(E.eagle_kvq_attention_workspace_bytes(kv, T))
    dc, ds, dq, dl = _dev(codes), _dev(scales), _dev_bf16(q), _dev(L.astype(np.int32))
    runs = []
    for _ in range(30):
        out = torch.empty(B, T, Hq, D, dtype=torch.bfloat16, device="cuda")
        E.eagle_kvq_tree_attention(kv, T, dq, dc, ds, 0, dl, None, None, out, ws)
        runs.append(out)
    torch.cuda.synchronize()
    assert E.eagle_status_fetch(ws) == 0
    want, tol = P.attention(kv, T, q, *P.views(kv, codes, scales), 0, L, None, None)
    assert (np.abs(runs[0].float().cpu().numpy() - want) <= tol).all()
    assert all((r == runs[0]).all() for r in runs)


# ------------------------------------------- small products, NaN, limits ---

@pytest.mark.parametrize("T,L", [(1, [20, 333]), (61, [20, 333]), (1, [3000]), (61, [3000])])
def test_attention_zero_and_tiny_rows_over_small_scales(T, L):
    """Rows of q that are zero or tiny over blocks of zero K (scale 2^-126, as the store writes it) and over small
    scales: the factor of a score underflows, and the row is the mean of the V rows that it sees. Whole items, and
    one of 3000 positions that many workers share."""
    E = _E()
    rng = np.random.default_rng(40 + T)
    B, Hq, H = len(L), 8, 2
    kv = E.kvq_contiguous(B, Hq, H, D, 1, max(L) + T, 16)
    codes, scales = _buffers(kv, rng)
    vc, vs = P.views(kv, codes, scales)
    vs[:, 0, 0] = 2.0 ** rng.choice([-126.0, -60.0, -24.0, -9.0], vs[:, 0, 0].shape)
    vs[:, 0, 0, -5:] = 2.0 ** -126 if T > 1 else 2.0 ** -24
    zero = np.repeat(vs[:, 0, 0] == 2.0 ** -126, 16, 1)[:, :kv.max_len]
    vc[:, 0, 0][zero] = 0
    q = _bf16(rng, (B, T, Hq, D), 2.0)
    size = 2.0 ** np.array([-200.0, -130.0, -100.0, -40.0, -20.0, -15.0, -14.0, 0.0])
    q = P.bf16_round(q * size[rng.permutation(B * T * Hq) % 8].reshape(B, T, Hq, 1))
    q[:, 0, ::2] = 0.0
    see = _tree(rng, B, T, [T] * B) if T > 1 else None
    want, tol = P.attention(kv, T, q, vc, vs, 0, L, see, None)
    got, status = _attend(E, kv, T, L, None, see, codes, scales, q, 0)
    assert status == 0
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4])


@pytest.mark.parametrize("T,L,where", [(T, L, where) for T, L in ((1, 40), (12, 40), (61, 40), (1, 5000), (61, 5000))
                                       for where in ("prefix", "slot", "q") if T > 1 or where != "slot"])
def test_attention_nan_in_k_or_q_reaches_the_rows_that_see_it_only(T, L, where):
    """A NaN among K's codes or in q: the rows that see it are zero or NaN, all others as without it, whether an
    item is one worker's or shared by many."""
    E = _E()
    rng = np.random.default_rng(50 + T)
    Hq, H = 2 if T == 12 else 8, 2
    G = Hq // H
    kv = E.kvq_contiguous(1, Hq, H, D, 1, L + T, 32)
    codes, scales = _buffers(kv, rng)
    vc, vs = P.views(kv, codes, scales)
    q = _bf16(rng, (1, T, Hq, D), 2.0)
    see = _tree(rng, 1, T, [T]) if T > 1 else None
    want, tol = P.attention(kv, T, q, vc, vs, 0, [L], see, None)
    hit = np.zeros((T, Hq), bool)
    if where == "q":
        q[0, T - 1, Hq - 1, 5] = np.nan
        hit[T - 1, Hq - 1] = True
    else:
        at = 3 if where == "prefix" else T // 2
        vc[0, 0, 0, at if where == "prefix" else L + at, 1, 77] = 0x7F
        hit[:, G:] = (np.ones(T, bool) if where == "prefix" else see[0, :, at])[:, None]
    got, status = _attend(E, kv, T, [L], None, see, codes, scales, q, 0)
    assert status == 0
    got, want, tol = got[0], want[0], tol[0]
    assert ((got[hit] == 0) | np.isnan(got[hit])).all()
    assert (np.abs(got - want) <= tol)[~hit].all()


def test_decode_steps_issued_back_to_back():
    """Sixty decode steps, store then attention, with nothing in between that waits: each attention reads the codes,
    the scales (which grow in most steps) and the lengths as the calls just before it left them."""
    import torch
    E = _E()
    rng = np.random.default_rng(70)
    B, Hq, H, steps = 3, 8, 2, 60
    kv = E.kvq_contiguous(B, Hq, H, D, 1, 700, 32)
    codes, scales = _buffers(kv, rng)
    vc, vs = P.views(kv, codes, scales)
    dc, ds = _dev(codes), _dev(scales)
    start = np.array([0, 30, 600])
    grow = (1.12 ** np.arange(steps))[:, None, None, None, None]
    rows, q = _bf16(rng, (steps, 2, B, H, D), 0.1) * grow, _bf16(rng, (steps, B, 1, Hq, D))
    rows = P.bf16_round(rows)
    d_rows, d_q = _dev_bf16(rows), _dev_bf16(q)
    out = torch.full((steps, B, 1, Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    d_start, one = _dev(start.astype(np.int32)), torch.ones(B, dtype=torch.int32, device="cuda")
    ws = E.alloc_workspace(E.eagle_kvq_attention_workspace_bytes(kv, 1))
    torch.cuda.synchronize()
    for s in range(steps):
        E.eagle_kvq_store(kv, 0, 1, d_rows[s, 0], d_rows[s, 1], H * D, None, d_start, None, dc, ds, ws)
        E.eagle_kvq_tree_attention(kv, 1, d_q[s], dc, ds, 0, d_start, None, None, out[s], ws)
        d_start.add_(one)
    torch.cuda.synchronize()
    assert E.eagle_status_fetch(ws) == 0
    got = out.float().cpu().numpy()
    for s in range(steps):
        P.store(kv, 0, 1, rows[s, 0], rows[s, 1], None, start + s, None, vc, vs)
        want, tol = P.attention(kv, 1, q[s], vc, vs, 0, start + s, None, None)
        assert (np.abs(got[s] - want) <= tol).all(), s
    assert (ds.cpu().numpy() == scales).all() and (dc.cpu().numpy() == codes).all()


@pytest.mark.parametrize("T,L", [(1, 40), (12, 40), (61, 40), (61, 5000)])
def test_attention_nan_in_v_stays_in_its_column_and_head(T, L):
    E = _E()
    rng = np.random.default_rng(60 + T)
    Hq, H = 2 if T == 12 else 8, 2
    G = Hq // H
    kv = E.kvq_contiguous(1, Hq, H, D, 1, L + T, 32)
    codes, scales = _buffers(kv, rng)
    vc, vs = P.views(kv, codes, scales)
    q = _bf16(rng, (1, T, Hq, D), 2.0)
    see = _tree(rng, 1, T, [T]) if T > 1 else None
    want, tol = P.attention(kv, T, q, vc, vs, 0, [L], see, None)
    vc[0, 0, 1, L + T // 2, 1, 77] = 0xFF
    got, status = _attend(E, kv, T, [L], None, see, codes, scales, q, 0)
    assert status == 0
    ok = np.abs(got[0] - want[0]) <= tol[0]
    assert np.isnan(got[0][:, G:, 77]).all()
    ok[:, G:, 77] = True
    assert ok.all()


def test_short_items_launched_again_and_again():
    """Workers with one tile or two, which leave right behind their last product, in launches that follow one another at
    once: every run is the first, bit for bit."""
    import torch
    E = _E()
    rng = np.random.default_rng(80)
    B, Hq, H, T = 5, 32, 8, 61
    L = np.array([0, 1, 3, 64, 130])
    kv = E.kvq_contiguous(B, Hq, H, D, 1, 256, 16)
    codes, scales = _buffers(kv, rng)
    q = _bf16(rng, (B, T, Hq, D), 2.0)
    want, tol = P.attention(kv, T, q, *P.views(kv, codes, scales), 0, L, None, None)
    ws = E.alloc_workspace(E.eagle_kvq_attention_workspace_bytes(kv, T))
    dc, ds, dq, dl = _dev(codes), _dev(scales), _dev_bf16(q), _dev(L.astype(np.int32))
    runs = torch.empty(200, B, T, Hq, D, dtype=torch.bfloat16, device="cuda")
    for out in runs:
        E.eagle_kvq_tree_attention(kv, T, dq, dc, ds, 0, dl, None, None, out, ws)
    torch.cuda.synchronize()
    assert E.eagle_status_fetch(ws) == 0
    assert (np.abs(runs[0].float().cpu().numpy() - want) <= tol).all()
    assert (runs == runs[0]).all()


@pytest.mark.parametrize("T,L", [(1, 40), (12, 40), (61, 40), (1, 5000), (61, 5000)])
@pytest.mark.parametrize("value", [np.inf, -np.inf])
def test_attention_infinities_in_q_do_not_pass_for_numbers(T, L, value):
    """A row of q with an infinity is zero or NaN, as one with a NaN; the others are as without it."""
    E = _E()
    rng = np.random.default_rng(90 + T)
    Hq, H = 2 if T == 12 else 8, 2
    kv = E.kvq_contiguous(1, Hq, H, D, 1, L + T, 32)
    codes, scales = _buffers(kv, rng, lo=-30, hi=-4)
    vc, vs = P.views(kv, codes, scales)
    vs[:, :, 0] = 2.0 ** -30 / np.float32(1.4426950408889634 / np.sqrt(128.0))  # factors of the scores: powers of two
    q = _bf16(rng, (1, T, Hq, D), 2.0)
    want, tol = P.attention(kv, T, q, vc, vs, 0, [L], None, None)
    q[0, T // 2, Hq - 1, 77] = value
    got, status = _attend(E, kv, T, [L], None, None, codes, scales, q, 0)
    assert status == 0
    ok = np.abs(got[0] - want[0]) <= tol[0]
    row = got[0, T // 2, Hq - 1]
    assert ((row == 0) | np.isnan(row)).all()
    ok[T // 2, Hq - 1] = True
    assert ok.all()


@pytest.mark.parametrize("T,L", [(1, 200), (12, 200), (61, 200), (1, 5000), (61, 5000)])
def test_attention_subnormal_and_huge_v_scales(T, L):
    """V scales from fp32's subnormal numbers to 2^100, whole sequences of one size and blocks of both."""
    E = _E()
    rng = np.random.default_rng(95 + T)
    B, Hq, H = 5, 2 if T == 12 else 8, 2
    kv = E.kvq_contiguous(B, Hq, H, D, 1, L + T, 32)
    codes, scales = _buffers(kv, rng)
    vc, vs = P.views(kv, codes, scales)
    sizes = (-149.0, -140.0, -127.0, 100.0)
    for b, e in enumerate(sizes):
        vs[b, :, 1] = 2.0 ** e
    vs[4, :, 1] = 2.0 ** rng.choice(np.array([-149.0, -130.0, -126.0, -120.0]), vs[4, :, 1].shape)
    q = _bf16(rng, (B, T, Hq, D), 1.0)
    want, tol = P.attention(kv, T, q, vc, vs, 0, [L] * B, None, None)
    got, status = _attend(E, kv, T, [L] * B, None, None, codes, scales, q, 0)
    assert status == 0
    # beside tol (without its 1e-30): half of bf16's subnormal step, half of fp32's in the partial results, the
    # normalisation and the products, and the weights' 2^-25 under the least reference of V's scales, 2^-126
    more = 2.0 ** -134 + 8 * 2.0 ** -150 + (L + T) * 2.0 ** -25 * 448 * 2.0 ** -126
    assert (np.abs(got - want) <= tol - 1e-30 + more).all()
