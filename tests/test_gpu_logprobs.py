"""Token log-probabilities, ranks, entropies and alternatives on the GPU against
a plain 64-bit form (plain64.logprobs).

Bounds. A row's sum S of V exponentials: each is off by 2^-22 (the
approximate exp2) and by its argument's rounding, 2^-24 of |y| (weighted by
2^y, at most a few units); partial sums per thread hold at most 2^9 terms and
are joined in fewer than 2^5 steps, so S is within 2^-14 relative and, its
errors being of either sign, far closer; ln S is then within 2^-14. What the
tests hold the outputs to is 2^-17 for ln S (a row of 2^18 entries summed by
2^11 threads or more: at most 2^7 + 2^5 sequential additions of 2^-24 each),
plus 2^-22 of the value itself for y and the final subtraction. The entropy is
a mean of |y| over the same sums: 2^-16 (1 + entropy). Ranks and ids are exact."""
import math

import numpy as np
import pytest

import plain64 as P

pytestmark = pytest.mark.gpu


def _E():
    from speculative_decoding_dynamic_gb300 import eagle as E
    return E


def _run(E, x, slots, tokens, n_alt, temperature, optional=True, ws=None):
    import torch
    n, rows, V = x.shape
    per = tokens.shape[1]
    cfg = E.TreeCfg(1, V, 1, 1, 1, 0.0, E.EAGLE_BF16 if x.dtype == torch.bfloat16 else E.EAGLE_F32)
    ws = E.alloc_workspace(E.eagle_workspace_bytes(cfg))
    f = lambda *s: torch.full(s, 777.0, device="cuda")  # noqa: E731
    i = lambda *s: torch.full(s, 777, dtype=torch.int32, device="cuda")  # noqa: E731
    lp, rank, ent, ids, alts = f(n, per), i(n, per), f(n, per), i(n, per, n_alt), f(n, per, n_alt)
    dev = lambda a: None if a is None else torch.from_numpy(np.asarray(a, np.int32)).cuda()  # noqa: E731
    E.eagle_token_logprobs(cfg, ws, n, per, rows, x, temperature, dev(slots), dev(tokens), n_alt, lp,
                           rank if optional else None, ent if optional else None, ids if n_alt else None,
                           alts if n_alt else None)
    status = E.eagle_status_fetch(ws)
    return [t.cpu().numpy() for t in (lp, rank, ent, ids, alts)], status


def _check(E, x, slots, tokens, n_alt, temperature):
    (lp, rank, ent, ids, alts), status = _run(E, x, slots, tokens, n_alt, temperature)
    assert status == 0
    host = x.double().cpu().numpy()
    for b in range(tokens.shape[0]):
        for j in range(tokens.shape[1]):
            s = j if slots is None else slots[b, j]
            if s < 0 or tokens[b, j] < 0:
                assert math.isnan(lp[b, j]) and math.isnan(ent[b, j]) and rank[b, j] == -1
                assert (ids[b, j] == -1).all() and np.isnan(alts[b, j]).all()
                continue
            wl, wr, we, wi, wa = P.logprobs(host[b, s], tokens[b, j], temperature, n_alt)
            at = (b, j)
            assert rank[at] == wr, at
            k = len(wi)
            assert (ids[at][:k] == wi).all() and (ids[at][k:] == -1).all(), at
            assert (alts[at][k:] == -np.inf).all()
            assert abs(ent[at] - we) <= 2.0 ** -16 * (1 + we), (at, ent[at], we)
            for got, want in [(lp[at], wl)] + list(zip(alts[at], wa)):
                assert got == want or abs(got - want) <= 2.0 ** -17 + 2.0 ** -22 * abs(want), (at, got, want)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,rows,per,V,k,temperature,slots", [
    (1, 1, 1, 8, 16, 1.0, False),            # fewer entries than alternatives
    (1, 3, 3, 1000, 0, 0.7, False),
    (2, 9, 7, 4096, 5, 1.0, True),
    (1, 1, 1, 128256, 16, 1.0, False),       # one row over eight CTAs
    (3, 5, 4, 131072, 1, 1.7, True),         # the longest fp32 row
    (700, 1, 1, 8200, 3, 1.0, False),        # one CTA per row
])
def test_random_rows(dtype, n, rows, per, V, k, temperature, slots):
    import torch
    E = _E()
    rng = np.random.default_rng(V + n)
    x = torch.from_numpy(rng.standard_normal((n, rows, V)).astype(np.float32) * 2.5).cuda()
    x = x.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    sl = rng.integers(-1, rows, (n, per)) if slots else None
    tokens = rng.integers(0, V, (n, per))
    tokens[:, ::2] = x[:, :1].float().argmax(-1).cpu().numpy()
    if per > 2:
        tokens[0, 2] = -1
    _check(E, x, sl, tokens, k, temperature)


def test_the_longest_bf16_row():
    import torch
    E = _E()
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.standard_normal((1, 2, 262144)).astype(np.float32) * 2.5).cuda().to(torch.bfloat16)
    _check(E, x, None, np.array([[262143, 0]]), 16, 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_ties_masks_and_extreme_rows(dtype):
    """Equal logits (more of them at the top than the candidate scratch holds), masked entries of -inf and of the
    type's lowest value, a row that is masked but for one entry, rows of one value, large logits, both zeros."""
    import torch
    E = _E()
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    rng = np.random.default_rng(2)
    V = 32768
    lowest = float(torch.finfo(dt).min)
    base = rng.standard_normal((12, V)).astype(np.float32)
    base[0] = np.round(base[0])              # thousands of ties
    base[1, rng.permutation(V)[:V // 2]] = -np.inf
    base[2, rng.permutation(V)[:V // 2]] = lowest
    base[3] = -np.inf
    base[3, 777] = 3.0                       # certain
    base[4] = 0.25                           # uniform
    base[5] = lowest                         # nothing but the lowest value: uniform
    base[6] = base[6] * 0.01 + 300.0
    base[7] = base[7] * 1e4
    base[8] = np.where(rng.random(V) < 0.5, 0.0, -0.0)
    base[9] = -np.inf
    base[9, 5:25] = lowest
    base[10, :-3] = -1e4
    base[11] = np.sort(base[11])             # ascending
    x = torch.from_numpy(base).cuda().to(dt)[None]
    tok = np.array([[17, 0, 1, 777, 9, 30000, 5, 6, 31999, 7, V - 1, 0]])
    masked = int(np.nonzero(np.isinf(base[1]))[0][5])
    tok[0, 1] = masked
    tok[0, 2] = int(np.nonzero(base[2] == np.float32(lowest))[0][9])
    _check(E, x, None, tok, 16, 1.0)
    _check(E, x[:, :5], None, tok[:, :5], 3, 1.3)
    (lp, rank, _, _, _), status = _run(E, x[:, 3:4].contiguous(), None, np.array([[778]]), 0, 1.0)
    # above token 778: the certain one, and the 777 masked ones of lower id
    assert status == 0 and lp[0, 0] == -np.inf and rank[0, 0] == 1 + 777


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_non_finite_rows_raise_status_1(value):
    import torch
    E = _E()
    for V, at in ((64, 3), (128256, 99999)):
        x = torch.zeros(1, 2, V, device="cuda")
        x[0, 1, at] = value
        (lp, _, _, _, _), status = _run(E, x, None, np.array([[1, 2]]), 4, 1.0)
        assert status == 1 and lp[0, 0] == np.float32(-math.log(V)) or abs(lp[0, 0] + math.log(V)) < 1e-5
        assert math.isnan(lp[0, 1])
    x = torch.full((1, 1, 64), float("-inf"), device="cuda")
    _, status = _run(E, x, None, np.array([[1]]), 4, 1.0)
    assert status == 1


def test_tokens_and_slots_out_of_range_raise_status_3():
    import torch
    E = _E()
    x = torch.zeros(2, 3, 64, device="cuda")
    for slots, tokens in (([[0, 1], [2, 3]], [[1, 1], [1, 1]]), ([[0, 1], [2, 0]], [[1, 64], [1, 1]])):
        (lp, rank, ent, ids, alts), status = _run(E, x, np.array(slots), np.array(tokens), 2, 1.0)
        assert status == 3
        bad = np.array([[False, tokens[0][1] == 64], [False, slots[1][1] == 3]])
        assert (np.isnan(lp) == bad).all() and ((rank == -1) == bad).all()


def test_optional_outputs_and_capture():
    import torch
    E = _E()
    rng = np.random.default_rng(4)
    x = torch.from_numpy(rng.standard_normal((2, 4, 4096)).astype(np.float32)).cuda()
    tokens = rng.integers(0, 4096, (2, 4))
    (lp, rank, _, _, _), status = _run(E, x, None, tokens, 0, 1.0, optional=False)
    assert status == 0 and (rank == 777).all()
    (want, *_), _ = _run(E, x, None, tokens, 8, 1.0)
    assert (lp == want).all()  # the other outputs change nothing
    cfg = E.TreeCfg(1, 4096, 1, 1, 1, 0.0, E.EAGLE_F32)
    ws = E.alloc_workspace(E.eagle_workspace_bytes(cfg))
    out, tok = torch.zeros(2, 4, device="cuda"), torch.from_numpy(tokens.astype(np.int32)).cuda()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        E.eagle_token_logprobs(cfg, ws, 2, 4, 4, x, 1.0, None, tok, 0, out)
    x.add_(torch.randn_like(x))
    (want, *_), _ = _run(E, x, None, tokens, 0, 1.0)
    g.replay()
    torch.cuda.synchronize()
    assert (out.cpu().numpy() == want).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("temperature", [2.0 ** -126, 1e-20, 1e-3, 1e30])
def test_extreme_temperatures(dtype, temperature):
    """Differences over the temperature past fp32's range: probability 0 for all but the largest, entropy 0."""
    import torch
    rng = np.random.default_rng(11)
    x = torch.from_numpy(rng.permutation(4096).astype(np.float32)[None, None] / 8 - 100).cuda()
    x[0, 0, 7] = 3e38
    x[0, 0, 9] = -3e38
    x = x.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    E = _E()
    (lp, rank, ent, _, _), status = _run(E, x, None, np.array([[7]]), 2, temperature)
    assert status == 0 and rank[0, 0] == 0
    if temperature < 1e10:
        assert lp[0, 0] == 0 and ent[0, 0] == 0
    else:  # 3e38 / 1e30 = 3e8 over the others
        assert lp[0, 0] == 0 and abs(ent[0, 0]) <= 2.0 ** -16


def test_rows_over_clusters_of_every_size_again_and_again():
    """Rows split over 2, 4 and 8 CTAs, as short as they are split at all, so that the shares meet with little
    work before; other values in every run."""
    import torch
    E = _E()
    rng = np.random.default_rng(13)
    for V in (8192, 16384, 32768):  # fp32: two, four and eight pieces of 16 KB
        for run in range(40):
            x = torch.from_numpy(rng.standard_normal((1, 5, V)).astype(np.float32) * 2.5).cuda()
            _check(E, x, None, rng.integers(0, V, (1, 5)), 4, 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("V", [64, 128256])
def test_rows_without_a_distribution_give_status_1_and_padding_values(dtype, value, V):
    """A row with one NaN or +inf, or with nothing but NaN, +inf or -inf: the status is 1, the row's outputs are
    those of padding, none is left as it was, and the other row is unharmed."""
    import torch
    E = _E()
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    for everywhere in (False, True):
        if value == float("-inf") and not everywhere:
            continue  # a masked entry
        x = torch.zeros(1, 2, V, device="cuda", dtype=dt)
        x[0, 1, slice(None) if everywhere else V - 3] = value
        (lp, rank, ent, ids, alts), status = _run(E, x, None, np.array([[1, 2]]), 4, 1.0)
        assert status == 1
        assert abs(lp[0, 0] + math.log(V)) < 2.0 ** -16 and rank[0, 0] == 1 and (ids[0, 0] == np.arange(4)).all()
        assert math.isnan(lp[0, 1]) and math.isnan(ent[0, 1]) and rank[0, 1] == -1
        assert (ids[0, 1] == -1).all() and np.isnan(alts[0, 1]).all()
