"""8-bit rows and products at sizes where a CTA (or a pair) goes round its loop more than once: a pair's second and
third tile, a norm's second turn with rows on their way. Tolerances as in test_gpu_fp8."""
import numpy as np
import pytest
import torch
import plain64 as P
import plain64_fp8 as F
from test_gpu_fp8 import DT, _check_codes, _check_linear, _code, _np, _operands, _round_to, _rows, _ws

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E():
    from speculative_decoding_dynamic_gb300 import eagle
    return eagle


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _pairs_of(rows, out_dim):
    """(rows of an accumulator, tiles) of the product by pairs of CTAs: accumulators of up to 224 rows, an even number of
    them, two to a tile of 256 weight rows."""
    subs = -(-rows // 224)
    per = -(-rows // (subs + subs % 2))
    nr = -(-per // 16) * 16
    return nr, -(-rows // (2 * nr)) * -(-out_dim // 256)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,out_dim,in_dim,nr,turns", [
    (225, 20000, 272, 128, 2), (300, 20001, 272, 160, 2), (300, 40000, 272, 160, 3),
    (448, 21000, 1040, 224, 2), (430, 39333, 656, 224, 3), (672, 20001, 640, 176, 3), (400, 20008, 528, 208, 2),
    (449, 10001, 4240, 128, 2), (449, 10004, 4240, 128, 2), (448, 19600, 4240, 224, 2)])
def test_pairs_with_several_tiles(E, dt, rows, out_dim, in_dim, nr, turns):
    """Even and odd output widths (bulk and plain stores), fp32 outputs added up over two parts of K."""
    got, tiles = _pairs_of(rows, out_dim)
    assert got == nr and tiles > (turns - 1) * (_sms() // 2)
    rng = np.random.default_rng(rows * 1021 + out_dim * 43 + in_dim)
    ops = _operands(rng, rows, out_dim, in_dim)
    around = torch.full((rows * out_dim + 128,), 7.0, dtype=DT[dt], device="cuda")
    out, ws = around[64:-64].view(rows, out_dim), _ws(E)
    dev = [torch.from_numpy(t).cuda() for t in ops]
    E.eagle_linear_fp8(rows, out_dim, in_dim, *dev, _code(E, dt), out, ws)
    assert E.eagle_status_fetch(ws) == 0
    _check_linear(out, *ops, dt)
    assert bool((around[:64] == 7).all()) and bool((around[-64:] == 7).all())
    again = torch.empty_like(out)
    for _ in range(2):
        E.eagle_linear_fp8(rows, out_dim, in_dim, *dev, _code(E, dt), again, ws)
        assert torch.equal(out, again)


@pytest.mark.parametrize("rows,out_dim", [(300, 20001), (448, 21000)])
def test_scales_and_nan_of_later_tiles(E, rows, out_dim):
    """One code a row picks a weight column under both scales: exact, so no tile has another's scales; a NaN scale of the
    last weight block reaches its own outputs."""
    rng = np.random.default_rng(rows)
    in_dim = 1168
    x, xs, w, wsc = _operands(rng, rows, out_dim, in_dim)
    x[:] = 0
    at = rng.integers(0, in_dim, rows)
    x[np.arange(rows), at] = 0x38  # 1.0
    out = torch.empty(rows, out_dim, device="cuda")
    dev = [torch.from_numpy(t).cuda() for t in (x, xs, w, wsc)]
    E.eagle_linear_fp8(rows, out_dim, in_dim, *dev, E.EAGLE_F32, out)
    want = F.dequant_weight(w, wsc)[:, at].T * 2.0 ** (xs[np.arange(rows), at // 128].astype(np.float64) - 127)[:, None]
    assert np.array_equal(_np(out), want)
    last = (out_dim - 1) // 128
    dev[3][last, 3] = 255
    E.eagle_linear_fp8(rows, out_dim, in_dim, *dev, E.EAGLE_F32, out)
    nan = torch.isnan(out)
    assert bool(nan[:, last * 128:].all()) and not bool(nan[:, :last * 128].any())


def test_pairs_captured(E):
    """A graph of two products by pairs, one after the other, replayed on other inputs."""
    rng = np.random.default_rng(17)
    shapes = ((300, 20001, 272), (448, 21000, 528))
    calls = []
    for s in shapes:
        calls.append([[torch.from_numpy(t).cuda() for t in _operands(rng, *s)], torch.empty(s[0], s[1], dtype=torch.bfloat16, device="cuda")])

    def run():
        for (rows, out_dim, in_dim), (ops, out) in zip(shapes, calls):
            E.eagle_linear_fp8(rows, out_dim, in_dim, *ops, E.EAGLE_BF16, out)

    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    new = [_operands(rng, *s) for s in shapes]
    for (ops, _), n in zip(calls, new):
        for a, b in zip(ops, n):
            a.copy_(torch.from_numpy(b))
    g.replay()
    torch.cuda.synchronize()
    for (_, out), n in zip(calls, new):
        _check_linear(out, *n, "bf16")


def _most_rows(dim, entries):
    """Rows that the norm can have at once at most: 64 warps an SM, a warp for `entries` of a row."""
    return _sms() * 64 // -(-dim // entries)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("form", ["norm", "residual", "codes", "codes_residual"])
@pytest.mark.parametrize("rows,dim", [(5003, 1040), (3301, 2064), (2500, 4096), (1303, 8208), (10007, 656), (20011, 272)])
def test_norm_goes_round(E, dt, form, rows, dim):
    """More rows than run at once, the last turn ragged; a row past fp32's squares and one with a NaN in later turns."""
    two = dim > 1024 and "residual" not in form  # two blocks of 128 a thread
    assert rows > _most_rows(dim, 1024 if two else 512)
    rng = np.random.default_rng(rows * 100019 + dim)
    x = _rows(rng, rows, dim, dt)
    far, bad = rows - 2, rows - 5
    x[far] = x[far] / x[far].abs().max() * 2e30
    x[bad, dim - 1] = float("nan")
    res = _rows(rng, rows, dim, dt) if "residual" in form else None
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(dim)).to(DT[dt]).cuda() if not form.startswith("codes") else None
    total = torch.empty_like(x) if res is not None else None
    codes, scales = E.alloc_fp8(rows + 1, dim)
    codes.fill_(99)
    scales.fill_(99)
    ws = _ws(E)
    E.eagle_rmsnorm_fp8(rows, dim, _code(E, dt), x, dim, res, total, w, 1e-5, codes, scales, ws)
    assert E.eagle_status_fetch(ws) == 1
    good = np.arange(rows) != bad
    s, y = F.norm_rows(_np(x)[good], None if res is None else _np(res)[good], None if w is None else _np(w),
                       float(np.float32(1e-5)), _round_to(dt))
    if total is not None:
        assert np.array_equal(_np(total)[good], s)
    keep = torch.from_numpy(np.nonzero(good)[0]).cuda()
    _check_codes(y, codes[keep], scales[keep])
    lost = (F.blocks(codes[bad:bad + 1].cpu().numpy())[0][:, 0] == 0x7F).sum()
    assert lost == (1 if w is None else -(-dim // 128))
    assert bool((codes[rows] == 99).all()) and bool((scales[rows] == 99).all())
