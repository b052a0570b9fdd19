"""Rows of 8-bit codes with power-of-two scales, their weights and their product
against plain 64-bit forms.

Tolerances. rmsnorm: y in fp32 is within 2^-19 of the exact one (at most 24
roundings of 2^-24 in the sum of squares, halved by the root, and four more), so
a code stands for a value within half a step of it plus that, and a scale is the
rule's for an amax within 2^-19. linear: fp32 sums in an unspecified order are
within in_dim 2^-23 of the sum of the products' magnitudes; a bf16 output is
rounded once more (half a step, 2^-8 of the value at most)."""
import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))
import plain64 as P  # noqa: E402
import plain64_fp8 as F  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS_Y = 2.0 ** -19


@pytest.fixture(scope="module")
def E():
    from speculative_decoding_dynamic_gb300 import eagle
    return eagle


def _code(E, dt):
    return E.EAGLE_BF16 if dt == "bf16" else E.EAGLE_F32


def _ws(E):
    return E.alloc_workspace(E.eagle_workspace_bytes(E.TreeCfg(1, 1024, 1, 1, 1, 0.0, E.EAGLE_F32)))


def _np(t):
    return t.double().cpu().numpy()


def _rows(rng, rows, dim, dt, scale=1.0):
    """Rows in a wide range of sizes, some blocks of zeros, one channel far above the others."""
    x = rng.standard_normal((rows, dim)) * np.exp(2 * rng.standard_normal((rows, 1))) * scale
    x[:, dim // 3] *= 50
    x[rows // 2, :min(dim, 256)] = 0
    return torch.from_numpy(x).to(DT[dt]).cuda()


def _round_to(dt):
    return P.bf16_round if dt == "bf16" else (lambda v: np.asarray(v, np.float32))


def _check_codes(y, codes, scales, eps=EPS_Y):
    codes, scales = codes.cpu().numpy(), scales.cpu().numpy()
    rows, dim = y.shape
    nb = (dim + 127) // 128
    assert scales.shape[1] == F.stride(dim) and not scales[:, nb:].any()
    amax = np.abs(F.blocks(y)).max(2)
    low, high = F.scale_bytes(amax * (1 - eps)), F.scale_bytes(amax * (1 + eps))
    assert np.all((scales[:, :nb] == low) | (scales[:, :nb] == high))
    v = y / 2.0 ** (np.repeat(scales[:, :nb].astype(np.float64), 128, 1)[:, :dim] - 127)
    assert np.all(np.abs(P.E4M3[codes] - v) <= F.half_step(v * (1 + eps)) + eps * np.abs(v))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,dim", [(1, 16), (3, 128), (9, 400), (10, 512), (33, 528), (2, 1040), (10, 4096), (5, 5120),
                                      (3, 8192), (2, 16384), (700, 656)])
@pytest.mark.parametrize("form", ["norm", "residual", "codes", "codes_residual"])
def test_rmsnorm(E, dt, rows, dim, form):
    rng = np.random.default_rng(rows * 100003 + dim)
    x = _rows(rng, rows, dim, dt)
    res = _rows(rng, rows, dim, dt) if "residual" in form else None
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(dim)).to(DT[dt]).cuda() if not form.startswith("codes") else None
    total = torch.empty_like(x) if res is not None else None
    codes, scales = E.alloc_fp8(rows, dim)
    scales.fill_(99)
    ws = _ws(E)
    E.eagle_rmsnorm_fp8(rows, dim, _code(E, dt), x, dim, res, total, w, 1e-5, codes, scales, ws)
    assert E.eagle_status_fetch(ws) == 0
    s, y = F.norm_rows(_np(x), None if res is None else _np(res), None if w is None else _np(w), float(np.float32(1e-5)),
                       _round_to(dt))
    if total is not None:
        assert np.array_equal(_np(total), s)
    _check_codes(y, codes, scales)


def test_rmsnorm_in_place_strided_and_untouched(E):
    """The sum over the residual, rows inside wider ones, bytes around the outputs left as they were."""
    rng = np.random.default_rng(5)
    rows, dim, stride = 13, 656, 1024
    wide = _rows(rng, 3 * rows, stride, "bf16").view(3, rows, stride)
    x, res = wide[0][:, 64:64 + dim], wide[1][:, 64:64 + dim]
    before, s0 = wide.clone(), _np(x) + _np(res)
    codes = torch.full((rows + 2, dim), 7, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows + 2, F.stride(dim)), 7, dtype=torch.uint8, device="cuda")
    w = torch.ones(dim, dtype=torch.bfloat16, device="cuda")
    E.eagle_rmsnorm_fp8(rows, dim, E.EAGLE_BF16, x, stride, res, res, w, 1e-5, codes[1:-1], scales[1:-1])
    s, y = F.norm_rows(s0, None, _np(w), float(np.float32(1e-5)), None)
    stored = P.bf16_round(s)
    assert np.array_equal(_np(wide[1][:, 64:64 + dim]), stored)
    _check_codes(F.norm_rows(stored, None, _np(w), float(np.float32(1e-5)), None)[1], codes[1:-1], scales[1:-1])
    before[1, :, 64:64 + dim] = wide[1, :, 64:64 + dim]
    assert torch.equal(before, wide)
    for t in (codes, scales):
        assert bool((t[0] == 7).all()) and bool((t[-1] == 7).all())


@pytest.mark.parametrize("dim", [256, 4096])
def test_rmsnorm_far_and_broken_rows(E, dim):
    """Squares past fp32's range, tiny rows, rows of zeros, infinities and NaN: the others are as they are alone."""
    rng = np.random.default_rng(dim)
    x = _rows(rng, 12, dim, "fp32")
    x[1] *= 1e30
    x[2] *= 1e-30
    x[3] = 0
    x[4, 5] = float("inf")
    x[5, dim - 1] = float("nan")
    x[6] = 3.0e38
    x[7] = torch.where(torch.arange(dim, device="cuda") % 2 == 0, 3.0e38, 1e-3)
    w = torch.ones(dim, device="cuda")
    codes, scales = E.alloc_fp8(12, dim)
    ws = _ws(E)
    E.eagle_rmsnorm_fp8(12, dim, E.EAGLE_F32, x, dim, None, None, w, 1e-6, codes, scales, ws)
    assert E.eagle_status_fetch(ws) == 1
    good = [i for i in range(12) if i not in (4, 5)]
    _, y = F.norm_rows(_np(x)[good], None, _np(w), float(np.float32(1e-6)), None)
    _check_codes(y, codes[good], scales[good])
    for i in (4, 5):
        assert bool((codes[i] == 0x7F).all()) and bool((scales[i, :dim // 128] == 127).all())
    # without a norm only the blocks that hold one are lost
    E.eagle_rmsnorm_fp8(12, dim, E.EAGLE_F32, x, dim, None, None, None, 0.0, codes, scales, ws)
    assert E.eagle_status_fetch(ws) == 1
    _check_codes(_np(x)[good], codes[good], scales[good])
    lost = (codes == 0x7F).view(12, -1, 128).all(2).sum(1).tolist()
    assert lost == [1 if i in (4, 5) else 0 for i in range(12)]


def test_scale_border(E):
    """Blocks whose largest value is at, just under and just over 448 times a power of two."""
    x = torch.zeros(6, 128, device="cuda")
    x[:, 3] = torch.tensor([448.0, 448.00003, 447.99997, 7.0, 7.0000005, 2.0 ** -130], device="cuda")
    codes, scales = E.alloc_fp8(6, 128)
    E.eagle_rmsnorm_fp8(6, 128, E.EAGLE_F32, x, 128, None, None, None, 0.0, codes, scales)
    assert scales[:, 0].tolist() == [127, 128, 127, 121, 122, 1]
    assert codes[:5, 3].tolist() == [0x7E, 0x76, 0x7E, 0x7E, 0x76]


@pytest.mark.parametrize("out_dim,in_dim", [(1, 16), (128, 128), (130, 144), (257, 400), (128, 1024), (300, 528)])
def test_pack(E, out_dim, in_dim):
    rng = np.random.default_rng(out_dim * 7 + in_dim)
    w = _rows(rng, out_dim, in_dim, "bf16", 0.02)
    codes, scales = E.alloc_fp8(out_dim, in_dim, -(-out_dim // 128))
    scales.fill_(9)
    E.eagle_linear_fp8_pack(out_dim, in_dim, w, codes, scales)
    y, sc = _np(w), scales.cpu().numpy()
    nb = -(-in_dim // 128)
    assert not sc[:, nb:].any()
    for i in range(sc.shape[0]):
        for j in range(nb):
            part = y[i * 128:(i + 1) * 128, j * 128:(j + 1) * 128]
            assert sc[i, j] == F.scale_bytes(np.abs(part).max())
            assert np.array_equal(P.E4M3[codes.cpu().numpy()[i * 128:(i + 1) * 128, j * 128:(j + 1) * 128]],
                                  P.E4M3[P.encode(part / 2.0 ** (int(sc[i, j]) - 127))])


def _operands(rng, rows, out_dim, in_dim):
    """Codes of every kind but NaN, scales of a wide range; unused scale bytes hold NaN (255)."""
    st = F.stride(in_dim)
    nb = -(-in_dim // 128)
    x = P.encode(rng.standard_normal((rows, in_dim)) * 60)
    w = P.encode(rng.standard_normal((out_dim, in_dim)) * 60)
    x[rng.random(x.shape) < 0.01] = 0x7E
    w[rng.random(w.shape) < 0.01] = 0xFE
    xs = np.full((rows, st), 255, np.uint8)
    wsc = np.full((-(-out_dim // 128), st), 255, np.uint8)
    xs[:, :nb] = rng.integers(117, 127, (rows, nb))
    wsc[:, :nb] = rng.integers(107, 127, (wsc.shape[0], nb))
    return x, xs, w, wsc


def _linear(E, dt, x, xs, w, wsc, ws=None):
    rows, in_dim = x.shape
    out = torch.full((rows, w.shape[0]), 7.0, dtype=DT[dt], device="cuda")
    dev = [torch.from_numpy(a).cuda() for a in (x, xs, w, wsc)]
    E.eagle_linear_fp8(rows, w.shape[0], in_dim, *dev, _code(E, dt), out, ws)
    return out


def _check_linear(out, x, xs, w, wsc, dt):
    a, b = F.dequant_rows(x, xs), F.dequant_weight(w, wsc)
    want = a @ b.T
    tol = x.shape[1] * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T)
    if dt == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    err = np.abs(_np(out) - want)
    assert np.all(err <= tol), (np.argwhere(err > tol)[:5], (err / np.maximum(tol, 1e-300)).max())


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,out_dim,in_dim", [
    (1, 8, 16), (1, 128, 128), (3, 129, 144), (16, 256, 512), (17, 300, 528), (10, 1000, 1040), (1, 4096, 4096),
    (33, 640, 2048), (100, 520, 640), (129, 384, 656), (224, 130, 512), (225, 257, 1152), (300, 1024, 384),
    (448, 300, 256), (700, 777, 912), (1000, 129, 2064), (2, 20000, 256), (513, 5000, 128),
    (65, 10100, 2512), (230, 10001, 1040), (449, 4000, 4224), (40, 20001, 2064), (20, 700, 8192), (672, 2500, 640)])
def test_linear(E, dt, rows, out_dim, in_dim):
    rng = np.random.default_rng(rows * 1009 + out_dim * 31 + in_dim)
    ops = _operands(rng, rows, out_dim, in_dim)
    ws = _ws(E)
    out = _linear(E, dt, *ops, ws)
    assert E.eagle_status_fetch(ws) == 0
    _check_linear(out, *ops, dt)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,out_dim,in_dim", [(1, 1, 32), (2, 5, 496), (1, 1003, 5120), (2, 1003, 4608), (1, 70, 16384),
                                                 (2, 333, 3600), (1, 11000, 4096), (2, 130, 16384), (1, 130000, 128)])
def test_linear_single_rows(E, dt, rows, out_dim, in_dim):
    """A row or two: K in chunks of 512 shared by one to eight warps, ends inside a chunk, weights across the rule's limit."""
    rng = np.random.default_rng(rows * 1013 + out_dim * 37 + in_dim)
    ops = _operands(rng, rows, out_dim, in_dim)
    _check_linear(_linear(E, dt, *ops), *ops, dt)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,out_dim,in_dim", [
    (66, 9729, 1040), (100, 14336, 528), (128, 20001, 4240), (113, 9800, 16),                # CTAs share the weight's rows
    (64, 4096, 4096), (90, 6100, 2064), (128, 130, 8192), (128, 8192, 1040), (97, 1000, 3600),  # parts of K
    (200, 2048, 4096), (257, 515, 5136), (500, 512, 4096),
    (129, 9729, 2064), (150, 10100, 2512), (224, 12000, 4240)])                              # pairs, one accumulator
def test_linear_dealt(E, dt, rows, out_dim, in_dim):
    """On both sides of the rules that deal the weight's rows, K or the rows of x to the CTAs; what lies before and
    behind the outputs is left."""
    rng = np.random.default_rng(rows * 1019 + out_dim * 41 + in_dim)
    ops = _operands(rng, rows, out_dim, in_dim)
    around = torch.full((rows * out_dim + 128,), 7.0, dtype=DT[dt], device="cuda")
    out = around[64:-64].view(rows, out_dim)
    ws = _ws(E)
    E.eagle_linear_fp8(rows, out_dim, in_dim, *[torch.from_numpy(t).cuda() for t in ops], _code(E, dt), out, ws)
    assert E.eagle_status_fetch(ws) == 0
    _check_linear(out, *ops, dt)
    assert bool((around[:64] == 7).all()) and bool((around[-64:] == 7).all())


@pytest.mark.parametrize("rows", [1, 2, 17, 130, 300])
def test_linear_scales_of_every_size(E, rows):
    """Scales from 2^-120 to 2^120 whose products are ordinary: each block's two exponents nearly cancel."""
    rng = np.random.default_rng(rows)
    out_dim, in_dim = 9000, 1040
    x, xs, w, wsc = _operands(rng, rows, out_dim, in_dim)
    nb = -(-in_dim // 128)
    xs[:, :nb] = np.array([7, 247, 127, 200, 50, 240, 14, 100, 180])[None]
    wsc[:, :nb] = 254 - xs[:1, :nb] + rng.integers(-3, 4, (wsc.shape[0], nb))
    _check_linear(_linear(E, "fp32", x, xs, w, wsc), x, xs, w, wsc, "fp32")


@pytest.mark.parametrize("rows", [1, 40, 300])
def test_linear_one_hot(E, rows):
    """A single code in each row of x picks a weight column under both scales: exact, so no scale is another's."""
    rng = np.random.default_rng(rows)
    out_dim, in_dim = 400, 1168
    x, xs, w, wsc = _operands(rng, rows, out_dim, in_dim)
    x[:] = 0
    at = rng.integers(0, in_dim, rows)
    x[np.arange(rows), at] = 0x38  # 1.0
    out = _linear(E, "fp32", x, xs, w, wsc)
    want = F.dequant_weight(w, wsc)[:, at].T * 2.0 ** (xs[np.arange(rows), at // 128].astype(np.float64) - 127)[:, None]
    assert np.array_equal(_np(out), want)


@pytest.mark.parametrize("rows", [1, 2, 20, 300])
def test_linear_nan_reaches_its_own_outputs(E, rows):
    rng = np.random.default_rng(8)
    for kind in ("x code", "x scale", "w code", "w scale"):
        x, xs, w, wsc = _operands(rng, rows, 10300, 512)
        want = np.zeros((rows, 10300), bool)
        if kind == "x code":
            x[rows - 1, 100] = 0x7F
            want[rows - 1] = True
        elif kind == "x scale":
            xs[rows - 1, 2] = 255
            want[rows - 1] = True
        elif kind == "w code":
            w[200, 7] = 0xFF
            want[:, 200] = True
        else:
            wsc[1, 3] = 255
            want[:, 128:256] = True
        assert np.array_equal(np.isnan(_np(_linear(E, "fp32", x, xs, w, wsc))), want), kind


def test_linear_captured_and_other_stream(E):
    """A graph replayed on changed inputs, beside the same call on another stream; outputs around it are untouched."""
    rng = np.random.default_rng(9)
    rows, out_dim, in_dim = 40, 900, 1024
    a, b = _operands(rng, rows, out_dim, in_dim), _operands(rng, rows, out_dim, in_dim)
    dev = [torch.from_numpy(t).cuda() for t in a]
    out = torch.full((rows + 2, out_dim), 7.0, device="cuda")
    call = lambda: E.eagle_linear_fp8(rows, out_dim, in_dim, *dev, E.EAGLE_F32, out[1:-1])  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for t, n in zip(dev, b):
        t.copy_(torch.from_numpy(n))
    other, side = torch.empty(rows, out_dim, device="cuda"), torch.cuda.Stream()
    dev2 = [torch.from_numpy(t).cuda() for t in a]
    torch.cuda.synchronize()
    g.replay()
    E.eagle_linear_fp8(rows, out_dim, in_dim, *dev2, E.EAGLE_F32, other, stream=side)
    torch.cuda.synchronize()
    _check_linear(out[1:-1], *b, "fp32")
    _check_linear(other, *a, "fp32")
    assert bool((out[0] == 7).all()) and bool((out[-1] == 7).all())


def test_linear_same_result_every_time(E):
    rng = np.random.default_rng(10)
    for shape in ((2, 4096, 4096), (5, 4096, 4096), (300, 1300, 1024), (300, 11000, 640)):
        ops = _operands(rng, *shape)
        first = _linear(E, "fp32", *ops)
        for _ in range(3):
            assert torch.equal(first, _linear(E, "fp32", *ops))


@pytest.mark.parametrize("rows,out_dim,dim", [(10, 3000, 1024), (260, 1000, 656)])
def test_norm_then_head(E, rows, out_dim, dim):
    """The operators together: residual, norm, codes, and the packed head's logits, against the same codes in 64 bits
    and, within the codes' rounding, against the head on the exact rows."""
    rng = np.random.default_rng(rows)
    x, res = _rows(rng, rows, dim, "bf16"), _rows(rng, rows, dim, "bf16")
    nw = torch.from_numpy(1 + 0.1 * rng.standard_normal(dim)).bfloat16().cuda()
    weight = (torch.from_numpy(rng.standard_normal((out_dim, dim))) * 0.03).bfloat16().cuda()
    wc = E.alloc_fp8(out_dim, dim, -(-out_dim // 128))
    xc = E.alloc_fp8(rows, dim)
    total, out = torch.empty_like(x), torch.empty(rows, out_dim, device="cuda")
    E.eagle_linear_fp8_pack(out_dim, dim, weight, *wc)
    E.eagle_rmsnorm_fp8(rows, dim, E.EAGLE_BF16, x, dim, res, total, nw, 1e-5, *xc)
    E.eagle_linear_fp8(rows, out_dim, dim, *xc, *wc, E.EAGLE_F32, out)
    x8, w8 = [t.cpu().numpy() for t in xc], [t.cpu().numpy() for t in wc]
    _check_linear(out, *x8, *w8, "fp32")
    _, y = F.norm_rows(_np(x), _np(res), _np(nw), float(np.float32(1e-5)), P.bf16_round)
    # each operand is off by 2^-4 of its value or half the smallest step of its block's scale (2^-10 of 2^e, where amax > 224 2^e)
    b = _np(weight)
    dy = 2.0 ** -4 * np.abs(y) + np.repeat(np.abs(F.blocks(y)).max(2), 128, 1)[:, :dim] * 2.0 ** -17
    db = 2.0 ** -4 * np.abs(b) + np.abs(b).max() * 2.0 ** -17
    tol = (dy @ np.abs(b).T + np.abs(y) @ db.T + dy @ db.T) * (1 + 2.0 ** -10)
    assert np.all(np.abs(_np(out) - y @ b.T) <= tol)
