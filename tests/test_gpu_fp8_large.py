"""The 8-bit operators and the loss at their arguments' largest values and with more than 2^31 entries, checked in 64
bits at the ends and in rows and columns picked at random. Tolerances as in test_gpu_fp8 and test_gpu_distill."""
import numpy as np
import pytest
import torch
import plain64 as P
import plain64_fp8 as F
from test_gpu_distill import _cfg, _check as _check_loss
from test_gpu_fp8 import DT, _check_codes, _code, _np, _ws

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E():
    from speculative_decoding_dynamic_gb300 import eagle
    yield eagle
    torch.cuda.empty_cache()


def _codes(n, dim, g):
    """Codes of every kind but NaN (0x7F and 0xFF become 0x7E)."""
    c = torch.randint(0, 256, (n, dim), device="cuda", generator=g, dtype=torch.uint8)
    return c.masked_fill_((c & 0x7F) == 0x7F, 0x7E)


def _scales(n, dim, low, g):
    return torch.randint(low, low + 10, (n, F.stride(dim)), device="cuda", generator=g, dtype=torch.uint8)


def _decoded(codes, scales, each):
    """float64 [n, dim] of code rows; each: the scale row of a code row."""
    dim = codes.shape[1]
    e = torch.exp2(scales[each].double() - 127).repeat_interleave(128, 1)[:, :dim]
    return codes.view(torch.float8_e4m3fn).float().double() * e


def _picked(n, count, rng):
    return torch.from_numpy(np.unique(np.concatenate([[0, n // 2, n - 1], rng.integers(0, n, count)]))).cuda()


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,out_dim,in_dim", [
    (1, 20, 1 << 20), (3, 130, 1 << 20), (300, 40, 1 << 20),  # the longest K
    (1 << 20, 5, 16), (1 << 20, 8, 48),                       # the most rows
    (2, 1 << 24, 16), (3, (1 << 24) - 5, 16),                 # the most outputs
    (40001, 60000, 16), (36000, 60001, 16),                   # more than 2^31 outputs
    (200, 12000000, 16), (1 << 20, 64, 2064)])                # more than 2^31 outputs or codes of x
def test_linear(E, dt, rows, out_dim, in_dim):
    rng = np.random.default_rng(rows + out_dim + in_dim)
    g = torch.Generator("cuda").manual_seed(rows + out_dim + in_dim)
    x, w = _codes(rows, in_dim, g), _codes(out_dim, in_dim, g)
    xs, wsc = _scales(rows, in_dim, 117, g), _scales(-(-out_dim // 128), in_dim, 107, g)
    out = torch.full((rows * out_dim + 64,), 7.0, dtype=DT[dt], device="cuda")
    ws = _ws(E)
    E.eagle_linear_fp8(rows, out_dim, in_dim, x, xs, w, wsc, _code(E, dt), out, ws)
    assert E.eagle_status_fetch(ws) == 0
    assert bool((out[rows * out_dim:] == 7).all())
    out = out[:rows * out_dim].view(rows, out_dim)
    m, n = _picked(rows, 60, rng), _picked(out_dim, 2000, rng)
    a, b = _decoded(x[m], xs, m), _decoded(w[n], wsc, n // 128)
    want, size = a @ b.T, a.abs() @ b.abs().T
    tol = in_dim * 2.0 ** -23 * size
    if dt == "bf16":
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
    assert bool(((out[m][:, n].double() - want).abs() <= tol).all())


@pytest.mark.parametrize("dt,rows,dim,stride", [("bf16", 1 << 24, 16, 16), ("bf16", 300001, 8192, 8192),
                                                ("fp32", 150001, 4096, 16384), ("bf16", 4, 656, (1 << 31) // 8 * 3)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(E, dt, rows, dim, stride, residual):
    g = torch.Generator("cuda").manual_seed(rows)
    n = (rows - 1) * stride + dim
    x = torch.empty(n, dtype=DT[dt], device="cuda").normal_(generator=g)
    res = torch.empty(n, dtype=DT[dt], device="cuda").normal_(generator=g) if residual else None
    w = torch.empty(dim, device="cuda").uniform_(0.5, 1.5, generator=g).to(DT[dt])
    pick = _picked(rows, 300, np.random.default_rng(rows))
    rows_of = lambda t: t.as_strided((rows, dim), (stride, 1))[pick]  # noqa: E731
    x64, r64 = _np(rows_of(x)), _np(rows_of(res)) if residual else None
    codes, scales = E.alloc_fp8(rows, dim)
    codes.fill_(99)
    scales.fill_(99)
    ws = _ws(E)
    E.eagle_rmsnorm_fp8(rows, dim, _code(E, dt), x, stride, res, res, w, 1e-5, codes, scales, ws)
    assert E.eagle_status_fetch(ws) == 0
    rounded = P.bf16_round if dt == "bf16" else (lambda v: np.asarray(v, np.float32))
    s, y = F.norm_rows(x64, r64, _np(w), float(np.float32(1e-5)), rounded)
    if residual:
        assert np.array_equal(_np(rows_of(res)), s)
    _check_codes(y, codes[pick], scales[pick])
    assert not bool((codes == 99).all(1).any())


def test_pack(E):
    out_dim, in_dim = 65535 * 128, 272
    g = torch.Generator("cuda").manual_seed(1)
    w = torch.empty(out_dim, in_dim, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    codes, scales = E.alloc_fp8(out_dim, in_dim, 65535)
    E.eagle_linear_fp8_pack(out_dim, in_dim, w, codes, scales)
    for block in (0, 31111, 65534):
        y = _np(w[block * 128:(block + 1) * 128])
        for j in range(3):
            part = y[:, j * 128:(j + 1) * 128]
            e = F.scale_bytes(np.abs(part).max())
            assert int(scales[block, j]) == e
            got = codes[block * 128:(block + 1) * 128, j * 128:(j + 1) * 128].cpu().numpy()
            assert np.array_equal(P.E4M3[got], P.E4M3[P.encode(part / 2.0 ** (int(e) - 127))])


@pytest.mark.parametrize("dt,rows,V,top", [("bf16", 1 << 24, 8, 1), ("bf16", 20001, 128256, 16), ("fp32", 70001, 32000, 64)])
def test_loss(E, dt, rows, V, top):
    g = torch.Generator("cuda").manual_seed(V)
    z = torch.empty(rows, V, dtype=DT[dt], device="cuda").normal_(0, 2, generator=g)
    ids = torch.randint(0, V // top, (rows, top), device="cuda", generator=g, dtype=torch.int32)
    ids += torch.arange(top, device="cuda", dtype=torch.int32) * (V // top)
    t = torch.empty(rows, top, device="cuda").normal_(generator=g)
    lse = torch.logsumexp(t, 1) + 0.5
    cfg = _cfg(E, V, dt)
    ws = E.alloc_workspace(E.eagle_workspace_bytes(cfg))
    pick = _picked(rows, 100, np.random.default_rng(V))
    z64 = _np(z[pick])
    loss = torch.full((rows,), float("nan"), device="cuda")
    E.eagle_distill_loss(cfg, ws, rows, top, z, ids, t, lse, 1.0, None, loss, z)  # the gradient in the logits' place
    assert E.eagle_status_fetch(ws) == 0
    want = F.distill(z64, ids[pick].cpu().numpy(), t[pick].cpu().numpy(), lse[pick].cpu().numpy(), 1.0, None)
    _check_loss(_np(loss[pick]), _np(z[pick]), want, V, dt)
    assert bool(torch.isfinite(loss).all()) and float(z.amax()) < 1.0  # (no row was left out: a gradient is below 1)
