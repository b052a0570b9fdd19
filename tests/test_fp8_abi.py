"""Host-side checks of the 8-bit rows and products and of the distillation loss:
every refusal happens before any CUDA call (pointers are fake addresses that a
refused call never follows), and the plain forms against hand-made values."""
import ctypes
import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))
import plain64 as P  # noqa: E402
import plain64_fp8 as F  # noqa: E402

PTR = 1 << 20  # an aligned fake address
f = ctypes.c_float


@pytest.fixture(scope="module")
def E():
    from speculative_decoding_dynamic_gb300 import build
    build.build()
    from speculative_decoding_dynamic_gb300 import eagle
    return eagle


def _each(E, name, good, bad):
    for at, value, code in bad:
        args = list(good)
        args[at] = value
        assert E.raw_call(name, *args) == code, (name, at, value)


def test_scale_stride(E):
    assert [E.eagle_fp8_scale_stride(d) for d in (0, -5, 1, 128, 512, 513, 4096, 5120)] == [0, 0, 4, 4, 4, 8, 32, 40]
    for d in (16, 400, 512, 528, 8192):
        assert E.eagle_fp8_scale_stride(d) == F.stride(d)


def test_rmsnorm_refusals(E):
    good = [4, 256, E.EAGLE_BF16, PTR, 256, PTR, PTR, PTR, f(1e-5), PTR, PTR, None, None]
    _each(E, "eagle_rmsnorm_fp8", good, [
        (0, 0, -1), (1, 0, -1), (2, 2, -1), (3, None, -1), (4, 255, -1), (4, -256, -1), (5, None, -1), (8, f(0.0), -1),
        (8, f(-1.0), -1), (8, f(float("nan")), -1), (8, f(float("inf")), -1), (9, None, -1), (10, None, -1),
        (0, (1 << 24) + 1, -2), (1, 248, -2), (4, 260, -2), (4, 1 << 32, -2)] +
        [(i, PTR + 8, -2) for i in (3, 5, 6, 7, 9)])
    big = [4, 16400, E.EAGLE_F32, PTR, 16400, None, None, None, f(0.0), PTR, PTR, None, None]
    assert E.raw_call("eagle_rmsnorm_fp8", *big) == -2


def test_linear_refusals(E):
    good = [4, 300, 256, PTR, PTR, PTR, PTR, E.EAGLE_BF16, PTR, None, None]
    _each(E, "eagle_linear_fp8", good, [(i, 0, -1) for i in (0, 1, 2)] + [(i, None, -1) for i in (3, 4, 5, 6, 8)] + [
        (7, 2, -1), (2, 248, -2), (3, PTR + 8, -2), (5, PTR + 8, -2), (8, PTR + 8, -2), (4, PTR + 2, -2), (6, PTR + 1, -2),
        (0, (1 << 20) + 1, -2), (1, (1 << 24) + 1, -2), (2, (1 << 20) + 16, -2)])
    _each(E, "eagle_linear_fp8_pack", [300, 256, PTR, PTR, PTR, None], [
        (0, 0, -1), (1, 0, -1), (2, None, -1), (3, None, -1), (4, None, -1), (1, 248, -2), (2, PTR + 2, -2), (3, PTR + 8, -2),
        (0, 65535 * 128 + 1, -2)])


def test_distill_refusals(E):
    cfg = E.TreeCfg(2, 1024, 4, 1, 1, 0.0, E.EAGLE_BF16)
    n = E.eagle_workspace_bytes(cfg)
    good = [ctypes.byref(cfg), PTR, n, 3, 16, PTR, PTR, PTR, PTR, f(1.0), PTR, PTR, PTR, None]
    _each(E, "eagle_distill_loss", good, [
        (0, None, -1), (1, None, -4), (1, PTR + 16, -4), (2, n - 1, -4), (3, 0, -1), (4, 0, -1), (5, None, -1), (6, None, -1),
        (7, None, -1), (11, None, -1), (9, f(0.0), -1), (9, f(-2.0), -1), (9, f(float("nan")), -1), (9, f(float("inf")), -1),
        (3, (1 << 24) + 1, -2), (4, 257, -2), (5, PTR + 8, -2), (12, PTR + 8, -2)])


def test_binding_refuses_tensors_that_do_not_fit(E):
    """Types and sizes are checked before the library is called (CPU tensors are refused for their device)."""
    u8, bf = torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x is torch.float32"):
        E.eagle_rmsnorm_fp8(4, 256, E.EAGLE_BF16, bf.float(), 256, None, None, bf[0], 1e-5, u8, u8)
    with pytest.raises(ValueError, match="w_codes|x_codes"):
        E.eagle_linear_fp8(4, 4, 256, u8, u8, bf, u8, E.EAGLE_F32, bf)
    with pytest.raises(ValueError, match="logits"):
        E.eagle_distill_loss(E.TreeCfg(1, 256, 1, 1, 1, 0.0, E.EAGLE_F32), None, 4, 4, bf, u8, u8, None, 1.0, None, u8)


def test_plain_scales_and_codes():
    assert F.scale_bytes(np.array([448.0, 449.0, 224.0, 0.0, 1.0, 1.75, 1.7500001])).tolist() == [127, 128, 126, 1, 119, 119, 120]
    y = np.array([[1.0, -448.0, 17.0, 2.0 ** -9]])
    v = P.E4M3[P.encode(y)]
    assert np.all(np.abs(v - y) <= F.half_step(y))


def test_plain_distill_gradient_is_the_difference_of_its_loss():
    rng = np.random.default_rng(3)
    z = rng.standard_normal((2, 24)) * 2
    ids = np.array([[3, 7, -1, 20], [1, 0, 2, -1]])
    t = rng.standard_normal((2, 4))
    for lse in (None, np.array([2.5, 3.0])):
        loss, grad, *_ = F.distill(z, ids, t, lse, 1.7, np.array([0.5, 2.0]))
        assert np.all(loss > 0)
        for j in range(24):
            d = np.zeros(24)
            d[j] = 1e-5
            up, down = (F.distill(z + s * d, ids, t, lse, 1.7, np.array([0.5, 2.0]))[0] for s in (1, -1))
            assert np.allclose((up - down) / 2e-5, grad[:, j], atol=1e-8)


def test_plain_distill_of_the_same_distribution_is_zero():
    z = np.random.default_rng(4).standard_normal((3, 40))
    ids = np.tile(np.arange(0, 16), (3, 1))
    t = z[:, :16]
    lse = np.log(np.exp(z).sum(1))
    loss, grad, *_ = F.distill(z, ids, t, lse, 1.0, None)
    assert np.abs(loss).max() < 1e-14 and np.abs(grad).max() < 1e-15
