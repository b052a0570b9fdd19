"""The 8-bit norm's eps over its whole range: beside rows whose squares leave fp32's range it counts as it does
elsewhere. Tolerances as in test_gpu_fp8 (y within 2^-19, a code within half a step)."""
import numpy as np
import pytest
import torch
import plain64_fp8 as F
from test_gpu_fp8 import DT, _check_codes, _code, _np, _ws

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E():
    from speculative_decoding_dynamic_gb300 import eagle
    return eagle


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("dim", [16, 256, 1040, 4096, 8192])
@pytest.mark.parametrize("eps", [2.0 ** -126, 1e-5, 1e30, 1e38, 3.4e38])
def test_eps(E, dt, dim, eps):
    rng = np.random.default_rng(dim)
    sizes = np.array([1e-30, 1.0, 1e15, 3e18, 1e19, 1.6e19, 3e19, 1e25])
    x = torch.from_numpy(rng.standard_normal((len(sizes), dim)) * sizes[:, None]).to(DT[dt]).cuda()
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(dim)).to(DT[dt]).cuda()
    codes, scales = E.alloc_fp8(len(sizes), dim)
    ws = _ws(E)
    E.eagle_rmsnorm_fp8(len(sizes), dim, _code(E, dt), x, dim, None, None, w, eps, codes, scales, ws)
    assert E.eagle_status_fetch(ws) == 0
    _, y = F.norm_rows(_np(x), None, _np(w), float(np.float32(eps)), None)
    low = np.abs(y).max(1) < 2.0 ** -100  # (rows whose y is near fp32's smallest numbers have zeros there)
    _check_codes(y[~low], codes[~torch.from_numpy(low)], scales[~torch.from_numpy(low)])
