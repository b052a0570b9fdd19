"""Rows of the distillation loss whose list gives no distribution: status, loss and gradient as the header has them."""
import numpy as np
import pytest
from test_gpu_distill import _case, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E():
    from speculative_decoding_dynamic_gb300 import eagle
    return eagle


def _faulty(E, z, ids, t, lse, weight, status):
    loss, grad, got = _run(E, z, ids, t, lse, 1.0, weight)
    assert got == status
    assert np.isnan(loss[0]) and not grad[0].any()
    assert np.isfinite(loss[1:]).all()


@pytest.mark.parametrize("V", [1024, 65536])
@pytest.mark.parametrize("rest", [True, False])
def test_no_id_of_the_vocabulary(E, V, rest):
    """Ids past the vocabulary alone, or with padding beside them."""
    z, ids, t, lse = _case(np.random.default_rng(V), 3, V, 4, "bf16", 1.0, rest)
    ids[0] = V
    _faulty(E, z, ids, t, lse, None, 3)
    ids[0] = (-1, V + 7, -1, -1)
    _faulty(E, z, ids, t, lse, None, 3)


@pytest.mark.parametrize("V", [1024, 65536])
def test_padding_alone_hides_no_other_fault(E, V):
    """A row without a list has loss and gradient 0, but not where its weight or its logits are at fault."""
    z, ids, t, lse = _case(np.random.default_rng(V + 1), 3, V, 4, "bf16", 1.0, False)
    ids[0] = -1
    t[0] = np.nan  # (padding's logits are not looked at)
    loss, grad, status = _run(E, z, ids, t, lse, 1.0, None)
    assert status == 0 and loss[0] == 0 and not grad[0].any()
    _faulty(E, z, ids, t, lse, np.array([np.nan, 1, 1], np.float32), 1)
    for bad in (float("nan"), float("inf")):
        broken = z.clone()
        broken[0, V - 3] = bad
        _faulty(E, broken, ids, t, lse, None, 1)
    broken[0] = -float("inf")
    _faulty(E, broken, ids, t, lse, None, 1)


@pytest.mark.parametrize("V", [1024, 65536])
@pytest.mark.parametrize("rest", [True, False])
def test_list_without_a_finite_logit(E, V, rest):
    z, ids, t, lse = _case(np.random.default_rng(V + 2), 3, V, 40, "fp32", 1.0, rest)
    t[0] = -np.inf
    _faulty(E, z, ids, t, lse, None, 1)
    ids[0, 1:] = -1  # a single entry, padding's logits finite
    t[0, 1:] = 1.0
    _faulty(E, z, ids, t, lse, None, 1)
    # one finite logit is a list; padding alone with an lse leaves everything to the rest
    t[0] = -np.inf
    t[0, 0] = 0.0
    if rest:
        lse[0] = 0.5
        ids[1] = -1
        t[1] = -np.inf
    loss, grad, status = _run(E, z, ids, t, lse, 1.0, None)
    assert status == 0 and np.isfinite(loss).all() and np.isfinite(grad).all()
    if rest:
        assert loss[1] == 0 and not grad[1].any()


@pytest.mark.parametrize("V", [1024, 65536])
@pytest.mark.parametrize("rest", [True, False])
def test_weight_over_temperature_past_fp32(E, V, rest):
    """A finite weight that divided by T is infinite has no gradient in 32 bits: refused where one is asked for."""
    T = 2.0 ** -126
    z, ids, t, _ = _case(np.random.default_rng(V + 3), 3, V, 4, "fp32", 1.0, rest)
    t = np.zeros_like(t)
    lse = np.full(3, 1.5, np.float32) if rest else None
    w = np.array([8.0, 1.0, -0.5], np.float32)
    loss, grad, status = _run(E, z, ids, t, lse, T, w)
    assert status == 1
    assert np.isnan(loss[0]) and not grad[0].any()
    assert not np.isnan(loss[1:]).any() and np.isfinite(grad).all()
    assert np.all(np.abs(grad[1:]).max(1) <= 2.0 ** 126 * np.abs(w[1:]) * 1.01) and np.all(grad[1:].any(1))
    alone, _, status = _run(E, z, ids, t, lse, T, w, grad=False)
    assert status == 0 and not np.isnan(alone).any() and np.array_equal(alone[1:], loss[1:])
