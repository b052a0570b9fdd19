"""What the 8-bit calls' host side says at the ends of its arguments' ranges, and of tensors whose rows lie otherwise
than the call says."""
import pytest
import torch


@pytest.fixture(scope="module")
def E():
    from speculative_decoding_dynamic_gb300 import build
    build.build()
    from speculative_decoding_dynamic_gb300 import eagle
    return eagle


def test_scale_stride_of_the_largest_dims(E):
    for dim in (2 ** 31 - 1, 2 ** 31 - 511, 2 ** 31 - 512, 2 ** 31 - 513, 1 << 30):
        assert E.eagle_fp8_scale_stride(dim) == (dim + 511) // 512 * 4
    assert E.eagle_fp8_scale_stride(-2 ** 31) == 0


def test_rows_that_lie_otherwise_than_the_call_says(E):
    """Rows inside wider ones: a tensor's own distance from row to row is the call's row_stride."""
    wide = torch.zeros(8, 1024, dtype=torch.bfloat16)
    codes, scales = E.alloc_fp8(4, 256, device="cpu")
    w = torch.ones(256, dtype=torch.bfloat16)

    def call(x, residual, total, stride):
        E.eagle_rmsnorm_fp8(4, 256, E.EAGLE_BF16, x, stride, residual, total, w, 1e-5, codes, scales)

    rows, every_other, across = wide[:4, 64:320], wide[::2, 64:320], wide.view(1024, 8).t()[:4, :256]
    for at in range(3):
        for other in (every_other, across, wide[:4, ::4]):
            args = [rows, rows, rows]
            args[at] = other
            with pytest.raises(ValueError, match="row_stride"):
                call(*args, 1024)
    # what lies as the call says, or whole tensors, go on to the checks of the device
    for x in (rows, wide, wide.view(2, 4, 1024)[:, :, 64:320], wide[:1, 64:320], wide.view(8, 8, 128)[:, 2:4],
              wide.view(8, 4, 256)[:, 1:3], wide[:, :900]):
        with pytest.raises(ValueError, match="current CUDA device"):
            call(x, rows, None, 1024)
    with pytest.raises(ValueError, match="current CUDA device"):
        call(every_other, None, None, 2048)
