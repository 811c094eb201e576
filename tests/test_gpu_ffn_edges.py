"""The feed-forward operators where they are easily wrong: rows without columns, in place, addresses, many rows of the
widest forms, values that are not finite, the kernels for few and for many tokens side by side, host threads, streams,
graphs.

Tolerances are those of test_gpu_ffn.py, and their derivation.
"""
import pytest
import torch

from fine_grained_block_b200 import binding as B

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _status():
    B.fp8_device_status(clear=True)
    yield
    assert B.fp8_device_status() == 0


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("stream", [False, True])
def test_norm_of_rows_without_columns(dtype, stream):
    """The mean of no elements is NaN, and so is rstd, whether the call makes it or is given it."""
    x, w = torch.empty(5, 0, dtype=dtype, device="cuda"), torch.empty(0, device="cuda")
    st = torch.cuda.Stream() if stream else None
    rstd = torch.full((7,), 3.0, device="cuda")
    torch.cuda.synchronize()
    q, s, h, y, given = B.fp8q_rmsnorm_quantize(x, w, x, rstd=rstd[1:6], want_y=True, stream=st)
    made = B.fp8q_rmsnorm_quantize(x, w, want_rstd=True, stream=st)[4]
    torch.cuda.synchronize()
    assert [tuple(t.shape) for t in (q, s, h, y)] == [(5, 0)] * 4
    assert bool(torch.isnan(given).all()) and bool(torch.isnan(made).all()) and made.shape == (5,)
    assert float(rstd[0]) == float(rstd[6]) == 3.0
    with pytest.raises(ValueError):
        B.fp8q_rmsnorm_quantize(x, w, rstd=rstd)
