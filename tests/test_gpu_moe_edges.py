"""The operators of a block of experts where a route is used in part or changed after the sort, and where offsets are not the
sort's.

Tolerances are those of test_gpu_moe.py, and their derivation.
"""
import pytest
import torch

from fine_grained_block_b200 import binding as B
from test_gpu_ffn import BF, FP, MAX
from test_gpu_moe import I32, guarded, untouched

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _status():
    B.fp8_device_status(clear=True)
    yield
    assert B.fp8_device_status() == 0


# -- products without columns of A ------------------------------------------------------------------------------------

@pytest.mark.parametrize("offsets", [[2, 4, 4, 7], [5, 5, 5, 5], [0, 3, 1, 6], [-4, 1, 9, 50]], ids=str)
def test_empty_sums_are_written_to_the_experts_rows_only(offsets):
    """K == 0: zeros on the rows of the experts, which need not start at row 0; every other row stays as it was."""
    R, N, E = 9, 256, 3
    off = torch.tensor(offsets, dtype=I32, device="cuda")
    hit = torch.zeros(R, dtype=torch.bool, device="cuda")
    for lo, hi in zip(offsets, offsets[1:]):
        hit[min(max(lo, 0), R):min(max(hi, 0), R)] = True
    empty = lambda *shape, dtype=torch.uint8: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    a, sa, b, sb = empty(R, 0), empty(R, 0, dtype=FP), empty(E, N, 0), empty(E, N // 128, 0, dtype=FP)
    for dtype in (BF, FP):
        out = [guarded((R, N // 2), torch.uint8), guarded((R, N // 256), FP), guarded((R, N), dtype), guarded((R, N), dtype)]
        B.fp8q_gemm_gated_grouped(a, sa, b, sb, off, q=out[0].t, scales=out[1].t, gu=out[2].t)
        B.fp8q_gemm_grouped(a, sa, b, sb, off, c=out[3].t)
        torch.cuda.synchronize()
        for o in out:
            o.check()
            assert untouched(o.t[~hit], 0)
        for o in (out[0], out[2], out[3]):
            assert int((o.t[hit] != 0).sum()) == 0
        assert bool((out[1].t[hit] == torch.tensor(MAX[B.E4M3], device="cuda") / 1e-12).all())
