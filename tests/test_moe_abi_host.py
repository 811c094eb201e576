"""The routed feed-forward operators' C ABI: bad arguments are refused on the host before anything is launched (no GPU
needed)."""
import pytest

from fine_grained_block_b200 import binding
from fine_grained_block_b200 import build as fbuild

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_FORMAT, ERR_DTYPE, ERR_CUDA, ERR_ARG = 0, -1, -2, -3, -4, -5, -6, -7

# Fake device addresses, far apart and never dereferenced.
X, O, P, S, Q, C, QT, CT, W, D = (0x7F0000000000 + (i << 37) for i in range(10))
F32, BF16, E4M3, E5M2 = 0, 1, 0, 1


@pytest.fixture(scope="module")
def L():
    fbuild.build()
    return binding.load_library()


def test_names_of_the_package(L):
    import fine_grained_block_b200 as pkg
    for name in ("MoeRoute", "fp8q_moe_rows", "fp8q_moe_sort", "fp8q_moe_dispatch", "fp8q_moe_dispatch_codes",
                 "fp8q_moe_combine", "fp8q_moe_combine_backward", "fp8q_gemm_grouped", "fp8q_gemm_gated_grouped",
                 "fp8q_gemm_grouped_wgrad"):
        assert getattr(pkg, name) is getattr(binding, name)


def test_rows_and_workspace(L):
    assert L.fp8q_moe_rows(0, 8, 64, 128) == 0
    assert L.fp8q_moe_rows(1, 8, 64, 1) == 8
    assert L.fp8q_moe_rows(1, 8, 64, 16) == 8 * 16
    assert L.fp8q_moe_rows(100, 2, 3, 128) == (200 + 3 * 127) // 128 * 128
    for bad in ((-1, 8, 64, 1), (1, 0, 64, 1), (1, 1, 0, 1), (1, 1, 1025, 1), (1 << 29, 4, 8, 1), (1 << 40, 1 << 40, 8, 1)):
        assert L.fp8q_moe_rows(*bad) == ERR_SHAPE
        assert L.fp8q_moe_sort_workspace(*bad[:3]) == ERR_SHAPE
    for align in (0, 3, -1, 256):
        assert L.fp8q_moe_rows(1, 8, 64, align) == ERR_ARG
    assert L.fp8q_moe_sort_workspace(512, 8, 64) == 0
    assert 0 < L.fp8q_moe_sort_workspace(513, 8, 64) <= 128 * 64 * 4
    assert 0 < L.fp8q_moe_sort_workspace(1 << 30, 1, 1024) <= 128 * 1024 * 4
    with pytest.raises(binding.FP8Error):
        binding.fp8q_moe_rows(1, 8, 64, 3)


SORT = dict(experts=X, tokens=100, top_k=8, num_experts=64, align=1, rows=800, offsets=O, pos=P, src=S, counts=C, workspace=None,
            bytes=0, stream=None)


@pytest.mark.parametrize("change, status", [
    (dict(tokens=-1), ERR_SHAPE), (dict(top_k=0), ERR_SHAPE), (dict(num_experts=0), ERR_SHAPE), (dict(num_experts=2000), ERR_SHAPE),
    (dict(rows=799), ERR_SHAPE), (dict(rows=1 << 40), ERR_SHAPE), (dict(align=128), ERR_SHAPE), (dict(align=3), ERR_ARG),
    (dict(align=0), ERR_ARG), (dict(tokens=1 << 31, top_k=1), ERR_SHAPE), (dict(experts=None), ERR_NULL), (dict(offsets=None), ERR_NULL),
    (dict(pos=None), ERR_NULL), (dict(src=None), ERR_NULL), (dict(tokens=1000, rows=8000), ERR_NULL),
    (dict(tokens=1000, rows=8000, workspace=W), ERR_ARG), (dict(tokens=1000, rows=8000, workspace=W + 4, bytes=1 << 20), ERR_ALIGN),
    (dict(experts=X + 2), ERR_ALIGN), (dict(pos=P + 1), ERR_ALIGN), (dict(counts=C + 2), ERR_ALIGN), (dict(pos=X), ERR_ARG),
    (dict(src=P), ERR_ARG), (dict(counts=O), ERR_ARG), (dict(offsets=X + 4), ERR_ARG),
    (dict(tokens=1000, rows=8000, workspace=X, bytes=1 << 20), ERR_ARG),
])
def test_sort_refusals(L, change, status):
    assert L.fp8q_moe_sort(*{**SORT, **change}.values()) == status


DISPATCH = dict(x=X, dtype=BF16, cols=256, offsets=O, num_experts=4, pos=P, src=S, tokens=100, top_k=2, rows=512, fmt=E4M3, q=Q,
                scales=C, qt=QT, scales_t=CT, stream=None)
ROUTE = [(dict(num_experts=0), ERR_SHAPE), (dict(num_experts=1025), ERR_SHAPE), (dict(tokens=-1), ERR_SHAPE),
         (dict(top_k=0), ERR_SHAPE), (dict(rows=-128), ERR_SHAPE), (dict(cols=200), ERR_SHAPE), (dict(cols=-128), ERR_SHAPE),
         (dict(cols=1 << 30), ERR_SHAPE), (dict(offsets=None), ERR_NULL), (dict(pos=None), ERR_NULL), (dict(src=None), ERR_NULL),
         (dict(offsets=O + 2), ERR_ALIGN), (dict(pos=P + 2), ERR_ALIGN), (dict(src=S + 1), ERR_ALIGN), (dict(q=None), ERR_NULL),
         (dict(scales=None), ERR_NULL), (dict(q=Q + 8), ERR_ALIGN), (dict(scales=C + 2), ERR_ALIGN), (dict(q=X), ERR_ARG),
         (dict(q=O), ERR_ARG), (dict(scales=P), ERR_ARG), (dict(q=S), ERR_ARG), (dict(scales=Q), ERR_ARG)]


@pytest.mark.parametrize("change, status", ROUTE + [
    (dict(fmt=2), ERR_FORMAT), (dict(dtype=2), ERR_DTYPE), (dict(x=None), ERR_NULL), (dict(x=X + 8), ERR_ALIGN),
    (dict(qt=None), ERR_NULL), (dict(scales_t=None), ERR_NULL), (dict(rows=500), ERR_SHAPE), (dict(qt=Q), ERR_ARG),
    (dict(scales_t=CT + 1), ERR_ALIGN), (dict(qt=QT + 4), ERR_ALIGN), (dict(tokens=0, x=None), OK), (dict(rows=0, q=None), OK),
    (dict(cols=0), OK)])
def test_dispatch_refusals(L, change, status):
    assert L.fp8q_moe_dispatch(*{**DISPATCH, **change}.values()) == status


CODES = dict(xq=X, xs=W, fmt=E4M3, cols=256, offsets=O, num_experts=4, pos=P, src=S, tokens=100, top_k=2, rows=500, q=Q, scales=C,
             stream=None)


@pytest.mark.parametrize("change, status", ROUTE + [
    (dict(fmt=2), ERR_FORMAT), (dict(xq=None), ERR_NULL), (dict(xs=None), ERR_NULL), (dict(xq=X + 8), ERR_ALIGN),
    (dict(xs=W + 1), ERR_ALIGN), (dict(q=W), ERR_ARG), (dict(tokens=0), OK)])
def test_dispatch_codes_refusals(L, change, status):
    assert L.fp8q_moe_dispatch_codes(*{**CODES, **change}.values()) == status


COMBINE = dict(x=X, dtype=BF16, rows=300, cols=256, pos=P, weights=W, residual=D, tokens=100, top_k=2, y=Q, stream=None)


@pytest.mark.parametrize("change, status", [
    (dict(dtype=2), ERR_DTYPE), (dict(rows=-1), ERR_SHAPE), (dict(cols=130), ERR_SHAPE), (dict(tokens=-1), ERR_SHAPE),
    (dict(top_k=0), ERR_SHAPE), (dict(x=None), ERR_NULL), (dict(pos=None), ERR_NULL), (dict(y=None), ERR_NULL),
    (dict(x=X + 8), ERR_ALIGN), (dict(residual=D + 8), ERR_ALIGN), (dict(y=Q + 8), ERR_ALIGN), (dict(pos=P + 2), ERR_ALIGN),
    (dict(weights=W + 2), ERR_ALIGN), (dict(y=X), ERR_ARG), (dict(y=D), ERR_ARG), (dict(y=P), ERR_ARG), (dict(y=W), ERR_ARG),
    (dict(tokens=0, x=None), OK), (dict(cols=0, y=None), OK)])
def test_combine_refusals(L, change, status):
    assert L.fp8q_moe_combine(*{**COMBINE, **change}.values()) == status


BACK = dict(dy=X, x=D, dtype=BF16, cols=256, offsets=O, num_experts=4, pos=P, src=S, tokens=100, top_k=2, rows=512, weights=W,
            fmt=E5M2, q=Q, scales=C, qt=QT, scales_t=CT, dweights=0x7F0000000000 + (10 << 37), stream=None)


@pytest.mark.parametrize("change, status", [r for r in ROUTE if r[0] not in ({"cols": 0},)] + [
    (dict(fmt=2), ERR_FORMAT), (dict(dtype=2), ERR_DTYPE), (dict(dy=None), ERR_NULL), (dict(x=None), ERR_NULL),
    (dict(weights=None), ERR_NULL), (dict(q=None, scales=None), ERR_NULL), (dict(q=None, scales=None, qt=None, scales_t=None,
                                                                                dweights=None), ERR_NULL),
    (dict(rows=500), ERR_SHAPE), (dict(dweights=W), ERR_ARG), (dict(dweights=X + 4), ERR_ARG), (dict(dweights=C), ERR_ARG),
    (dict(dy=X + 8), ERR_ALIGN), (dict(x=D + 8), ERR_ALIGN), (dict(weights=W + 2), ERR_ALIGN), (dict(tokens=0), OK)])
def test_combine_backward_refusals(L, change, status):
    assert L.fp8q_moe_combine_backward(*{**BACK, **change}.values()) == status


GEMM = dict(a=X, sa=S, a_fmt=E4M3, b=W, sb=D, b_fmt=E4M3, offsets=O, num_experts=4, rows=100, N=256, K=256, c=Q, c_dtype=BF16,
            stream=None)
PRODUCT = [(dict(a_fmt=3), ERR_FORMAT), (dict(b_fmt=3), ERR_FORMAT), (dict(num_experts=0), ERR_SHAPE),
           (dict(num_experts=1025), ERR_SHAPE), (dict(rows=-1), ERR_SHAPE), (dict(K=100), ERR_SHAPE), (dict(rows=1 << 31), ERR_SHAPE),
           (dict(a=None), ERR_NULL), (dict(sa=None), ERR_NULL), (dict(b=None), ERR_NULL), (dict(sb=None), ERR_NULL),
           (dict(offsets=None), ERR_NULL), (dict(a=X + 8), ERR_ALIGN), (dict(b=W + 8), ERR_ALIGN), (dict(sa=S + 2), ERR_ALIGN),
           (dict(sb=D + 2), ERR_ALIGN), (dict(offsets=O + 2), ERR_ALIGN), (dict(rows=0, a=None), OK)]


@pytest.mark.parametrize("change, status", PRODUCT + [
    (dict(c_dtype=2), ERR_DTYPE), (dict(N=200), ERR_SHAPE), (dict(N=1 << 29, num_experts=8), ERR_SHAPE), (dict(c=None), ERR_NULL),
    (dict(c=Q + 8), ERR_ALIGN), (dict(c=X), ERR_ARG), (dict(c=W), ERR_ARG), (dict(c=O), ERR_ARG), (dict(N=0, c=None), OK)])
def test_gemm_grouped_refusals(L, change, status):
    assert L.fp8q_gemm_grouped(*{**GEMM, **change}.values()) == status


GATED = dict(a=X, sa=S, a_fmt=E4M3, b=W, sb=D, b_fmt=E4M3, offsets=O, num_experts=4, rows=100, F=256, K=256, act=0, fmt=E4M3, q=Q,
             scales=C, gu=QT, gu_dtype=BF16, stream=None)


@pytest.mark.parametrize("change, status", PRODUCT + [
    (dict(fmt=3), ERR_FORMAT), (dict(gu_dtype=3), ERR_DTYPE), (dict(act=2), ERR_ARG), (dict(F=192), ERR_SHAPE),
    (dict(F=1 << 29), ERR_SHAPE), (dict(F=1 << 28, num_experts=8), ERR_SHAPE), (dict(q=None), ERR_NULL), (dict(scales=None), ERR_NULL),
    (dict(q=None, scales=None, gu=None), ERR_NULL), (dict(q=Q + 8), ERR_ALIGN), (dict(gu=QT + 8), ERR_ALIGN),
    (dict(scales=C + 2), ERR_ALIGN), (dict(gu=Q), ERR_ARG), (dict(scales=D), ERR_ARG), (dict(F=0), OK)])
def test_gemm_gated_grouped_refusals(L, change, status):
    assert L.fp8q_gemm_gated_grouped(*{**GATED, **change}.values()) == status


WGRAD = dict(at=X, sat=S, a_fmt=E4M3, bt=W, sbt=D, b_fmt=E4M3, offsets=O, num_experts=4, rows=512, N=256, K=384, dw=Q, dw_dtype=F32,
             stream=None)


@pytest.mark.parametrize("change, status", [
    (dict(a_fmt=3), ERR_FORMAT), (dict(b_fmt=3), ERR_FORMAT), (dict(dw_dtype=3), ERR_DTYPE), (dict(num_experts=0), ERR_SHAPE),
    (dict(rows=500), ERR_SHAPE), (dict(N=200), ERR_SHAPE), (dict(K=200), ERR_SHAPE), (dict(N=1 << 29, num_experts=8), ERR_SHAPE),
    (dict(at=None), ERR_NULL), (dict(sat=None), ERR_NULL), (dict(bt=None), ERR_NULL), (dict(sbt=None), ERR_NULL),
    (dict(offsets=None), ERR_NULL), (dict(dw=None), ERR_NULL), (dict(at=X + 8), ERR_ALIGN), (dict(bt=W + 8), ERR_ALIGN),
    (dict(dw=Q + 8), ERR_ALIGN), (dict(sat=S + 2), ERR_ALIGN), (dict(offsets=O + 2), ERR_ALIGN), (dict(dw=X), ERR_ARG),
    (dict(dw=O), ERR_ARG), (dict(N=0, dw=None), OK), (dict(K=0), OK)])
def test_wgrad_refusals(L, change, status):
    assert L.fp8q_gemm_grouped_wgrad(*{**WGRAD, **change}.values()) == status
