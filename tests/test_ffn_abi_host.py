"""The feed-forward operators' C ABI and binding: what include/fp8q_ffn.h declares is exported and bound, and bad
arguments are refused on the host before anything is launched (no GPU needed)."""
import ctypes
import os
import re

import pytest
import torch

from fine_grained_block_b200 import binding
from fine_grained_block_b200 import build as fbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp8q_ffn.h")
OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_FORMAT, ERR_DTYPE, ERR_CUDA, ERR_ARG = 0, -1, -2, -3, -4, -5, -6, -7

# Fake device addresses, far apart and never dereferenced.
X, R, W, Q, S, H, Y, D = (0x7F0000000000 + (i << 36) for i in range(8))
F32, BF16, E4M3, E5M2 = 0, 1, 0, 1


@pytest.fixture(scope="module")
def L():
    fbuild.build()
    return binding.load_library()


def test_declared_exported_and_bound(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = set(re.findall(r"^\s*(?:int|int64_t)\s+(fp8q_\w+)\s*\(", text, flags=re.M))
    exported = set(re.findall(r" T (fp8q_\w+)$", os.popen(f"nm -D --defined-only {binding.LIB_PATH}").read(), flags=re.M))
    assert declared == exported == set(binding.FFN_SIGNATURES)
    import fine_grained_block_b200 as pkg
    for name in ("fp8q_rmsnorm_quantize", "fp8q_rmsnorm_backward", "fp8q_gemm_gated", "fp8q_gated_backward"):
        assert getattr(pkg, name) is getattr(binding, name)


NORM = dict(x=X, dtype=BF16, residual=R, weight=W, w_dtype=BF16, rows=4, cols=256, eps=1e-6, fmt=E4M3, q=Q, scales=S, h=H,
            y=Y, rstd=D, stream=None)


@pytest.mark.parametrize("change, status", [
    (dict(fmt=2), ERR_FORMAT), (dict(dtype=2), ERR_DTYPE), (dict(w_dtype=-1), ERR_DTYPE), (dict(rows=-1), ERR_SHAPE),
    (dict(cols=-1), ERR_SHAPE), (dict(rows=1 << 40, cols=1 << 40), ERR_SHAPE), (dict(eps=0.0), ERR_ARG),
    (dict(eps=-1.0), ERR_ARG), (dict(eps=float("inf")), ERR_ARG), (dict(eps=float("nan")), ERR_ARG),
    (dict(x=None), ERR_NULL), (dict(weight=None), ERR_NULL), (dict(q=None), ERR_NULL), (dict(scales=None), ERR_NULL),
    (dict(h=None), ERR_NULL), (dict(x=X + 8), ERR_ALIGN), (dict(residual=R + 2), ERR_ALIGN), (dict(weight=W + 8), ERR_ALIGN),
    (dict(q=Q + 1), ERR_ALIGN), (dict(h=H + 4), ERR_ALIGN), (dict(y=Y + 4), ERR_ALIGN), (dict(scales=S + 2), ERR_ALIGN),
    (dict(rstd=D + 1), ERR_ALIGN), (dict(h=X + 16), ERR_ARG), (dict(h=R - 16), ERR_ARG), (dict(q=X), ERR_ARG),
    (dict(y=H), ERR_ARG), (dict(y=X), ERR_ARG), (dict(rstd=S), ERR_ARG), (dict(q=S), ERR_ARG), (dict(h=W), ERR_ARG),
    (dict(rows=0, x=None, q=None), OK), (dict(cols=0, x=None, weight=None), OK),
])
def test_rmsnorm_quantize_refusals(L, change, status):
    assert L.fp8q_rmsnorm_quantize(*{**NORM, **change}.values()) == status


BACK = dict(dy=X, h=H, dtype=BF16, rstd=D, weight=W, w_dtype=F32, dh=R, rows=400, cols=256, dx=Y, dweight=Q, workspace=S,
            bytes=1 << 30, stream=None)


@pytest.mark.parametrize("change, status", [
    (dict(dtype=9), ERR_DTYPE), (dict(w_dtype=9), ERR_DTYPE), (dict(rows=-4), ERR_SHAPE), (dict(dy=None), ERR_NULL),
    (dict(h=None), ERR_NULL), (dict(rstd=None), ERR_NULL), (dict(weight=None), ERR_NULL), (dict(dx=None), ERR_NULL),
    (dict(workspace=None), ERR_NULL), (dict(bytes=16), ERR_ARG), (dict(dy=X + 8), ERR_ALIGN), (dict(h=H + 8), ERR_ALIGN),
    (dict(dh=R + 8), ERR_ALIGN), (dict(dx=Y + 8), ERR_ALIGN), (dict(dweight=Q + 2), ERR_ALIGN),
    (dict(workspace=S + 4), ERR_ALIGN), (dict(rstd=D + 2), ERR_ALIGN), (dict(dx=H), ERR_ARG), (dict(dx=X + 16), ERR_ARG),
    (dict(dweight=W), ERR_ARG), (dict(workspace=X), ERR_ARG), (dict(dweight=S), ERR_ARG),
    (dict(cols=0, dy=None, dweight=None), OK), (dict(rows=0, dy=None, dweight=None), OK),
])
def test_rmsnorm_backward_refusals(L, change, status):
    assert L.fp8q_rmsnorm_backward(*{**BACK, **change}.values()) == status


def test_rmsnorm_backward_workspace(L):
    assert L.fp8q_rmsnorm_backward_workspace(0, 256) == 0
    assert L.fp8q_rmsnorm_backward_workspace(3, 256) == 0  # few rows need none
    assert L.fp8q_rmsnorm_backward_workspace(400, 256) == 400 * 256 * 4
    big = L.fp8q_rmsnorm_backward_workspace(1 << 20, 256)
    assert 0 < big < 1 << 22 and big % (256 * 4) == 0
    assert L.fp8q_rmsnorm_backward_workspace(-1, 256) == ERR_SHAPE


GEMM = dict(a=X, sa=S, a_fmt=E4M3, b=W, sb=R, b_fmt=E4M3, M=4, F=256, K=256, act=0, fmt=E4M3, q=Q, scales=H, gu=Y,
            gu_dtype=BF16, stream=None)


@pytest.mark.parametrize("change, status", [
    (dict(a_fmt=3), ERR_FORMAT), (dict(b_fmt=3), ERR_FORMAT), (dict(fmt=3), ERR_FORMAT), (dict(gu_dtype=3), ERR_DTYPE),
    (dict(act=2), ERR_ARG), (dict(act=-1), ERR_ARG), (dict(M=-1), ERR_SHAPE), (dict(F=192), ERR_SHAPE),
    (dict(K=100), ERR_SHAPE), (dict(M=1 << 31), ERR_SHAPE), (dict(M=(1 << 30) - 1, K=(1 << 30) - 128), ERR_SHAPE),
    (dict(a=None), ERR_NULL), (dict(sa=None), ERR_NULL), (dict(b=None), ERR_NULL), (dict(sb=None), ERR_NULL),
    (dict(q=None), ERR_NULL), (dict(scales=None), ERR_NULL), (dict(q=None, scales=None, gu=None), ERR_NULL),
    (dict(a=X + 8), ERR_ALIGN), (dict(b=W + 8), ERR_ALIGN), (dict(q=Q + 8), ERR_ALIGN), (dict(gu=Y + 8), ERR_ALIGN),
    (dict(sa=S + 2), ERR_ALIGN), (dict(sb=R + 2), ERR_ALIGN), (dict(scales=H + 2), ERR_ALIGN), (dict(q=X), ERR_ARG),
    (dict(gu=W), ERR_ARG), (dict(gu=Q), ERR_ARG), (dict(scales=S), ERR_ARG),
    (dict(M=0, a=None, q=None), OK), (dict(F=0, q=None, scales=None, gu=None), OK),
])
def test_gemm_gated_refusals(L, change, status):
    assert L.fp8q_gemm_gated(*{**GEMM, **change}.values()) == status


GATED = dict(gu=X, dh=R, dtype=BF16, M=4, F=256, act=1, fmt=E5M2, q=Q, scales=S, qt=H, scales_t=Y, ht=W, ht_scales=D,
             stream=None)


@pytest.mark.parametrize("change, status", [
    (dict(fmt=5), ERR_FORMAT), (dict(dtype=5), ERR_DTYPE), (dict(act=5), ERR_ARG), (dict(F=100), ERR_SHAPE),
    (dict(M=-1), ERR_SHAPE), (dict(M=1 << 31), ERR_SHAPE), (dict(gu=None), ERR_NULL), (dict(dh=None), ERR_NULL),
    (dict(q=None), ERR_NULL), (dict(scales=None), ERR_NULL), (dict(qt=None), ERR_NULL), (dict(scales_t=None), ERR_NULL),
    (dict(ht=None), ERR_NULL), (dict(ht_scales=None), ERR_NULL), (dict(gu=X + 8), ERR_ALIGN), (dict(dh=R + 8), ERR_ALIGN),
    (dict(q=Q + 8), ERR_ALIGN), (dict(qt=H + 8), ERR_ALIGN), (dict(ht=W + 8), ERR_ALIGN), (dict(scales=S + 2), ERR_ALIGN),
    (dict(scales_t=Y + 2), ERR_ALIGN), (dict(ht_scales=D + 2), ERR_ALIGN), (dict(q=X), ERR_ARG), (dict(qt=R), ERR_ARG),
    (dict(ht=Q), ERR_ARG), (dict(ht_scales=Y), ERR_ARG),
    (dict(M=0, gu=None, q=None), OK), (dict(F=0, gu=None), OK),
])
def test_gated_backward_refusals(L, change, status):
    assert L.fp8q_gated_backward(*{**GATED, **change}.values()) == status


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, 128)
    for call in (lambda: binding.fp8q_rmsnorm_quantize(x, torch.ones(128)),
                 lambda: binding.fp8q_rmsnorm_backward(x, x, torch.ones(2), torch.ones(128)),
                 lambda: binding.fp8q_gemm_gated(x.to(torch.uint8), torch.ones(2, 1), x.to(torch.uint8), torch.ones(1, 1)),
                 lambda: binding.fp8q_gated_backward(torch.zeros(2, 256), x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
