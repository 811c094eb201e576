"""The feed-forward operators against plain implementations in 64 bits.

Tolerances.  u = 2^-24 is half an fp32 step.  A code is v * s rounded to nearest: half a step is 2^-4 (E4M3) or 2^-3
(E5M2) of the value, and 2^-10 or 2^-17 in the subnormal range, so with the returned scale s
    |decode(q) / s - v| <= half * |v| + sub / s + e_v,   e_v the error of the fp32 value before its rounding,
and |MAX / s - amax| <= max e_v + 4 u amax.
Norm: the row's sum of squares has at most 100 dependent additions (a thread's elements, then the reductions) at the
widths used here, so rstd is off by (100 / 2 + 8) u and y by 64 u = 2^-18, relative.  Backward: every term's error is
within 2^-17 of B = rstd (|a| + |n| mean|a n|) + |dh| (the same count for the mean, and n's, a's and the last sums' roundings),
dweight's within 2^-17 of the sum of |dy n| (at most 100 dependent additions in all).
Gated product: a chunk's sum of 128 products carries 2^-14 of its absolute sum at most (as allowed for the blockwise
GEMM), the two roundings of the factor 2^-22, the sum over chunks (K / 128) u and up to 8 ranks 8 u: e = (2^-14 + 2^-22 +
(K/128 + 8) u) S with S the product over absolute values.  exp(-p) is off by |p| 2^-22 relative (p's own rounding) and
2 more units, 1 / (1 + x) by 2: act is off by (1 + |p|) 2^-20 relative; act' is bounded by 1.13 for both activations.
A bf16 output adds 2^-8 relative.
"""
import math

import pytest
import torch

from fine_grained_block_b200 import binding as B
from parity_util import Guarded

pytestmark = pytest.mark.gpu

F8 = {B.E4M3: torch.float8_e4m3fn, B.E5M2: torch.float8_e5m2}
HALF = {B.E4M3: 2.0 ** -4, B.E5M2: 2.0 ** -3}
SUB = {B.E4M3: 2.0 ** -10, B.E5M2: 2.0 ** -17}
MAX = {B.E4M3: 448.0, B.E5M2: 57344.0}
U = 2.0 ** -24
BF, FP = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _status():
    B.fp8_device_status(clear=True)
    yield
    assert B.fp8_device_status() == 0


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * std


def guarded(*specs):
    return [Guarded(s, d) for s, d in specs]


def spread(scales, cols):
    return scales.double().repeat_interleave(128, dim=1)[:, :cols]


def check_codes(q, scales, v, e, fmt, what):
    """Codes and scales of v [R, C] (fp64), whose fp32 value is off by at most e."""
    R, C = v.shape
    nb = -(-C // 128)
    pad = lambda t: torch.nn.functional.pad(t, (0, nb * 128 - C)).view(R, nb, 128)  # noqa: E731
    amax, emax = pad(v.abs()).amax(2), pad(e).amax(2)
    assert scales.shape == (R, nb) and bool((scales > 0).all()), what
    got = MAX[fmt] / scales.double()
    assert bool(((got - amax.clamp_min(1e-12)).abs() <= emax + 4 * U * amax.clamp_min(1e-12)).all()), f"{what}: scales"
    s = spread(scales, C)
    d = q.view(F8[fmt]).double()
    err = (d / s - v).abs()
    tol = HALF[fmt] * (v.abs() + e) + SUB[fmt] / s + e
    assert bool((err <= tol).all()), f"{what}: codes off by {float((err / tol).max()):.3g} of the bound"


def check_close(got, want, tol, what):
    if got.dtype == BF:
        tol = tol + 2.0 ** -8 * want.abs()
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), f"{what}: off by {float((err / tol.clamp_min(1e-300)).max()):.3g} of the bound"


# -- the norm ---------------------------------------------------------------------------------------------------------

def norm_reference(x, residual, w, eps=1e-6):
    h = x if residual is None else (x.double() + residual.double()).to(x.dtype)
    hd = h.double()
    rstd = (hd.square().mean(1) + eps).rsqrt()
    return h, rstd, hd * rstd[:, None] * w.double()


def run_norm(x, residual, w, fmt, y=True, **kw):
    R, C = x.shape
    out = guarded(((R, C), torch.uint8), ((R, -(-C // 128)), FP), ((R, C), x.dtype), ((R, C), x.dtype), ((R,), FP))
    q, s, h, yo, rstd = B.fp8q_rmsnorm_quantize(x, w, residual, fmt=fmt, q=out[0].t, scales=out[1].t,
                                                h=out[2].t if residual is not None else None, y=out[3].t if y else None,
                                                rstd=out[4].t, **kw)
    torch.cuda.synchronize()
    for o in out:
        o.check()
    return q, s, h, yo, rstd


def check_norm(x, residual, w, fmt, what):
    q, s, h, y, rstd = run_norm(x, residual, w, fmt)
    rh, rr, ry = norm_reference(x, residual, w)
    assert torch.equal(h, rh), what
    check_close(rstd, rr, 2.0 ** -18 * rr, what + " rstd")
    e = 2.0 ** -18 * ry.abs()
    check_close(y, ry, e, what + " y")
    check_codes(q, s, ry, e, fmt, what)
    if x.dtype == FP:  # the codes of the fp32 y, exactly
        q2, s2 = B.fp8_quantize_blockwise(y, (1, 128), fmt)
        assert torch.equal(q, q2) and torch.equal(s, s2), what


NORM_SHAPES = [(1, 1), (3, 5), (2, 127), (1, 128), (5, 129), (300, 64), (9, 512), (1, 4096), (257, 1024), (33, 4104),
               (1200, 520), (17, 7168), (3, 8208), (2, 16384), (2, 16400), (5, 20001), (1000, 144), (700, 7168), (600, 4100),
               (500, 3001), (2500, 301), (3, 4096), (16, 7168), (17, 7168), (13, 1001), (16, 8191), (60, 512), (128, 64),
               (129, 64), (50, 9000), (1800, 2048), (2101, 8192)]


@pytest.mark.parametrize("rows, cols", NORM_SHAPES)
@pytest.mark.parametrize("dtype, fmt", [(BF, B.E4M3), (BF, B.E5M2), (FP, B.E4M3), (FP, B.E5M2)])
@pytest.mark.parametrize("with_residual", [True, False])
def test_norm(rows, cols, dtype, fmt, with_residual):
    g = gen(rows * 31 + cols)
    x = normal(g, rows, cols)
    x[:, 0] *= 30
    r = normal(g, rows, cols, std=2.0).to(dtype) if with_residual else None
    w = (1 + normal(g, cols, std=0.2)).to(FP if cols % 2 else BF)  # weights of either type with either input
    check_norm(x.to(dtype), r, w, fmt, f"{rows}x{cols} {dtype}")


@pytest.mark.parametrize("dtype", [BF, FP])
def test_norm_sixteen_byte_aligned_views(dtype):
    """Rows of whole 32-byte vectors at an address that is only 16-byte aligned."""
    g = gen(5)
    e = 16 // torch.empty(0, dtype=dtype).element_size()
    rows, cols = 12, 2048
    x, r = (normal(g, rows * cols + e).to(dtype)[e:].view(rows, cols) for _ in range(2))
    assert x.data_ptr() % 32 == 16
    check_norm(x, r, torch.ones(cols, dtype=dtype, device="cuda"), B.E4M3, "unaligned")


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("cols", [512, 4096, 777])
def test_norm_in_place(dtype, cols):
    g = gen(cols)
    x, r = normal(g, 40, cols).to(dtype), normal(g, 40, cols).to(dtype)
    w = torch.ones(cols, device="cuda")
    want = run_norm(x, r, w, B.E4M3)
    for target in (0, 1):
        pair = [x.clone(), r.clone()]
        q, s, h, y, rstd = B.fp8q_rmsnorm_quantize(pair[0], w, pair[1], h=pair[target], want_y=True, want_rstd=True)
        assert h.data_ptr() == pair[target].data_ptr()
        for a, b in zip((q, s, h, y, rstd), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("cols", [256, 4096, 300])
def test_norm_zero_rows_and_values_that_are_not_finite(cols):
    x = torch.randn(6, cols, device="cuda")
    x[1] = 0
    x[2, 3] = float("nan")
    x[3, 7] = float("inf")
    x[4] *= 1e25  # the squares overflow
    w = torch.ones(cols, device="cuda")
    q, s, h, y, rstd = run_norm(x, None, w, B.E4M3)
    assert float(rstd[1]) == pytest.approx(1e3, rel=1e-6) and bool((q[1] == 0).all()) and bool((y[1] == 0).all())
    assert bool((s[1] == torch.tensor(448.0) / torch.tensor(1e-12)).all())
    assert bool(torch.isnan(y[2]).all()) and bool((q[2] & 0x7F == 0x7F).all())
    assert float(rstd[3]) == 0 and bool(torch.isnan(y[3, 7])) and bool((y[3, :7] == 0).all())
    assert float(rstd[4]) == 0 and bool((y[4] == 0).all())
    rr = norm_reference(x, None, w)[1]
    check_close(rstd[[0, 5]], rr[[0, 5]], 2.0 ** -18 * rr[[0, 5]], "the other rows")


def test_norm_without_rows_or_columns():
    w = torch.ones(256, device="cuda")
    q, s, *_ = B.fp8q_rmsnorm_quantize(torch.empty(0, 256, device="cuda"), w)
    assert q.shape == (0, 256) and s.shape == (0, 2)
    q, s, *_ = B.fp8q_rmsnorm_quantize(torch.empty(3, 0, device="cuda"), w[:0])
    assert q.shape == (3, 0) and s.shape == (3, 0)
    dx, dw = B.fp8q_rmsnorm_backward(torch.empty(0, 256, device="cuda"), torch.empty(0, 256, device="cuda"),
                                     torch.empty(0, device="cuda"), w)
    assert dx.shape == (0, 256) and bool((dw == 0).all())


def backward_reference(dy, h, rstd, w, dh):
    hd, dyd, r = h.double(), dy.double(), rstd.double()[:, None]
    n, a = hd * r, dyd * w.double()
    dx = r * (a - n * (a * n).mean(1, keepdim=True)) + (0 if dh is None else dh.double())
    b = r * (a.abs() + n.abs() * (a * n).abs().mean(1, keepdim=True)) + (0 if dh is None else dh.double().abs())
    return dx, b, (dyd * n).sum(0), (dyd * n).abs().sum(0)


@pytest.mark.parametrize("rows, cols", NORM_SHAPES)
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("with_dh", [True, False])
def test_norm_backward(rows, cols, dtype, with_dh):
    g = gen(rows * 17 + cols)
    dy, h = normal(g, rows, cols, std=0.01).to(dtype), normal(g, rows, cols, std=3.0).to(dtype)
    dh = normal(g, rows, cols, std=0.01).to(dtype) if with_dh else None
    w = (1 + normal(g, cols, std=0.2)).to(FP if cols % 2 else BF)
    rstd = (h.double().square().mean(1) + 1e-6).rsqrt().float()
    out = guarded(((rows, cols), dtype), ((cols,), FP))
    ws = Guarded((B.load_library().fp8q_rmsnorm_backward_workspace(rows, cols),), torch.uint8)  # 0xA5: any content
    dx, dw = B.fp8q_rmsnorm_backward(dy, h, rstd, w, dh, dx=out[0].t, dweight=out[1].t, workspace=ws.t)
    torch.cuda.synchronize()
    for o in (*out, ws):
        o.check()
    rdx, b, rdw, bw = backward_reference(dy, h, rstd, w, dh)
    check_close(dx, rdx, 2.0 ** -17 * b, "dx")
    check_close(dw, rdw, 2.0 ** -17 * bw, "dweight")
    # again: the same bits; without the weight gradient and in place: the same dx
    dx2, dw2 = B.fp8q_rmsnorm_backward(dy, h, rstd, w, dh)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    for target in [dy] + ([dh] if with_dh else []):
        t = target.clone()
        args = [t if a is target else a for a in (dy, h, rstd, w, dh)]
        dx3, none = B.fp8q_rmsnorm_backward(*args, dx=t, want_dweight=False)
        assert none is None and torch.equal(dx3, dx)


@pytest.mark.parametrize("rows, cols", [(2, 256), (3, 4096), (2, 77), (5, 7168), (13, 2048), (14, 4101), (100, 128), (2, 9000)])
def test_norm_backward_of_few_rows_into_a_four_byte_aligned_weight_gradient(rows, cols):
    """One CTA may write the weight gradient itself, 16 bytes at a time: not where it lies on a 4-byte boundary."""
    g = gen(rows + cols)
    dy, h = normal(g, rows, cols), normal(g, rows, cols)
    w, rstd = torch.ones(cols, device="cuda"), torch.rand(rows, device="cuda", generator=g)
    store = torch.full((cols + 2,), 7.0, device="cuda")
    dx, dw = B.fp8q_rmsnorm_backward(dy, h, rstd, w, dweight=store[1:-1])
    assert float(store[0]) == float(store[-1]) == 7.0
    rdx, b, rdw, bw = backward_reference(dy, h, rstd, w, None)
    check_close(dx, rdx, 2.0 ** -17 * b, "dx")
    check_close(dw, rdw, 2.0 ** -17 * bw, "dweight")
    assert torch.equal(dw, B.fp8q_rmsnorm_backward(dy, h, rstd, w)[1])


def test_norm_gradient_against_differences():
    """Central differences of the 64-bit forward pass: their own error is step^2 times a third derivative, 1e-8 here."""
    g = gen(77)
    h, w, dy = normal(g, 3, 40).double(), (1 + normal(g, 40, std=0.1)).double(), normal(g, 3, 40).double()

    def loss(h, w):
        return float((h * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w * dy).sum())

    h32, w32, dy32 = h.float(), w.float(), dy.float()
    dx, dw = B.fp8q_rmsnorm_backward(dy32, h32, (h.square().mean(1) + 1e-6).rsqrt().float(), w32)
    step = 1e-4
    for i, j in [(0, 0), (1, 17), (2, 39), (0, 20)]:
        d = torch.zeros_like(h)
        d[i, j] = step
        assert (loss(h + d, w) - loss(h - d, w)) / (2 * step) == pytest.approx(float(dx[i, j]), abs=1e-5)
        e = torch.zeros_like(w)
        e[j] = step
        assert (loss(h, w + e) - loss(h, w - e)) / (2 * step) == pytest.approx(float(dw[j]), abs=1e-5)


# -- the gated projections ----------------------------------------------------------------------------------------------

def decode(q, scales, block_rows, fmt):
    v = q.view(F8[fmt]).double()
    s = scales.double().repeat_interleave(block_rows, 0)[:v.shape[0]].repeat_interleave(128, 1)[:, :v.shape[1]]
    return v / s


def act64(g, act):
    """act(g), act'(g), p(g) in 64 bits."""
    if act == B.ACT_SILU:
        sg = torch.sigmoid(g)
        return g * sg, sg * (1 + g * (1 - sg)), g
    c = math.sqrt(2 / math.pi)
    z = c * (g + 0.044715 * g ** 3)
    sg = torch.sigmoid(2 * z)  # 0.5 (1 + tanh z)
    return g * sg, sg + g * sg * (1 - sg) * 2 * c * (1 + 3 * 0.044715 * g ** 2), 2 * z


def projections(a, sa, a_fmt, b, sb, b_fmt):
    av, bv = decode(a, sa, 1, a_fmt), decode(b, sb, 128, b_fmt)
    return av @ bv.T, av.abs() @ bv.abs().T


def check_gated(M, F, K, act=B.ACT_SILU, fmt=B.E4M3, a_fmt=B.E4M3, b_fmt=B.E4M3, gu_dtype=FP, want_q=True, seed=0):
    g = gen(M * 7 + F + K + seed)
    a, sa = B.fp8_quantize_blockwise(normal(g, M, K), (1, 128), a_fmt)
    b, sb = B.fp8_quantize_blockwise(normal(g, 2 * F, K, std=2 / math.sqrt(K)), (128, 128), b_fmt)
    out = guarded(((M, F), torch.uint8), ((M, F // 128), FP), ((M, 2 * F), gu_dtype or FP))
    kw = dict(q=out[0].t, scales=out[1].t) if want_q else dict(want_q=False)
    q, s, gu = B.fp8q_gemm_gated(a, sa, b, sb, a_fmt, b_fmt, act, fmt, gu=out[2].t if gu_dtype else None, **kw)
    torch.cuda.synchronize()
    for o in out:
        o.check()
    G, S = projections(a, sa, a_fmt, b, sb, b_fmt)
    e = (2.0 ** -14 + 2.0 ** -22 + (K / 128 + 8) * U) * S
    what = f"{M}x{F}x{K}"
    if gu_dtype:
        check_close(gu, G, e, what + " gu")
    if want_q:
        (gg, uu), (eg, eu) = G.split(F, 1), e.split(F, 1)
        av, _, p = act64(gg, act)
        H = av * uu
        eh = 1.13 * eg * uu.abs() + av.abs() * eu + 1.13 * eg * eu + 2.0 ** -20 * (1 + p.abs()) * H.abs()
        check_codes(q, s, H, eh, fmt, what)
    return a, sa, b, sb, q, s, gu


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 32, 33, 64, 65, 127, 128, 129, 255, 256, 257, 600])
@pytest.mark.parametrize("F, K", [(128, 128), (384, 640)])
def test_gated_tokens(M, F, K):
    check_gated(M, F, K, act=M % 2, fmt=M // 2 % 2)


@pytest.mark.parametrize("M", [3, 40, 100, 300])
@pytest.mark.parametrize("act", [B.ACT_SILU, B.ACT_GELU_TANH])
@pytest.mark.parametrize("a_fmt, b_fmt, fmt", [(B.E4M3, B.E5M2, B.E4M3), (B.E5M2, B.E4M3, B.E5M2), (B.E5M2, B.E5M2, B.E4M3)])
def test_gated_formats(M, act, a_fmt, b_fmt, fmt):
    check_gated(M, 256, 512, act, fmt, a_fmt, b_fmt, gu_dtype=BF)


@pytest.mark.parametrize("M", [5, 30, 50, 90, 700])
@pytest.mark.parametrize("gu_dtype, want_q", [(None, True), (BF, False), (FP, False)])
def test_gated_outputs(M, gu_dtype, want_q):
    check_gated(M, 256, 1024, gu_dtype=gu_dtype, want_q=want_q)


@pytest.mark.parametrize("M, F, K", [
    (1, 4096, 7168),    # K split over a cluster
    (4, 128, 16384),    # one tile, the widest split
    (2, 128 * 300, 128),  # more tiles than CTAs at a time, one chunk
    (20, 128 * 180, 256),
    (60, 2048, 1152), (128, 1408, 896), (100, 128 * 150, 128),
    (1024, 4096, 256),  # more tiles than CTA pairs
    (5000, 512, 384),   # 20 rows of tiles: a group of 16 and one of 4
])
def test_gated_sizes(M, F, K):
    check_gated(M, F, K, act=B.ACT_GELU_TANH)


# Shapes whose CTAs fill more than half the SMs go to the CTA pairs: 2432 columns from 257 tokens on.
@pytest.mark.parametrize("M", [257, 300, 384, 511, 700])
@pytest.mark.parametrize("act, fmt, gu_dtype, want_q", [(B.ACT_SILU, B.E4M3, BF, True), (B.ACT_GELU_TANH, B.E5M2, BF, True),
                                                        (B.ACT_SILU, B.E4M3, BF, False), (B.ACT_GELU_TANH, B.E4M3, None, True),
                                                        (B.ACT_SILU, B.E5M2, FP, True)])
def test_gated_pairs(M, act, fmt, gu_dtype, want_q):
    check_gated(M, 2432, 256, act, fmt, gu_dtype=gu_dtype, want_q=want_q)


# More than 12 chunks of K and few tiles: two pairs share one.
@pytest.mark.parametrize("M, F, K", [(512, 1280, 1664), (449, 1280, 2176), (600, 1280, 1792), (257, 2560, 1664), (1000, 1024, 2048),
                                     (256, 4608, 1664)])
@pytest.mark.parametrize("act, fmt, gu_dtype, want_q", [(B.ACT_SILU, B.E4M3, BF, True), (B.ACT_GELU_TANH, B.E5M2, FP, True),
                                                        (B.ACT_SILU, B.E4M3, FP, False), (B.ACT_GELU_TANH, B.E4M3, None, True)])
def test_gated_two_pairs_a_tile(M, F, K, act, fmt, gu_dtype, want_q):
    a, sa, b, sb, q, s, gu = check_gated(M, F, K, act, fmt, gu_dtype=gu_dtype, want_q=want_q)
    again = B.fp8q_gemm_gated(a, sa, b, sb, act=act, fmt=fmt, gu_dtype=gu_dtype or BF, want_q=want_q, want_gu=gu_dtype is not None)
    for first, second in zip((q, s, gu), again):
        assert first is None or torch.equal(first, second)  # the halves meet in a fixed order


@pytest.mark.parametrize("a_fmt, b_fmt", [(B.E4M3, B.E5M2), (B.E5M2, B.E4M3), (B.E5M2, B.E5M2)])
def test_gated_pairs_formats(a_fmt, b_fmt):
    check_gated(430, 2432, 640, B.ACT_SILU, B.E4M3, a_fmt, b_fmt, gu_dtype=BF)


def test_gated_pairs_with_many_tiles_each():
    check_gated(1500, 2432, 1152, gu_dtype=BF)  # 6 x 19 tiles of 74 pairs
    check_gated(6000, 640, 128, gu_dtype=BF)    # one chunk of K: the epilogues follow one another


def test_gated_pairs_nan_and_far_out():
    g = gen(4)
    M, F, K = 300, 2432, 256
    a, sa = B.fp8_quantize_blockwise(normal(g, M, K))
    b, sb = B.fp8_quantize_blockwise(normal(g, 2 * F, K, std=0.1), (128, 128))
    clean = B.fp8q_gemm_gated(a, sa, b, sb, want_gu=True)
    a = a.clone()
    a[299, 3] = 0x7F
    q, s, gu = B.fp8q_gemm_gated(a, sa, b, sb, want_gu=True)
    assert bool((q[299] & 0x7F == 0x7F).all()) and bool(torch.isnan(gu[299]).all())
    for x, y in ((q, clean[0]), (s, clean[1]), (gu, clean[2])):
        assert torch.equal(x[:299], y[:299])
    for act in (B.ACT_SILU, B.ACT_GELU_TANH):
        x = torch.zeros(M, 128, device="cuda")
        x[:, 0] = torch.linspace(-200, 200, M, device="cuda")
        a, sa = B.fp8_quantize_blockwise(x)
        w = torch.zeros(2 * F, 128, device="cuda")
        w[:, 0] = 1
        b, sb = B.fp8_quantize_blockwise(w, (128, 128))
        q, s, _ = B.fp8q_gemm_gated(a, sa, b, sb, act=act)
        gg = projections(a, sa, B.E4M3, b, sb, B.E4M3)[0][:, :F]
        av, _, p = act64(gg, act)
        H = av * gg
        check_codes(q, s, H, 2.0 ** -19 * (1 + p.abs()) * H.abs() + 1e-30, B.E4M3, "far out")


@pytest.mark.parametrize("M", [8, 200])
def test_gated_empty_sums(M):
    F = 256
    a, b = torch.empty(M, 0, dtype=torch.uint8, device="cuda"), torch.empty(2 * F, 0, dtype=torch.uint8, device="cuda")
    q, s, gu = B.fp8q_gemm_gated(a, torch.empty(M, 0, device="cuda"), b, torch.empty(2 * F // 128, 0, device="cuda"),
                                 want_gu=True)
    assert bool((q == 0).all()) and bool((gu == 0).all()) and bool((s == torch.tensor(448.0) / torch.tensor(1e-12)).all())
    q, s, _ = B.fp8q_gemm_gated(a[:0], torch.empty(0, 0, device="cuda"), b, torch.empty(2 * F // 128, 0, device="cuda"))
    assert q.shape == (0, F) and s.shape == (0, 2)


@pytest.mark.parametrize("M", [6, 20, 64, 128, 300])
def test_gated_projections_are_those_of_the_blockwise_gemm(M):
    """Within the two calls' accumulation bounds; rows behind the last token stay as they were (guard bands above)."""
    a, sa, b, sb, q, s, gu = check_gated(M, 256, 2048)
    c = B.fp8_gemm_blockwise(a, sa, b, sb, out_dtype=FP)
    S = projections(a, sa, B.E4M3, b, sb, B.E4M3)[1]
    assert bool(((gu - c).abs() <= 2.0 ** -12 * S).all())


@pytest.mark.parametrize("M", [9, 50, 200])
def test_gated_nan_code_reaches_its_row_only(M):
    g = gen(3)
    a, sa = B.fp8_quantize_blockwise(normal(g, M, 256))
    b, sb = B.fp8_quantize_blockwise(normal(g, 512, 256, std=0.1), (128, 128))
    clean = B.fp8q_gemm_gated(a, sa, b, sb)
    a = a.clone()
    a[4, 200] = 0x7F
    q, s, _ = B.fp8q_gemm_gated(a, sa, b, sb)
    assert bool((q[4] & 0x7F == 0x7F).all())
    keep = [m for m in range(M) if m != 4]
    assert torch.equal(q[keep], clean[0][keep]) and torch.equal(s[keep], clean[1][keep])


@pytest.mark.parametrize("act", [B.ACT_SILU, B.ACT_GELU_TANH])
def test_gate_values_far_out(act):
    """One weight per column makes G the activation itself: from -200 to 200, where exp overflows and underflows."""
    M, F, K = 401, 128, 128
    v = torch.linspace(-200, 200, M, device="cuda")
    x = torch.zeros(M, K, device="cuda")
    x[:, 0] = v
    a, sa = B.fp8_quantize_blockwise(x)
    b = torch.zeros(2 * F, K, device="cuda")
    b[:, 0] = 1
    b, sb = B.fp8_quantize_blockwise(b, (128, 128))
    for rows in (slice(0, 100), slice(0, M)):  # both kernels
        q, s, gu = B.fp8q_gemm_gated(a[rows], sa[rows], b, sb, act=act, want_gu=True, gu_dtype=FP)
        G, _ = projections(a[rows], sa[rows], B.E4M3, b, sb, B.E4M3)
        gg = G[:, :F]
        av, _, p = act64(gg, act)
        H = av * gg
        # fp32's smallest normal number bounds what flushing to zero can lose
        check_codes(q, s, H, 2.0 ** -19 * (1 + p.abs()) * H.abs() + 1e-30, B.E4M3, "far out")


# -- the gated backward pass ---------------------------------------------------------------------------------------------

def gated_backward_reference(gu, dh, act):
    F = dh.shape[1]
    g, u, d = gu[:, :F].double(), gu[:, F:].double(), dh.double()
    a, da, p = act64(g, act)
    sg = torch.sigmoid(p)
    c = 1.0 if act == B.ACT_SILU else 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g ** 2)
    rel = 2.0 ** -19 * (1 + p.abs())  # act's, and the three products'
    mag = sg + (a * (1 - sg) * c).abs()  # the terms of act'
    dg, du, H = d * u * da, d * a, a * u
    tiny = 1e-37
    return (torch.cat([dg, du], 1), torch.cat([(d * u).abs() * mag * rel, du.abs() * rel], 1) + tiny, H,
            H.abs() * rel + tiny)


def pad_t(v):
    return torch.nn.functional.pad(v, (0, 0, 0, -v.shape[0] % 128)).t().contiguous()


def check_gated_backward(gu, dh, act, fmt, what):
    M, F = dh.shape
    Mt = -(-M // 128) * 128
    u8 = torch.uint8
    out = guarded(((M, 2 * F), u8), ((M, 2 * F // 128), FP), ((2 * F, Mt), u8), ((2 * F, Mt // 128), FP), ((F, Mt), u8),
                  ((F, Mt // 128), FP))
    t = [o.t for o in out]
    B.fp8q_gated_backward(gu, dh, act, fmt, q=t[0], scales=t[1], qt=t[2], scales_t=t[3], ht=t[4], ht_scales=t[5])
    torch.cuda.synchronize()
    for o in out:
        o.check()
    D, e, H, eh = gated_backward_reference(gu, dh, act)
    check_codes(t[0], t[1], D, e, fmt, what)
    check_codes(t[2], t[3], pad_t(D), pad_t(e), fmt, what + " transposed")
    check_codes(t[4], t[5], pad_t(H), pad_t(eh), fmt, what + " H")
    assert bool((t[2][:, M:] == 0).all()) and bool((t[4][:, M:] == 0).all())
    rows = B.fp8q_gated_backward(gu, dh, act, fmt, transposed=False)
    assert torch.equal(rows[0], t[0]) and torch.equal(rows[1], t[1]) and rows[2:] == (None,) * 4
    return t


@pytest.mark.parametrize("M, F", [(1, 128), (3, 384), (127, 128), (128, 256), (129, 128), (300, 640), (1000, 1024)])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("act, fmt", [(B.ACT_SILU, B.E4M3), (B.ACT_GELU_TANH, B.E5M2)])
def test_gated_backward(M, F, dtype, act, fmt):
    g = gen(M + F)
    gu, dh = normal(g, M, 2 * F, std=2.0).to(dtype), normal(g, M, F, std=1e-3).to(dtype)
    check_gated_backward(gu, dh, act, fmt, f"{M}x{F} {dtype}")


@pytest.mark.parametrize("dtype", [BF, FP])
def test_gated_backward_sixteen_byte_aligned_views(dtype):
    g = gen(9)
    e = 16 // torch.empty(0, dtype=dtype).element_size()
    M, F = 140, 256
    gu = normal(g, M * 2 * F + e).to(dtype)[e:].view(M, 2 * F)
    dh = normal(g, M * F + e).to(dtype)[e:].view(M, F)
    assert gu.data_ptr() % 32 == 16
    check_gated_backward(gu, dh, B.ACT_SILU, B.E4M3, "unaligned")


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("act", [B.ACT_SILU, B.ACT_GELU_TANH])
def test_gated_backward_far_out_and_not_finite(act, dtype):
    M, F = 130, 128
    g = gen(11)
    gu, dh = normal(g, M, 2 * F).to(dtype), normal(g, M, F).to(dtype)
    gu[:, 0] = torch.linspace(-300, 300, M, device="cuda")
    gu[0] = 0
    dh[1] = 0
    check_gated_backward(gu, dh, act, B.E4M3, "far out")
    clean = B.fp8q_gated_backward(gu, dh, act)
    dh[5, 7] = float("nan")
    q, s, qt, st, ht, hs = B.fp8q_gated_backward(gu, dh, act)
    nan = torch.zeros(M, 2 * F, dtype=torch.bool, device="cuda")
    nan[5, 7] = nan[5, F + 7] = True
    assert torch.equal(q & 0x7F == 0x7F, nan) and torch.equal(qt[:, :M] & 0x7F == 0x7F, nan.t())
    assert torch.equal(ht, clean[4]) and torch.equal(hs, clean[5])  # H does not see dH
    other = [m for m in range(M) if m != 5]
    assert torch.equal(q[other], clean[0][other])


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("act", [B.ACT_SILU, B.ACT_GELU_TANH])
def test_gated_backward_of_gates_whose_square_is_infinite(act, dtype):
    """The slope is 1 above and 0 below, also where g^2 or its cubic leaves fp32."""
    M, F = 4, 128
    far = torch.tensor([1e4, 1e9, 1e15, 3e18, 1.8e19, 1e20, 1e25, 1e30, 1e37, 3e38], device="cuda").to(dtype)
    gate = torch.cat([far, -far]).repeat(7)[:F].repeat(M, 1)
    one = torch.ones(M, F, device="cuda", dtype=dtype)
    q, s, qt, st, *_ = B.fp8q_gated_backward(torch.cat([gate, one], 1).contiguous(), one, act)
    want = torch.where(gate > 0, 0x7E, 0).to(torch.uint8)  # dG = act'(g), and 1 is its block's maximum
    assert torch.equal(q[:, :F] & 0x7F, want) and torch.equal(qt[:F, :M] & 0x7F, want.t())
    assert bool((s[:, 0] == 448).all())


@pytest.mark.parametrize("dtype", [BF, FP])
def test_gated_backward_with_several_tiles_a_cta(dtype):
    """17 x 12 and 33 x 16 tiles: more than the SMs."""
    for M, F in ((2100, 1536), (4200, 2048)):
        g = gen(M)
        check_gated_backward(normal(g, M, 2 * F, std=1.5).to(dtype), normal(g, M, F, std=1e-2).to(dtype), B.ACT_SILU, B.E4M3,
                             f"{M}x{F} {dtype}")


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("which", ["qt", "ht"])
def test_gated_backward_with_one_transposed_output(dtype, which):
    """The C call takes either pair without the other."""
    M, F = 200, 256
    g = gen(41)
    gu, dh = normal(g, M, 2 * F).to(dtype), normal(g, M, F).to(dtype)
    q, s, qt, st, ht, hs = B.fp8q_gated_backward(gu, dh)
    one, one_s = (qt, st) if which == "qt" else (ht, hs)
    out = guarded((one.shape, torch.uint8), (one_s.shape, FP), (q.shape, torch.uint8), (s.shape, FP))
    p = [o.t.data_ptr() for o in out]
    pairs = (p[0], p[1], None, None) if which == "qt" else (None, None, p[0], p[1])
    rc = B.load_library().fp8q_gated_backward(gu.data_ptr(), dh.data_ptr(), B.BF16 if dtype == BF else B.F32, M, F, 0, 0, p[2],
                                              p[3], *pairs, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0
    for o, want in zip(out, (one, one_s, q, s)):
        o.check()
        assert torch.equal(o.t, want)


def test_gated_gradient_against_differences():
    """The returned codes stand for the gradients within half a step: central differences of the 64-bit forward pass."""
    M, F, step = 2, 128, 1e-5
    g = gen(21)
    gu, dh = normal(g, M, 2 * F), normal(g, M, F)
    for act in (B.ACT_SILU, B.ACT_GELU_TANH):
        q, s, *_ = B.fp8q_gated_backward(gu, dh, act, transposed=False)
        d = decode(q, s, 1, B.E4M3)

        def each(v):
            return act64(v[:, :F], act)[0] * v[:, F:] * dh.double()

        lo, hi = gu.double(), gu.double()
        for part in (slice(0, F), slice(F, 2 * F)):
            dlo, dhi = lo.clone(), hi.clone()
            dlo[:, part] -= step
            dhi[:, part] += step
            want = (each(dhi) - each(dlo)) / (2 * step)
            tol = HALF[B.E4M3] * want.abs() + SUB[B.E4M3] / spread(s, 2 * F)[:, part] + 1e-6 * (1 + want.abs())
            assert bool(((d[:, part] - want).abs() <= tol).all())


def test_gated_backward_without_tokens():
    out = B.fp8q_gated_backward(torch.empty(0, 256, device="cuda"), torch.empty(0, 128, device="cuda"))
    assert [tuple(t.shape) for t in out] == [(0, 256), (0, 2), (256, 0), (256, 0), (128, 0), (128, 0)]


# -- together, as a feed-forward block uses them ---------------------------------------------------------------------------

def block_inputs(M, D, F, seed=0):
    g = gen(1000 + seed)
    x, res = normal(g, M, D).to(BF), normal(g, M, D).to(BF)
    w = (1 + normal(g, D, std=0.1)).to(BF)
    wgu, wd = normal(g, 2 * F, D, std=1 / math.sqrt(D)), normal(g, D, F, std=1 / math.sqrt(F))
    dout = normal(g, M, D, std=0.1).to(BF)
    return x, res, w, wgu, wd, dout


def feed_forward(x, res, w, bgu, bd):
    q, s, h, y, rstd = B.fp8q_rmsnorm_quantize(x, w, res, want_y=True, want_rstd=True)
    qh, sh, gu = B.fp8q_gemm_gated(q, s, *bgu, want_gu=True)
    return B.fp8_gemm_blockwise(qh, sh, *bd), (q, s, h, y, rstd, qh, sh, gu)


def feed_forward_backward(dout, kept, w, bgu_t, bd_t, dres):
    q, s, h, y, rstd, qh, sh, gu = kept
    qo, so, qot, sot = B.fp8_quantize_blockwise_transpose(dout)
    dh = B.fp8_gemm_blockwise(qo, so, *bd_t)
    qd, sd, qdt, sdt, ht, hts = B.fp8q_gated_backward(gu, dh)
    dwd = B.fp8_gemm_blockwise(qot, sot, ht, hts, out_dtype=FP, b_block=1)
    dy = B.fp8_gemm_blockwise(qd, sd, *bgu_t)
    _, _, yt, syt = B.fp8_quantize_blockwise_transpose(y)
    dwgu = B.fp8_gemm_blockwise(qdt, sdt, yt, syt, out_dtype=FP, b_block=1)
    dx, dw = B.fp8q_rmsnorm_backward(dy, h, rstd, w, dres)
    return dx, dw, dwgu, dwd, dh, dy


def test_feed_forward_block():
    """Forward and backward through the library alone, against 64-bit products of the same values.  A product of two
    quantized operands is off by at most (2 * 2^-4 + 2^-8) of the product of absolute values, and a bf16 result by 2^-8 of it."""
    M, D, F = 256, 512, 768
    x, res, w, wgu, wd, dout = block_inputs(M, D, F)
    bgu, bd = B.fp8_quantize_blockwise(wgu, (128, 128)), B.fp8_quantize_blockwise(wd, (128, 128))
    bgu_t = B.fp8_quantize_blockwise(wgu.t().contiguous(), (128, 128))
    bd_t = B.fp8_quantize_blockwise(wd.t().contiguous(), (128, 128))
    out, kept = feed_forward(x, res, w, bgu, bd)
    dx, dw, dwgu, dwd, dh, dy = feed_forward_backward(dout, kept, w, bgu_t, bd_t, dout)
    torch.cuda.synchronize()
    q, s, h, y, rstd, qh, sh, gu = kept

    def near(got, a, b, what):
        a, b = a.double(), b.double()
        tol = (2 * 2.0 ** -4 + 2.0 ** -7) * (a.abs() @ b.abs().T) + 1e-30
        # the sub-normal codes of a block: 2^-10 of the scaled values, 2^-10 * amax / 448 of either operand
        tol += 2.0 ** -18 * (a.abs().amax() * b.abs().sum(1)[None, :] + b.abs().amax() * a.abs().sum(1)[:, None])
        assert bool(((got.double() - a @ b.T).abs() <= tol).all()), what

    near(gu, y, wgu, "projections")
    H = act64(gu[:, :F].double(), B.ACT_SILU)[0] * gu[:, F:].double()
    near(out, H, wd, "out")
    near(dh, dout, wd.t(), "dH")
    near(dwd, dout.t(), H.t(), "dWd")
    Dgu = gated_backward_reference(gu, dh, B.ACT_SILU)[0]
    near(dy, Dgu, wgu.t(), "dy")
    near(dwgu, Dgu.t(), y.t(), "d[Wg; Wu]")
    rdx, b, rdw, bw = backward_reference(dy, h, rstd, w, dout)
    check_close(dx, rdx, 2.0 ** -17 * b, "dx")
    check_close(dw, rdw, 2.0 ** -17 * bw, "dw")


@pytest.mark.parametrize("M", [3, 256])
def test_block_captured_and_replayed(M):
    """The forward block in a CUDA graph: replays on new inputs give what eager calls give."""
    D, F = 512, 256
    x, res, w, wgu, wd, _ = block_inputs(M, D, F, seed=2)
    bgu, bd = B.fp8_quantize_blockwise(wgu, (128, 128)), B.fp8_quantize_blockwise(wd, (128, 128))
    feed_forward(x, res, w, bgu, bd)  # first use outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, kept = feed_forward(x, res, w, bgu, bd)
        dx, dw = B.fp8q_rmsnorm_backward(kept[3], kept[2], kept[4], w, res)
    for seed in (3, 4):
        x.copy_(block_inputs(M, D, F, seed=seed)[0])
        graph.replay()
        torch.cuda.synchronize()
        want, wkept = feed_forward(x, res, w, bgu, bd)
        wdx, wdw = B.fp8q_rmsnorm_backward(wkept[3], wkept[2], wkept[4], w, res)
        assert torch.equal(out, want) and torch.equal(dx, wdx) and torch.equal(dw, wdw)
        for a, b in zip(kept, wkept):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    """Calls on two streams at a time, repeated, give the same bits as one after the other (outputs and workspaces
    allocated by the calls belong to their stream)."""
    g = gen(31)
    sets = []
    for M in (5, 40, 300, 1200):
        a, sa = B.fp8_quantize_blockwise(normal(g, M, 2048))
        b, sb = B.fp8_quantize_blockwise(normal(g, 1024, 2048, std=0.05), (128, 128))
        x = normal(g, M * 8, 1024).to(BF)
        sets.append((a, sa, b, sb, x, torch.ones(1024, device="cuda"), torch.full((M * 8,), 0.5, device="cuda"),
                     x[:, :512].contiguous()))

    def work(t, stream=None):
        a, sa, b, sb, x, w, r, half = t
        q, s, gu = B.fp8q_gemm_gated(a, sa, b, sb, want_gu=True, stream=stream)
        dx, dw = B.fp8q_rmsnorm_backward(x, x, r, w, stream=stream)
        n = B.fp8q_rmsnorm_quantize(x, w, x, stream=stream)
        gb = B.fp8q_gated_backward(x, half, stream=stream)
        return (q, s, gu, dx, dw, *n[:3], *gb)

    want = [work(t) for t in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [work(t, st) for t, st in zip(sets, streams)]
    torch.cuda.synchronize()
    for w_, g_ in zip(want, got):
        for a, b in zip(w_, g_):
            assert torch.equal(a, b)


def test_binding_refusals():
    x = torch.zeros(4, 256, device="cuda")
    w = torch.ones(256, device="cuda")
    u8 = torch.zeros(4, 256, dtype=torch.uint8, device="cuda")
    s = torch.ones(4, 2, device="cuda")
    b, sb = torch.zeros(256, 256, dtype=torch.uint8, device="cuda"), torch.ones(2, 2, device="cuda")
    bad = [
        lambda: B.fp8q_rmsnorm_quantize(x[0], w),
        lambda: B.fp8q_rmsnorm_quantize(x, w[:255]),
        lambda: B.fp8q_rmsnorm_quantize(x, w.double()),
        lambda: B.fp8q_rmsnorm_quantize(x.half(), w),
        lambda: B.fp8q_rmsnorm_quantize(x.t(), w),
        lambda: B.fp8q_rmsnorm_quantize(x, w, residual=x.to(BF)),
        lambda: B.fp8q_rmsnorm_quantize(x, w, residual=x[:2]),
        lambda: B.fp8q_rmsnorm_quantize(x, w, h=torch.empty_like(x)),
        lambda: B.fp8q_rmsnorm_quantize(x, w, q=torch.empty(4, 256, device="cuda")),
        lambda: B.fp8q_rmsnorm_quantize(x, w, scales=torch.empty(4, 3, device="cuda")),
        lambda: B.fp8q_rmsnorm_quantize(x, w.cpu()),
        lambda: B.fp8q_rmsnorm_backward(x, x.to(BF), w[:4], w),
        lambda: B.fp8q_rmsnorm_backward(x, x, w[:3], w),
        lambda: B.fp8q_rmsnorm_backward(x, x, w[:4], w, dweight=torch.empty(255, device="cuda")),
        lambda: B.fp8q_gemm_gated(u8, s, b[:, :128], sb),
        lambda: B.fp8q_gemm_gated(u8, s[:, :1], b, sb),
        lambda: B.fp8q_gemm_gated(u8, s, b, s),
        lambda: B.fp8q_gemm_gated(u8, s, b, sb, q=u8[:, :128].contiguous()),
        lambda: B.fp8q_gemm_gated(u8.float(), s, b, sb),
        lambda: B.fp8q_gated_backward(x, x),
        lambda: B.fp8q_gated_backward(x, x[:, :128].contiguous().to(BF)),
        lambda: B.fp8q_gated_backward(x[:, :255].contiguous(), x),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(B.FP8Error):
        B.fp8q_rmsnorm_quantize(x, w, eps=0.0)
    with pytest.raises(B.FP8Error):
        B.fp8q_rmsnorm_quantize(x, w, fmt=7)
    with pytest.raises(B.FP8Error):
        big = torch.zeros(400, 256, device="cuda")
        B.fp8q_rmsnorm_backward(big.clone(), big, torch.ones(400, device="cuda"), w,
                                workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(B.FP8Error):
        B.fp8q_rmsnorm_quantize(x, w, y=x)
    with pytest.raises(B.FP8Error):
        B.fp8q_gemm_gated(u8, s, b, sb, act=9)
    with pytest.raises(B.FP8Error):
        B.fp8q_gated_backward(torch.zeros(2, 200, device="cuda"), torch.zeros(2, 100, device="cuda"), transposed=False)


# -- past 2^31 elements ---------------------------------------------------------------------------------------------------

def around(rows, per_row):
    """Rows at both ends and on both sides of element 2^31."""
    at = 2 ** 31 // per_row
    assert at + 1 < rows
    return torch.tensor(sorted({0, 1, at - 1, at, at + 1, rows - 2, rows - 1}), device="cuda")


def test_norm_past_two_to_the_31_elements():
    R, C = 300100, 7168
    x = torch.randn(R, C, dtype=BF, device="cuda", generator=gen(51))
    r = torch.randn(R, C, dtype=BF, device="cuda", generator=gen(52))
    w = torch.ones(C, device="cuda")
    q, s, h, y, rstd = B.fp8q_rmsnorm_quantize(x, w, r, want_y=True, want_rstd=True)
    i = around(R, C)
    rh, rr, ry = norm_reference(x[i], r[i], w)
    assert torch.equal(h[i], rh)
    check_close(rstd[i], rr, 2.0 ** -18 * rr, "rstd")
    check_close(y[i], ry, 2.0 ** -18 * ry.abs(), "y")
    check_codes(q[i], s[i], ry, 2.0 ** -18 * ry.abs(), B.E4M3, "codes")
    dx, dw = B.fp8q_rmsnorm_backward(x, h, rstd, w, r)
    rdx, b, _, _ = backward_reference(x[i], h[i], rstd[i], w, r[i])
    check_close(dx[i], rdx, 2.0 ** -17 * b, "dx")
    # the weight gradient's sum has R / 148 dependent additions a CTA, then the CTAs': 2^-12 of the absolute sum
    want = sum((x[k:k + 20000].double() * h[k:k + 20000].double() * rstd[k:k + 20000, None].double()).sum(0)
               for k in range(0, R, 20000))
    size = sum((x[k:k + 20000].double() * h[k:k + 20000].double() * rstd[k:k + 20000, None].double()).abs().sum(0)
               for k in range(0, R, 20000))
    check_close(dw, want, 2.0 ** -12 * size, "dweight")


def test_gated_past_two_to_the_31_elements():
    M, F, K = 264000, 4096, 128
    a, sa = B.fp8_quantize_blockwise(torch.randn(M, K, device="cuda", generator=gen(53)))
    b, sb = B.fp8_quantize_blockwise(torch.randn(2 * F, K, device="cuda", generator=gen(54)) * 0.2, (128, 128))
    q, s, gu = B.fp8q_gemm_gated(a, sa, b, sb, want_gu=True)
    i = around(M, 2 * F)
    G, S = projections(a[i], sa[i], B.E4M3, b, sb, B.E4M3)
    e = (2.0 ** -14 + 2.0 ** -22 + 9 * U) * S
    check_close(gu[i], G, e, "gu")
    (gg, uu), (eg, eu) = G.split(F, 1), e.split(F, 1)
    av, _, p = act64(gg, B.ACT_SILU)
    H = av * uu
    check_codes(q[i], s[i], H, 1.13 * eg * uu.abs() + av.abs() * eu + 1.13 * eg * eu + 2.0 ** -20 * (1 + p.abs()) * H.abs(),
                B.E4M3, "codes")
    dh = torch.randn(M, F, dtype=BF, device="cuda", generator=gen(55))
    q, s, qt, st, ht, hs = B.fp8q_gated_backward(gu, dh)
    D, e, H, eh = gated_backward_reference(gu[i], dh[i], B.ACT_SILU)
    check_codes(q[i], s[i], D, e, B.E4M3, "backward codes")
    # a block of 128 tokens of every column: the last one, whose codes lie past 2^31 in qt
    t = slice(M // 128 * 128 - 128, M // 128 * 128)
    D, e, H, eh = gated_backward_reference(gu[t], dh[t], B.ACT_SILU)
    check_codes(qt[:, t].contiguous(), st[:, t.start // 128:t.stop // 128].contiguous(), D.t().contiguous(), e.t().contiguous(),
                B.E4M3, "transposed codes")
    check_codes(ht[:, t].contiguous(), hs[:, t.start // 128:t.stop // 128].contiguous(), H.t().contiguous(),
                eh.t().contiguous(), B.E4M3, "H codes")
