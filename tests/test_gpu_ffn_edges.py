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


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * std


# Several rows a CTA in every form: vectors of 32 and 16 bytes, odd widths (whose rows share memory sectors), the widest.
IN_PLACE = [(3000, 256), (3000, 2048), (2500, 7168), (3000, 520), (4000, 301), (3000, 1001), (2000, 7001), (700, 8201),
            (700, 16400)]


@pytest.mark.parametrize("rows, cols", IN_PLACE)
@pytest.mark.parametrize("dtype", [BF, FP])
def test_norm_in_place_of_many_rows(rows, cols, dtype):
    g = gen(rows + cols)
    x, r, w = normal(g, rows, cols).to(dtype), normal(g, rows, cols).to(dtype), torch.ones(cols, device="cuda")
    want = B.fp8q_rmsnorm_quantize(x, w, r, want_y=True, want_rstd=True)
    for target in (0, 1):
        pair = [x.clone(), r.clone()]
        got = B.fp8q_rmsnorm_quantize(pair[0], w, pair[1], h=pair[target], want_y=True, want_rstd=True)
        assert got[2].data_ptr() == pair[target].data_ptr()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    same = x.clone()  # one tensor as input, residual and h
    got, want = B.fp8q_rmsnorm_quantize(same, w, same, h=same), B.fp8q_rmsnorm_quantize(x, w, x)
    for a, b in zip(got[:3], want[:3]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("rows, cols", IN_PLACE)
@pytest.mark.parametrize("dtype", [BF, FP])
def test_norm_backward_in_place_of_many_rows(rows, cols, dtype):
    g = gen(rows * 3 + cols)
    dy, h, dh = (normal(g, rows, cols).to(dtype) for _ in range(3))
    w, rstd = torch.ones(cols, device="cuda"), torch.rand(rows, device="cuda", generator=g)
    want = B.fp8q_rmsnorm_backward(dy, h, rstd, w, dh)
    for target in (0, 1):
        pair = [dy.clone(), dh.clone()]
        dx, dw = B.fp8q_rmsnorm_backward(pair[0], h, rstd, w, pair[1], dx=pair[target])
        assert dx.data_ptr() == pair[target].data_ptr() and torch.equal(dx, want[0]) and torch.equal(dw, want[1])
    same = dy.clone()  # one tensor as both gradients and dx
    got, want = B.fp8q_rmsnorm_backward(same, h, rstd, w, same, dx=same), B.fp8q_rmsnorm_backward(dy, h, rstd, w, dy)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def shifted(t):
    """t's values at an address that is 16-byte but not 32-byte aligned."""
    e = 16 // t.element_size()
    s = torch.empty(t.numel() + 2 * e, dtype=t.dtype, device="cuda")
    s = s[e if s.data_ptr() % 32 == 0 else 2 * e:][:t.numel()].view_as(t)
    assert s.data_ptr() % 32 == 16
    return s.copy_(t)


@pytest.mark.parametrize("cols", [64, 256, 512, 1024, 2048, 2560, 4096, 7168, 8192, 12288, 16384, 16400, 136, 4104, 301])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("with_residual", [True, False])
def test_norm_does_not_depend_on_the_address(cols, dtype, with_residual):
    """The order of a row's sum is that of its shape: bit for bit the same at any permitted alignment of any tensor."""
    rows = 900 if cols <= 8192 else 30
    g = gen(cols)
    x, w = normal(g, rows, cols).to(dtype), normal(g, cols)
    r = normal(g, rows, cols).to(dtype) if with_residual else None
    want = B.fp8q_rmsnorm_quantize(x, w, r, want_y=True, want_rstd=True)
    if cols % 8 == 0:
        new = lambda: torch.empty_like(x)  # noqa: E731
        sh = lambda: shifted(new())  # noqa: E731
        h = (lambda f: f()) if with_residual else (lambda f: None)
        for args, kw in (((shifted(x), w, r if r is None else shifted(r)), dict(h=h(sh), y=sh())),
                         ((shifted(x), w, r), dict(h=h(new), y=new())), ((x, w, r), dict(h=h(sh), y=new())),
                         ((x, w, r), dict(h=h(new), y=sh())), ((x, shifted(w), r), dict(h=h(new), y=new()))):
            got = B.fp8q_rmsnorm_quantize(*args, want_rstd=True, **kw)
            for a, b in zip(got, want):
                assert torch.equal(a, b)
    no_y = B.fp8q_rmsnorm_quantize(x, w, r, want_rstd=True)
    for a, b in zip(no_y[:3] + no_y[4:], want[:3] + want[4:]):
        assert torch.equal(a, b)
    one = B.fp8q_rmsnorm_quantize(x[7:8].clone(), w, None if r is None else r[7:8].clone(), want_rstd=True)
    assert torch.equal(one[0], want[0][7:8]) and torch.equal(one[4], want[4][7:8])  # nor on the number of rows


# 2432 columns: 300 tokens go to the CTA pairs, fewer than 65 to the few-token kernel, which splits K from 512 on.
@pytest.mark.parametrize("K", [128, 256, 384])
@pytest.mark.parametrize("a_fmt, b_fmt", [(B.E4M3, B.E4M3), (B.E5M2, B.E4M3)])
def test_gated_tokens_do_not_depend_on_their_number(K, a_fmt, b_fmt):
    """One formula for the factors of the block scales: where K is summed in one piece, both kernels give the same bits."""
    M, F = 300, 2432
    g = gen(K)
    a, sa = B.fp8_quantize_blockwise(normal(g, M, K) * torch.rand(M, 1, device="cuda", generator=g), (1, 128), a_fmt)
    b, sb = B.fp8_quantize_blockwise(normal(g, 2 * F, K, std=0.1), (128, 128), b_fmt)
    want = B.fp8q_gemm_gated(a, sa, b, sb, a_fmt, b_fmt, want_gu=True, gu_dtype=FP)
    for rows in (1, 16, 17, 33, 64):
        got = B.fp8q_gemm_gated(a[:rows], sa[:rows], b, sb, a_fmt, b_fmt, want_gu=True, gu_dtype=FP)
        for x, y in zip(got, want):
            assert torch.equal(x, y[:rows])
