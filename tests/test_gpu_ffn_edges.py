"""The feed-forward operators where they are easily wrong: rows without columns, in place, addresses, many rows of the
widest forms, values that are not finite, the kernels for few and for many tokens side by side, host threads, streams,
graphs.

Tolerances are those of test_gpu_ffn.py, and their derivation.
"""
import math
import threading

import pytest
import torch

from fine_grained_block_b200 import binding as B
from test_gpu_ffn import backward_reference, check_close, check_codes, check_gated, check_norm, gated_backward_reference
from test_gpu_ffn import act64, block_inputs, feed_forward, projections

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


# -- many rows of the widest forms ------------------------------------------------------------------------------------

# Beyond 8192 columns a CTA takes whole rows, at most 4 CTAs an SM: 1500 rows are 2 or 3 a CTA.
WIDEST = [(1500, 8200, BF), (1500, 9001, BF), (1500, 8200, FP), (1300, 9001, FP), (1200, 16400, BF)]


@pytest.mark.parametrize("rows, cols, dtype", WIDEST)
@pytest.mark.parametrize("with_residual", [True, False])
def test_norm_of_many_wide_rows(rows, cols, dtype, with_residual):
    g = gen(rows + cols)
    x, w = normal(g, rows, cols).to(dtype), 1 + normal(g, cols, std=0.2)
    r = normal(g, rows, cols, std=2.0).to(dtype) if with_residual else None
    check_norm(x, r, w, B.E4M3, f"{rows}x{cols}")


@pytest.mark.parametrize("rows, cols, dtype", WIDEST)
@pytest.mark.parametrize("with_dh", [True, False])
def test_norm_backward_of_many_wide_rows(rows, cols, dtype, with_dh):
    """dweight: at most 3 rows a CTA, 592 / 32 partial rows a warp and 5 steps between lanes are dependent additions."""
    g = gen(rows + cols + 1)
    dy, h = normal(g, rows, cols, std=0.01).to(dtype), normal(g, rows, cols, std=3.0).to(dtype)
    dh = normal(g, rows, cols, std=0.01).to(dtype) if with_dh else None
    w = 1 + normal(g, cols, std=0.2)
    rstd = (h.double().square().mean(1) + 1e-6).rsqrt().float()
    dx, dw = B.fp8q_rmsnorm_backward(dy, h, rstd, w, dh)
    rdx, b, rdw, bw = backward_reference(dy, h, rstd, w, dh)
    check_close(dx, rdx, 2.0 ** -17 * b, "dx")
    check_close(dw, rdw, 2.0 ** -17 * bw, "dweight")
    again = B.fp8q_rmsnorm_backward(dy, h, rstd, w, dh)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


# -- values that are not finite -----------------------------------------------------------------------------------------

@pytest.mark.parametrize("rows, cols", [(6, 256), (40, 4096), (700, 301), (14, 1001), (9, 8200), (650, 9001)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_norm_backward_of_values_that_are_not_finite(rows, cols, dtype):
    g = gen(rows + 2 * cols)
    dy, h, dh = normal(g, rows, cols).to(dtype), normal(g, rows, cols).to(dtype), normal(g, rows, cols).to(dtype)
    w = 1 + normal(g, cols, std=0.2)
    rstd = (h.double().square().mean(1) + 1e-6).rsqrt().float()
    rstd[4] = 0  # as for a row whose squares overflow: n = 0
    clean = B.fp8q_rmsnorm_backward(dy, h, rstd, w, dh)
    dy[0, 5] = float("nan")   # its row, and its column of dweight
    dy[1, 6] = float("inf")
    dh[2, 7] = float("inf")   # its element
    h[3, 9] = float("nan")    # its row and column
    dx, dw = B.fp8q_rmsnorm_backward(dy, h, rstd, w, dh)
    rdx, b, rdw, bw = backward_reference(dy, h, rstd, w, dh)
    rows_hit = torch.zeros(rows, dtype=torch.bool, device="cuda")
    rows_hit[[0, 1, 3]] = True
    assert bool((~torch.isfinite(dx[rows_hit])).all()) and bool(torch.isnan(dx[[0, 3]]).all())
    other = dx.clone()
    other[2, 7] = clean[0][2, 7]
    assert torch.equal(other[~rows_hit], clean[0][~rows_hit]) and math.isinf(float(dx[2, 7]))
    assert torch.equal(dx[4], dh[4])
    hit = torch.zeros(cols, dtype=torch.bool, device="cuda")
    hit[[5, 6, 9]] = True
    assert torch.equal(torch.isfinite(dw), ~hit) and torch.equal(dw[~hit], clean[1][~hit])
    assert torch.equal(torch.isnan(dw), torch.isnan(rdw))


# -- the gated product's CTA pairs ---------------------------------------------------------------------------------------

# 30 tiles that the few-token form does not take (9 token blocks x 10 x 2 CTAs), K of 13 chunks: two pairs a tile.
@pytest.mark.parametrize("act, fmt, gu_dtype, want_q", [(B.ACT_SILU, B.E4M3, BF, True), (B.ACT_GELU_TANH, B.E5M2, FP, True),
                                                        (B.ACT_SILU, B.E5M2, None, True), (B.ACT_GELU_TANH, B.E4M3, BF, False)])
@pytest.mark.parametrize("K", [1664, 1792])
def test_gated_two_pairs_a_tile_of_513_tokens(act, fmt, gu_dtype, want_q, K):
    check_gated(513, 1280, K, act, fmt, gu_dtype=gu_dtype, want_q=want_q)


@pytest.mark.parametrize("act", [B.ACT_SILU, B.ACT_GELU_TANH])
@pytest.mark.parametrize("M, F, K", [(64, 128, 128), (300, 2432, 128), (513, 1280, 1664)])
def test_gate_values_far_out_in_each_kernel(act, M, F, K):
    """One weight per column makes G the activation itself, from -200 to 200, and a NaN code reaches its row only: in the
    few-token kernel, the CTA pairs, and two pairs a tile."""
    x = torch.zeros(M, K, device="cuda")
    x[:, 0] = torch.linspace(-200, 200, M, device="cuda")
    a, sa = B.fp8_quantize_blockwise(x)
    w = torch.zeros(2 * F, K, device="cuda")
    w[:, 0] = 1
    b, sb = B.fp8_quantize_blockwise(w, (128, 128))
    q, s, gu = B.fp8q_gemm_gated(a, sa, b, sb, act=act, want_gu=True)
    gg = projections(a, sa, B.E4M3, b, sb, B.E4M3)[0][:, :F]
    av, _, p = act64(gg, act)
    H = av * gg
    check_codes(q, s, H, 2.0 ** -19 * (1 + p.abs()) * H.abs() + 1e-30, B.E4M3, "far out")
    a = a.clone()
    a[M - 1, K - 1] = 0x7F
    q2, s2, gu2 = B.fp8q_gemm_gated(a, sa, b, sb, act=act, want_gu=True)
    assert bool((q2[M - 1] & 0x7F == 0x7F).all()) and bool(torch.isnan(gu2[M - 1]).all())
    for got, want in ((q2, q), (s2, s), (gu2, gu)):
        assert torch.equal(got[:M - 1], want[:M - 1])


# -- graphs, blocks, streams, host threads ---------------------------------------------------------------------------------

# Tokens x model width x F: the CTA pairs; two pairs a tile; and the few-token kernel with K split.
BLOCKS = [(300, 512, 2560), (513, 1792, 1280), (40, 2048, 1024)]


def weights(wgu, wd):
    quantize = lambda t: B.fp8_quantize_blockwise(t.contiguous(), (128, 128))  # noqa: E731
    return quantize(wgu), quantize(wd), quantize(wgu.t()), quantize(wd.t())


def block_backward(dout, kept, w, bgu_t, bd_t, dres):
    """The backward pass for any number of tokens: what the sums over the tokens take is padded with zero rows to whole
    blocks of 128, as fp8q_gated_backward pads its transposed codes."""
    q, s, h, y, rstd, qh, sh, gu = kept
    pad = lambda t: torch.nn.functional.pad(t, (0, 0, 0, -t.shape[0] % 128))  # noqa: E731
    dh = B.fp8_gemm_blockwise(*B.fp8_quantize_blockwise(dout), *bd_t)
    qd, sd, qdt, sdt, ht, hts = B.fp8q_gated_backward(gu, dh)
    _, _, qot, sot = B.fp8_quantize_blockwise_transpose(pad(dout))
    _, _, yt, syt = B.fp8_quantize_blockwise_transpose(pad(y))
    dwd = B.fp8_gemm_blockwise(qot, sot, ht, hts, out_dtype=FP, b_block=1)
    dwgu = B.fp8_gemm_blockwise(qdt, sdt, yt, syt, out_dtype=FP, b_block=1)
    dy = B.fp8_gemm_blockwise(qd, sd, *bgu_t)
    dx, dw = B.fp8q_rmsnorm_backward(dy, h, rstd, w, dres)
    return dx, dw, dwgu, dwd, dh, dy


@pytest.mark.parametrize("M, D, F", BLOCKS)
def test_block_forward_and_backward_captured_and_replayed(M, D, F):
    """A whole block in a CUDA graph, two graphs of it replayed on two streams at once: what eager calls give, and the
    gradients those of the 64-bit forms of the same values."""
    x, res, w, wgu, wd, dout = block_inputs(M, D, F, seed=5)
    bgu, bd, bgu_t, bd_t = weights(wgu, wd)
    xs, graphs, outs = [x.clone(), x.clone()], [], []
    block_backward(dout, feed_forward(x, res, w, bgu, bd)[1], w, bgu_t, bd_t, dout)  # first use outside the capture
    torch.cuda.synchronize()
    for xi in xs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out, kept = feed_forward(xi, res, w, bgu, bd)
            outs.append((out, *kept, *block_backward(dout, kept, w, bgu_t, bd_t, dout)))
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for seed in (6, 7):
        for i, xi in enumerate(xs):
            xi.copy_(block_inputs(M, D, F, seed=seed + 10 * i)[0])
        torch.cuda.synchronize()
        for _ in range(3):
            for graph, stream in zip(graphs, streams):
                with torch.cuda.stream(stream):
                    graph.replay()
        torch.cuda.synchronize()
        for xi, got in zip(xs, outs):
            out, kept = feed_forward(xi, res, w, bgu, bd)
            want = (out, *kept, *block_backward(dout, kept, w, bgu_t, bd_t, dout))
            for a, b in zip(got, want):
                assert torch.equal(a, b)
    q, s, h, y, rstd, qh, sh, gu = kept
    dx, dw, dwgu, dwd, dh, dy = want[-6:]
    rdx, b, rdw, bw = backward_reference(dy, h, rstd, w, dout)
    check_close(dx, rdx, 2.0 ** -17 * b, "dx")
    check_close(dw, rdw, 2.0 ** -17 * bw, "dw")
    qd, sd = B.fp8q_gated_backward(gu, dh)[:2]
    ref, e = gated_backward_reference(gu, dh, B.ACT_SILU)[:2]
    check_codes(qd, sd, ref, e, B.E4M3, "dG | dU")
    # a product of two quantized operands: (2 * 2^-4 + 2^-8) of the product of absolute values, rounded up, and the
    # subnormal codes of a block, 2^-10 of its scaled values
    H = act64(gu[:, :F].double(), B.ACT_SILU)[0] * gu[:, F:].double()
    for got, a, b_ in ((dwd, dout, H), (dwgu, ref, y)):
        a, b_ = a.double().T, b_.double().T
        tol = (2 * 2.0 ** -4 + 2.0 ** -7) * (a.abs() @ b_.abs().T) + 1e-30
        tol += 2.0 ** -18 * (a.abs().amax() * b_.abs().sum(1)[None, :] + b_.abs().amax() * a.abs().sum(1)[:, None])
        assert bool(((got.double() - a @ b_.T).abs() <= tol).all())


def call_set(seed, M):
    """One call of each operator at a size of its own, and what it gives when nothing else runs."""
    g = gen(seed)
    K, F = 2048, 1280
    a, sa = B.fp8_quantize_blockwise(normal(g, M, K))
    b, sb = B.fp8_quantize_blockwise(normal(g, 2 * F, K, std=0.05), (128, 128))
    x, w = normal(g, M * 3, 1024).to(BF), torch.ones(1024, device="cuda")
    r, half = torch.rand(M * 3, device="cuda", generator=g), normal(g, M * 3, 512).to(BF)

    def work(stream=None):
        q, s, gu = B.fp8q_gemm_gated(a, sa, b, sb, want_gu=True, stream=stream)
        n = B.fp8q_rmsnorm_quantize(x, w, x, want_y=True, want_rstd=True, stream=stream)
        return (q, s, gu, *n, *B.fp8q_rmsnorm_backward(x, x, r, w, stream=stream),
                *B.fp8q_gated_backward(x, half, stream=stream))

    return work


SIZES = (1, 40, 300, 513, 1200)


def test_streams_at_once_in_every_round():
    sets = [call_set(60 + i, M) for i, M in enumerate(SIZES)]
    want = [work() for work in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    rounds = [[work(st) for work, st in zip(sets, streams)] for _ in range(12)]
    torch.cuda.synchronize()
    for got in rounds:
        for w_, g_ in zip(want, got):
            for a, b in zip(w_, g_):
                assert torch.equal(a, b)


def test_host_threads_at_once():
    """Calls from several host threads, each on its stream: the launchers' per-device notes are shared."""
    sets = [call_set(80 + i, M) for i, M in enumerate(SIZES)]
    want = [work() for work in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    results, errors = [[] for _ in sets], []
    start = threading.Barrier(len(sets))

    def run(i):
        try:
            torch.cuda.set_device(0)
            start.wait(30)
            with torch.cuda.stream(streams[i]):
                for _ in range(12):
                    results[i].append(sets[i]())
        except Exception as e:  # noqa: BLE001 -- told by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    torch.cuda.synchronize()
    assert not errors and not any(t.is_alive() for t in threads)
    for w_, rounds in zip(want, results):
        assert len(rounds) == 12
        for got in rounds:
            for a, b in zip(w_, got):
                assert torch.equal(a, b)
