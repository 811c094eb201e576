"""The operators of a block of experts against plain implementations in 64 bits.

Tolerances.  u = 2^-24 is half an fp32 step.  The sort and the movement of codes are exact.  Codes made of rows follow
    |decode(q) / s - v| <= half * |v| + sub / s + e_v       (test_gpu_ffn)
with e_v = u |v| for a token times its weight and 0 for a token alone; and a token alone gives the bits of
fp8_quantize_blockwise.  Combine: residual and top_k terms are one fused sum, each step rounded once, so
    |y - exact| <= (top_k + 1) u (|residual| + sum |w x|), bf16 adds 2^-8 |y|.
The weights' gradients: a thread adds 16 products for every 2048 columns, then come 5 + 2 additions, so
    |dw - exact| <= (16 ceil(cols / 2048) + 8) u sum |dy x|.
Products: as for fp8q_gemm_gated, e = (2^-14 + 2^-22 + (K / 128 + 8) u) S with S the product over absolute values; the
weights' gradients have two roundings of the reciprocal scales and one of their product, 2^-22 as well.
"""
import math
import threading

import pytest
import torch

from fine_grained_block_b200 import binding as B
from parity_util import Guarded
from test_gpu_ffn import BF, FP, MAX, U, act64, check_close, check_codes, decode, gated_backward_reference, gen, normal

pytestmark = pytest.mark.gpu

I32 = torch.int32
NONE = -(2 ** 31)


@pytest.fixture(scope="module", autouse=True)
def _status():
    B.fp8_device_status(clear=True)
    yield
    assert B.fp8_device_status() == 0


def guarded(shape, dtype):
    return Guarded(shape, dtype)


def sorted_pairs(experts, E, align, rows):
    """The sort, by a loop over the pairs."""
    order = [[] for _ in range(E)]
    for p, e in enumerate(experts.reshape(-1).tolist()):
        if 0 <= e < E:
            order[e].append(p)
    offsets, pos, src = [0], [-1] * experts.numel(), [-1] * rows
    for pairs in order:
        for i, p in enumerate(pairs):
            pos[p] = offsets[-1] + i
            src[pos[p]] = p
        offsets.append(offsets[-1] + -(-len(pairs) // align) * align)
    t = lambda v: torch.tensor(v, dtype=I32)  # noqa: E731
    return t(offsets), t(pos).view(experts.shape), t(src), t([len(p) for p in order])


def make_experts(T, K, E, kind="random", seed=0):
    g = torch.Generator().manual_seed(seed + 7 * T + E)
    e = torch.randint(0, E, (T, K), generator=g, dtype=I32)
    if kind == "one":
        e.fill_(E - 1)
    elif kind == "none":
        e.fill_(-1)
    elif kind == "some":
        bad = torch.tensor([-1, E, 2 ** 31 - 1, NONE], dtype=I32)[torch.randint(0, 4, (T, K), generator=g)]
        e = torch.where(torch.rand(T, K, generator=g) < 0.3, bad, e)
    elif kind == "skewed":
        e = (e.float() * torch.rand(T, K, generator=g) ** 3).to(I32)
    return e


# -- the sort ---------------------------------------------------------------------------------------------------------

SORTS = [(0, 2, 4, 1), (1, 1, 1, 1), (1, 8, 8, 128), (5, 3, 7, 16), (64, 8, 256, 1), (31, 1, 33, 2), (1000, 6, 64, 128),
         (4097, 1, 3, 2), (512, 8, 1, 64), (513, 8, 1024, 128), (600, 7, 1000, 1), (16384, 8, 256, 128), (3000, 2, 1023, 4),
         (131073, 1, 17, 32), (140000, 3, 60, 1)]


@pytest.mark.parametrize("T, K, E, align", SORTS)
@pytest.mark.parametrize("kind", ["random", "some", "one", "none", "skewed"])
def test_sort(T, K, E, align, kind):
    experts = make_experts(T, K, E, kind)
    rows = B.fp8q_moe_rows(T, K, E, align) + (5 if T % 2 else 0)  # also more rows than any routing needs
    out = [guarded(s, I32) for s in ((E + 1,), (T, K), (rows,), (E,))]
    ws = guarded((B.load_library().fp8q_moe_sort_workspace(T, K, E),), torch.uint8)
    route = B.fp8q_moe_sort(experts.cuda(), E, align, offsets=out[0].t, pos=out[1].t, src=out[2].t, counts=out[3].t,
                            workspace=ws.t if ws.n else None)
    torch.cuda.synchronize()
    for o in (*out, ws):
        o.check()
    for got, want, name in zip(route, sorted_pairs(experts, E, align, rows), route._fields):
        assert torch.equal(got.cpu(), want), name
    bare = B.fp8q_moe_sort(experts.cuda(), E, align, want_counts=False)
    assert bare.counts is None and torch.equal(bare.offsets, route.offsets) and torch.equal(bare.pos, route.pos)
    assert torch.equal(bare.src, route.src[:bare.src.numel()])


def test_rows_hold_any_routing():
    for T, K, E, align in [(1, 8, 64, 16), (3, 2, 2, 128), (100, 4, 7, 8)]:
        rows = B.fp8q_moe_rows(T, K, E, align)
        worst = 0
        for kind in ("random", "one", "skewed"):
            worst = max(worst, int(sorted_pairs(make_experts(T, K, E, kind), E, align, rows)[0][-1]))
        assert worst <= rows and rows % align == 0
    assert B.fp8q_moe_rows(1, 8, 64, 16) == 128  # eight experts with one row each


# -- rows -------------------------------------------------------------------------------------------------------------

def make_route(T, K, E, align, kind="some", seed=0, spare=0):
    """A route on the device with spare rows behind any that it uses."""
    rows = B.fp8q_moe_rows(T, K, E, align) + spare
    route = [t.cuda() for t in sorted_pairs(make_experts(T, K, E, kind, seed), E, align, rows)]
    return B.MoeRoute(*route)


def token_rows(x, route):
    """Row src[r] // K of x (fp64) for the rows in use, zeros where there is no pair."""
    used = int(route.offsets[-1])
    src = route.src[:used].long()
    return torch.where((src >= 0)[:, None], x.double()[src.clamp_min(0) // route.pos.shape[1]], 0.0), used


ROUTES = [(1, 1, 1, 1), (1, 8, 16, 1), (3, 2, 5, 16), (33, 4, 8, 128), (200, 8, 20, 128), (257, 3, 64, 1), (130, 11, 6, 8)]


def untouched(t, rows, dim=0):
    """The bytes that stood in t before, from row (or column) `rows` on."""
    rest = t.narrow(dim, rows, t.shape[dim] - rows).contiguous()
    return bool((rest.view(torch.uint8) == 0xA5).all())


@pytest.mark.parametrize("T, K, E, align", ROUTES)
@pytest.mark.parametrize("cols", [128, 640])
@pytest.mark.parametrize("dtype, fmt", [(BF, B.E4M3), (FP, B.E5M2), (BF, B.E5M2), (FP, B.E4M3)])
@pytest.mark.parametrize("transposed", [False, True])
def test_dispatch(T, K, E, align, cols, dtype, fmt, transposed):
    route = make_route(T, K, E, align, spare=-B.fp8q_moe_rows(T, K, E, align) % 128 + 128)
    g = gen(T + cols)
    x = normal(g, T, cols)
    x[:, 1] *= 50
    x[T // 2, :128] = 0
    x = x.to(dtype)
    R = route.src.numel()
    out = [guarded((R, cols), torch.uint8), guarded((R, cols // 128), FP)]
    if transposed:
        out += [guarded((cols, R), torch.uint8), guarded((cols, R // 128), FP)]
    kw = dict(zip(("q", "scales", "qt", "scales_t"), (o.t for o in out)))
    q, s, qt, st = B.fp8q_moe_dispatch(x, route, fmt=fmt, transposed=transposed, **kw)
    torch.cuda.synchronize()
    for o in out:
        o.check()
    v, used = token_rows(x, route)
    v = v.to(dtype)
    if used:
        wq, ws = B.fp8_quantize_blockwise(v, (1, 128), fmt)
        assert torch.equal(q[:used], wq) and torch.equal(s[:used], ws)
    assert untouched(q, used) and untouched(s, used)
    if transposed:
        blocks = -(-used // 128)
        if blocks:
            padded = torch.nn.functional.pad(v, (0, 0, 0, blocks * 128 - used)).t().contiguous()
            wq, ws = B.fp8_quantize_blockwise(padded, (1, 128), fmt)
            assert torch.equal(qt[:, :blocks * 128], wq) and torch.equal(st[:, :blocks], ws)
        assert untouched(qt, blocks * 128, 1) and untouched(st, blocks, 1)


@pytest.mark.parametrize("T, K, E, align", ROUTES)
@pytest.mark.parametrize("cols", [128, 640])
@pytest.mark.parametrize("fmt", [B.E4M3, B.E5M2])
def test_dispatch_codes(T, K, E, align, cols, fmt):
    route = make_route(T, K, E, align, spare=3)
    g = gen(T + cols)
    xq = torch.randint(0, 256, (T, cols), generator=g, device="cuda", dtype=torch.uint8)
    xs = torch.rand(T, cols // 128, generator=g, device="cuda")
    R = route.src.numel()
    out = [guarded((R, cols), torch.uint8), guarded((R, cols // 128), FP)]
    q, s = B.fp8q_moe_dispatch_codes(xq, xs, route, fmt=fmt, q=out[0].t, scales=out[1].t)
    torch.cuda.synchronize()
    for o in out:
        o.check()
    used = int(route.offsets[-1])
    src = route.src[:used].long()
    real = (src >= 0)[:, None]
    t = src.clamp_min(0) // K
    assert torch.equal(q[:used], torch.where(real, xq[t], 0).to(torch.uint8))
    zero = torch.tensor(MAX[fmt], device="cuda") / 1e-12
    assert torch.equal(s[:used], torch.where(real, xs[t], zero))
    assert untouched(q, used) and untouched(s, used)


@pytest.mark.parametrize("T, K, E, align", ROUTES)
@pytest.mark.parametrize("cols", [128, 4224])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("weighted, with_residual", [(True, False), (True, True), (False, False), (False, True)])
def test_combine(T, K, E, align, cols, dtype, weighted, with_residual):
    route = make_route(T, K, E, align)
    g = gen(T + cols)
    R = route.src.numel()
    rows = normal(g, R, cols).to(dtype)
    rows[(route.src < 0)] = math.nan  # rows without a pair are not read as results
    weights = normal(g, T, K)
    weights[route.pos < 0] = math.nan
    residual = normal(g, T, cols, std=3.0).to(dtype) if with_residual else None
    y = guarded((T, cols), dtype)
    got = B.fp8q_moe_combine(rows, route, weights if weighted else None, residual, y=y.t)
    torch.cuda.synchronize()
    y.check()
    want = torch.zeros(T, cols, dtype=torch.float64, device="cuda") if residual is None else residual.double()
    size = want.abs()
    for k in range(K):
        at = route.pos[:, k].long()
        w = weights[:, k].double() if weighted else torch.ones(T, dtype=torch.float64, device="cuda")
        term = torch.where((at >= 0)[:, None], w[:, None] * rows[at.clamp_min(0)].double(), 0.0)
        want, size = want + term, size + term.abs()
    check_close(got, want, (K + 1) * U * size, f"{T}x{cols}")


@pytest.mark.parametrize("T, K, E, align", ROUTES)
@pytest.mark.parametrize("cols", [128, 4224])
@pytest.mark.parametrize("dtype, fmt", [(BF, B.E5M2), (FP, B.E4M3)])
@pytest.mark.parametrize("transposed", [False, True])
def test_combine_backward(T, K, E, align, cols, dtype, fmt, transposed):
    route = make_route(T, K, E, align, spare=-B.fp8q_moe_rows(T, K, E, align) % 128)
    g = gen(T + cols)
    R = route.src.numel()
    rows = normal(g, R, cols).to(dtype)
    rows[(route.src < 0)] = math.nan
    weights = normal(g, T, K)
    dy = normal(g, T, cols, std=1e-3).to(dtype)
    out = [guarded((T, K), FP), guarded((R, cols), torch.uint8), guarded((R, cols // 128), FP)]
    kw = dict(dweights=out[0].t, q=out[1].t, scales=out[2].t)
    if transposed:
        out += [guarded((cols, R), torch.uint8), guarded((cols, R // 128), FP)]
        kw.update(qt=out[3].t, scales_t=out[4].t)
    q, s, qt, st, dw = B.fp8q_moe_combine_backward(dy, rows, route, weights, fmt=fmt, transposed=transposed, **kw)
    torch.cuda.synchronize()
    for o in out:
        o.check()
    v, used = token_rows(dy, route)
    w = weights.double().reshape(-1)[route.src[:used].long().clamp_min(0)]
    v = v * w[:, None]
    if used:
        check_codes(q[:used], s[:used], v, U * v.abs(), fmt, "rows")
        if transposed:
            blocks = -(-used // 128)
            vt = torch.nn.functional.pad(v, (0, 0, 0, blocks * 128 - used)).t().contiguous()
            check_codes(qt[:, :blocks * 128], st[:, :blocks], vt, U * vt.abs(), fmt, "transposed")
    assert untouched(q, used) and untouched(s, used)
    at = route.pos.long()
    x = torch.where((at >= 0)[..., None], rows[at.clamp_min(0)].double(), 0.0)
    want, size = (x * dy.double()[:, None]).sum(2), (x * dy.double()[:, None]).abs().sum(2)
    check_close(dw, want, (16 * math.ceil(cols / 2048) + 8) * U * size, "dweights")
    # each output alone
    alone = B.fp8q_moe_combine_backward(dy, None, route, weights, fmt=fmt, transposed=transposed, want_dweights=False)
    assert alone[4] is None and torch.equal(alone[0][:used], q[:used]) and torch.equal(alone[1][:used], s[:used])
    if transposed and align == 128:
        assert torch.equal(alone[2][:, :used], qt[:, :used]) and torch.equal(alone[3][:, :used // 128], st[:, :used // 128])


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_values_that_are_not_finite(dtype, transposed):
    """A NaN or infinite element or weight reaches its own blocks only, and NaN does not count toward an amax; the form by
    tokens and the one by tiles give the same bits."""
    T, K, E, cols = 40, 3, 4, 256
    route = make_route(T, K, E, 128, "random")
    g = gen(3)
    dy = normal(g, T, cols).to(dtype)
    weights = normal(g, T, K)
    dy[3, 5], dy[4, 200], dy[5, :] = math.nan, math.inf, 0
    weights[6, 0], weights[7, 1], weights[5, 0], weights[8, 2] = math.nan, math.inf, math.inf, 0
    q, s, qt, st, _ = B.fp8q_moe_combine_backward(dy, None, route, weights, transposed=transposed, want_dweights=False)
    used = int(route.offsets[-1])
    src = route.src[:used].long()
    v = dy.float()[src.clamp_min(0) // K] * weights.reshape(-1)[src.clamp_min(0)][:, None]
    v[src < 0] = 0
    wq, ws = B.fp8_quantize_blockwise(v, (1, 128))
    assert torch.equal(q[:used], wq) and torch.equal(s[:used], ws)
    if transposed:
        wq, ws = B.fp8_quantize_blockwise(v.t().contiguous(), (1, 128))
        assert torch.equal(qt[:, :used], wq) and torch.equal(st[:, :used // 128], ws)
    x, xs, xt, xst = B.fp8q_moe_dispatch(dy, route, transposed=transposed)
    v = dy[src.clamp_min(0) // K]
    v[src < 0] = 0
    wq, ws = B.fp8_quantize_blockwise(v, (1, 128))
    assert torch.equal(x[:used], wq) and torch.equal(xs[:used], ws)
    y = B.fp8q_moe_combine(dy, B.MoeRoute(route.offsets, torch.arange(T, device="cuda", dtype=I32)[:, None].contiguous(),
                                          route.src, None))
    assert torch.equal(y.isnan(), dy.isnan()) and torch.equal(y.nan_to_num(0, 9e9, -9e9), dy.nan_to_num(0, 9e9, -9e9))


def test_indices_that_no_sort_makes_are_not_followed():
    """Positions, pairs and offsets outside their range have no row: nothing outside the tensors is touched."""
    T, K, E, cols, R = 9, 2, 3, 256, 128
    g = gen(4)
    x = normal(g, T, cols).to(BF)
    far = torch.tensor([R, 2 ** 31 - 1, NONE, -2], dtype=I32, device="cuda")
    pos = torch.full((T, K), -1, dtype=I32, device="cuda")
    pos[0], pos[1], pos[2, 0] = far[:2], far[2:], 7
    src = torch.full((R,), -1, dtype=I32, device="cuda")
    src[0], src[1], src[2], src[7] = T * K, 2 ** 31 - 1, NONE, 4
    offsets = torch.tensor([NONE, 5, 2, 2 ** 31 - 1], dtype=I32, device="cuda")  # used: all of R
    route = B.MoeRoute(offsets, pos, src, None)
    for transposed in (False, True):
        out = [guarded((R, cols), torch.uint8), guarded((R, cols // 128), FP)]
        kw = dict(q=out[0].t, scales=out[1].t)
        if transposed:
            out += [guarded((cols, R), torch.uint8), guarded((cols, 1), FP)]
            kw.update(qt=out[2].t, scales_t=out[3].t)
        q = B.fp8q_moe_dispatch(x, route, transposed=transposed, **kw)[0]
        torch.cuda.synchronize()
        for o in out:
            o.check()
        wq, _ = B.fp8_quantize_blockwise(x)
        assert torch.equal(q[7], wq[2])
        if transposed:
            assert int(q[:7].sum()) == int(q[8:].sum()) == 0
    rows = normal(g, R, cols).to(BF)
    y = B.fp8q_moe_combine(rows, route)
    assert torch.equal(y[2], rows[7]) and int(y[:2].abs().sum() + y[3:].abs().sum()) == 0
    dw = B.fp8q_moe_combine_backward(x, rows, route, torch.ones(T, K, device="cuda"), transposed=False)[4]
    assert int((dw != 0).sum()) == 1
    # products: expert 0 rows 0..4, expert 1 none (its end comes first), expert 2 rows 2..127
    a, sa = B.fp8_quantize_blockwise(rows)
    b, sb = B.fp8_quantize_blockwise(normal(g, E * 256, cols), (128, 128))
    c = guarded((R, 256), BF)
    B.fp8q_gemm_grouped(a, sa, b.view(E, 256, cols), sb.view(E, 2, 2), offsets, c=c.t)
    torch.cuda.synchronize()
    c.check()


# -- products ---------------------------------------------------------------------------------------------------------

def segments(lengths, align=1, spare=0):
    """Offsets of experts with these many rows, and the rows of tensors that hold them."""
    off = [0]
    for n in lengths:
        off.append(off[-1] + -(-n // align) * align)
    return torch.tensor(off, dtype=I32, device="cuda"), off, off[-1] + spare


def make_products(lengths, N, K, align=1, spare=0, a_fmt=B.E4M3, b_fmt=B.E4M3, seed=0):
    offsets, off, R = segments(lengths, align, spare)
    g = gen(N + K + len(lengths) + seed)
    a, sa = B.fp8_quantize_blockwise(normal(g, R, K), (1, 128), a_fmt)
    E = len(lengths)
    b, sb = B.fp8_quantize_blockwise(normal(g, E * N, K, std=2 / math.sqrt(K)), (128, 128), b_fmt)
    return a, sa, b.view(E, N, K), sb.view(E, N // 128, K // 128), offsets, off


def expert_products(a, sa, b, sb, off, a_fmt, b_fmt):
    R, N = a.shape[0], b.shape[1]
    c, S = (torch.zeros(R, N, dtype=torch.float64, device="cuda") for _ in range(2))
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        if hi > lo:
            av, bv = decode(a[lo:hi], sa[lo:hi], 1, a_fmt), decode(b[e], sb[e], 128, b_fmt)
            c[lo:hi], S[lo:hi] = av @ bv.T, av.abs() @ bv.abs().T
    return c, S


def bound(S, K):
    return (2.0 ** -14 + 2.0 ** -22 + (K / 128 + 8) * U) * S


def check_grouped(lengths, N, K, align=1, spare=0, a_fmt=B.E4M3, b_fmt=B.E4M3, dtype=FP):
    a, sa, b, sb, offsets, off = make_products(lengths, N, K, align, spare, a_fmt, b_fmt)
    c = guarded((a.shape[0], N), dtype)
    got = B.fp8q_gemm_grouped(a, sa, b, sb, offsets, a_fmt, b_fmt, c=c.t)
    torch.cuda.synchronize()
    c.check()
    want, S = expert_products(a, sa, b, sb, off, a_fmt, b_fmt)
    used = off[-1]
    check_close(got[:used], want[:used], bound(S[:used], K), f"{lengths} {N}x{K}")
    assert untouched(got, used)
    return got


LENGTHS = [[1], [3, 0, 5], [0, 0, 7, 0], [1] * 8, [16, 17, 15, 33], [64, 1, 65, 0, 2], [20] * 5, [40, 63, 64, 66],  # few rows
           [128, 127, 129, 0, 1, 300], [256, 257, 255], [70, 500], [1000], [0, 513, 31, 0, 97, 32]]                # many


@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
@pytest.mark.parametrize("N, K", [(128, 128), (256, 640), (640, 384), (1152, 2176)])
def test_products_of_any_rows(lengths, N, K):
    check_grouped(lengths, N, K, spare=3)


@pytest.mark.parametrize("lengths", LENGTHS[8:], ids=str)
@pytest.mark.parametrize("N, K", [(4096, 128), (4224, 640)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_products_of_many_rows_and_columns(lengths, N, K, dtype):
    """So many tiles that every SM has one: the kernel for many rows, whatever the lengths."""
    check_grouped(lengths, N, K, spare=3, dtype=dtype)


@pytest.mark.parametrize("lengths, align", [([1, 3, 9, 0], 16), ([100, 300, 0, 129], 128), ([33, 2, 190], 32), ([5, 5], 2)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_products_of_aligned_rows(lengths, align, dtype):
    check_grouped(lengths, 512, 384, align, spare=align, dtype=dtype)


@pytest.mark.parametrize("lengths", [[2, 9], [30, 41, 0, 50], [300, 20, 129]], ids=str)
@pytest.mark.parametrize("a_fmt, b_fmt", [(B.E4M3, B.E5M2), (B.E5M2, B.E4M3), (B.E5M2, B.E5M2)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_products_formats(lengths, a_fmt, b_fmt, dtype):
    for N in (384, 4096):
        check_grouped(lengths, N, 256, a_fmt=a_fmt, b_fmt=b_fmt, dtype=dtype)


@pytest.mark.parametrize("E", [256, 1000, 1024])
@pytest.mark.parametrize("most", [3, 70])
def test_products_of_many_experts(E, most):
    g = torch.Generator().manual_seed(E)
    lengths = (torch.randint(0, most + 1, (E,), generator=g) * (torch.rand(E, generator=g) < 0.7)).tolist()
    check_grouped(lengths, 128, 128, dtype=BF)
    if most > 64:  # enough rows an expert for the other kernel
        check_grouped([n * 3 for n in lengths], 128, 128, dtype=BF)
        check_grouped([n * 3 for n in lengths], 256, 128, align=16, dtype=BF)


@pytest.mark.parametrize("K", [128, 384])
def test_products_are_those_of_the_blockwise_gemm(K):
    """K < 512: an expert's rows have the bits of the plain product of them alone, in either kernel."""
    for lengths, N in (([3, 10, 0, 1], 512), ([200, 300, 130], 512), ([200, 300, 130], 4096)):
        a, sa, b, sb, offsets, off = make_products(lengths, N, K)
        got = B.fp8q_gemm_grouped(a, sa, b, sb, offsets, out_dtype=FP)
        for e, (lo, hi) in enumerate(zip(off, off[1:])):
            if hi > lo:
                want = B.fp8_gemm_blockwise(a[lo:hi].contiguous(), sa[lo:hi].contiguous(), b[e], sb[e], out_dtype=FP)
                assert torch.equal(got[lo:hi], want)


def check_gated_grouped(lengths, F, K, align=1, spare=0, act=B.ACT_SILU, fmt=B.E4M3, a_fmt=B.E4M3, b_fmt=B.E4M3, gu_dtype=FP,
                        want_q=True):
    a, sa, b, sb, offsets, off = make_products(lengths, 2 * F, K, align, spare, a_fmt, b_fmt)
    R, used = a.shape[0], off[-1]
    out = [guarded((R, F), torch.uint8), guarded((R, F // 128), FP), guarded((R, 2 * F), gu_dtype or FP)]
    kw = dict(q=out[0].t, scales=out[1].t) if want_q else dict(want_q=False)
    q, s, gu = B.fp8q_gemm_gated_grouped(a, sa, b, sb, offsets, a_fmt, b_fmt, act, fmt, gu=out[2].t if gu_dtype else None, **kw)
    torch.cuda.synchronize()
    for o in out:
        o.check()
        assert untouched(o.t, used)
    G, S = expert_products(a, sa, b, sb, off, a_fmt, b_fmt)
    G, e = G[:used], bound(S[:used], K)
    what = f"{lengths} {F}x{K}"
    if gu_dtype:
        check_close(gu[:used], G, e, what + " gu")
    if want_q and used:
        (gg, uu), (eg, eu) = G.split(F, 1), e.split(F, 1)
        av, _, p = act64(gg, act)
        H = av * uu
        eh = 1.13 * eg * uu.abs() + av.abs() * eu + 1.13 * eg * eu + 2.0 ** -20 * (1 + p.abs()) * H.abs()
        check_codes(q[:used], s[:used], H, eh, fmt, what)


@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
@pytest.mark.parametrize("F, K", [(128, 128), (384, 640), (640, 2176)])
def test_gated_products_of_any_rows(lengths, F, K):
    check_gated_grouped(lengths, F, K, spare=3)


@pytest.mark.parametrize("lengths", LENGTHS[8:], ids=str)
@pytest.mark.parametrize("act, fmt, gu_dtype, want_q", [(B.ACT_SILU, B.E4M3, BF, True), (B.ACT_GELU_TANH, B.E5M2, FP, True),
                                                        (B.ACT_SILU, B.E5M2, None, True), (B.ACT_GELU_TANH, B.E4M3, BF, False)])
def test_gated_products_of_many_rows_and_columns(lengths, act, fmt, gu_dtype, want_q):
    check_gated_grouped(lengths, 4096, 384, spare=3, act=act, fmt=fmt, gu_dtype=gu_dtype, want_q=want_q)


@pytest.mark.parametrize("lengths, align", [([1, 3, 9, 0], 16), ([100, 300, 0, 129], 128), ([33, 2, 190], 32)])
@pytest.mark.parametrize("act, fmt, gu_dtype, want_q", [(B.ACT_SILU, B.E4M3, BF, True), (B.ACT_GELU_TANH, B.E5M2, BF, True),
                                                        (B.ACT_SILU, B.E5M2, None, True), (B.ACT_GELU_TANH, B.E4M3, BF, False)])
def test_gated_products_outputs(lengths, align, act, fmt, gu_dtype, want_q):
    check_gated_grouped(lengths, 256, 384, align, spare=align, act=act, fmt=fmt, gu_dtype=gu_dtype, want_q=want_q)


@pytest.mark.parametrize("lengths", [[2, 9], [30, 41, 0, 50], [300, 20, 129]], ids=str)
@pytest.mark.parametrize("a_fmt, b_fmt", [(B.E4M3, B.E5M2), (B.E5M2, B.E4M3)])
def test_gated_products_formats(lengths, a_fmt, b_fmt):
    for F in (256, 4096):
        check_gated_grouped(lengths, F, 256, a_fmt=a_fmt, b_fmt=b_fmt)


@pytest.mark.parametrize("lengths, F", [([3, 1, 0, 12], 256), ([200, 150, 300], 256), ([200, 150, 300], 4096)])
def test_gated_products_are_those_of_the_gated_gemm(lengths, F):
    """K < 512: an expert's rows have the bits of fp8q_gemm_gated of them alone."""
    a, sa, b, sb, offsets, off = make_products(lengths, 2 * F, 384)
    q, s, gu = B.fp8q_gemm_gated_grouped(a, sa, b, sb, offsets, want_gu=True)
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        if hi > lo:
            want = B.fp8q_gemm_gated(a[lo:hi].contiguous(), sa[lo:hi].contiguous(), b[e], sb[e], want_gu=True)
            for x, y in zip((q, s, gu), want):
                assert torch.equal(x[lo:hi], y)


@pytest.mark.parametrize("lengths, N", [([3, 4], 512), ([150, 300], 512), ([150, 300], 8192)])
def test_nan_code_reaches_its_row_only(lengths, N):
    a, sa, b, sb, offsets, off = make_products(lengths, N, 256)
    clean = B.fp8q_gemm_grouped(a, sa, b, sb, offsets, out_dtype=FP)
    row = off[1]  # the first of the second expert, in the same tile as rows of the first
    a[row, 7] = 0x7F
    q, s, gu = B.fp8q_gemm_gated_grouped(a, sa, b, sb, offsets, want_gu=True, gu_dtype=FP)
    got = B.fp8q_gemm_grouped(a, sa, b, sb, offsets, out_dtype=FP)
    assert bool(got[row].isnan().all()) and bool(gu[row].isnan().all()) and bool(((q[row] & 0x7F) == 0x7F).all())
    keep = torch.arange(a.shape[0], device="cuda") != row
    assert torch.equal(got[keep], clean[keep]) and torch.equal(gu[keep], clean[keep])


def test_products_without_rows_or_sums():
    a, sa, b, sb, offsets, off = make_products([2, 0, 3], 256, 128, spare=2)
    none = torch.zeros(4, dtype=I32, device="cuda")  # no expert has a row: nothing is written
    c = guarded((7, 256), FP)
    B.fp8q_gemm_grouped(a, sa, b, sb, none, c=c.t)
    assert untouched(c.t, 0)
    empty = lambda *shape, dtype=torch.uint8: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    c = guarded((7, 256), FP)
    B.fp8q_gemm_grouped(empty(7, 0), empty(7, 0, dtype=FP), empty(3, 256, 0), empty(3, 2, 0, dtype=FP), offsets, c=c.t)
    assert int(c.t[:5].abs().sum()) == 0 and untouched(c.t, 5)
    q, s, gu = B.fp8q_gemm_gated_grouped(empty(7, 0), empty(7, 0, dtype=FP), empty(3, 256, 0), empty(3, 2, 0, dtype=FP), offsets,
                                         want_gu=True)
    assert int(q[:5].sum()) == 0 and bool((s[:5] == torch.tensor(448.0, device="cuda") / 1e-12).all())
    assert int(gu[:5].abs().sum()) == 0
    c = B.fp8q_gemm_grouped(a[:0], sa[:0], b, sb, none)
    assert c.shape == (0, 256)


# -- the weights' gradients -------------------------------------------------------------------------------------------

def check_wgrad(lengths, N, K, spare=0, a_fmt=B.E4M3, b_fmt=B.E4M3, dtype=FP):
    offsets, off, R = segments(lengths, 128, spare)
    E = len(lengths)
    g = gen(N + K + E)
    at, sat = B.fp8_quantize_blockwise(normal(g, N, R, std=1e-3), (1, 128), a_fmt)
    bt, sbt = B.fp8_quantize_blockwise(normal(g, K, R), (1, 128), b_fmt)
    dw = guarded((E, N, K), dtype)
    got = B.fp8q_gemm_grouped_wgrad(at, sat, bt, sbt, offsets, a_fmt, b_fmt, dw=dw.t)
    torch.cuda.synchronize()
    dw.check()
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        av, bv = (decode(q[:, lo:hi], s[:, lo // 128:hi // 128], 1, f) for q, s, f in ((at, sat, a_fmt), (bt, sbt, b_fmt)))
        S = av.abs() @ bv.abs().T
        check_close(got[e], av @ bv.T, (2.0 ** -14 + 2.0 ** -22 + ((hi - lo) / 128 + 8) * U) * S, f"{lengths} {N}x{K} {e}")
    return at, sat, bt, sbt, off, got


@pytest.mark.parametrize("lengths", [[1], [0], [128, 0, 300], [1000, 5, 0, 129, 640], [0, 0], [2900]], ids=str)
@pytest.mark.parametrize("N, K", [(128, 128), (256, 256), (384, 640), (1024, 768)])
@pytest.mark.parametrize("spare", [0, 256])
def test_wgrad(lengths, N, K, spare):
    check_wgrad(lengths, N, K, spare)


@pytest.mark.parametrize("a_fmt, b_fmt", [(B.E4M3, B.E5M2), (B.E5M2, B.E4M3), (B.E5M2, B.E5M2)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_wgrad_formats(a_fmt, b_fmt, dtype):
    check_wgrad([200, 0, 700, 130], 384, 256, 128, a_fmt, b_fmt, dtype)


def test_wgrad_is_that_of_the_blockwise_gemm():
    at, sat, bt, sbt, off, got = check_wgrad([300, 513, 0, 256], 512, 256)
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        if hi > lo:
            want = B.fp8_gemm_blockwise(at[:, lo:hi].contiguous(), sat[:, lo // 128:hi // 128].contiguous(),
                                        bt[:, lo:hi].contiguous(), sbt[:, lo // 128:hi // 128].contiguous(), out_dtype=FP, b_block=1)
            assert torch.equal(got[e], want)


def test_wgrad_of_many_experts():
    g = torch.Generator().manual_seed(1)
    check_wgrad((torch.randint(0, 200, (300,), generator=g)).tolist(), 128, 256, dtype=BF)


# -- together ---------------------------------------------------------------------------------------------------------

def block_inputs(T, K, E, D, F, seed=0):
    g = gen(500 + seed)
    x = normal(g, T, D).to(BF)
    w = (1 + normal(g, D, std=0.1)).to(BF)
    scores, experts = normal(g, T, E).topk(K, dim=1)
    gates = torch.softmax(scores, dim=1).contiguous()
    wgu, wd = normal(g, E, 2 * F, D, std=1 / math.sqrt(D)), normal(g, E, D, F, std=1 / math.sqrt(F))
    dout = normal(g, T, D, std=0.1).to(BF)
    return x, w, experts.to(I32).contiguous(), gates, wgu, wd, dout


def by_blocks(w):
    """128x128 codes of every expert's weights, as they are and transposed."""
    E, N, K = w.shape
    parts = [B.fp8_quantize_blockwise_transpose(w[e].contiguous(), (128, 128)) for e in range(E)]
    return [torch.stack(t) for t in zip(*parts)]


def block_forward(x, w, experts, gates, wgu, wd, align):
    E = wgu[0].shape[0]
    q, s, h, y, rstd = B.fp8q_rmsnorm_quantize(x, w, want_y=True, want_rstd=True)
    route = B.fp8q_moe_sort(experts, E, align)
    qx, sx = B.fp8q_moe_dispatch_codes(q, s, route)
    qh, sh, gu = B.fp8q_gemm_gated_grouped(qx, sx, wgu[0], wgu[1], route.offsets, want_gu=True)
    rows = B.fp8q_gemm_grouped(qh, sh, wd[0], wd[1], route.offsets)
    out = B.fp8q_moe_combine(rows, route, gates, residual=x)
    return out, (h, y, rstd, route, gu, rows)


def block_backward(dout, kept, w, gates, wgu, wd):
    h, y, rstd, route, gu, rows = kept
    qr, sr, qrt, srt, dgates = B.fp8q_moe_combine_backward(dout, rows, route, gates)
    dh = B.fp8q_gemm_grouped(qr, sr, wd[2], wd[3], route.offsets)
    qd, sd, qdt, sdt, ht, hts = B.fp8q_gated_backward(gu, dh)
    dwd = B.fp8q_gemm_grouped_wgrad(qrt, srt, ht, hts, route.offsets)
    drows = B.fp8q_gemm_grouped(qd, sd, wgu[2], wgu[3], route.offsets)
    _, _, xt, sxt = B.fp8q_moe_dispatch(y, route, transposed=True)
    dwgu = B.fp8q_gemm_grouped_wgrad(qdt, sdt, xt, sxt, route.offsets)
    dy = B.fp8q_moe_combine(drows, route)
    dx, dw = B.fp8q_rmsnorm_backward(dy, h, rstd, w, dout)
    return dx, dw, dgates, dwgu, dwd, dh, drows, dy


def near(got, a, b, what):
    """A product of two quantized operands is off by at most (2 * 2^-4 + 2^-8) of the product of absolute values, a bf16
    result by 2^-8 of it, and by the subnormal codes of a block: 2^-10 of the scaled values, 2^-10 amax / 448 of an operand."""
    a, b = a.double(), b.double()
    tol = (2 * 2.0 ** -4 + 2.0 ** -7) * (a.abs() @ b.abs().T) + 1e-30
    tol += 2.0 ** -18 * (a.abs().amax() * b.abs().sum(1)[None, :] + b.abs().amax() * a.abs().sum(1)[:, None])
    assert bool(((got.double() - a @ b.T).abs() <= tol).all()), what


@pytest.mark.parametrize("T, K, E", [(200, 2, 6), (1, 2, 4), (300, 3, 3)])
def test_block_of_experts(T, K, E):
    """Forward and backward through the library alone, every step against 64-bit products of the same values."""
    D, F = 384, 256
    x, w, experts, gates, wgu, wd, dout = block_inputs(T, K, E, D, F)
    bgu, bd = by_blocks(wgu), by_blocks(wd)
    out, kept = block_forward(x, w, experts, gates, bgu, bd, 128)
    dx, dw, dgates, dwgu, dwd, dh, drows, dy = block_backward(dout, kept, w, gates, bgu, bd)
    torch.cuda.synchronize()
    h, y, rstd, route, gu, rows = kept
    off = route.offsets.tolist()
    src = route.src.long()
    token, gate = src.clamp_min(0) // K, torch.where(src >= 0, gates.reshape(-1)[src.clamp_min(0)], 0.0).double()
    X = torch.where((src >= 0)[:, None], y[token].double(), 0.0)
    dR = dout[token].double() * gate[:, None]
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        r = slice(lo, hi)
        if hi > lo:
            near(gu[r], X[r], wgu[e], "projections")
            H = act64(gu[r, :F].double(), B.ACT_SILU)[0] * gu[r, F:].double()
            near(rows[r], H, wd[e], "rows")
            near(dh[r], dR[r], wd[e].t(), "dH")
            near(dwd[e], dR[r].t(), H.t(), "dWd")
            dgu = gated_backward_reference(gu[r], dh[r], B.ACT_SILU)[0]
            near(drows[r], dgu, wgu[e].t(), "dX")
            near(dwgu[e], dgu.t(), X[r].t(), "d[Wg; Wu]")
        else:
            assert int(dwd[e].abs().sum() + dwgu[e].abs().sum()) == 0
    at = route.pos.long()
    assert bool((at >= 0).all())
    picked = rows.double()[at]
    want = x.double() + (gates.double()[..., None] * picked).sum(1)
    size = x.double().abs() + (gates.double()[..., None] * picked).abs().sum(1)
    check_close(out, want, (K + 1) * U * size, "out")
    terms = picked * dout.double()[:, None]
    check_close(dgates, terms.sum(2), 24 * U * terms.abs().sum(2), "dgates")
    check_close(dy, drows.double()[at].sum(1), (K + 1) * U * drows.double()[at].abs().sum(1), "dy")
    # a serving program's packed rows: the same tokens within the bf16 results' roundings and the order of the sums
    packed, pkept = block_forward(x, w, experts, gates, bgu, bd, 1)
    assert pkept[3].src.numel() == T * K
    assert bool(((packed.double() - out.double()).abs() <= 2.0 ** -3 * size + 1e-3).all())


def test_gradient_against_differences():
    """<d loss / d gates> and <d loss / d rows> of loss = sum(dout * combine(rows, gates)) against central differences: the
    loss is linear in each, so a difference is exact up to fp32 sums."""
    T, K, E, cols = 20, 3, 5, 256
    route = make_route(T, K, E, 128, "random")
    g = gen(9)
    rows, dout, gates = normal(g, route.src.numel(), cols), normal(g, T, cols), normal(g, T, K)
    q, s, _, _, dw = B.fp8q_moe_combine_backward(dout, rows, route, gates)
    drows = decode(q, s, 1, B.E4M3)

    def loss(rows, gates):
        return float((B.fp8q_moe_combine(rows, route, gates).double() * dout.double()).sum())

    dg = normal(g, T, K)
    diff = (loss(rows, gates + dg) - loss(rows, gates - dg)) / 2
    want = float((dw.double() * dg.double()).sum())
    size = float((rows.double()[route.pos.long()] * dout.double()[:, None]).abs().sum(2).mul(dg.abs().double() + gates.abs().double()).sum())
    assert abs(diff - want) <= 64 * U * size
    d = normal(g, *rows.shape)
    diff = (loss(rows + d, gates) - loss(rows - d, gates)) / 2
    used = int(route.offsets[-1])
    want = float((drows[:used] * d[:used].double()).sum())
    src = route.src[:used].long()
    exact = torch.where((src >= 0)[:, None], gates.reshape(-1)[src.clamp_min(0)].double()[:, None] * dout.double()[src.clamp_min(0) // K], 0.0)
    tol = float((2.0 ** -4 * (exact * d[:used].double()).abs()).sum() + 2.0 ** -10 / 448 * (exact.abs().amax() * d[:used].abs().double().sum()))
    assert abs(diff - want) <= tol + 64 * U * float((exact.abs() * (d[:used].abs() + rows[:used].abs()).double()).sum())


@pytest.mark.parametrize("T, align", [(3, 1), (70, 1), (64, 128), (1500, 128)])
def test_block_captured_and_replayed(T, align):
    """Forward (and, on rows aligned for it, backward) in a CUDA graph: replays with other tokens and another routing give
    what eager calls give, and two graphs at a time do not disturb one another."""
    D, F, K, E = 384, 256, 4, 8
    x, w, experts, gates, wgu, wd, dout = block_inputs(T, K, E, D, F)
    bgu, bd = by_blocks(wgu), by_blocks(wd)

    def step():
        out, kept = block_forward(x, w, experts, gates, bgu, bd, align)
        return (out, *(block_backward(dout, kept, w, gates, bgu, bd)[:5] if align == 128 else ()))

    step()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step())
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for seed in (1, 2, 3):
        nx, _, ne, ng, *_ = block_inputs(T, K, E, D, F, seed)
        x.copy_(nx), experts.copy_(ne), gates.copy_(ng)
        if seed == 3:
            experts.fill_(E - 1)  # everything to one expert
        want = step()
        torch.cuda.synchronize()
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        for out in outs:
            for a, b in zip(out, want):
                assert torch.equal(a, b)


def test_streams_at_once():
    sets = [block_inputs(T, 2, 6, 384, 256, seed=T) for T in (5, 60, 700)]
    coded = [(by_blocks(t[4]), by_blocks(t[5])) for t in sets]

    def work(t, c):
        x, w, experts, gates, _, _, dout = t
        out, kept = block_forward(x, w, experts, gates, *c, 128)
        return (out, *block_backward(dout, kept, w, gates, *c)[:5])

    want = [work(t, c) for t, c in zip(sets, coded)]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    rounds = []
    for _ in range(8):
        for t, c, st in zip(sets, coded, streams):
            with torch.cuda.stream(st):
                rounds.append(work(t, c))
    torch.cuda.synchronize()
    for i, got in enumerate(rounds):
        for a, b in zip(got, want[i % len(sets)]):
            assert torch.equal(a, b)


def test_given_stream_and_results_repeat():
    T, K, E, D, F = 90, 2, 6, 384, 256
    x, w, experts, gates, wgu, wd, dout = block_inputs(T, K, E, D, F)
    route = B.fp8q_moe_sort(experts, E, 128)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    other = B.fp8q_moe_sort(experts, E, 128, stream=st)
    q, s, qt, stt = B.fp8q_moe_dispatch(x, other, transposed=True, stream=st)
    y = B.fp8q_moe_combine(x.repeat(route.src.numel() // T + 1, 1)[:route.src.numel()].contiguous(), other, gates, stream=st)
    st.synchronize()
    used = int(route.offsets[-1])
    q2, s2, qt2, st2 = B.fp8q_moe_dispatch(x, route, transposed=True)
    y2 = B.fp8q_moe_combine(x.repeat(route.src.numel() // T + 1, 1)[:route.src.numel()].contiguous(), route, gates)
    for a, b in zip(route, other):
        assert torch.equal(a, b)
    assert torch.equal(q[:used], q2[:used]) and torch.equal(qt[:, :used], qt2[:, :used]) and torch.equal(y, y2)


def test_host_threads_at_once():
    sets = [block_inputs(T, 2, 6, 384, 256, seed=T) for T in (7, 90, 500)]
    coded = [(by_blocks(t[4]), by_blocks(t[5])) for t in sets]

    def work(i):
        x, w, experts, gates, _, _, dout = sets[i]
        out, kept = block_forward(x, w, experts, gates, *coded[i], 128)
        return (out, *block_backward(dout, kept, w, gates, *coded[i])[:5])

    want = [work(i) for i in range(len(sets))]
    torch.cuda.synchronize()
    got = [[] for _ in sets]

    def run(i):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(6):
                got[i].append(work(i))
        st.synchronize()

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for w, g in zip(want, got):
        assert len(g) == 6
        for r in g:
            for a, b in zip(r, w):
                assert torch.equal(a, b)


def test_offsets_that_do_not_ascend():
    """Every second expert is said to have all rows: nothing outside the tensors is touched, and every call ends."""
    E, R, N, K = 1000, 2000, 512, 128
    offsets = torch.zeros(E + 1, dtype=I32, device="cuda")
    offsets[1::2] = R
    g = gen(6)
    a, sa = B.fp8_quantize_blockwise(normal(g, R, K))
    b, sb = B.fp8_quantize_blockwise(normal(g, E * N, K), (128, 128))
    for r in (R, 100):
        c, out = guarded((r, N), BF), [guarded((r, N // 2), torch.uint8), guarded((r, N // 256), FP)]
        B.fp8q_gemm_grouped(a[:r], sa[:r], b.view(E, N, K), sb.view(E, N // 128, 1), offsets, c=c.t)
        B.fp8q_gemm_gated_grouped(a[:r], sa[:r], b.view(E, N, K), sb.view(E, N // 128, 1), offsets, q=out[0].t, scales=out[1].t)
        torch.cuda.synchronize()
        for o in (c, *out):
            o.check()


def test_past_two_to_the_31_elements():
    """Rows whose elements lie behind 2^31: the first, the last and those around the border."""
    T, K, E, cols = 40000, 8, 8, 7168
    g = gen(12)
    experts = torch.rand(T, E, generator=g, device="cuda").argsort(dim=1).to(I32).contiguous()  # every token to every expert
    route = B.fp8q_moe_sort(experts, E, 128)
    used, R = int(route.offsets[-1]), route.src.numel()
    assert used * cols > 2 ** 31 and used == E * -(-T // 128) * 128
    border = 2 ** 31 // cols
    at = torch.tensor([0, 1, border - 1, border, border + 1, used - 200, used - 65], device="cuda")
    src = route.src[at].long()
    assert bool((src >= 0).all())
    x = normal(g, T, cols).to(BF)
    gates = normal(g, T, K)
    q, s, qt, st = B.fp8q_moe_dispatch(x, route, transposed=True)
    wq, ws = B.fp8_quantize_blockwise(x[src // K])
    assert torch.equal(q[at], wq) and torch.equal(s[at], ws)
    for col in (0, cols - 1):  # columns of 320256 rows: the last lies behind 2^31
        block = at[-1] // 128
        v = torch.where((route.src >= 0)[:, None], x[:, col:col + 1][route.src.long().clamp_min(0) // K], 0).t().contiguous()
        wq, ws = B.fp8_quantize_blockwise(v)
        assert torch.equal(qt[col:col + 1, :used], wq[:, :used]) and torch.equal(st[col, :block + 1], ws[0, :block + 1])
    rows = torch.empty(R, cols, dtype=BF, device="cuda").normal_(generator=g)
    y = B.fp8q_moe_combine(rows, route, gates)
    dw = B.fp8q_moe_combine_backward(x, rows, route, gates, transposed=False)
    for t in (0, T // 2, T - 1):
        picked = rows[route.pos[t].long()].double()
        terms = gates[t].double()[:, None] * picked
        check_close(y[t], terms.sum(0), (K + 1) * U * terms.abs().sum(0), "combine")
        prod = picked * x[t].double()
        check_close(dw[4][t], prod.sum(1), (16 * 4 + 8) * U * prod.abs().sum(1), "dweights")
    check_codes(dw[0][at], dw[1][at], x[src // K].double() * gates.reshape(-1)[src].double()[:, None],
                U * (x[src // K].double() * gates.reshape(-1)[src].double()[:, None]).abs(), B.E4M3, "rows' gradient")
    del rows, y, dw
    # products whose results lie behind 2^31, and weights' gradients whose operands do
    b, sb = B.fp8_quantize_blockwise(normal(g, E * cols, 128), (128, 128))
    a, sa = q[:, :128].contiguous(), s[:, :1].contiguous()
    c = B.fp8q_gemm_grouped(a, sa, b.view(E, cols, 128), sb.view(E, cols // 128, 1), route.offsets)
    for r in at.tolist():
        e = int((route.offsets <= r).sum()) - 1
        av, bv = decode(a[r:r + 1], sa[r:r + 1], 1, B.E4M3), decode(b.view(E, cols, 128)[e], sb.view(E, cols // 128, 1)[e], 128, B.E4M3)
        check_close(c[r:r + 1], av @ bv.T, bound(av.abs() @ bv.abs().T, 128), "products")
    del c
    dwt = B.fp8q_gemm_grouped_wgrad(qt, st, qt[-128:].contiguous(), st[-128:].contiguous(), route.offsets)
    lo, hi = route.offsets[-2:].tolist()
    rowsn = torch.tensor([0, cols - 1], device="cuda")
    av = decode(qt[rowsn, lo:hi], st[rowsn, lo // 128:hi // 128], 1, B.E4M3)
    bv = decode(qt[-128:, lo:hi], st[-128:, lo // 128:hi // 128], 1, B.E4M3)
    check_close(dwt[-1][rowsn], av @ bv.T, (2.0 ** -14 + 2.0 ** -22 + ((hi - lo) / 128 + 8) * U) * (av.abs() @ bv.abs().T), "weights' gradients")


def test_binding_refusals():
    T, K, E, D = 6, 2, 4, 256
    experts = make_experts(T, K, E).cuda()
    x = torch.zeros(T, D, device="cuda", dtype=BF)
    route = B.fp8q_moe_sort(experts, E, 128)
    R = route.src.numel()
    gates = torch.ones(T, K, device="cuda")
    rows = torch.zeros(R, D, device="cuda", dtype=BF)
    code = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    ones = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    for call, match in [
            (lambda: B.fp8q_moe_sort(experts.long(), E), "dtype"), (lambda: B.fp8q_moe_sort(experts[0], E), "experts"),
            (lambda: B.fp8q_moe_sort(experts.t(), E), "contiguous"), (lambda: B.fp8q_moe_sort(experts.cpu(), E), "CUDA"),
            (lambda: B.fp8q_moe_sort(experts, E, pos=experts[:3].clone()), "pos has shape"),
            (lambda: B.fp8q_moe_dispatch(x[:3], route), "pos has shape"),
            (lambda: B.fp8q_moe_dispatch(x.half(), route), "dtype"), (lambda: B.fp8q_moe_dispatch(x[0], route), "takes x"),
            (lambda: B.fp8q_moe_dispatch(x, route, qt=code(D, R), scales_t=ones(D, R // 128)), "only with transposed"),
            (lambda: B.fp8q_moe_dispatch(x, route, q=code(R, D + 128)), "q has shape"),
            (lambda: B.fp8q_moe_dispatch_codes(code(T, D), ones(T, 1), route), "xs has shape"),
            (lambda: B.fp8q_moe_combine(rows, route, gates.double()), "weights has dtype"),
            (lambda: B.fp8q_moe_combine(rows, route, gates, residual=x.float()), "residual has dtype"),
            (lambda: B.fp8q_moe_combine_backward(x, None, route, gates), "needs the rows"),
            (lambda: B.fp8q_moe_combine_backward(x, rows[:-1], route, gates), "rows has shape"),
            (lambda: B.fp8q_gemm_grouped(code(R, D), ones(R, 2), code(E, 256, 128), ones(E, 2, 1), route.offsets), "takes a"),
            (lambda: B.fp8q_gemm_grouped(code(R, D), ones(R, 2), code(E, 256, D), ones(E, 2, 2), route.offsets[:-1].clone()),
             "offsets has shape"),
            (lambda: B.fp8q_gemm_grouped(code(R, D), ones(R, 1), code(E, 256, D), ones(E, 2, 2), route.offsets), "sa has shape"),
            (lambda: B.fp8q_gemm_gated_grouped(code(R, D), ones(R, 2), code(E, 255, D), ones(E, 1, 2), route.offsets), "2F"),
            (lambda: B.fp8q_gemm_gated_grouped(code(R, D), ones(R, 2), code(E, 256, D), ones(E, 2, 2), route.offsets,
                                               q=code(R, 128)), "go together"),
            (lambda: B.fp8q_gemm_grouped_wgrad(code(D, R), ones(D, R // 128), code(D, R - 128), ones(D, R // 128), route.offsets),
             "takes at")]:
        with pytest.raises(ValueError, match=match):
            call()
    for call in (lambda: B.fp8q_moe_sort(experts, E, 3), lambda: B.fp8q_moe_sort(experts, E, src=experts.view(-1)[:2].clone()),
                 lambda: B.fp8q_moe_sort(experts, 1025), lambda: B.fp8q_moe_dispatch(x[:, :192].contiguous(), route),
                 lambda: B.fp8q_moe_dispatch(x, B.fp8q_moe_sort(experts, E, 1), transposed=True),
                 lambda: B.fp8q_moe_combine(rows, route, gates, residual=x, y=x),
                 lambda: B.fp8q_gemm_grouped(code(R, 192), ones(R, 1), code(E, 256, 192), ones(E, 2, 1), route.offsets),
                 lambda: B.fp8q_gemm_gated_grouped(code(R, D), ones(R, 2), code(E, 256, D), ones(E, 2, 2), route.offsets, act=7)):
        with pytest.raises(B.FP8Error):
            call()


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two GPUs")
def test_tensors_of_another_device_than_the_current_one():
    experts = make_experts(9, 2, 4).to("cuda:1")
    route = B.fp8q_moe_sort(experts, 4)
    assert route.pos.device == experts.device
