"""The operators of a block of experts where a route is used in part or changed after the sort, and where offsets are not the
sort's.

Tolerances are those of test_gpu_moe.py, and their derivation.
"""
import pytest
import torch

from fine_grained_block_b200 import binding as B
from test_gpu_ffn import BF, FP, MAX, check_close, decode, gen, normal
from test_gpu_moe import I32, bound, check_gated_grouped, check_grouped, guarded, make_route, untouched

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


# -- K split over a cluster -------------------------------------------------------------------------------------------

# Few tiles and at least 32 chunks of K: clusters of 8, whose ranks take unlike numbers of chunks for K = 4224 (33) and
# 4992 (39); 16, 24 and 31 chunks: clusters of 4.  Up to 8 rows an expert blocks of 16 rows, else of 32.
SPLIT = [([1], 1), ([3, 0, 5], 1), ([8, 8], 16), ([20], 1), ([17, 0, 31], 1), ([64, 2], 1)]


@pytest.mark.parametrize("K", [2048, 3968, 4096, 4224, 4992, 7168])
@pytest.mark.parametrize("N", [128, 384, 512])
@pytest.mark.parametrize("lengths, align", SPLIT, ids=str)
def test_products_of_long_rows_split(lengths, align, N, K):
    for dtype in (BF, FP):
        got = [check_grouped(lengths, N, K, align, spare=3, dtype=dtype) for _ in range(2)]
        assert torch.equal(*got)  # the ranks' sums are joined in a fixed order


@pytest.mark.parametrize("K", [2048, 4096, 4224, 7168])
@pytest.mark.parametrize("F", [128, 384, 512])
@pytest.mark.parametrize("lengths, align", SPLIT, ids=str)
@pytest.mark.parametrize("act, fmt", [(B.ACT_SILU, B.E4M3), (B.ACT_GELU_TANH, B.E5M2)])
def test_gated_products_of_long_rows_split(lengths, align, F, K, act, fmt):
    check_gated_grouped(lengths, F, K, align, spare=3, act=act, fmt=fmt)


# -- offsets that no sort makes ---------------------------------------------------------------------------------------

# Rows 0 and 1 are the first expert's alone, 5 and on the last one's; the second has none, since its end comes first.
@pytest.mark.parametrize("R, N", [(128, 256), (128, 8192), (700, 256), (2000, 4096)])
@pytest.mark.parametrize("offsets", [[-2 ** 31, 5, 2, 2 ** 31 - 1], [-1, 5, 2, 5000], [0, 5, -7, 4000]], ids=str)
def test_products_where_an_expert_has_its_rows_alone(R, N, offsets):
    K, E = 256, 3
    off = torch.tensor(offsets, dtype=I32, device="cuda")
    g = gen(R + N)
    a, sa = B.fp8_quantize_blockwise(normal(g, R, K))
    b, sb = B.fp8_quantize_blockwise(normal(g, E * N, K), (128, 128))
    c = guarded((R, N), FP)
    B.fp8q_gemm_grouped(a, sa, b.view(E, N, K), sb.view(E, N // 128, K // 128), off, c=c.t)
    torch.cuda.synchronize()
    c.check()
    first = max(offsets[2], 0)  # of the last expert
    for e, rows in ((0, slice(0, first)), (2, slice(5, R)))[first == 0:]:
        av = decode(a[rows], sa[rows], 1, B.E4M3)
        bv = decode(b[e * N:(e + 1) * N], sb[e * N // 128:(e + 1) * N // 128], 128, B.E4M3)
        check_close(c.t[rows], av @ bv.T, bound(av.abs() @ bv.abs().T, K), f"expert {e}")


@pytest.mark.parametrize("offsets", [[-5, 130, 100, 2 ** 31 - 1], [1, 200, 383], [127, 128, 129, 255, 256], [640, 0, 640],
                                     [-2 ** 31, -1, 384], [300, 300, 500]], ids=str)
@pytest.mark.parametrize("N, K", [(128, 128), (384, 640)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_wgrad_of_offsets_that_are_no_multiples(offsets, N, K, dtype):
    """Offsets are held inside 0 .. rows and rounded down to a block of 128; an expert whose end comes first has no rows."""
    R, E = 384, len(offsets) - 1
    g = gen(N + K)
    at, sat = B.fp8_quantize_blockwise(normal(g, N, R))
    bt, sbt = B.fp8_quantize_blockwise(normal(g, K, R))
    dw = guarded((E, N, K), dtype)
    B.fp8q_gemm_grouped_wgrad(at, sat, bt, sbt, torch.tensor(offsets, dtype=I32, device="cuda"), dw=dw.t)
    torch.cuda.synchronize()
    dw.check()
    block = [min(max(o, 0), R) // 128 for o in offsets]
    for e, (lo, hi) in enumerate(zip(block, block[1:])):
        if hi <= lo:
            assert int((dw.t[e] != 0).sum()) == 0
            continue
        av, bv = (decode(q[:, lo * 128:hi * 128], s[:, lo:hi], 1, B.E4M3) for q, s in ((at, sat), (bt, sbt)))
        check_close(dw.t[e], av @ bv.T, bound(av.abs() @ bv.abs().T, (hi - lo) * 128), f"expert {e}")


# -- rows of a route --------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("experts", [0, 1, 3])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_rows_behind_the_last_expert_named(experts, dtype):
    """A route cut to its first experts: rows behind theirs are left as they were, though pairs have them."""
    T, K, E, cols = 70, 3, 5, 256
    route = make_route(T, K, E, 128, "random")
    used = int(route.offsets[experts])
    first = B.MoeRoute(route.offsets[:max(experts, 1) + 1].clone(), *route[1:])
    if experts == 0:
        first.offsets[1] = 0
    R = route.src.numel()
    g = gen(experts)
    x, weights = normal(g, T, cols).to(dtype), normal(g, T, K)
    q, s, qt, st = B.fp8q_moe_dispatch(x, route, transposed=True)
    dq, ds, dqt, dst, _ = B.fp8q_moe_combine_backward(x, None, route, weights, want_dweights=False)
    cq, cs = B.fp8q_moe_dispatch_codes(*B.fp8_quantize_blockwise(x), route)

    def outputs(transposed):
        shapes = [((R, cols), torch.uint8), ((R, cols // 128), FP)]
        return [guarded(*v) for v in (*shapes, *((((cols, R), torch.uint8), ((cols, R // 128), FP)) if transposed else ()))]

    for transposed in (False, True):
        for call, want in ((lambda **kw: B.fp8q_moe_dispatch(x, first, transposed=transposed, **kw), (q, s, qt, st)),
                           (lambda **kw: B.fp8q_moe_combine_backward(x, None, first, weights, transposed=transposed,
                                                                     want_dweights=False, **kw), (dq, ds, dqt, dst)),
                           (lambda **kw: B.fp8q_moe_dispatch_codes(*B.fp8_quantize_blockwise(x), first, **kw), (cq, cs))):
            if transposed and len(want) == 2:
                continue
            out = outputs(transposed)
            call(**dict(zip(("q", "scales", "qt", "scales_t"), (o.t for o in out))))
            torch.cuda.synchronize()
            for i, (o, w) in enumerate(zip(out, want)):
                o.check()
                dim, n = (0, used) if i < 2 else (1, used if i == 2 else used // 128)
                assert torch.equal(o.t.narrow(dim, 0, n), w.narrow(dim, 0, n)) and untouched(o.t, n, dim), i


def dropped_by_pos(route, kind, seed):
    """The route with some pairs' pos set to -1 (src as it was), and the same with their rows' src set to -1 too."""
    g = torch.Generator().manual_seed(seed)
    pos, src = route.pos.cpu(), route.src.cpu()
    drop = {"some": torch.rand(pos.shape, generator=g) < 0.3, "all": torch.ones(pos.shape, dtype=torch.bool),
            "one": torch.arange(pos.numel()).view(pos.shape) == pos.numel() // 2,
            "capacity": torch.zeros(pos.shape, dtype=torch.bool)}[kind]
    if kind == "capacity":  # the second half of the rows of the fullest expert, and as many rows elsewhere at most
        first = route.offsets.cpu()[torch.bucketize(pos, route.offsets.cpu()[1:], right=True)]
        drop = pos - first > int((pos - first).max()) // 2
    drop &= pos >= 0
    assert bool(drop.any())
    src[pos[drop].long()] = -1
    pos = torch.where(drop, -1, pos).to(I32)
    return B.MoeRoute(route.offsets, pos.cuda(), route.src, route.counts), B.MoeRoute(route.offsets, pos.cuda(), src.cuda(), None)


@pytest.mark.parametrize("T, K, E, align, cols", [(5, 2, 3, 1, 128), (70, 3, 5, 128, 256), (300, 8, 9, 128, 1152), (2000, 4, 8, 16, 640)])
@pytest.mark.parametrize("kind", ["some", "all", "one", "capacity"])
@pytest.mark.parametrize("dtype, fmt", [(BF, B.E4M3), (FP, B.E5M2)])
def test_pairs_dropped_after_the_sort(T, K, E, align, cols, kind, dtype, fmt):
    """A pair whose pos is set to -1 gives up its row: zeros in every output, as if src said so too."""
    route = make_route(T, K, E, align, "random", spare=-B.fp8q_moe_rows(T, K, E, align) % 128)
    by_pos, by_both = dropped_by_pos(route, kind, T)
    used, R = int(route.offsets[-1]), route.src.numel()
    g = gen(T)
    x, weights = normal(g, T, cols).to(dtype), normal(g, T, K)
    rows = normal(g, R, cols).to(dtype)
    codes = B.fp8_quantize_blockwise(x, (1, 128), fmt)
    blocks = -(-used // 128)
    for call in (lambda r, **kw: B.fp8q_moe_dispatch(x, r, fmt, True, **kw),
                 lambda r, **kw: B.fp8q_moe_combine_backward(x, rows, r, weights, fmt, True, **kw),
                 lambda r, **kw: B.fp8q_moe_dispatch(x, r, fmt, **kw),
                 lambda r, **kw: B.fp8q_moe_dispatch_codes(*codes, r, fmt, **kw)):
        want = [t for t in call(by_both) if t is not None]
        out = [guarded(tuple(t.shape), t.dtype) for t in want]
        call(by_pos, **dict(zip(("q", "scales", "qt", "scales_t", "dweights"), (o.t for o in out))))
        torch.cuda.synchronize()
        for i, (o, w) in enumerate(zip(out, want)):
            o.check()
            dim, n = ((0, used), (0, used), (1, blocks * 128), (1, blocks), (0, T))[i]
            assert torch.equal(o.t.narrow(dim, 0, n), w.narrow(dim, 0, n)), i
            if i < 4:
                assert untouched(o.t, n, dim), i
    empty = (by_both.src[:used] < 0)
    q, s, *_ = B.fp8q_moe_dispatch(x, by_pos, fmt)
    assert int(q[:used][empty].sum()) == 0 and bool((s[:used][empty] == torch.tensor(MAX[fmt], device="cuda") / 1e-12).all())
    dweights = B.fp8q_moe_combine_backward(x, rows, by_pos, weights, transposed=False)[4]
    assert int((dweights[by_pos.pos < 0] != 0).sum()) == 0
