"""The operators of a feed-forward block of experts in FP8, as they are measured: what each case stands for, its inputs, its
plain form in elementary torch operations, and the calls that a program makes of the library.

Five operators: the sort of (token, expert) pairs by expert; the dispatch of tokens to their rows as FP8 codes; the combine
of the experts' rows with the router's weights, and its gradient; the gated projections of every expert; and the experts'
plain products, forward and for the weights' gradients.

With ``own`` false, ``run`` computes the plain form in fp32; with ``own`` true it calls the library.  Codes are returned
as float8 tensors, the values that they stand for, beside their scales.

Rows are laid out expert after expert.  A serving program packs them (align 1); a training program starts each expert at a
multiple of 128 rows (align 128), the blocks of the weights' gradients, and the rows in between are zeros.
"""
import math

import torch

own = False

AMAX_FLOOR = 1e-12
F8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# -- cases ------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # a decode batch is routed: latency
        dict(name="sort decode", op="sort", tokens=64, top_k=8, experts=256, align=1, drop=False),
        # a training step's tokens, each expert at a multiple of 128 rows
        dict(name="sort training", op="sort", tokens=16384, top_k=8, experts=256, align=128, drop=False),
        # a decode batch whose codes the norm has made: each token's codes go to the rows of its experts
        dict(name="dispatch decode codes", op="dispatch", tokens=64, top_k=8, experts=256, align=1, drop=False, cols=7168,
             dtype="codes", fmt="e4m3", train=False),
        # a training step: codes of the rows, and of their transpose for the weights' gradients
        dict(name="dispatch training", op="dispatch", tokens=16384, top_k=8, experts=64, align=128, drop=False, cols=7168,
             dtype="bf16", fmt="e4m3", train=True),
        # a prompt of odd length in fp32, some pairs dropped (experts over their capacity)
        dict(name="combine odd f32", op="combine", tokens=1001, top_k=6, experts=64, align=1, drop=True, cols=4096,
             dtype="f32", residual=False),
        # a training step, onto the shared expert's output
        dict(name="combine training", op="combine", tokens=16384, top_k=8, experts=64, align=128, drop=False, cols=7168,
             dtype="bf16", residual=True),
        # its gradient: the rows' as codes in both directions, and the weights'
        dict(name="combine backward training", op="combine_bwd", tokens=16384, top_k=8, experts=64, align=128, drop=True,
             cols=4096, dtype="bf16", fmt="e5m2", train=True),
        # decode: one token against the projections of its eight experts, bound by reading them
        dict(name="gated experts one token", op="gated", tokens=1, top_k=8, experts=64, align=1, drop=False, k=7168, f=2048,
             act="silu", fmt="e4m3", train=False),
        # a training step: the projections are kept for the backward pass
        dict(name="gated experts training", op="gated", tokens=8192, top_k=8, experts=32, align=128, drop=False, k=4096,
             f=2048, act="silu", fmt="e4m3", train=True),
        # the down projection of a decode batch
        dict(name="products decode", op="gemm", tokens=48, top_k=4, experts=32, align=1, drop=False, k=2048, n=7168,
             dtype="bf16"),
        # the down projection of a prompt of odd length, some pairs dropped
        dict(name="products prompt", op="gemm", tokens=1001, top_k=8, experts=64, align=1, drop=True, k=2048, n=7168,
             dtype="bf16"),
        # a training step: the gradients of every expert's projections
        dict(name="weight gradients training", op="wgrad", tokens=8192, top_k=8, experts=32, align=128, drop=False, k=4096,
             n=4096, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["sort", "dispatch", "dispatch", "combine", "combine_bwd", "gated", "gated", "gemm", "gemm", "wgrad"])
    experts = _log(rng, 2, 256)
    c = dict(op=op, tokens=_log(rng, 1, 16384), top_k=rng.randint(1, min(8, experts)), experts=experts,
             align=rng.choice([1, 1, 16, 128]), drop=rng.random() < 0.3)
    if op in ("dispatch", "combine", "combine_bwd"):
        c.update(cols=128 * _log(rng, 1, 56), dtype=rng.choice(["bf16", "bf16", "f32"]))
        if op == "combine":
            c.update(residual=rng.random() < 0.5)
        else:
            c.update(fmt=rng.choice(["e4m3", "e5m2"]), train=rng.random() < 0.5)
            if op == "dispatch" and not c["train"] and rng.random() < 0.5:
                c["dtype"] = "codes"
            if c["train"]:
                c["align"] = 128
        if c["dtype"] == "f32":
            c["tokens"] = max(1, c["tokens"] // 2)
        if op == "combine_bwd" and c["cols"] > 4096:
            c["tokens"] = max(1, c["tokens"] // 2)
    elif op in ("gated", "gemm", "wgrad"):
        c["k"] = 128 * _log(rng, 2, 56)
        if op == "gated":
            c.update(f=128 * _log(rng, 1, 32), act=rng.choice(["silu", "gelu"]), fmt=rng.choice(["e4m3", "e4m3", "e5m2"]),
                     train=rng.random() < 0.5)
        else:
            c.update(n=128 * _log(rng, 1, 56), dtype=rng.choice(["bf16", "f32"]))
        if op == "wgrad":  # rows in blocks of 128 tokens, columns in the tiles of the library's weight gradients
            c.update(align=128, n=max(256, c["n"] // 256 * 256), k=max(256, c["k"] // 256 * 256))
        wide = 2 * c["f"] if op == "gated" else c["n"]
        while c["experts"] * wide * c["k"] > (1 << 29):  # the weights of the listed training steps
            c["experts"] //= 2
        c["top_k"] = min(c["top_k"], c["experts"])
        rows_most = (1 << 16) * 4096 * 4096 // (wide * c["k"])  # and their rows, by the work
        c["tokens"] = max(1, min(c["tokens"], rows_most // c["top_k"]))
    return c


def _capacity(c):
    """Rows that hold any routing of the case's pairs."""
    pairs = c["tokens"] * c["top_k"]
    return (pairs + min(c["experts"], pairs) * (c["align"] - 1)) // c["align"] * c["align"]


def work(case):
    c, op = case, case["op"]
    pairs = c["tokens"] * c["top_k"]
    if op == "sort":
        return {"bytes": 4 * (2 * pairs + _capacity(c) + 2 * c["experts"] + 1), "flops": 2 * pairs}
    if op in ("dispatch", "combine", "combine_bwd"):
        t, d = c["tokens"], c["cols"]
        e = {"bf16": 2, "f32": 4, "codes": 1}[c["dtype"]]
        codes = pairs * d + 4 * pairs * (d // 128)
        if op == "dispatch":
            b = t * d * e + (4 * t * (d // 128) if c["dtype"] == "codes" else 0) + 4 * pairs + codes * (2 if c["train"] else 1)
            return {"bytes": b, "flops": 4 * t * d}
        if op == "combine":
            return {"bytes": (pairs + t * (2 if c["residual"] else 1)) * d * e + 8 * pairs, "flops": 2 * pairs * d}
        return {"bytes": (pairs + t) * d * e + codes * (2 if c["train"] else 1) + 12 * pairs, "flops": 4 * pairs * d}
    n, k = (2 * c["f"] if op == "gated" else c["n"]), c["k"]
    hit = c["experts"] * (1.0 - (1.0 - c["top_k"] / c["experts"]) ** c["tokens"])  # experts with a token, on average
    weights = round(hit) * (n * k + 4 * (n // 128) * (k // 128))
    rows = pairs * k + 4 * pairs * (k // 128)
    if op == "gated":
        b = rows + weights + pairs * c["f"] + 4 * pairs * (c["f"] // 128) + (2 * pairs * n if c["train"] else 0)
    elif op == "gemm":
        b = rows + weights + pairs * n * (2 if c["dtype"] == "bf16" else 4)
    else:
        b = rows + pairs * n + 4 * pairs * (n // 128) + c["experts"] * n * k * (2 if c["dtype"] == "bf16" else 4)
    return {"bytes": b, "flops": 2 * pairs * n * k}


# -- inputs -----------------------------------------------------------------------------------------------------------

def _codes(x, block_rows, fmt="e4m3"):
    """Codes and scales of x [R, C] (multiples of the block), in blocks of block_rows x 128."""
    ty, top = F8[fmt]
    R, C = x.shape
    v = x.view(R // block_rows, block_rows, C // 128, 128)
    s = top / v.abs().amax(dim=(1, 3)).clamp_min(AMAX_FLOOR)
    q = (v * s[:, None, :, None]).clamp(-top, top).view(R, C).to(ty)
    return q.view(torch.uint8), s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c, op = case, case["op"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    def empty(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda")

    # The router: scores of a token, some experts liked more than others; the best top_k and their shares.  How many tokens
    # share an expert is the case's; which tokens and which expert is the seed's.
    t, k, E = c["tokens"], c["top_k"], c["experts"]
    sizes = torch.Generator(device="cuda")
    sizes.manual_seed(t * 65536 + k * 4096 + E)
    liked = torch.randn(t, E, generator=sizes, device="cuda") + 0.5 * torch.randn(E, generator=sizes, device="cuda")
    experts = torch.randperm(E, generator=g, device="cuda")[liked.topk(k, dim=1).indices]
    if c["drop"]:  # pairs over an expert's capacity
        over = torch.rand(t, k, generator=sizes, device="cuda") < 0.05
        over[0, 0] = False
        experts[over] = -1
    experts = experts[torch.randperm(t, generator=g, device="cuda")].to(torch.int32).contiguous()
    weights = torch.softmax(normal(t, k).sort(dim=1, descending=True).values, dim=1).contiguous()
    s = {"case": c}
    if op == "sort":
        s["experts"] = experts
        i32 = dict(dtype=torch.int32)
        s["offsets"], s["pos"], s["src"], s["counts"] = empty(E + 1, **i32), empty(t, k, **i32), empty(_capacity(c), **i32), empty(E, **i32)
        return s

    # the plan that the program keeps from its sort; the rows' number is what the plan needs, and known to it
    offsets, pos, src, counts = _sorted(experts, E, c["align"], _capacity(c))
    s["bounds"] = offsets.tolist()
    R = s["bounds"][-1]
    s["offsets"], s["pos"], s["src"], s["counts"] = offsets, pos, src[:R].contiguous(), counts
    real = s["src"] >= 0  # the other rows are zeros

    if op in ("dispatch", "combine", "combine_bwd"):
        d = c["cols"]
        if op == "dispatch":
            x = normal(t, d)
            x[:, torch.randint(0, d, (8,), generator=g, device="cuda")] *= 20.0  # a few outlier channels
            if c["dtype"] == "codes":
                s["x"], s["sx"] = _codes(x, 1, c["fmt"])
            else:
                s["x"] = x.to(DT[c["dtype"]])
        else:
            dt = DT[c["dtype"]]
            s["weights"] = weights
            s["rows"] = (normal(R, d) * real[:, None]).to(dt)
            if op == "combine":
                s["residual"] = normal(t, d, std=2.0).to(dt) if c["residual"] else None
                s["y"] = empty(t, d, dtype=dt)
                return s
            s["dy"] = normal(t, d, std=1e-3).to(dt)
            s["dweights"] = empty(t, k)
        s["q"], s["scales"] = empty(R, d, dtype=torch.uint8), empty(R, d // 128)
        s["qt"], s["scales_t"] = (empty(d, R, dtype=torch.uint8), empty(d, R // 128)) if c["train"] else (None, None)
        return s

    if op == "wgrad":
        live = real.float()
        s["at"], s["sat"] = _codes((normal(R, c["n"], std=1e-3) * live[:, None]).t().contiguous(), 1)
        s["bt"], s["sbt"] = _codes((normal(R, c["k"]) * live[:, None]).t().contiguous(), 1)
        s["dw"] = empty(E, c["n"], c["k"], dtype=DT[c["dtype"]])
        return s
    n = 2 * c["f"] if op == "gated" else c["n"]
    s["a"], s["sa"] = _codes(normal(R, c["k"]) * real[:, None], 1)
    b, sb = _codes(normal(E * n, c["k"], std=0.02), 128)
    s["b"], s["sb"] = b.view(E, n, c["k"]), sb.view(E, n // 128, c["k"] // 128)
    if op == "gated":
        s["q"], s["scales"] = empty(R, c["f"], dtype=torch.uint8), empty(R, c["f"] // 128)
        s["gu"] = empty(R, n, dtype=torch.bfloat16) if c["train"] else None
    else:
        s["c"] = empty(R, n, dtype=DT[c["dtype"]])
    return s


# -- one pass ---------------------------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"sort": _own_sort, "dispatch": _own_dispatch, "combine": _own_combine, "combine_bwd": _own_combine_bwd,
                "gated": _own_gated, "gemm": _own_gemm, "wgrad": _own_wgrad}[op](state)
    return {"sort": _sort, "dispatch": _dispatch, "combine": _combine, "combine_bwd": _combine_bwd, "gated": _gated,
            "gemm": _gemm, "wgrad": _wgrad}[op](state)


def _route(B, s):
    return B.MoeRoute(s["offsets"], s["pos"], s["src"], s["counts"])


def _code_outputs(c, q, scales, qt, scales_t):
    ty = F8[c["fmt"]][0]
    out = {"q": q.view(ty), "scales": scales}
    if c["train"]:
        out["qt"], out["scales_t"] = qt.view(ty), scales_t
    return out


def _own_sort(s):
    from fine_grained_block_b200 import binding as B
    c = s["case"]
    r = B.fp8q_moe_sort(s["experts"], c["experts"], align=c["align"], offsets=s["offsets"], pos=s["pos"], src=s["src"],
                        counts=s["counts"])
    return {"offsets": r.offsets, "pos": r.pos, "src": r.src, "counts": r.counts}


def _own_dispatch(s):
    from fine_grained_block_b200 import binding as B
    c = s["case"]
    if c["dtype"] == "codes":
        q, scales = B.fp8q_moe_dispatch_codes(s["x"], s["sx"], _route(B, s), fmt=B.E4M3 if c["fmt"] == "e4m3" else B.E5M2,
                                              q=s["q"], scales=s["scales"])
        return _code_outputs(c, q, scales, None, None)
    return _code_outputs(c, *B.fp8q_moe_dispatch(s["x"], _route(B, s), fmt=B.E4M3 if c["fmt"] == "e4m3" else B.E5M2,
                                                 transposed=c["train"], q=s["q"], scales=s["scales"], qt=s["qt"],
                                                 scales_t=s["scales_t"]))


def _own_combine(s):
    from fine_grained_block_b200 import binding as B
    return B.fp8q_moe_combine(s["rows"], _route(B, s), weights=s["weights"], residual=s["residual"], y=s["y"])


def _own_combine_bwd(s):
    from fine_grained_block_b200 import binding as B
    c = s["case"]
    q, scales, qt, scales_t, dweights = B.fp8q_moe_combine_backward(
        s["dy"], s["rows"], _route(B, s), s["weights"], fmt=B.E4M3 if c["fmt"] == "e4m3" else B.E5M2, transposed=c["train"],
        q=s["q"], scales=s["scales"], qt=s["qt"], scales_t=s["scales_t"], dweights=s["dweights"])
    return dict(_code_outputs(c, q, scales, qt, scales_t), dweights=dweights)


def _own_gated(s):
    from fine_grained_block_b200 import binding as B
    c = s["case"]
    q, scales, gu = B.fp8q_gemm_gated_grouped(
        s["a"], s["sa"], s["b"], s["sb"], s["offsets"], act=B.ACT_SILU if c["act"] == "silu" else B.ACT_GELU_TANH,
        fmt=B.E4M3 if c["fmt"] == "e4m3" else B.E5M2, q=s["q"], scales=s["scales"], gu=s["gu"])
    out = {"q": q.view(F8[c["fmt"]][0]), "scales": scales}
    if c["train"]:
        out["gu"] = gu
    return out


def _own_gemm(s):
    from fine_grained_block_b200 import binding as B
    return B.fp8q_gemm_grouped(s["a"], s["sa"], s["b"], s["sb"], s["offsets"], c=s["c"])


def _own_wgrad(s):
    from fine_grained_block_b200 import binding as B
    return B.fp8q_gemm_grouped_wgrad(s["at"], s["sat"], s["bt"], s["sbt"], s["offsets"], dw=s["dw"])


# -- plain forms ------------------------------------------------------------------------------------------------------

def _sorted(experts, E, align, rows):
    t, k = experts.shape
    e = experts.reshape(-1).long()
    hit = e[:, None] == torch.arange(E, device=e.device)[None, :]  # a pair's expert, at most one
    upto = hit.to(torch.int32).cumsum(dim=0)                       # pairs of the expert up to here
    counts = upto[-1].long()
    ends = ((counts + align - 1) // align * align).cumsum(dim=0)
    offsets = torch.cat([ends.new_zeros(1), ends])
    routed = hit.any(dim=1)
    own_e = e.clamp(0, E - 1)
    pos = offsets[own_e] + upto.gather(1, own_e[:, None])[:, 0].long() - 1
    pos = torch.where(routed, pos, torch.full_like(pos, -1))
    src = torch.full((rows + 1,), -1, dtype=torch.int64, device=e.device)
    src[torch.where(routed, pos, torch.full_like(pos, rows))] = torch.arange(t * k, device=e.device)
    i32 = torch.int32
    return offsets.to(i32), pos.view(t, k).to(i32), src[:rows].to(i32), counts.to(i32)


def _quantize(v, fmt):
    """fp32 [R, C], C % 128 == 0, in blocks of 1x128: float8 codes and fp32 scales."""
    ty, top = F8[fmt]
    R, C = v.shape
    w = v.view(R, -1, 128)
    s = top / w.abs().amax(dim=2).clamp_min(AMAX_FLOOR)
    return (w * s[:, :, None]).clamp(-top, top).view(R, C).to(ty), s


def _act(g, kind):
    """act(g) = g * sigmoid(p(g)); the tanh GELU is this with p = 2c(g + 0.044715 g^3)."""
    p = g if kind == "silu" else 2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)
    return g / (1.0 + torch.exp(-p))


def _sort(s):
    c = s["case"]
    return dict(zip(("offsets", "pos", "src", "counts"), _sorted(s["experts"], c["experts"], c["align"], _capacity(c))))


def _token_rows(x, s):
    """Row src[r] // top_k of x for every row, zeros for the rows between the experts."""
    src = s["src"].long()
    return x[src.clamp_min(0) // s["case"]["top_k"]] * (src >= 0)[:, None].to(x.dtype)


def _both(v, c):
    out = dict(zip(("q", "scales"), _quantize(v, c["fmt"])))
    if c["train"]:
        out.update(zip(("qt", "scales_t"), _quantize(v.t().contiguous(), c["fmt"])))
    return out


def _dispatch(s):
    c = s["case"]
    if c["dtype"] == "codes":  # the bytes of the codes; a zero block's scale on the rows between the experts
        ty, top = F8[c["fmt"]]
        real = (s["src"] >= 0)[:, None]
        scales = torch.where(real, _token_rows(s["sx"], s), s["sx"].new_tensor(top) / AMAX_FLOOR)
        return {"q": _token_rows(s["x"], s).view(ty), "scales": scales}
    return _both(_token_rows(s["x"].float(), s), c)


def _combine(s):
    y = torch.zeros_like(s["y"], dtype=torch.float32) if s["residual"] is None else s["residual"].float()
    for j in range(s["case"]["top_k"]):
        at = s["pos"][:, j].long()
        w = torch.where(at >= 0, s["weights"][:, j], 0.0)
        y = y + w[:, None] * s["rows"][at.clamp_min(0)].float()
    return y.to(s["y"].dtype)


def _combine_bwd(s):
    c = s["case"]
    dy = s["dy"].float()
    w = s["weights"].reshape(-1)[s["src"].long().clamp_min(0)]
    out = _both(_token_rows(dy, s) * w[:, None], c)
    dw = []
    for j in range(c["top_k"]):
        at = s["pos"][:, j].long()
        dw.append(torch.where(at >= 0, (dy * s["rows"][at.clamp_min(0)].float()).sum(dim=1), 0.0))
    out["dweights"] = torch.stack(dw, dim=1)
    return out


def _by_expert(s, n):
    """A_e B_e^T of every expert's rows, fp32."""
    ty = torch.float8_e4m3fn
    R, k = s["a"].shape
    gu = torch.zeros(R, n, device="cuda")
    for e, (lo, hi) in enumerate(zip(s["bounds"], s["bounds"][1:])):
        if hi > lo:
            a = (s["a"][lo:hi].view(ty).float().view(hi - lo, -1, 128) / s["sa"][lo:hi, :, None]).view(hi - lo, k)
            b = (s["b"][e].view(ty).float().view(n // 128, 128, k // 128, 128) / s["sb"][e][:, None, :, None]).view(n, k)
            gu[lo:hi] = a @ b.t()
    return gu


def _gated(s):
    c = s["case"]
    gu = _by_expert(s, 2 * c["f"])
    g, u = gu.chunk(2, dim=1)
    q, scales = _quantize(_act(g, c["act"]) * u, c["fmt"])
    return {"q": q, "scales": scales, "gu": gu.to(torch.bfloat16)} if c["train"] else {"q": q, "scales": scales}


def _gemm(s):
    return _by_expert(s, s["case"]["n"]).to(s["c"].dtype)


def _wgrad(s):
    ty = torch.float8_e4m3fn
    dw = torch.zeros(s["dw"].shape, device="cuda")
    for e, (lo, hi) in enumerate(zip(s["bounds"], s["bounds"][1:])):
        if hi > lo:
            a, b = ((v[:, lo:hi].view(ty).float().reshape(v.shape[0], -1, 128) / sc[:, lo // 128:hi // 128, None]).flatten(1)
                    for v, sc in ((s["at"], s["sat"]), (s["bt"], s["sbt"])))
            dw[e] = a @ b.t()
    return dw.to(s["dw"].dtype)


# -- the definitions in 64 bits ---------------------------------------------------------------------------------------

def _scaled(v, fmt):
    """The numbers that the codes of v (fp64 [R, C]) stand for, before their rounding, and the scales.  No numbers for
    E5M2: its two bits put every code about 5 % off, as far as half of what a comparison of 8-bit values allows."""
    R, C = v.shape
    s = F8[fmt][1] / torch.maximum(v.abs().reshape(R, C // 128, 128).max(dim=2).values, v.new_tensor(AMAX_FLOOR))
    return v * s.repeat_interleave(128, dim=1) if fmt == "e4m3" else None, s


def _scaled_both(v, c):
    out = dict(zip(("q", "scales"), _scaled(v, c["fmt"])))
    if c["train"]:
        out.update(zip(("qt", "scales_t"), _scaled(v.T.contiguous(), c["fmt"])))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "sort":
        e = s["experts"].reshape(-1).cpu()
        order = [[] for _ in range(c["experts"])]
        for p, x in enumerate(e.tolist()):
            if x >= 0:
                order[x].append(p)
        offsets, src, pos = [0], [-1] * _capacity(c), [-1] * e.numel()
        for pairs in order:
            for i, p in enumerate(pairs):
                pos[p] = offsets[-1] + i
                src[pos[p]] = p
            offsets.append(offsets[-1] + math.ceil(len(pairs) / c["align"]) * c["align"])
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        return {"offsets": i32(offsets), "pos": i32(pos).view(c["tokens"], c["top_k"]), "src": i32(src),
                "counts": i32([len(p) for p in order])}
    pair = s["src"].long()
    real = torch.nonzero(pair >= 0)[:, 0]
    if op in ("dispatch", "combine_bwd"):
        x = s["x"] if op == "dispatch" else s["dy"]
        v = torch.zeros(pair.numel(), c["cols"], dtype=torch.float64, device="cuda")
        if c["dtype"] == "codes":
            v[real] = x.view(F8[c["fmt"]][0]).double()[pair[real] // c["top_k"]]
            scales = torch.full_like(s["scales"], F8[c["fmt"]][1], dtype=torch.float64) / AMAX_FLOOR
            scales[real] = s["sx"].double()[pair[real] // c["top_k"]]
            return {"q": v, "scales": scales}
        v[real] = x.double()[pair[real] // c["top_k"]]
        if op == "dispatch":
            return _scaled_both(v, c)
        dots = torch.zeros(c["tokens"] * c["top_k"], dtype=torch.float64, device="cuda")
        dots[pair[real]] = torch.einsum("rd,rd->r", v[real], s["rows"][real].double())
        v[real] *= s["weights"].double().reshape(-1)[pair[real], None]
        return dict(_scaled_both(v, c), dweights=dots.view(c["tokens"], c["top_k"]))
    if op == "combine":
        y = torch.zeros(c["tokens"], c["cols"], dtype=torch.float64, device="cuda")
        if s["residual"] is not None:
            y += s["residual"].double()
        y.index_add_(0, pair[real] // c["top_k"],
                     s["weights"].double().reshape(-1)[pair[real], None] * s["rows"][real].double())
        return y
    ty = torch.float8_e4m3fn
    wide = lambda v, by: v.double().repeat_interleave(by, dim=0).repeat_interleave(128, dim=1)  # noqa: E731
    spans = [(e, slice(lo, hi)) for e, (lo, hi) in enumerate(zip(s["bounds"], s["bounds"][1:])) if hi > lo]
    if op == "wgrad":
        dw = torch.zeros(s["dw"].shape, dtype=torch.float64, device="cuda")
        for e, r in spans:
            blocks = slice(r.start // 128, r.stop // 128)
            dw[e] = torch.einsum("nr,kr->nk", s["at"][:, r].view(ty).double() / wide(s["sat"][:, blocks], 1),
                                 s["bt"][:, r].view(ty).double() / wide(s["sbt"][:, blocks], 1))
        return dw
    n = s["b"].shape[1]
    y = torch.zeros(pair.numel(), n, dtype=torch.float64, device="cuda")
    for e, r in spans:
        y[r] = torch.mm(s["a"][r].view(ty).double() / wide(s["sa"][r], 1), (s["b"][e].view(ty).double() / wide(s["sb"][e], 128)).T)
    if op == "gemm":
        return y
    g, u = y[:, :c["f"]], y[:, c["f"]:]
    p = g if c["act"] == "silu" else math.sqrt(8.0 / math.pi) * (g + 0.044715 * g ** 3)
    out = dict(zip(("q", "scales"), _scaled(g * torch.special.expit(p) * u, c["fmt"])))
    return dict(out, gu=y) if c["train"] else out
