"""The operators of a feed-forward block in FP8, as they are measured: what each case stands for, its inputs, its plain
form in elementary torch operations, and the calls that a program makes of the library.

Four operators, of two kinds: the root-mean-square norm with the residual's addition and an FP8 output (forward and
backward), and the gated feed-forward product (both projections, activation and product; and its backward pass).

With ``own`` false, ``run`` computes the plain form in fp32; with ``own`` true it calls the library.  Codes are returned
as float8 tensors, the values that they stand for, beside their scales.
"""
import math

import torch

own = False

EPS = 1e-6
AMAX_FLOOR = 1e-12
F8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# -- cases ------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one token of a decode step enters the feed-forward block: latency
        dict(name="norm one token", op="norm", rows=1, cols=4096, dtype="bf16", fmt="e4m3", residual=True, train=False),
        # a training step's activations, the widest rows of this repository's workloads
        dict(name="norm training", op="norm", rows=16384, cols=7168, dtype="bf16", fmt="e4m3", residual=True, train=True),
        # a ragged width in fp32 without a residual (the first norm of a stack)
        dict(name="norm ragged f32", op="norm", rows=1000, cols=4100, dtype="f32", fmt="e5m2", residual=False, train=True),
        # the same training step's backward pass, with the residual stream's gradient
        dict(name="norm backward training", op="norm_bwd", rows=16384, cols=7168, dtype="bf16", residual=True),
        # a ragged width in fp32
        dict(name="norm backward ragged f32", op="norm_bwd", rows=1000, cols=4100, dtype="f32", residual=False),
        # decode: one token against both projections, bound by reading the weights
        dict(name="gate/up one token", op="gemm", m=1, k=7168, f=4096, act="silu", fmt="e4m3", train=False),
        # a decode batch
        dict(name="gate/up 48 tokens", op="gemm", m=48, k=4096, f=8192, act="silu", fmt="e4m3", train=False),
        # a prompt of odd length
        dict(name="gate/up prompt 1000", op="gemm", m=1000, k=4096, f=4096, act="gelu", fmt="e4m3", train=False),
        # a training step: the projections are kept for the backward pass
        dict(name="gate/up training", op="gemm", m=16384, k=7168, f=4096, act="silu", fmt="e4m3", train=True),
        # its backward pass: codes for the data gradient and both weight gradients
        dict(name="gated backward training", op="gated_bwd", m=16384, f=4096, dtype="bf16", act="silu", fmt="e4m3", train=True),
        # odd token count, fp32, gradients in the wide-range format
        dict(name="gated backward odd f32", op="gated_bwd", m=1000, f=2048, dtype="f32", act="gelu", fmt="e5m2", train=True),
        # a short batch whose weights are frozen: only the data gradient's codes
        dict(name="gated backward frozen", op="gated_bwd", m=200, f=4096, dtype="bf16", act="silu", fmt="e4m3", train=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "gemm", "gemm", "gated_bwd"])
    if op in ("norm", "norm_bwd"):
        cols = _log(rng, 64, 7168)
        if rng.random() < 0.7:
            cols = max(64, cols // 16 * 16)
        c = dict(op=op, rows=_log(rng, 1, 16384), cols=cols, dtype=rng.choice(["bf16", "bf16", "f32"]),
                 residual=rng.random() < 0.6)
        if c["dtype"] == "f32":
            c["rows"] = max(1, c["rows"] // 2)
        if op == "norm":
            c.update(fmt=rng.choice(["e4m3", "e4m3", "e5m2"]), train=rng.random() < 0.5)
        return c
    if op == "gemm":
        return dict(op=op, m=_log(rng, 1, 16384), k=128 * _log(rng, 2, 56), f=128 * _log(rng, 2, 32),
                    act=rng.choice(["silu", "gelu"]), fmt=rng.choice(["e4m3", "e4m3", "e5m2"]), train=rng.random() < 0.5)
    # a training batch comes in whole runs of 16 tokens; without weight gradients any count
    c = dict(op=op, m=_log(rng, 1, 16384), f=128 * _log(rng, 1, 32), dtype=rng.choice(["bf16", "bf16", "f32"]),
             act=rng.choice(["silu", "gelu"]), fmt=rng.choice(["e4m3", "e5m2"]), train=rng.random() < 0.7)
    if c["dtype"] == "f32":
        c["m"] = max(1, c["m"] // 2)
    if c["train"]:
        c["m"] = max(16, c["m"] // 16 * 16)
    return c


def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        r, c, e = case["rows"], case["cols"], 2 if case["dtype"] == "bf16" else 4
        if op == "norm":
            b = r * c * (e + 1) + 4 * r * math.ceil(c / 128) + c * e
            b += 2 * r * c * e if case["residual"] else 0
            b += (r * c * e + 4 * r) if case["train"] else 0
            return {"bytes": b, "flops": 8 * r * c}
        b = r * c * e * (4 if case["residual"] else 3) + 4 * r + c * (e + 4)
        return {"bytes": b, "flops": 10 * r * c}
    m, f = case["m"], case["f"]
    if op == "gemm":
        k = case["k"]
        b = m * k + 4 * m * (k // 128) + 2 * f * k + 4 * (2 * f // 128) * (k // 128) + m * f + 4 * m * (f // 128)
        b += 2 * m * 2 * f if case["train"] else 0
        return {"bytes": b, "flops": 2 * m * k * 2 * f}
    e, mt = 2 if case["dtype"] == "bf16" else 4, -(-m // 128) * 128
    b = 3 * m * f * e + 2 * m * f + 4 * m * (2 * f // 128)
    b += (3 * mt * f + 4 * 3 * f * (mt // 128)) if case["train"] else 0
    return {"bytes": b, "flops": 30 * m * f}


# -- inputs -----------------------------------------------------------------------------------------------------------

def _codes(x, block_rows, fmt):
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

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    def empty(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda")

    s = {"case": case}
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        r, c, dt = case["rows"], case["cols"], DT[case["dtype"]]
        x = normal(r, c)
        x[:, torch.randint(0, c, (8,), generator=g, device="cuda")] *= 20.0  # a few outlier channels
        s["weight"] = (1.0 + normal(c, std=0.1)).to(dt)
        if op == "norm":
            s["x"] = x.to(dt)
            s["residual"] = normal(r, c, std=2.0).to(dt) if case["residual"] else None
            s["q"], s["scales"] = empty(r, c, dtype=torch.uint8), empty(r, -(-c // 128))
            s["h"] = empty(r, c, dtype=dt) if case["residual"] else None
            s["y"], s["rstd"] = (empty(r, c, dtype=dt), empty(r)) if case["train"] else (None, None)
        else:
            s["h"] = x.to(dt)
            s["rstd"] = torch.rsqrt(s["h"].float().square().mean(dim=1) + EPS)
            s["dy"] = normal(r, c, std=1e-3).to(dt)
            s["dh"] = normal(r, c, std=1e-3).to(dt) if case["residual"] else None
            s["dx"], s["dweight"] = empty(r, c, dtype=dt), empty(c)
    elif op == "gemm":
        m, k, f = case["m"], case["k"], case["f"]
        s["a"], s["sa"] = _codes(normal(m, k), 1, "e4m3")
        s["b"], s["sb"] = _codes(normal(2 * f, k, std=0.02), 128, "e4m3")
        s["q"], s["scales"] = empty(m, f, dtype=torch.uint8), empty(m, f // 128)
        s["gu"] = empty(m, 2 * f, dtype=torch.bfloat16) if case["train"] else None
    else:
        m, f, dt = case["m"], case["f"], DT[case["dtype"]]
        mt = -(-m // 128) * 128
        s["gu"] = normal(m, 2 * f, std=1.5).to(dt)
        s["dh"] = normal(m, f, std=1e-3).to(dt)
        s["q"], s["scales"] = empty(m, 2 * f, dtype=torch.uint8), empty(m, 2 * f // 128)
        if case["train"]:
            s["qt"], s["scales_t"] = empty(2 * f, mt, dtype=torch.uint8), empty(2 * f, mt // 128)
            s["ht"], s["ht_scales"] = empty(f, mt, dtype=torch.uint8), empty(f, mt // 128)
        else:
            s["qt"] = s["scales_t"] = s["ht"] = s["ht_scales"] = None
    return s


# -- one pass ---------------------------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "norm_bwd": _own_norm_bwd, "gemm": _own_gemm, "gated_bwd": _own_gated_bwd}[op](state)
    return {"norm": _norm, "norm_bwd": _norm_bwd, "gemm": _gemm, "gated_bwd": _gated_bwd}[op](state)


def _own_norm(s):
    from fine_grained_block_b200 import binding as B
    c = s["case"]
    fmt = B.E4M3 if c["fmt"] == "e4m3" else B.E5M2
    q, scales, h, y, rstd = B.fp8q_rmsnorm_quantize(s["x"], s["weight"], residual=s["residual"], eps=EPS, fmt=fmt, q=s["q"],
                                                    scales=s["scales"], h=s["h"], y=s["y"], rstd=s["rstd"])
    out = {"q": q.view(F8[c["fmt"]][0]), "scales": scales}
    if c["residual"]:
        out["h"] = h
    if c["train"]:
        out["y"], out["rstd"] = y, rstd
    return out


def _own_norm_bwd(s):
    from fine_grained_block_b200 import binding as B
    dx, dw = B.fp8q_rmsnorm_backward(s["dy"], s["h"], s["rstd"], s["weight"], dh=s["dh"], dx=s["dx"], dweight=s["dweight"])
    return {"dx": dx, "dweight": dw}


def _own_gemm(s):
    from fine_grained_block_b200 import binding as B
    c = s["case"]
    q, scales, gu = B.fp8q_gemm_gated(s["a"], s["sa"], s["b"], s["sb"], act=B.ACT_SILU if c["act"] == "silu" else B.ACT_GELU_TANH,
                                      fmt=B.E4M3 if c["fmt"] == "e4m3" else B.E5M2, q=s["q"], scales=s["scales"], gu=s["gu"])
    out = {"q": q.view(F8[c["fmt"]][0]), "scales": scales}
    if c["train"]:
        out["gu"] = gu
    return out


def _own_gated_bwd(s):
    from fine_grained_block_b200 import binding as B
    c = s["case"]
    ty = F8[c["fmt"]][0]
    q, scales, qt, scales_t, ht, ht_scales = B.fp8q_gated_backward(
        s["gu"], s["dh"], act=B.ACT_SILU if c["act"] == "silu" else B.ACT_GELU_TANH, fmt=B.E4M3 if c["fmt"] == "e4m3" else B.E5M2,
        transposed=c["train"], q=s["q"], scales=s["scales"], qt=s["qt"], scales_t=s["scales_t"], ht=s["ht"],
        ht_scales=s["ht_scales"])
    out = {"q": q.view(ty), "scales": scales}
    if c["train"]:
        out.update(qt=qt.view(ty), scales_t=scales_t, ht=ht.view(ty), ht_scales=ht_scales)
    return out


# -- plain forms ------------------------------------------------------------------------------------------------------

def _quantize(v, fmt):
    """fp32 [R, C] in blocks of 1x128 (the last of a row may be short): float8 codes and fp32 scales."""
    ty, top = F8[fmt]
    R, C = v.shape
    pad = -C % 128
    w = torch.nn.functional.pad(v, (0, pad)) if pad else v
    w = w.view(R, -1, 128)
    s = top / w.abs().amax(dim=2).clamp_min(AMAX_FLOOR)
    q = (w * s[:, :, None]).clamp(-top, top).view(R, C + pad)[:, :C].to(ty).contiguous()
    return q, s


def _act(g, kind):
    """act(g) = g * sigmoid(p(g)) and its derivative, fp32.  The tanh GELU is this with p = 2c(g + 0.044715 g^3): written with
    tanh it loses its small values to cancellation."""
    if kind == "silu":
        p, slope = g, 1.0
    else:
        c = 2.0 * math.sqrt(2.0 / math.pi)
        p, slope = c * (g + 0.044715 * g * g * g), c * (1.0 + 3.0 * 0.044715 * g * g)
    sg = 1.0 / (1.0 + torch.exp(-p))
    return g * sg, sg + g * sg * (1.0 - sg) * slope


def _norm(s):
    c = s["case"]
    dt = s["x"].dtype
    h = (s["x"].float() + s["residual"].float()).to(dt) if c["residual"] else s["x"]
    hf = h.float()
    rstd = 1.0 / torch.sqrt((hf * hf).mean(dim=1) + EPS)
    y = hf * rstd[:, None] * s["weight"].float()
    q, scales = _quantize(y, c["fmt"])
    out = {"q": q, "scales": scales}
    if c["residual"]:
        out["h"] = h
    if c["train"]:
        out["y"], out["rstd"] = y.to(dt), rstd
    return out


def _norm_bwd(s):
    dt = s["dy"].dtype
    n = s["h"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    a = dy * s["weight"].float()
    dx = s["rstd"][:, None] * (a - n * (a * n).mean(dim=1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(dt), "dweight": (dy * n).sum(dim=0)}


def _gemm(s):
    c = s["case"]
    ty = torch.float8_e4m3fn
    m, k = s["a"].shape
    f2 = s["b"].shape[0]
    a = (s["a"].view(ty).float().view(m, -1, 128) / s["sa"][:, :, None]).view(m, k)
    b = (s["b"].view(ty).float().view(f2 // 128, 128, k // 128, 128) / s["sb"][:, None, :, None]).view(f2, k)
    gu = a @ b.t()
    g, u = gu.chunk(2, dim=1)
    q, scales = _quantize(_act(g, c["act"])[0] * u, c["fmt"])
    out = {"q": q, "scales": scales}
    if c["train"]:
        out["gu"] = gu.to(torch.bfloat16)
    return out


def _gated_bwd(s):
    c = s["case"]
    g, u = s["gu"].float().chunk(2, dim=1)
    dh = s["dh"].float()
    act, dact = _act(g, c["act"])
    d = torch.cat([dh * u * dact, dh * act], dim=1)
    q, scales = _quantize(d, c["fmt"])
    out = {"q": q, "scales": scales}
    if c["train"]:
        pad = -c["m"] % 128
        out["qt"], out["scales_t"] = _quantize(torch.nn.functional.pad(d, (0, 0, 0, pad)).t().contiguous(), c["fmt"])
        out["ht"], out["ht_scales"] = _quantize(torch.nn.functional.pad(act * u, (0, 0, 0, pad)).t().contiguous(), c["fmt"])
    return out


# -- the definitions in 64 bits ---------------------------------------------------------------------------------------

def _scaled(v, fmt):
    """The numbers that the codes of v (fp64 [R, C]) stand for, before their rounding, and the scales.  No numbers for
    E5M2: its two bits put every code about 5 % off, as far as half of what a comparison of 8-bit values allows."""
    top = F8[fmt][1]
    R, C = v.shape
    nb = -(-C // 128)
    w = v.new_zeros(R, nb * 128)
    w[:, :C] = v
    s = top / torch.maximum(w.abs().reshape(R, nb, 128).max(dim=2).values, v.new_tensor(AMAX_FLOOR))
    return v * s.repeat_interleave(128, dim=1)[:, :C] if fmt == "e4m3" else None, s


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        dt = s["x"].dtype
        h = s["x"].double()
        if case["residual"]:
            h = (h + s["residual"].double()).to(dt).double()  # the sum is stored in the input's type, and that is normed
        rstd = (h.pow(2).sum(dim=1) / case["cols"] + EPS).pow(-0.5)
        y = torch.einsum("rc,r,c->rc", h, rstd, s["weight"].double())
        q, scales = _scaled(y, case["fmt"])
        out = {"q": q, "scales": scales}
        if case["residual"]:
            out["h"] = h
        if case["train"]:
            out["y"], out["rstd"] = y, rstd
        return out
    if op == "norm_bwd":
        h, r, dy, w = (s[n].double() for n in ("h", "rstd", "dy", "weight"))
        r = r[:, None]
        dot = (dy * w * h).sum(dim=1, keepdim=True)
        dx = r * dy * w - r.pow(3) * h * dot / case["cols"]
        if s["dh"] is not None:
            dx += s["dh"].double()
        return {"dx": dx, "dweight": torch.einsum("rc,rc,ri->c", dy, h, r)}
    sigma = lambda z: torch.special.expit(z)  # noqa: E731
    slope = lambda g: g if case["act"] == "silu" else math.sqrt(8.0 / math.pi) * (g + 0.044715 * g ** 3)  # noqa: E731
    if op == "gemm":
        ty = torch.float8_e4m3fn
        a = s["a"].view(ty).double() / s["sa"].double().repeat_interleave(128, dim=1)
        b = s["b"].view(ty).double() / s["sb"].double().repeat_interleave(128, dim=0).repeat_interleave(128, dim=1)
        gu = torch.mm(a, b.T)
        g, u = gu[:, :case["f"]], gu[:, case["f"]:]
        q, scales = _scaled(g * sigma(slope(g)) * u, case["fmt"])
        return {"q": q, "scales": scales, "gu": gu} if case["train"] else {"q": q, "scales": scales}
    g, u, dh = s["gu"][:, :case["f"]].double(), s["gu"][:, case["f"]:].double(), s["dh"].double()
    p = sigma(slope(g))
    grow = 1.0 if case["act"] == "silu" else math.sqrt(8.0 / math.pi) * (1.0 + 3.0 * 0.044715 * g ** 2)
    d = torch.cat([dh * u * (p + g * p * (1.0 - p) * grow), dh * g * p], dim=1)
    out = dict(zip(("q", "scales"), _scaled(d, case["fmt"])))
    if case["train"]:
        mt = -(-case["m"] // 128) * 128
        for v, names in ((d, ("qt", "scales_t")), (g * p * u, ("ht", "ht_scales"))):
            w = v.new_zeros(v.shape[1], mt)
            w[:, :case["m"]] = v.T
            out.update(zip(names, _scaled(w, case["fmt"])))
    return out
