"""What a run cannot show of the feed-forward kernels is read from their source (no GPU needed)."""
import math
import os
import re

import numpy as np

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fine_grained_block_b200", "csrc")


def test_norm_reads_what_it_may_overwrite_with_coherent_loads():
    """h may be x or residual and dx may be dy or dh, while non-coherent loads (__ldg, ld.global.nc) are defined for memory
    only that nobody writes during the kernel: they are left to the weight, rstd, the backward pass's h and the partial sums."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "rmsnorm.cu")).read())
    assert ".nc" not in text
    loads = set(re.findall(r"(?:ld_words_stream|__ldg)\(\s*((?:static_cast<[^>]*>\()?[\w.]+)", text))
    assert loads <= {"h", "p.rstd", "static_cast<const uint16_t*>(w", "static_cast<const float*>(w"}, loads
    forward = text[:text.index("k_rmsnorm_backward")]
    assert "ld_words_stream(h" not in forward


def test_rounding_of_the_activations_exponent():
    """t = -p log2(e) as gated_act.cuh forms it, in fp32: 2^t is off by ln 2 times t's absolute error, which the comment
    there bounds by 1.3 (SiLU) and 4 (GELU) |p| 2^-24.  (A product in 64 bits stands for the fused one's exact part.)"""
    text = open(os.path.join(CSRC, "gated_act.cuh")).read()
    f = np.float32
    log2e, c, a = (f(re.search(name + r" = ([\d.]+)f;", text).group(1)) for name in ("kLog2e", "kGeluC", "kGeluA"))
    rng = np.random.default_rng(1)
    g = np.concatenate([rng.uniform(-12, 12, 300000), np.exp(rng.uniform(-20, 3, 300000))]).astype(f)
    x = g.astype(np.float64)
    exact = {"silu": x, "gelu": 2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)}
    c1, c0 = f(f(-log2e * c) * a), f(-log2e * c)
    inner = ((g * g).astype(np.float64) * np.float64(c1) + np.float64(c0)).astype(f)
    for name, t, units in (("silu", g * -log2e, 1.3), ("gelu", g * inner, 4.0)):
        err = np.abs(t.astype(np.float64) * math.log(2) + exact[name])
        assert bool((err <= units * 2.0 ** -24 * np.abs(exact[name])).all()), name
