"""What a run cannot show of the feed-forward kernels is read from their source (no GPU needed)."""
import os
import re

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
