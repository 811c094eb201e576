"""The bounds with which the smoke run compares the feed-forward operators tell a right result from a wrong one (no GPU
needed: the results are made here, the mistakes are in the expected values)."""
import pytest
import torch

import __graft_entry__ as entry


def quantize(v):
    s = 448.0 / v.float().abs().view(v.shape[0], -1, 128).amax(2).clamp_min(1e-12)
    q = (v.float() * s.repeat_interleave(128, 1)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(torch.uint8), s


@pytest.fixture(scope="module")
def gated():
    """H and its parts for values as the smoke run has them: most of H lies far below its largest element."""
    torch.manual_seed(3)
    g, u = torch.randn(384, 2432).double() * 1.5, torch.randn(384, 2432).double() * 1.5
    return g, u, g * torch.sigmoid(g) * u


def test_right_codes_pass(gated):
    H = gated[2]
    q, s = quantize(H)
    entry.codes_close(q, s, H, 2.0 ** -20 * H.abs(), "H")
    entry.close(H.to(torch.bfloat16), H, 2.0 ** -20 * H.abs(), "H")


@pytest.mark.parametrize("mistake", ["gelu", "no activation", "one element", "small elements zero", "block scale"])
def test_wrong_codes_do_not(gated, mistake):
    g, u, H = gated
    q, s = quantize(H)
    if mistake == "gelu":
        want = torch.nn.functional.gelu(g, approximate="tanh") * u
    elif mistake == "no activation":
        want = g * u
    elif mistake == "one element":
        want = H.clone()
        want[17, 1000] += 0.25 * want[17, 1000].abs() + 0.05
    elif mistake == "small elements zero":
        want = torch.where(H.abs() <= 0.06 * H.abs().max(), 0.0, H)
    else:
        want = H
        s = s.clone()
        s[5, 3] *= 1.5
    with pytest.raises(AssertionError, match="smoke"):
        entry.codes_close(q, s, want, 2.0 ** -20 * want.abs(), "H")
    if mistake != "block scale":
        with pytest.raises(AssertionError, match="smoke"):
            entry.close(H.to(torch.bfloat16), want, 2.0 ** -20 * want.abs(), "H")
