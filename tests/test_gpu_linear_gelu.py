"""gelu far out on the left: its values are small there, but a bf16 output has
the range to hold them, and they have to be as good as its rounding."""
import math

import pytest
import torch

import gated_deltanet_linear_03_amd as gdn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M", [1, 40, 300])
def test_left_tail_keeps_its_relative_precision(M, dtype):
    """x w^T = 0, so the bias is the pre-activation, exactly.  The value p
    Phi(p) is off by 9e-4 of itself (outputs in bf16: what the polynomial is
    good for) or 2^-16 (fp32: p^2 log2(e) / 2 up to 120 rounds to 2^-18, times
    ln 2, in the argument of 2^x), then it is rounded.  Past |p| = 12.9 Phi is
    below 2^-126: next to nothing."""
    p = torch.cat([-torch.linspace(0.01, 14, 3001), torch.tensor([-20.0, -1e3, -1e30]), torch.linspace(0, 14, 997)]).cuda()
    N = p.numel()
    x = torch.zeros((M, 8), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((N, 8), dtype=torch.bfloat16, device="cuda")
    y = gdn.linear(x, w, bias=p, act=gdn.GDN_ACT_GELU, out_dtype=dtype).double()
    q = p.double()
    want = q * 0.5 * torch.erfc(-q / math.sqrt(2))
    rel, half = (9e-4, 2.0 ** -8) if dtype == torch.bfloat16 else (2.0 ** -16, 2.0 ** -24)
    lim = want.abs() * (rel + half * (1 + rel) + 2.0 ** -22) + 14 * 2.0 ** -126
    bad = ~((y - want).abs() <= lim)
    assert not bad.any(), (int(bad.sum()), p[bad.any(0)][:5].tolist(), float(((y - want).abs() / lim).max()))
    assert (y == y[:1]).all()
