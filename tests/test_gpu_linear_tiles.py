"""The linear layer's tile loops, each size in its steady state (several rounds
of the reduction, an odd and an even number of its 64-wide stages, a rest of 8)
and with every form of the epilogue, forward and backward, against 64 bits.
The sizes are chosen by their cost, so each test asserts which tiles it ran."""
import pytest
import torch

import gated_deltanet_linear_03_amd as gdn
from test_gpu_linear import ACTS, HALF, _gradients, close, data, reference

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
FORWARD = [
    # M, N, K, tiles, act, y, bias, residual, preact
    (4096, 4104, 328, (256, 256), "gelu", BF16, True, True, True),
    (4090, 4096, 712, (256, 256), "gelu", FP32, True, True, False),
    (4096, 4000, 576, (256, 256), "none", BF16, False, False, False),
    (3850, 4104, 640, (256, 256), "gelu_tanh", FP32, True, False, True),
    (4096, 1064, 584, (256, 128), "gelu", BF16, True, True, True),
    (2000, 2100, 712, (256, 128), "silu", FP32, False, True, True),
    (2048, 2056, 512, (256, 128), "relu", BF16, True, False, False),
    (1030, 2050, 520, (128, 128), "gelu", FP32, True, True, True),
    (1500, 1500, 712, (128, 128), "gelu_tanh", BF16, True, True, False),
    (300, 300, 1000, (64, 64), "gelu", BF16, True, True, True),
    (700, 500, 328, (64, 64), "silu", FP32, True, True, False),
]


@pytest.mark.parametrize("M, N, K, tiles, act, dt, bias, residual, preact", FORWARD,
                         ids=[f"{c[0]}x{c[1]}x{c[2]}-{c[4]}" for c in FORWARD])
def test_forward(M, N, K, tiles, act, dt, bias, residual, preact):
    assert gdn.linear_tiles(M, N, K) == tiles
    g, x, w = data(M, N, K, 31, pad=8)
    b = torch.randn(N, generator=g, device="cuda") if bias else None
    res = torch.randn((M, N + 3), generator=g, device="cuda").to(dt)[:, :N] if residual else None
    pre = torch.empty((M, N + 1), dtype=BF16, device="cuda")[:, :N] if preact else None
    y = gdn.linear(x, w, bias=b, act=ACTS[act], residual=res, out_dtype=dt, preact=pre)
    p, plim, want, lim = reference(x, w, b, act, res)
    close("y", y, want, lim + (want.abs() + lim) * HALF[dt] + 1e-37)
    if preact:
        close("preact", pre, p, plim + (p.abs() + plim) * HALF[BF16] + 1e-37)
    if residual:                                  # the output in the residual's place
        assert gdn.linear(x, w, bias=b, act=ACTS[act], residual=res, out=res) is res and torch.equal(res, y)


BACKWARD = [
    (4096, 4104, 1032, (256, 256), "gelu_tanh", BF16), (4090, 4000, 1096, (256, 256), "none", BF16),
    (2048, 2040, 1032, (256, 128), "silu", FP32), (2056, 2056, 1032, (256, 128), "relu", BF16),
    (1100, 1200, 1304, (128, 128), "gelu", FP32), (2000, 4100, 1032, (128, 128), "gelu", BF16),
]


@pytest.mark.parametrize("M, N, K, tiles, act, dt", BACKWARD, ids=[f"{c[0]}x{c[1]}x{c[2]}-{c[4]}" for c in BACKWARD])
def test_backward(M, N, K, tiles, act, dt):
    assert gdn.linear_tiles(M, N, K, backward=True) == tiles
    g, x, w = data(M, N, K, 32)
    dy = torch.randn((M, N), generator=g, device="cuda").to(dt)
    pre = torch.randn((M, N), generator=g, device="cuda").to(BF16)
    r = gdn.linear_backward(dy, x, w, preact=None if act == "none" else pre, act=ACTS[act], want_dbias=True)
    _gradients(r, dy, x, w, pre, act)
