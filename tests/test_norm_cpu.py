"""The norms on the host: calls that are refused before anything is enqueued,
and the reference's gradients against differences."""
import ctypes

import pytest
import torch

import gated_deltanet_linear_03_amd as gdn
from train_helpers import norm64, norm_backward64

FAKE = 0x10000            # never dereferenced
FAR = 1 << 36
WS, NWS = FAKE + 20 * FAR, 1 << 34


def _io(**kw):
    io = gdn.CNormIO()
    io.M, io.D, io.eps = 100, 72, 1e-5
    io.x, io.weight, io.bias, io.y, io.stats = (FAKE + i * FAR for i in range(1, 6))
    io.x_dtype, io.y_dtype = gdn.GDN_DTYPE_FP32, gdn.GDN_DTYPE_BF16
    for k, v in kw.items():
        setattr(io, k, v)
    return io


@pytest.mark.parametrize("change, word", [
    (dict(M=-1), "M (-1)"), (dict(M=1 << 31), "M ("), (dict(D=0), "D (0)"), (dict(D=(1 << 22) + 1), "D ("),
    (dict(kind=2), "kind"), (dict(x_dtype=2), "x_dtype"), (dict(y_dtype=-1), "y_dtype"), (dict(eps=-1.0), "eps"),
    (dict(eps=float("nan")), "eps"), (dict(x=None), "x is NULL"), (dict(y=None), "y is NULL"),
    (dict(x=FAKE + FAR + 2), "element aligned"), (dict(y=FAKE + 4 * FAR + 1), "element aligned"),
    (dict(x_stride=71), "x_stride"), (dict(y_stride=8), "y_stride"), (dict(weight=FAKE + 2), "weight"),
    (dict(bias=FAKE + 1), "bias"), (dict(stats=FAKE + 3), "stats"), (dict(y=FAKE + FAR), "overlaps"),
    (dict(y=FAKE + FAR + 4 * 7199), "overlaps"), (dict(stats=FAKE + 4 * FAR + 14000), "overlaps"),
    (dict(stats=FAKE + 2 * FAR), "overlaps"),
])
def test_norm_refuses(change, word):
    assert gdn.lib().gdn_norm(ctypes.byref(_io(**change)), None) == gdn.GDN_ERR_INVALID_ARGUMENT
    assert word in gdn.lib().gdn_last_error().decode()


def test_no_rows_are_no_call():
    assert gdn.lib().gdn_norm(ctypes.byref(_io(M=0, x=None, y=None)), None) == gdn.GDN_OK
    assert gdn.lib().gdn_norm(None, None) == gdn.GDN_ERR_INVALID_ARGUMENT


def _grad(**kw):
    gr = gdn.CNormGrad()
    gr.M, gr.D = 100, 72
    gr.dy, gr.x, gr.weight, gr.stats, gr.d_residual, gr.dx, gr.dweight, gr.dbias = (FAKE + i * FAR for i in range(1, 9))
    gr.x_dtype, gr.dy_dtype = gdn.GDN_DTYPE_FP32, gdn.GDN_DTYPE_BF16
    for k, v in kw.items():
        setattr(gr, k, v)
    return gr


@pytest.mark.parametrize("change, word", [
    (dict(M=-2), "M (-2)"), (dict(D=0), "D (0)"), (dict(kind=-1), "kind"), (dict(x_dtype=5), "x_dtype"),
    (dict(dy_dtype=5), "dy_dtype"), (dict(dy=None), "dy is NULL"), (dict(x=None), "x is NULL"),
    (dict(stats=None), "stats is NULL"), (dict(dx=FAKE + 6 * FAR + 2), "element aligned"),
    (dict(dx_stride=71), "dx_stride"), (dict(dy_stride=71), "dy_stride"), (dict(d_residual_stride=71), "d_residual_stride"),
    (dict(dweight=FAKE + 2), "dweight"), (dict(dbias=FAKE + 2), "dbias"), (dict(dx=FAKE + 2 * FAR), "overlaps"),
    (dict(dx=FAKE + FAR), "overlaps"), (dict(dx=FAKE + 5 * FAR + 4), "overlaps"),
    (dict(dx=FAKE + 5 * FAR, dx_stride=73), "overlaps"), (dict(dweight=FAKE + 8 * FAR), "overlaps"),
    (dict(dbias=WS), "overlaps"), (dict(dweight=FAKE + 4 * FAR), "overlaps"),
])
def test_backward_refuses(change, word):
    st = gdn.lib().gdn_norm_backward(ctypes.byref(_grad(**change)), WS, NWS, None)
    assert st == gdn.GDN_ERR_INVALID_ARGUMENT
    assert word in gdn.lib().gdn_last_error().decode()


def test_backward_workspace():
    L = gdn.lib()
    need = L.gdn_norm_backward_workspace_bytes(100, 72)
    assert need >= 8 * 72 and need % 256 == 0
    assert L.gdn_norm_backward_workspace_bytes(0, 72) == 256
    assert L.gdn_norm_backward_workspace_bytes(5, 0) == 0 and L.gdn_last_error()
    for ws, n in ((None, NWS), (WS + 8, NWS), (WS, need - 1)):
        assert L.gdn_norm_backward(ctypes.byref(_grad()), ws, n, None) == gdn.GDN_ERR_WORKSPACE
    assert L.gdn_norm_backward(None, WS, NWS, None) == gdn.GDN_ERR_INVALID_ARGUMENT
    assert L.gdn_norm_backward(ctypes.byref(_grad(dx=None, dweight=None, dbias=None)), None, 0, None) == gdn.GDN_OK


@pytest.mark.parametrize("layer", [True, False])
def test_reference_gradients(layer):
    """Differences of the definition: central, of 1e-5, so off by about 1e-9 of the third derivative."""
    g = torch.Generator().manual_seed(3)
    M, D, eps = 4, 11, 1e-2
    x, w, b, dy = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((M, D), (D,), (D,), (M, D)))
    y, mean, rstd = norm64(x, w, b, layer, eps)
    (dx, dw, db), _ = norm_backward64(dy, x, w, mean, rstd, layer, None)

    def loss(x, w, b):
        return float((norm64(x, w, b, layer, eps)[0] * dy).sum())

    h = 1e-5
    for t, grad, at in ((x, dx, 0), (w, dw, 1), (b, db, 2)):
        for i in range(t.numel()):
            e = torch.zeros_like(t).view(-1)
            e[i] = h
            e = e.view(t.shape)
            args = [x, w, b]
            args[at] = t + e
            up = loss(*args)
            args[at] = t - e
            assert abs((up - loss(*args)) / (2 * h) - float(grad.reshape(-1)[i])) < 1e-7
