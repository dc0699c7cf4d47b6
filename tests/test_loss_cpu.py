"""The cross entropy of a linear layer's outputs on the host: calls that are
refused before anything is enqueued, workspaces, and the reference's gradients
against differences."""
import ctypes

import pytest
import torch

import gated_deltanet_linear_03_amd as gdn
from train_helpers import loss64, loss_backward64

FAKE = 0x10000            # never dereferenced
FAR = 1 << 36
WS, NWS = FAKE + 20 * FAR, 1 << 34


def _io(**kw):
    io = gdn.CLossIO()
    io.M, io.V, io.K = 100, 72, 64
    io.x, io.w, io.bias, io.targets, io.loss, io.lse, io.status = (FAKE + i * FAR for i in range(1, 8))
    io.target_bytes, io.ignore_index = 8, -100
    for k, v in kw.items():
        setattr(io, k, v)
    return io


def _grad(**kw):
    gr = gdn.CLossGrad()
    gr.dloss, gr.dx, gr.dw, gr.dbias = (FAKE + i * FAR for i in range(8, 12))
    for k, v in kw.items():
        setattr(gr, k, v)
    return gr


BOTH = [
    (dict(M=-1), "M, N, K"), (dict(K=60), "multiple of 8"), (dict(K=0), "K (0)"), (dict(V=0), "V (0)"), (dict(V=1 << 31), "M, N, K"),
    (dict(M=1 << 26), "too large"), (dict(M=1 << 20, V=1 << 20), "too large"), (dict(target_bytes=2), "target_bytes"),
    (dict(label_smoothing=1.0), "label_smoothing"), (dict(label_smoothing=-0.1), "label_smoothing"), (dict(z_loss=-1.0), "z_loss"),
    (dict(z_loss=float("nan")), "z_loss"), (dict(x=None), "x is NULL"), (dict(w=None), "w is NULL"), (dict(targets=None), "targets"),
    (dict(targets=FAKE + 4 * FAR + 4), "targets"), (dict(x=FAKE + FAR + 8), "16-byte"), (dict(w_stride=68), "multiple of 8"),
    (dict(x_stride=56), "x_stride"), (dict(bias=FAKE + 2), "bias"), (dict(lse=FAKE + 2), "lse"),
]


@pytest.mark.parametrize("change, word", BOTH + [
    (dict(loss=FAKE + 1), "loss"), (dict(status=FAKE + 1), "status"), (dict(loss=FAKE + 6 * FAR + 396), "overlaps"),
    (dict(lse=FAKE + FAR), "overlaps"), (dict(loss=FAKE + 4 * FAR), "overlaps"), (dict(status=FAKE + 5 * FAR), "overlaps"),
    (dict(lse=WS), "overlaps"),
])
def test_forward_refuses(change, word):
    st = gdn.lib().gdn_linear_cross_entropy(ctypes.byref(_io(**change)), WS, NWS, None)
    assert st == gdn.GDN_ERR_INVALID_ARGUMENT and word in gdn.lib().gdn_last_error().decode()


@pytest.mark.parametrize("change, word", BOTH + [(dict(lse=None), "lse"), (dict(V=1 << 28, M=1, K=4096), "too large")])
def test_backward_refuses(change, word):
    st = gdn.lib().gdn_linear_cross_entropy_backward(ctypes.byref(_io(**change)), ctypes.byref(_grad()), WS, NWS, None)
    assert st == gdn.GDN_ERR_INVALID_ARGUMENT and word in gdn.lib().gdn_last_error().decode()


@pytest.mark.parametrize("change, word", [
    (dict(dloss=None), "dloss"), (dict(dloss=FAKE + 2), "dloss"), (dict(dx=FAKE + 9 * FAR + 1), "element aligned"),
    (dict(dx_stride=63), "dx_stride"), (dict(dw_stride=8), "dw_stride"), (dict(dbias=FAKE + 2), "dbias"),
    (dict(dx=FAKE + FAR), "overlaps"), (dict(dw=FAKE + 2 * FAR), "overlaps"), (dict(dbias=FAKE + 3 * FAR), "overlaps"),
    (dict(dbias=FAKE + 8 * FAR), "overlaps"), (dict(dw=WS + 1024), "overlaps"), (dict(dx=FAKE + 10 * FAR), "overlaps"),
])
def test_gradient_refuses(change, word):
    st = gdn.lib().gdn_linear_cross_entropy_backward(ctypes.byref(_io()), ctypes.byref(_grad(**change)), WS, NWS, None)
    assert st == gdn.GDN_ERR_INVALID_ARGUMENT and word in gdn.lib().gdn_last_error().decode()


def test_workspaces():
    L = gdn.lib()
    for name, call in (("gdn_linear_cross_entropy", lambda ws, n: L.gdn_linear_cross_entropy(ctypes.byref(_io()), ws, n, None)),
                       ("gdn_linear_cross_entropy_backward",
                        lambda ws, n: L.gdn_linear_cross_entropy_backward(ctypes.byref(_io()), ctypes.byref(_grad()), ws, n, None))):
        size = getattr(L, name + "_workspace_bytes")
        need = size(100, 72, 64)
        assert need > 0 and need % 256 == 0 and size(0, 72, 64) == 256
        assert size(1, 1, 3) == 0 and L.gdn_last_error()
        for ws, n in ((None, NWS), (WS + 8, NWS), (WS, need - 1)):
            assert call(ws, n) == gdn.GDN_ERR_WORKSPACE
    # nothing of the size rows x vocabulary
    assert L.gdn_linear_cross_entropy_workspace_bytes(4096, 248320, 2048) < 4096 * 248320 // 16
    assert L.gdn_linear_cross_entropy_backward_workspace_bytes(4096, 248320, 2048) < 4096 * 248320 // 4


def test_no_calls():
    L = gdn.lib()
    assert L.gdn_linear_cross_entropy(ctypes.byref(_io(M=0, x=None, w=None, targets=None)), None, 0, None) == gdn.GDN_OK
    assert L.gdn_linear_cross_entropy(ctypes.byref(_io(loss=None, lse=None)), None, 0, None) == gdn.GDN_OK
    assert L.gdn_linear_cross_entropy(None, None, 0, None) == gdn.GDN_ERR_INVALID_ARGUMENT
    none = _grad(dx=None, dw=None, dbias=None)
    assert L.gdn_linear_cross_entropy_backward(ctypes.byref(_io()), ctypes.byref(none), None, 0, None) == gdn.GDN_OK
    assert L.gdn_linear_cross_entropy_backward(ctypes.byref(_io()), None, WS, NWS, None) == gdn.GDN_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("smooth, z", [(0.0, 0.0), (0.1, 0.01)])
def test_reference_gradients(smooth, z):
    """Central differences of 1e-5: off by about 1e-9."""
    g = torch.Generator().manual_seed(5)
    M, V, K = 5, 7, 8
    x, w, b = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((M, K), (V, K), (V,)))
    t = torch.tensor([0, 6, -100, 3, 9])
    dloss = torch.randn(M, generator=g, dtype=torch.float64)
    loss, lse = loss64(x, w, b, t, smooth, z)[:2]
    assert float(loss[2]) == 0 and bool(loss[4].isnan()) and bool(loss[[0, 1, 3]].isfinite().all())
    grads, _ = loss_backward64(dloss, x, w, b, t, lse, smooth, z)

    def total(x, w, b):
        return float((loss64(x, w, b, t, smooth, z)[0] * dloss).nan_to_num(0.0).sum())

    h = 1e-5
    for k, (p, grad) in enumerate(zip((x, w, b), grads)):
        for i in range(p.numel()):
            e = torch.zeros(p.numel(), dtype=torch.float64)
            e[i] = h
            args = [x, w, b]
            args[k] = p + e.view(p.shape)
            up = total(*args)
            args[k] = p - e.view(p.shape)
            assert abs((up - total(*args)) / (2 * h) - float(grad.reshape(-1)[i])) < 1e-7
