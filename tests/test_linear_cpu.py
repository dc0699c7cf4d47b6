"""The linear layer with its epilogue on the host: struct layouts, workspace
sizes and calls that are refused before anything is enqueued."""
import ctypes
import os
import shutil
import subprocess

import pytest

import gated_deltanet_linear_03_amd as gdn

FAKE = 0x10000            # never dereferenced
FAR = 1 << 36
WS, NWS = FAKE + 20 * FAR, 1 << 34


def _io(**kw):
    io = gdn.CLinearIO()
    io.M, io.N, io.K = 100, 72, 64
    io.x, io.w, io.bias, io.residual, io.y, io.preact = (FAKE + i * FAR for i in range(1, 7))
    io.act, io.y_dtype = gdn.GDN_ACT_SILU, gdn.GDN_DTYPE_BF16
    for k, v in kw.items():
        setattr(io, k, v)
    return io


@pytest.mark.parametrize("change, word", [
    (dict(K=63), "multiple of 8"), (dict(M=-1), "M, N, K"), (dict(N=1 << 31), "M, N, K"), (dict(act=5), "act"),
    (dict(act=-1), "act"), (dict(y_dtype=2), "y_dtype"), (dict(x=None), "x is NULL"), (dict(w=None), "w is NULL"),
    (dict(y=None), "y is NULL"), (dict(x=FAKE + FAR + 8), "16-byte"), (dict(x_stride=68), "multiple of 8"),
    (dict(w_stride=56), "w_stride"), (dict(y_stride=71), "y_stride"), (dict(residual_stride=8), "residual_stride"),
    (dict(preact_stride=8), "preact_stride"), (dict(bias=FAKE + 2), "bias"), (dict(y=FAKE + 5 * FAR + 1), "element aligned"),
    (dict(y=FAKE + FAR), "overlaps"), (dict(preact=FAKE + 5 * FAR), "overlaps"), (dict(residual=FAKE + 5 * FAR + 2), "overlaps"),
    (dict(residual=FAKE + 5 * FAR, residual_stride=80), "overlaps"), (dict(M=1 << 30, N=1 << 30), "too large"),
])
def test_linear_refuses(change, word):
    assert gdn.lib().gdn_linear(ctypes.byref(_io(**change)), WS, NWS, None) == gdn.GDN_ERR_INVALID_ARGUMENT
    assert word in gdn.lib().gdn_last_error().decode()


def test_empty_outputs_are_no_calls():
    for kw in (dict(M=0), dict(N=0)):
        assert gdn.lib().gdn_linear(ctypes.byref(_io(**kw)), None, 0, None) == gdn.GDN_OK
    assert gdn.lib().gdn_linear(None, None, 0, None) == gdn.GDN_ERR_INVALID_ARGUMENT


def test_forward_workspace():
    """Rows 17 .. 64 keep [parts][M][N] fp32 sums when K is at least 512, rows
    65 .. 256 when it is at least 2048 and N is small."""
    L = gdn.lib()
    for M, N, K in ((16, 2048, 4096), (257, 2048, 4096), (65, 12352, 4096), (256, 2048, 2040), (32, 2048, 504), (0, 64, 4096)):
        assert L.gdn_linear_workspace_bytes(M, N, K) == 0 and L.gdn_last_error() == b""
    need = L.gdn_linear_workspace_bytes(40, 72, 1024)
    assert need > 0 and need % 256 == 0 and need % (4 * 40 * 72) < 256
    need_some = L.gdn_linear_workspace_bytes(70, 72, 2048)
    assert need_some > 0 and need_some % (4 * 70 * 72) < 256
    assert L.gdn_linear_workspace_bytes(1, 1, 3) == 0 and L.gdn_last_error()
    for ws, n in ((None, NWS), (WS + 8, NWS), (WS, need - 1)):
        assert L.gdn_linear(ctypes.byref(_io(M=40, K=1024)), ws, n, None) == gdn.GDN_ERR_WORKSPACE
    assert L.gdn_linear(ctypes.byref(_io(M=40, K=1024)), FAKE + 5 * FAR, NWS, None) == gdn.GDN_ERR_INVALID_ARGUMENT
    assert b"workspace overlaps" in L.gdn_last_error()


def _grad(**kw):
    gr = gdn.CLinearGrad()
    gr.M, gr.N, gr.K = 100, 72, 64
    gr.dy, gr.x, gr.w, gr.preact, gr.dx, gr.dw, gr.dbias = (FAKE + i * FAR for i in range(1, 8))
    gr.dy_dtype, gr.act = gdn.GDN_DTYPE_BF16, gdn.GDN_ACT_GELU
    for k, v in kw.items():
        setattr(gr, k, v)
    return gr


@pytest.mark.parametrize("change, word", [
    (dict(K=60), "multiple of 8"), (dict(act=9), "act"), (dict(dy_dtype=3), "dy_dtype"), (dict(dy=None), "dy is NULL"),
    (dict(preact=None), "preact is NULL"), (dict(x=None), "x is NULL"), (dict(w=None), "w is NULL"),
    (dict(x=FAKE + 2 * FAR + 2), "16-byte"), (dict(w_stride=66), "multiple of 8"), (dict(dx_stride=63), "dx_stride"),
    (dict(dw_stride=8), "dw_stride"), (dict(dbias=FAKE + 1), "dbias"), (dict(dx=FAKE + FAR), "overlaps"),
    (dict(dw=FAKE + 5 * FAR + 64), "overlaps"), (dict(dbias=WS), "overlaps"),
])
def test_backward_refuses(change, word):
    st = gdn.lib().gdn_linear_backward(ctypes.byref(_grad(**change)), WS, NWS, None)
    assert st == gdn.GDN_ERR_INVALID_ARGUMENT
    assert word in gdn.lib().gdn_last_error().decode()


def test_backward_workspace():
    L = gdn.lib()
    need = L.gdn_linear_backward_workspace_bytes(100, 72, 64)
    assert need >= 2 * 100 * 72
    for ws, n in ((None, NWS), (WS + 8, NWS), (WS, need - 1)):
        assert L.gdn_linear_backward(ctypes.byref(_grad()), ws, n, None) == gdn.GDN_ERR_WORKSPACE
    assert L.gdn_linear_backward_workspace_bytes(1, 2, 3) == 0 and L.gdn_last_error()
    assert L.gdn_linear_backward(ctypes.byref(_grad(dx=None, dw=None, dbias=None)), None, 0, None) == gdn.GDN_OK


@pytest.mark.parametrize("M, N, K, fits", [
    (16, (1 << 27) - 16, 8, True), (16, (1 << 27) - 15, 8, False), (1, (1 << 31) - 1, 8, False), (17, (1 << 30) - 64, 8, True),
    (17, (1 << 30) - 63, 8, False), ((1 << 30) - 64, 64, 8, True), ((1 << 30) - 63, 64, 8, False), (1 << 18, 1 << 18, 8, False),
    (1 << 25, 64, 1 << 22, True),
])
def test_forward_fits_one_launch(M, N, K, fits):
    """A launch of 2^32 work-items or more would run a part of them: refused."""
    L = gdn.lib()
    assert L.gdn_linear_workspace_bytes(M, N, K) == 0 and (L.gdn_last_error() == b"") == fits
    if not fits:
        io = _io(M=M, N=N, K=K, x_stride=0, residual=None, preact=None)
        assert L.gdn_linear(ctypes.byref(io), WS, NWS, None) == gdn.GDN_ERR_INVALID_ARGUMENT
        assert b"too large" in L.gdn_last_error()


@pytest.mark.parametrize("M, N, K, fits", [
    (1 << 29, 8, 8, False), ((1 << 29) - 32, 8, 8, True), (1 << 24, 8, 4096, False), (1 << 23, 1 << 16, 8, False),
    ((1 << 21) - 32, 1 << 16, 64, True), (1 << 21, 1 << 16, 64, False), (1 << 12, 1 << 22, 1 << 14, False), (4096, 4096, 4096, True),
])
def test_backward_fits_one_launch(M, N, K, fits):
    L = gdn.lib()
    assert (L.gdn_linear_backward_workspace_bytes(M, N, K) > 0) == fits
    if not fits:
        gr = _grad(M=M, N=N, K=K)
        assert L.gdn_linear_backward(ctypes.byref(gr), WS, 1 << 62, None) == gdn.GDN_ERR_INVALID_ARGUMENT
        assert b"too large" in L.gdn_last_error()


def test_tiles():
    assert gdn.linear_tiles(1, 4096, 512) == (16, 16) and gdn.linear_tiles(40, 4096, 2048) == (64, 64)
    with pytest.raises(gdn.GdnError, match="multiple of 8"):
        gdn.linear_tiles(64, 64, 60)
    with pytest.raises(gdn.GdnError, match="too large"):
        gdn.linear_tiles(1 << 20, 1 << 20, 64)
    with pytest.raises(gdn.GdnError, match="2\\^22"):
        gdn.linear_tiles(64, (1 << 22) + 8, 64, backward=True)
    rows = ctypes.c_int32()
    assert gdn.lib().gdn_linear_tiles(64, 64, 64, 0, ctypes.byref(rows), None) == gdn.GDN_ERR_INVALID_ARGUMENT


def test_one_rows_stride_is_not_looked_at():
    """hidden[:, -1] of a long prompt: one row, with whatever stride.  (The
    calls are refused for what is checked last.)"""
    L = gdn.lib()
    odd = dict(x_stride=(1 << 23) + 4, y_stride=5, residual_stride=3, preact_stride=1)
    assert L.gdn_linear(ctypes.byref(_io(M=1, preact=FAKE + 5 * FAR, **odd)), WS, NWS, None) == gdn.GDN_ERR_INVALID_ARGUMENT
    assert b"overlaps" in L.gdn_last_error()
    assert L.gdn_linear(ctypes.byref(_io(N=1, w_stride=12, preact=FAKE + 5 * FAR)), WS, NWS, None) == gdn.GDN_ERR_INVALID_ARGUMENT
    assert b"overlaps" in L.gdn_last_error()
    odd = dict(dy_stride=1, x_stride=(1 << 23) + 4, preact_stride=2, dx_stride=7)
    for g in (dict(M=1, **odd), dict(N=1, w_stride=12, dw_stride=3)):
        st = L.gdn_linear_backward(ctypes.byref(_grad(dbias=WS, **g)), WS, NWS, None)
        assert st == gdn.GDN_ERR_INVALID_ARGUMENT and b"overlaps" in L.gdn_last_error()


def test_struct_layouts(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    checks = {"gdn_linear_io": gdn.CLinearIO, "gdn_linear_grad": gdn.CLinearGrad}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "gdn.h"', "int main(void) {"]
    for name, cls in checks.items():
        lines.append(f'  printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'  printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["  return 0;\n}"]))
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run([cc, "-std=c11", "-I", inc, str(src), "-o", str(tmp_path / "layout")], check=True)
    got = dict(line.split() for line in subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True,
                                                       check=True).stdout.splitlines())
    for name, cls in checks.items():
        assert int(got[name]) == ctypes.sizeof(cls), name
        for f, _ in cls._fields_:
            assert int(got[f"{name}.{f}"]) == getattr(cls, f).offset, (name, f)
