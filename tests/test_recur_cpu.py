"""The diagonal gated recurrence on the host: the reference's gradient against
differences, sizes of workspaces and saved states, struct layouts, and calls
that are refused before anything is enqueued."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import gated_deltanet_linear_03_amd as gdn
import recur_helpers as rh

FAKE = 0x10000            # never dereferenced: validation fails before any device use
FAR = 1 << 33


def test_reference_gradient_matches_differences():
    """d(loss)/d(each input) by central differences of the fp64 forward."""
    rng = np.random.default_rng(0)
    lens, D = [5, 0, 3], 2
    T, N = sum(lens), len(lens)
    inp = {k: rh.rows(rng, T, D) for k in ("x", "a", "b", "z")}
    A_log, dt_bias = rng.uniform(-1, 1, D), rng.uniform(-2, 1, D)
    h0, dy, dhT = rh.rows(rng, N, D), rh.rows(rng, T, D), rh.rows(rng, N, D)
    args = dict(inp, A_log=A_log, dt_bias=dt_bias, h0=h0)

    def loss(**kw):
        v, _ = rh.reference(lens, **kw)
        return (v["y"] * dy).sum() + (v["final"] * dhT).sum()

    val, _ = rh.reference(lens, dy=dy, dhT=dhT, **args)
    for name, key in (("x", "dx"), ("a", "da"), ("b", "db"), ("z", "dz"), ("A_log", "dA_log"),
                      ("dt_bias", "ddt_bias"), ("h0", "d_initial")):
        base = args[name]
        for i in np.ndindex(*base.shape):
            eps = 1e-6
            hi, lo = base.copy(), base.copy()
            hi[i] += eps
            lo[i] -= eps
            diff = (loss(**dict(args, **{name: hi})) - loss(**dict(args, **{name: lo}))) / (2 * eps)
            # the difference is good to about 1e-16 / eps plus eps^2
            assert abs(diff - val[key][i]) < 1e-7 * max(1.0, abs(diff)), (name, i)


def _recur(D=128, act=gdn.GDN_DTYPE_BF16, A_log=FAKE, dt_bias=FAKE):
    return gdn.CRecur(D, act, A_log, dt_bias)


def test_sizes():
    L = gdn.lib()
    r = _recur(D=100)
    # units of 128 rows, one at least per sequence: T / 128 + N bounds their number; two states each
    for N, T in ((1, 1), (1, 4096), (8, 5000), (600, 10)):
        assert L.gdn_recur_saved_bytes(ctypes.byref(r), N, T) == 2 * (T // 128 + N) * 100 * 4
    # short calls run without a workspace, and say so without an error
    assert L.gdn_recur_workspace_bytes(ctypes.byref(r), 3, 512) == 0 and L.gdn_last_error() == b""
    assert L.gdn_recur_workspace_bytes(ctypes.byref(r), 3, 513) > 0
    assert L.gdn_recur_workspace_bytes(ctypes.byref(r), 513, 512) > 0
    assert L.gdn_recur_backward_workspace_bytes(ctypes.byref(r), 3, 16) > 0
    for bad in (_recur(D=0), _recur(act=7)):
        assert L.gdn_recur_saved_bytes(ctypes.byref(bad), 1, 16) == 0 and L.gdn_last_error()
    for N, T in ((-1, 4), (1, -1), (0, 3), (1, 1 << 31)):
        assert L.gdn_recur_workspace_bytes(ctypes.byref(r), N, T) == 0 and L.gdn_last_error()


def _io(**kw):
    io = gdn.CRecurIO()
    io.N, io.T_total, io.cu_seqlens = 2, 1024, FAKE
    io.x, io.a, io.b, io.z, io.y = (FAKE + i * FAR for i in range(1, 6))
    io.initial_state, io.final_state = FAKE + 6 * FAR, FAKE + 7 * FAR
    for k, v in kw.items():
        setattr(io, k, v)
    return io


WS, NWS = FAKE + 20 * FAR, 1 << 30


@pytest.mark.parametrize("change, word", [
    (dict(x=None), "x is NULL"), (dict(b=None), "b is NULL"), (dict(y=None), "y is NULL"),
    (dict(x=FAKE + FAR + 1), "element aligned"), (dict(x_stride=100), "x_stride"),
    (dict(y_stride=127), "y_stride"), (dict(a_stride=(1 << 22) + 1), "2^22"), (dict(N=-1), "N"), (dict(T_total=-3), "T_total"),
    (dict(N=0), "N == 0"), (dict(T_total=1 << 31), "2^31"), (dict(cu_seqlens=None), "cu_seqlens"),
    (dict(cu_seqlens=FAKE + 2), "cu_seqlens"), (dict(status=FAKE + 1), "status"),
    (dict(state_slots=FAKE, num_slots=0), "num_slots"),
    (dict(final_state=FAKE + 6 * FAR + 4), "partially overlaps"),
    (dict(final_state=FAKE + 5 * FAR + 64), "y overlaps a state"),
    (dict(final_state=FAKE + FAR + 64, initial_state=None), "final_state overlaps"),
    (dict(y=FAKE + FAR + 128), "y overlaps an input"),
    (dict(y=FAKE + FAR, y_stride=256), "y overlaps an input"),
    (dict(saved=FAKE + 5 * FAR), "saved overlaps"), (dict(saved=FAKE + 1), "saved"),
    (dict(saved=WS + 64), "workspace overlaps"), (dict(status=FAKE + 5 * FAR), "status overlaps"),
])
def test_forward_refuses(change, word):
    st = gdn.lib().gdn_recur_forward(ctypes.byref(_recur()), ctypes.byref(_io(**change)), WS, NWS, None)
    assert st == gdn.GDN_ERR_INVALID_ARGUMENT
    assert word in gdn.lib().gdn_last_error().decode()


def test_forward_refuses_layer_and_workspace():
    L = gdn.lib()
    io = _io()
    for r in (_recur(D=0), _recur(act=5), _recur(A_log=None), _recur(dt_bias=FAKE + 2)):
        assert L.gdn_recur_forward(ctypes.byref(r), ctypes.byref(io), WS, NWS, None) == gdn.GDN_ERR_INVALID_ARGUMENT
    assert L.gdn_recur_forward(None, ctypes.byref(io), WS, NWS, None) == gdn.GDN_ERR_INVALID_ARGUMENT
    assert L.gdn_recur_forward(ctypes.byref(_recur()), None, WS, NWS, None) == gdn.GDN_ERR_INVALID_ARGUMENT
    need = L.gdn_recur_workspace_bytes(ctypes.byref(_recur()), 2, 1024)
    for ws, n in ((None, NWS), (WS + 4, NWS), (WS, need - 1)):
        assert L.gdn_recur_forward(ctypes.byref(_recur()), ctypes.byref(io), ws, n, None) == gdn.GDN_ERR_WORKSPACE


def _grad(**kw):
    gr = gdn.CRecurGrad()
    gr.dy, gr.dx, gr.da, gr.db, gr.dz = (FAKE + i * FAR for i in range(8, 13))
    gr.dA_log, gr.ddt_bias, gr.d_initial_state = FAKE + 13 * FAR, FAKE + 14 * FAR, FAKE + 15 * FAR
    for k, v in kw.items():
        setattr(gr, k, v)
    return gr


@pytest.mark.parametrize("change, io, word", [
    (dict(dy=None), {}, "dy is NULL"), (dict(dz=None), {}, "dz is NULL"), (dict(dx_stride=5), {}, "dx_stride"),
    (dict(dx=FAKE + FAR), {}, "overlap an input"), (dict(da=FAKE + 9 * FAR + 128), {}, "two gradients"),
    (dict(d_initial_state=FAKE + 9 * FAR), {}, "another buffer"), (dict(dA_log=FAKE + 2), {}, "4-byte"),
    (dict(d_final_state=FAKE + 15 * FAR + 4), {}, "partially overlaps"),
    ({}, dict(saved=None), "saved"), (dict(dx=FAKE + 16 * FAR), {}, "another buffer"),
    (dict(d_initial_state=WS), {}, "must not overlap"),
    (dict(dA_log=FAKE + 14 * FAR), {}, "dA_log and ddt_bias"), (dict(ddt_bias=WS), {}, "dA_log and ddt_bias"),
])
def test_backward_refuses(change, io, word):
    io = _io(**dict(dict(saved=FAKE + 16 * FAR), **io))
    st = gdn.lib().gdn_recur_backward(ctypes.byref(_recur()), ctypes.byref(io), ctypes.byref(_grad(**change)), WS, NWS, None)
    assert st == gdn.GDN_ERR_INVALID_ARGUMENT
    assert word in gdn.lib().gdn_last_error().decode()


def test_backward_refuses_workspace():
    L = gdn.lib()
    io = _io(saved=FAKE + 16 * FAR)
    need = L.gdn_recur_backward_workspace_bytes(ctypes.byref(_recur()), 2, 1024)
    for ws, n in ((None, NWS), (WS + 4, NWS), (WS, need - 1)):
        st = L.gdn_recur_backward(ctypes.byref(_recur()), ctypes.byref(io), ctypes.byref(_grad()), ws, n, None)
        assert st == gdn.GDN_ERR_WORKSPACE


def test_decode_refuses():
    L = gdn.lib()
    for change in (dict(final_state=None), dict(N=-1), dict(x=None), dict(y=FAKE + 7 * FAR)):
        st = L.gdn_recur_decode(ctypes.byref(_recur()), ctypes.byref(_io(**change)), None)
        assert st == gdn.GDN_ERR_INVALID_ARGUMENT, change
    assert L.gdn_recur_decode(ctypes.byref(_recur()), ctypes.byref(_io(N=0)), None) == gdn.GDN_OK


# FAKE: cu_seqlens and the parameters; FAKE + i FAR: x, a, b, z
@pytest.mark.parametrize("change, word", [
    (dict(saved=FAKE + FAR), "saved overlaps"), (dict(saved=FAKE + 4 * FAR + 1024), "saved overlaps"), (dict(saved=FAKE), "saved overlaps"),
    (dict(x=WS + 4096), "workspace overlaps"), (dict(z=WS), "workspace overlaps"), (dict(cu_seqlens=WS + 64), "workspace overlaps"),
    (dict(y=FAKE), "y overlaps an input"), (dict(final_state=FAKE), "final_state overlaps"), (dict(status=FAKE + 4), "status overlaps"),
    (dict(status=FAKE + 2 * FAR), "status overlaps"),
    (dict(state_slots=FAKE + 9 * FAR, num_slots=4, final_state=FAKE + 9 * FAR, initial_state=None), "final_state overlaps"),
])
def test_forward_refuses_what_shares_bytes_with_its_inputs(change, word):
    st = gdn.lib().gdn_recur_forward(ctypes.byref(_recur()), ctypes.byref(_io(**change)), WS, NWS, None)
    assert st == gdn.GDN_ERR_INVALID_ARGUMENT and word in gdn.lib().gdn_last_error().decode()


@pytest.mark.parametrize("grad, io, word", [
    ({}, dict(x=WS + 64), "overlaps an input"), ({}, dict(b=WS), "overlaps an input"), (dict(dy=WS + 4096), {}, "overlaps an input"),
    ({}, dict(cu_seqlens=WS), "overlaps an input"), (dict(dA_log=FAKE), {}, "overlaps an input"),
    (dict(dA_log=FAKE + 2 * FAR), {}, "overlaps an input"), (dict(ddt_bias=FAKE + 16 * FAR), {}, "overlaps an input"),
    (dict(d_initial_state=FAKE + 8 * FAR), {}, "overlaps an input"), (dict(d_initial_state=FAKE), {}, "overlaps an input"),
    (dict(dx=FAKE), {}, "overlaps an input"), (dict(dA_log=FAKE + 17 * FAR, d_final_state=FAKE + 17 * FAR), {}, "overlaps an input"),
    ({}, dict(status=FAKE + 9 * FAR), "status overlaps"), ({}, dict(status=WS + 8), "status overlaps"),
    ({}, dict(status=FAKE + 16 * FAR), "status overlaps"),
])
def test_backward_refuses_what_shares_bytes_with_its_inputs(grad, io, word):
    io = _io(**dict(dict(saved=FAKE + 16 * FAR), **io))
    st = gdn.lib().gdn_recur_backward(ctypes.byref(_recur()), ctypes.byref(io), ctypes.byref(_grad(**grad)), WS, NWS, None)
    assert st == gdn.GDN_ERR_INVALID_ARGUMENT and word in gdn.lib().gdn_last_error().decode()


def test_decode_refuses_what_shares_bytes_with_its_inputs():
    L = gdn.lib()
    for change in (dict(y=FAKE), dict(final_state=FAKE), dict(status=FAKE + 3 * FAR), dict(status=FAKE),
                   dict(state_slots=FAKE + 5 * FAR, num_slots=2)):
        io = _io(**dict(dict(cu_seqlens=None), **change))
        st = L.gdn_recur_decode(ctypes.byref(_recur()), ctypes.byref(io), None)
        assert st == gdn.GDN_ERR_INVALID_ARGUMENT and b"overlaps an input" in L.gdn_last_error(), change


def test_one_rows_stride_is_not_looked_at():
    """One token's row, with whatever stride.  (The calls are refused for what
    is checked last.)"""
    L = gdn.lib()
    odd = {k + "_stride": v for k, v in zip("xabzy", ((1 << 22) + 1, 3, 1 << 30, 127, 1))}
    io = _io(N=1, T_total=1, status=FAKE + 7 * FAR, **odd)
    for st in (L.gdn_recur_decode(ctypes.byref(_recur()), ctypes.byref(io), None),
               L.gdn_recur_forward(ctypes.byref(_recur()), ctypes.byref(io), WS, NWS, None)):
        assert st == gdn.GDN_ERR_INVALID_ARGUMENT and b"status overlaps" in L.gdn_last_error()
    io = _io(N=1, T_total=1, saved=FAKE + 16 * FAR, **odd)
    gr = _grad(ddt_bias=WS, **{k + "_stride": v for k, v in zip(("dy", "dx", "da", "db", "dz"), (1, 2, 3, 1 << 23, 5))})
    assert L.gdn_recur_backward(ctypes.byref(_recur()), ctypes.byref(io), ctypes.byref(gr), WS, NWS, None) == gdn.GDN_ERR_INVALID_ARGUMENT
    assert b"dA_log and ddt_bias" in L.gdn_last_error()


def test_binding_refuses_host_tensors():
    import torch
    r = gdn.Recur(D=4, A_log=torch.zeros(4), dt_bias=torch.zeros(4))
    with pytest.raises(ValueError, match="device tensor"):
        r.c()


def test_struct_layouts(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    checks = {"gdn_recur": gdn.CRecur, "gdn_recur_io": gdn.CRecurIO, "gdn_recur_grad": gdn.CRecurGrad}
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
