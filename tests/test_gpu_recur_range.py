"""The recurrence's backward pass where 1 - alpha^2 is next to nothing: the
gradients divide by its root, and every factor on the way has to stay inside
the range of 32 bits."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_03_amd as gdn
import recur_helpers as rh
from test_gpu_recur import DT, HALF, check

pytestmark = pytest.mark.gpu

# A_log, and logits around the place where 1 - alpha^2 = 2 exp(A_log + v) falls below 2^-126 and e^v below 2^-126
WINDOWS = [(-3.0, -89.0, -83.0), (-10.0, -89.0, -76.0), (-20.0, -86.0, -66.0), (-60.0, -46.0, -26.0), (0.0, -89.0, -83.0),
           (4.0, -89.0, -84.0), (-80.0, -10.0, 0.0), (-87.0, -3.0, 3.0)]


def _far(val, err, lens, v, A_log, x, b, z, h0, dy, dhT):
    """What the range and the logits' size add to the bounds of recur_helpers.

    1 - alpha^2 below 2^-126 counts as 0, and with it w and 1 / w: what is lost
    is the value itself, below 2^-63 of the other factors.  Next to that border
    either side may be taken (its error is below 2^-10).  e^-|v| is off by a
    relative tv = |v| 2^-23 (the rounded argument of 2^x), and so are softplus,
    1 - alpha^2 and sigmoid(v) down there; w and 1 / w by half of it.  Below
    v = -87.33 the hardware's 2^x gives 0 for e^v, and g and sigmoid(v) are 0
    (recur_helpers counts v < -87 so): the terms of da, dA_log and ddt_bias are
    lost whole, each below 2^-126 of G h and 2^-63 of G x."""
    rate, beta = np.exp(A_log), rh.sigmoid(b)
    g = -rate * rh.softplus(v)
    al, q = np.exp(g), -np.expm1(2 * g)
    w, sv, tv = np.sqrt(q), rate * rh.sigmoid(v), np.abs(v) * 2.0 ** -23
    gone = (q < 2.0 ** -126 * (1 + 2.0 ** -10)).astype(np.float64)
    swish = np.ones_like(x) if z is None else z * rh.sigmoid(z)
    lost = (v < -87.0) + tv
    u = np.abs(w * beta * x)
    eu = u * (gone + tv / 2)
    hp, G, eh, at = np.zeros_like(x), np.zeros_like(x), np.zeros_like(x), 0
    for n, L in enumerate(lens):
        s, e = h0[n].copy(), np.zeros_like(h0[n])
        for t in range(at, at + L):
            hp[t] = s
            s = al[t] * s + w[t] * beta[t] * x[t]
            e = al[t] * e + eu[t]
            eh[t] = e
        err["final"][n] += e
        c = dhT[n].copy()
        for t in range(at + L - 1, at - 1, -1):
            G[t] = np.abs(dy[t] * swish[t]) + np.abs(c)      # (its terms' size)
            c = al[t] * (dy[t] * swish[t] + c)
        at += L
    r = np.abs(beta * x * al / w)
    edg = al * G * (eh + r * (gone + tv / 2))
    eda = edg * sv + al * G * (np.abs(hp) + r) * sv * lost
    err["y"] += eh * np.abs(swish)
    if z is not None:
        err["dz"] += np.abs(dy) * eh * (1 + np.abs(z))
    for k in ("dx", "db"):
        err[k] += np.abs(val[k]) * (gone + tv / 2)
    err["da"] += eda
    err["dA_log"] += (edg * np.abs(g) + al * G * (np.abs(hp) + r) * np.abs(g) * lost).sum(0)
    err["ddt_bias"] += eda.sum(0)
    return err


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("gate", [True, False], ids=["gate", "plain"])
def test_gradients_where_the_decay_is_next_to_one(gate, dtype):
    lens, per = [150, 0, 75], 12
    T, N, D = sum(lens), len(lens), len(WINDOWS) * per
    rng = np.random.default_rng(31)
    A_log = np.repeat([wd[0] for wd in WINDOWS], per).astype(np.float32)
    dt_bias = np.zeros(D, np.float32)
    host = {n: rh.rows(rng, T, D) for n in ("x", "b", "z", "dy")}
    host["a"] = np.concatenate([rng.uniform(lo, hi, (T, per)) for _, lo, hi in WINDOWS], axis=1)
    for k, s in enumerate((0.0, 1.0, 100.0, 3e4)):           # (the fifth kind as drawn)
        host["x"][:, k::5] *= s
    t = {n: torch.from_numpy(v).to("cuda", DT[dtype]) for n, v in host.items()}
    if not gate:
        t["z"] = None
    f64 = {n: None if v is None else v.double().cpu().numpy() for n, v in t.items()}
    h0, dhT = (rh.rows(rng, N, D).astype(np.float32) for _ in range(2))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    rec = gdn.Recur(D=D, A_log=torch.from_numpy(A_log).cuda(), dt_bias=torch.from_numpy(dt_bias).cuda(),
                    act_dtype=gdn.GDN_DTYPE_BF16 if dtype == "bf16" else gdn.GDN_DTYPE_FP32)
    f = gdn.recur_forward(rec, *(t[k] for k in "xabz"), cu, initial_state=torch.from_numpy(h0).cuda(), want_saved=True)
    g = gdn.recur_backward(rec, *(t[k] for k in "xabz"), t["dy"], f["saved"], cu, d_final_state=torch.from_numpy(dhT).cuda(),
                           want_d_initial=True)
    up = lambda v: v.astype(np.float64)  # noqa: E731
    args = (f64["x"], f64["a"], f64["b"], f64["z"], up(A_log), up(dt_bias), up(h0), f64["dy"], up(dhT))
    val, err = rh.reference(lens, *args)
    err = _far(val, err, lens, f64["a"], up(A_log), f64["x"], f64["b"], f64["z"], up(h0), f64["dy"], up(dhT))
    check("y", f["out"], val["y"], err["y"], HALF[dtype])
    check("final_state", f["final_state"], val["final"], err["final"], HALF["fp32"])
    for n in ("dx", "da", "db") + (("dz",) if gate else ()):
        check(n, g[n], val[n], err[n], HALF[dtype])
    check("d_initial_state", g["d_initial_state"], val["d_initial"], err["d_initial"], HALF["fp32"])
    for n in ("dA_log", "ddt_bias"):
        check(n, g[n], val[n], err[n], HALF["fp32"])
