"""fp64 reference of the diagonal gated recurrence and its gradient, token by
token in numpy, with bounds on what a 32-bit evaluation may be off.

The bounds follow the error through the recurrence.  Per step the decay may be
off by a relative (2^-22 + |g| 2^-20) (2^x to 1 ulp, its argument g log2(e) to
a few roundings of softplus, and the roundings of the products that compose
steps), the input u by 2^-20 (square root, sigmoid, series and three
products), and each product-sum rounds to 2^-24:

    E_t = alpha_t E_{t-1} + |alpha_t h_{t-1}| (2^-22 + |g_t| 2^-20) + |u_t| 2^-20 + |h_t| 2^-24

and the same from the other end for G.  Outputs add their own factors'
roundings (2^-19 for up to eight of them) and half a step of their type."""
import numpy as np

U = 2.0 ** -24


def softplus(v):
    return np.logaddexp(v, 0.0)


def sigmoid(v):
    return np.exp(-np.logaddexp(0.0, -v))          # keeps its relative precision far out on the left


def reference(lens, x, a, b, z, A_log, dt_bias, h0=None, dy=None, dhT=None):
    """Arrays in float64: x, a, b, z (or None), dy [T, D]; h0, dhT [N, D] or
    None.  Returns (values, bounds): dicts with y, final and, with dy, dx, da,
    db, dz, dA_log, ddt_bias, d_initial; the bounds without the outputs'
    own rounding."""
    N, D = len(lens), x.shape[1]
    T = x.shape[0]
    rate = np.exp(A_log)
    v = a + dt_bias
    g = -rate * softplus(v)
    al = np.exp(g)
    w = np.sqrt(-np.expm1(2 * g))
    beta = sigmoid(b)
    u = w * beta * x
    sz = None if z is None else sigmoid(z)
    swish = np.ones_like(x) if z is None else z * sz
    rel = 2.0 ** -22 + np.abs(g) * 2.0 ** -20
    # The hardware 2^x gives no denormals: e^v below 2^-126 (v < -87.3) counts
    # as 0, and so do sigmoid(v), w and what they multiply.  What is lost is
    # the value itself: w is at most sqrt(2 exp(A_log) 2^-126) < 2^-60 there.
    gone = (v < -87.0).astype(np.float64)
    # sigmoid(t) = 1 / (1 + 2^(-t log2 e)): the product rounds to 2^-24 and
    # log2 e is off by 2^-25.8, so 2^(..) is off by a relative |t| 2^-23.5, of
    # which sigmoid takes the share 1 - sigmoid
    def tail(t, st):
        return np.abs(t) * (1 - st) * 2.0 ** -23
    tb = tail(b, beta)
    tz = 0.0 if z is None else tail(z, sz)
    tv = tail(v, sigmoid(v))
    h, hp, E, Ep = (np.zeros((T, D)) for _ in range(4))
    final = np.zeros((N, D)) if h0 is None else h0.copy()
    Ef = np.zeros((N, D))
    at = np.concatenate([[0], np.cumsum(lens)])
    for n, L in enumerate(lens):
        s, e = final[n].copy(), np.zeros(D)
        for t in range(at[n], at[n] + L):
            hp[t], Ep[t] = s, e
            new = al[t] * s + u[t]
            e = al[t] * e + np.abs(al[t] * s) * rel[t] + np.abs(u[t]) * (2.0 ** -20 + gone[t] + tb[t]) + np.abs(new) * U
            s = new
            h[t], E[t] = s, e
        final[n], Ef[n] = s, e
    val = {"y": h * swish, "final": final}
    err = {"y": E * np.abs(swish) + np.abs(h * swish) * (2.0 ** -19 + tz), "final": Ef}
    if dy is None:
        return val, err
    G, EG = np.zeros((T, D)), np.zeros((T, D))
    dinit = np.zeros((N, D)) if dhT is None else dhT.copy()
    Ed = np.zeros((N, D))
    e_y = dy * swish
    tzs = np.zeros_like(x) + tz
    for n, L in enumerate(lens):
        c, e = dinit[n].copy(), np.zeros(D)
        for t in range(at[n] + L - 1, at[n] - 1, -1):
            G[t] = e_y[t] + c
            EG[t] = e + np.abs(e_y[t]) * (2.0 ** -20 + tzs[t]) + np.abs(G[t]) * U
            c = al[t] * G[t]
            e = al[t] * EG[t] + np.abs(c) * rel[t] + np.abs(c) * U
        dinit[n], Ed[n] = c, e
    with np.errstate(divide="ignore", invalid="ignore"):
        over = np.where(w > 0, 1.0 / w, 0.0)
    r = beta * x * al * over
    dg = al * G * (hp - r)
    Edg = al * (EG * (np.abs(hp) + np.abs(r)) + np.abs(G) * Ep + np.abs(G) * (np.abs(hp) + np.abs(r)) * (2.0 ** -19 + rel + tb))
    sv = rate * sigmoid(v)
    val.update(dx=G * w * beta, da=-dg * sv, db=G * w * x * beta * (1 - beta), d_initial=dinit,
               dA_log=(dg * g).sum(0), ddt_bias=(-dg * sv).sum(0))
    # 1 - beta is off by up to 2^-22 of 1
    err.update(dx=EG * w * beta + np.abs(val["dx"]) * (2.0 ** -19 + gone + tb),
               da=Edg * sv + np.abs(val["da"]) * (2.0 ** -19 + gone + tv + tb),
               db=(EG * (1 - beta) + np.abs(G) * 2.0 ** -22) * w * np.abs(x) * beta
               + np.abs(val["db"]) * (2.0 ** -19 + gone + tb),
               d_initial=Ed)
    # sums over T rows: depth of the summation at most 32 + T / 128
    depth = (64 + T / 128) * U
    for name, each, ev in (("dA_log", dg * g, Edg * np.abs(g)), ("ddt_bias", dg * sv, Edg * sv)):
        err[name] = ev.sum(0) + np.abs(each).sum(0) * (depth + 2.0 ** -19)
    if z is not None:
        ds = sz * (1 + z * (1 - sz))
        val["dz"] = dy * h * ds
        # silu' passes through zero: its error is one of sigmoid and of z (1 - sigmoid)
        err["dz"] = np.abs(dy) * (E * np.abs(ds) + np.abs(h) * sz * (1 + np.abs(z)) * (2.0 ** -19 + tz))
    return val, err


def rows(rng, T, D, scale=1.0):
    return rng.standard_normal((T, D)) * scale


def parameters(rng, D):
    """A_log and dt_bias with decay rates from 1e-3 to about 1.6."""
    rate = np.exp(rng.uniform(np.log(1e-3), np.log(1e-1), D))
    return (rng.uniform(0, np.log(16.0), D).astype(np.float32),
            (rate + np.log(-np.expm1(-rate))).astype(np.float32))
