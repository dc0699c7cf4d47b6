"""The norms, the AdamW step and the cross entropy of a linear layer's outputs
from their definitions in float64 on the CPU, with bounds on what 32-bit
arithmetic may be off by (U: half a step of 32 bits, relative)."""
import numpy as np
import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
GOLDEN = 0x9E3779B1


def close(name, got, want, lim):
    got = got.detach().double().cpu()
    assert got.shape == want.shape, f"{name}: {tuple(got.shape)}, not {tuple(want.shape)}"
    bad = ~((got - want).abs() <= lim) & ~(got.isnan() & want.isnan())
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float(((got - want).abs() / lim)[bad].max()):.2f} of the bound at {bad.nonzero()[:3].tolist()}")


# ---- norms ---------------------------------------------------------------------

def norm64(x, weight, bias, layer, eps):
    """y, mean, rstd."""
    x = x.double()
    mean = x.mean(1) if layer else torch.zeros(x.shape[0], dtype=torch.float64)
    d = x - mean[:, None]
    rstd = (d.square().mean(1) + eps) ** -0.5
    y = d * rstd[:, None]
    y = y if weight is None else y * weight.double()
    return y if bias is None else y + bias.double(), mean, rstd


def norm_bounds(x, weight, bias, layer, eps):
    """Bounds for norm64's results.  A row is summed by at least 64 threads
    (16 where D is at most 128), each at most 64 or D / 512 values, and then in
    at most 10 + 16 steps: every value goes through at most `steps` additions."""
    x = x.double()
    D = x.shape[1]
    steps = 90 + D / 512
    y, mean, rstd = norm64(x, None, None, layer, eps)
    e_mean = (steps + 2) * U * x.abs().mean(1) if layer else torch.zeros_like(mean)
    d = (x - mean[:, None]).abs()
    e_d = e_mean[:, None] + U * (d + e_mean[:, None])
    # the mean square of d + e_d, its sum's rounding, the root's, the quotient's
    var = d.square().mean(1)
    e_var = (2 * d * e_d + e_d.square()).mean(1) + (steps + 4) * U * (var + eps)
    rel = 0.5 * e_var / (var + eps) * (1 + e_var / (var + eps)) + 4 * U
    e = (e_d * rstd[:, None] + d * (rstd * rel)[:, None]) * (1 + rel[:, None]) + 2 * U * y.abs()
    if weight is not None:
        e = e * weight.double().abs()
        y = y * weight.double()
        e = e + U * y.abs()
    if bias is not None:
        e = e + U * (y + bias.double()).abs() + U * e
    return e + 1e-37, e_mean + 1e-37, rstd * rel + 1e-37


def norm_backward64(dy, x, weight, mean, rstd, layer, skip):
    """dx, dweight, dbias from the statistics given, and bounds on 32 bits' errors."""
    dy, x, rstd = dy.double(), x.double(), rstd.double()[:, None]
    M, D = x.shape
    steps = 90 + D / 512
    xh = (x - mean.double()[:, None]) * rstd
    q = dy if weight is None else dy * weight.double()
    b = (q * xh).mean(1, keepdim=True)
    a = q.mean(1, keepdim=True) if layer else torch.zeros_like(b)
    dx = rstd * (q - a - xh * b)
    # x - mean may lose U of x itself
    e_xh = 3 * U * (xh.abs() + (x.abs() + mean.double().abs()[:, None]) * rstd)
    e_b = (steps + 6) * U * (q * xh).abs().mean(1, keepdim=True) + (q.abs() * e_xh).mean(1, keepdim=True)
    e_a = (steps + 4) * U * q.abs().mean(1, keepdim=True)
    e = rstd * (2 * U * q.abs() + e_a + xh.abs() * e_b + e_xh * (b.abs() + e_b) + 6 * U * (q.abs() + a.abs() + (xh * b).abs()))
    if skip is not None:
        dx = dx + skip.double()
        e = e + U * dx.abs()
    e_w = (M + 8) * U * (dy * xh).abs().sum(0) + (dy.abs() * e_xh).sum(0)
    return (dx, (dy * xh).sum(0), dy.sum(0)), (e + 1e-37, e_w + 1e-37, (M + 8) * U * dy.abs().sum(0) + 1e-37)


# ---- AdamW ---------------------------------------------------------------------

def mix(h):
    """The finaliser of MurmurHash3 on uint32 arrays (products wrap)."""
    h = np.asarray(h, dtype=np.uint32)
    with np.errstate(over="ignore"):
        h = (h ^ (h >> np.uint32(16))) * np.uint32(0x85EBCA6B)
        h = (h ^ (h >> np.uint32(13))) * np.uint32(0xC2B2AE35)
    return h ^ (h >> np.uint32(16))


def random_halves(seed, step, tensor, n, first=0):
    """The low and the high 16 random bits of elements first .. first + n - 1."""
    with np.errstate(over="ignore"):
        key = mix(np.array([(seed + step * GOLDEN) & 0xFFFFFFFF], dtype=np.uint32))
        key = mix(key + np.uint32((tensor * GOLDEN) & 0xFFFFFFFF))
        i = np.arange(first, first + n, dtype=np.uint64)
        h = mix(key[0] + mix((i >> np.uint64(32)).astype(np.uint32)) + i.astype(np.uint32) * np.uint32(GOLDEN))
    return h & np.uint32(0xFFFF), h >> np.uint32(16)


def up_or_down(ratio, u):
    """|ratio| <= 448 to a value of e4m3, and whether the choice is closer to
    its border than 32 bits tell."""
    a = np.abs(ratio)
    unit = np.exp2(np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    at = a / unit + u / 65536.0
    value = np.sign(ratio) * np.minimum(np.floor(at) * unit, 448.0)
    # a is off by some steps of 32 bits, the units' own limits included
    near = np.minimum(at - np.floor(at), np.ceil(at) - at) < 16 * 8 * U * 16
    return value, near


def adamw64(p, g, m, v, lr, b1, b2, eps, decay, k):
    """p', m', v' and bounds, all float64 arrays; m and v as they stand (8 bits: multiplied out)."""
    m1, v1 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    c1, c2 = 1 - b1 ** k, 1 - b2 ** k
    den = np.sqrt(v1 / c2) + eps
    step = m1 / c1 / den
    e_m = 5 * U * (np.abs(b1 * m) + np.abs((1 - b1) * g))
    e_v = 8 * U * v1
    # c1: 6 U, the root 6 U, c2 6 U, the reciprocal 2 U, products
    e_p = lr * (e_m / c1 / den + 24 * U * np.abs(step)) + 2 * U * np.abs(p) + 4 * U * lr * decay * np.abs(p)
    return (p - lr * (step + decay * p), m1, v1), (e_p + 1e-37, e_m + 1e-37, e_v + 1e-37)


# ---- the cross entropy of a linear layer's outputs --------------------------------

def loss64(x, w, bias, targets, smooth, z, ignore=-100):
    """loss, lse and bounds on 32 bits' errors, and the logits with theirs.  A
    logit is a sum of K products of bf16 values (exact in 32 bits each), rounded
    at most K times in any order."""
    x, w = x.double(), w.double()
    K, V = x.shape[1], w.shape[0]
    l = x @ w.t().contiguous()
    e_l = (x.abs() @ w.abs().t().contiguous()) * (K * U)
    if bias is not None:
        l = l + bias.double()
        e_l = e_l + U * l.abs()
    lse = torch.logsumexp(l, 1)
    # off by no more than the logits are; then 2^(l log2 e - top): the product
    # and the difference to 2 U of l each, v_exp_f32 to 2 U; all terms are
    # positive, each through at most `steps` additions and joins (of 6 U)
    steps = 200 + V / 512
    e_lse = e_l.amax(1) + U * (6 * l.abs().amax(1) + 6 * lse.abs() + steps)
    counts = (targets != ignore) & (targets >= 0) & (targets < V)
    rows = torch.arange(x.shape[0], device=x.device)
    at = targets.long().clamp(0, V - 1)
    lt, e_lt = l[rows, at], e_l[rows, at]
    mean = l.mean(1)
    loss = (1 - smooth) * (lse - lt) + smooth * (lse - mean) + z * lse * lse
    e_mean = e_l.mean(1) + steps * U * l.abs().mean(1)
    e = (1 - smooth) * (e_lse + e_lt) + smooth * (e_lse + e_mean) + z * (2 * lse.abs() + e_lse) * e_lse
    e = e + 6 * U * (lse.abs() + lt.abs() + mean.abs() + z * lse * lse)
    bad = ~counts & (targets != ignore)
    loss = torch.where(counts, loss, torch.where(bad, float("nan"), 0.0))
    return loss, lse, e, e_lse, l, e_l, counts


def loss_backward64(dloss, x, w, bias, targets, lse, smooth, z, ignore=-100):
    """dx, dw, dbias from the lse given, and bounds that count dl's rounding to bf16."""
    _, _, _, _, l, e_l, counts = loss64(x, w, bias, targets, smooth, z, ignore)
    x, w, lse = x.double(), w.double(), lse.double()
    M, V = l.shape
    g = torch.where(counts, dloss.double().expand(M), 0.0)[:, None]
    c = 1 + 2 * z * lse[:, None]
    p = torch.exp(l - lse[:, None])
    rel = e_l + U * (6 * l.abs() + 6 * lse.abs()[:, None] + 6)
    hot = torch.zeros_like(p)
    hot[torch.arange(M, device=x.device), targets.long().clamp(0, V - 1)] = 1 - smooth
    dl = g * (c * p - hot - smooth / V)
    e = g.abs() * (c.abs() * p * (rel + rel * rel) + 4 * U * (c.abs() * p + hot + smooth / V)) + 1e-37
    r = e + HALF[torch.bfloat16] * (dl.abs() + e)                # of dl as the products see it
    d = dl.abs() + r
    dx, dw = dl @ w, dl.t().contiguous() @ x
    e_dx = r @ w.abs() + (V + 64) * U * (d @ w.abs())
    e_dw = r.t().contiguous() @ x.abs() + (M + 64) * U * (d.t().contiguous() @ x.abs())
    return (dx, dw, dl.sum(0)), (e_dx + 1e-37, e_dw + 1e-37, e.sum(0) + (M + 64) * U * dl.abs().sum(0))
