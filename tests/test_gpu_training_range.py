"""Sizes whose offsets pass 32 bits: rows of the norms, a tensor of the AdamW
step, a vocabulary; and grids beyond what one launch holds."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_03_amd as gdn
from train_helpers import HALF, close, loss64, norm64, norm_backward64, norm_bounds, random_halves, up_or_down

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M, D", [(1100000, 4096), (2200000, 2056), (70000000, 64)])
def test_norm_rows_past_4_gib(M, D):
    """bf16 rows of more than 2^32 values in all (64 columns: more rows than a
    launch has work-groups): the first, middle and last rows."""
    x = torch.empty((M, D), dtype=BF16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    at = torch.tensor([0, 1, M // 2, M - 2, M - 1], device="cuda")
    x.zero_()
    x[at] = torch.randn((5, D), generator=g, device="cuda").to(BF16)
    w = torch.randn(D, generator=g, device="cuda")
    stats = torch.empty((2, M), device="cuda")
    y = gdn.norm(x, w, None, stats=stats)
    want, _, _ = norm64(x[at].cpu(), w.cpu(), None, True, 1e-5)
    e, _, _ = norm_bounds(x[at].cpu(), w.cpu(), None, True, 1e-5)
    close("y", y[at], want, e + (want.abs() + e) * HALF[BF16])
    # y is the gradient now: rows of zeros add nothing
    r = gdn.norm_backward(y, x, w, stats, want_dbias=True)
    (dx, dw, db), (ex, ew, eb) = norm_backward64(y[at].cpu(), x[at].cpu(), w.cpu(), stats[0, at].cpu(), stats[1, at].cpu(), True, None)
    close("dx", r["dx"][at], dx, ex + (dx.abs() + ex) * HALF[BF16])
    close("dweight", r["dweight"], dw, ew)
    close("dbias", r["dbias"], db, eb)


def test_adamw_past_4_gib():
    """A tensor of more than 2^32 elements with 8-bit states: the random bits
    know the index's upper word."""
    n = (1 << 32) + 777
    p, g = torch.zeros(n, device="cuda"), torch.zeros(n, dtype=BF16, device="cuda")
    blocks = -(-n // 256)
    st = {k: [torch.zeros(n, dtype=torch.uint8, device="cuda")] for k in ("m", "v")}
    st.update({k + "_scale": [torch.zeros(blocks, device="cuda")] for k in ("m", "v")})
    at = [0, (1 << 32) - 256, 1 << 32, n - 777 // 256 * 256 - 9]
    at[3] = at[3] // 256 * 256
    values = {}
    for k, a in enumerate(at):
        v = torch.randn(min(256, n - a), generator=torch.Generator(device="cuda").manual_seed(k), device="cuda").to(BF16)
        g[a:a + v.numel()] = v
        values[a] = v.double().cpu().numpy()
    opt = gdn.AdamW([p], **st, seed=11)
    gdn.adamw_step(opt, [g], lr=0.5, step=1)
    for a, v in values.items():
        close("p", p[a:a + len(v)], torch.from_numpy(-0.5 * v / (np.abs(v) + 1e-8)), torch.full((len(v),), 1e-5))
        lo, hi = random_halves(11, 1, 0, len(v), first=a)
        for name, x, u in (("m", 0.1 * v, lo), ("v", np.sqrt(0.001 * v * v), hi)):
            scale = float(np.float32(np.abs(x).max() / 448))
            want, near = up_or_down(np.clip(x / scale, -448, 448), u)
            got = st[name][0][a:a + len(v)].view(torch.float8_e4m3fn).float().double().cpu().numpy()
            want = np.where((want == 0) & (x > 0) & (name == "v"), 2.0 ** -9, want)
            assert not ((got != want) & ~near).any(), (name, a)
    assert float(p[1 << 20:1 << 21].abs().max()) == 0 and int(st["v"][0][1 << 20:1 << 21].max()) == 0


@pytest.mark.parametrize("M", [3, 40])
def test_vocabulary_past_4_gib(M):
    """A vocabulary whose weights pass 2^32 bytes (and 2^31 elements): targets
    at its ends."""
    V, K = 2200003, 1024
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.zeros((V, K), dtype=BF16, device="cuda")
    rows = torch.tensor([0, 5, V // 2, V - 2, V - 1], device="cuda")
    w[rows] = (torch.randn((5, K), generator=g, device="cuda") / 8).to(BF16)
    x = torch.randn((M, K), generator=g, device="cuda").to(BF16)
    t = rows[torch.arange(M, device="cuda") % 5]
    r = gdn.linear_cross_entropy(x, w, t)
    # the other entries' logits are 0
    loss, lse, e, e_lse, l, *_ = loss64(x.cpu(), w[rows].cpu(), None, (torch.arange(M) % 5), 0.0, 0.0)
    total = torch.logsumexp(torch.cat([l, torch.full((M, 1), float(np.log(V - 5)), dtype=torch.float64)], 1), 1)
    slack = 2.0 ** -24 * (6 * l.abs().amax(1) + 6 * total + 200 + V / 512)
    close("lse", r["lse"], total, e_lse + slack)
    close("loss", r["loss"], total - l[torch.arange(M), torch.arange(M) % 5], 2 * e_lse + e + slack)
    b = gdn.linear_cross_entropy_backward(torch.ones(1, device="cuda"), x, w, t, r["lse"])
    p = torch.exp(l - r["lse"].double().cpu()[:, None])
    hot = torch.zeros_like(p)
    hot[torch.arange(M), torch.arange(M) % 5] = 1
    dl = p - hot
    lim = dl.abs() * 2.0 ** -7 + 1e-4
    want = dl.t() @ x.double().cpu()
    close("dw", b["dw"][rows], want, lim.t() @ x.double().cpu().abs() + want.abs() * HALF[BF16])
    want = dl @ w[rows].double().cpu()
    close("dx", b["dx"], want, lim @ w[rows].double().cpu().abs() + want.abs() * HALF[BF16])
