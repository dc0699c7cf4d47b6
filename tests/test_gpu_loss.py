"""The cross entropy of a linear layer's outputs on the device against its
definition in 64 bits, forward and backward: single rows, vocabularies that end
inside a tile and of one entry, several pieces, ignored and bad targets, masked
vocabulary entries; nothing written outside; the same bits from call to call."""
import ctypes

import pytest
import torch

import gated_deltanet_linear_03_amd as gdn
from train_helpers import HALF, close, loss64, loss_backward64

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def data(M, V, K, seed, pad=0, scale=2.0, ignored=True, dtype=torch.int64, device="cuda"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((M, K + pad), generator=g, device="cuda").to(BF16)[:, :K]
    w = (torch.randn((V, K + pad), generator=g, device="cuda") * (scale / K ** 0.5)).to(BF16)[:, :K]
    t = torch.randint(0, V, (M,), generator=g, device="cuda").to(dtype)
    if ignored:
        t[torch.rand(M, generator=g, device="cuda") < 0.2] = -100
    return g, x, w, t


SHAPES = [(1, 1, 8), (1, 2, 8), (1, 1000, 72), (2, 65, 16), (3, 4099, 200), (16, 16, 64), (16, 300, 1000), (5, 70001, 16),
          (17, 5, 8), (17, 64, 64), (33, 257, 72), (64, 1000, 136), (65, 63, 8), (100, 129, 264), (130, 3001, 200), (200, 250, 520),
          (257, 512, 64), (300, 5000, 72), (600, 1023, 136), (1100, 70, 40)]


@pytest.mark.parametrize("i", range(len(SHAPES)), ids=["x".join(map(str, s)) for s in SHAPES])
@pytest.mark.parametrize("turn", range(2))
def test_against_64_bits(i, turn):
    M, V, K = SHAPES[i]
    k = i + turn
    g, x, w, t = data(M, V, K, 300 + i, pad=8 * (k % 3), scale=(2, 6)[turn], ignored=M > 2, dtype=(torch.int64, torch.int32)[k % 2])
    bias = torch.randn(V, generator=g, device="cuda") if k % 3 else None
    smooth, z = (0.0, 0.1)[(i + turn) % 2], (0.0, 1e-3)[turn]
    how = dict(bias=bias, label_smoothing=smooth, z_loss=z)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = gdn.linear_cross_entropy(x, w, t, status=status, **how)
    cpu = [v.cpu() if v is not None else None for v in (x, w, bias, t)]
    loss, lse, e, e_lse = loss64(*cpu, smooth, z)[:4]
    close("loss", r["loss"], loss, e)
    close("lse", r["lse"], lse, e_lse)
    assert int(status) == 0
    again = gdn.linear_cross_entropy(x, w, t, **how)
    assert torch.equal(again["loss"], r["loss"]) and torch.equal(again["lse"], r["lse"])

    one = turn == 1
    dloss = torch.randn(1 if one else M, generator=g, device="cuda")
    b = gdn.linear_cross_entropy_backward(dloss, x, w, t, r["lse"], want_dbias=True, **how)
    assert set(b) == {"dx", "dw", "dbias"}
    want, lim = loss_backward64(dloss.cpu(), *cpu, r["lse"].cpu(), smooth, z)
    for name, v, l in zip(("dx", "dw", "dbias"), want, lim):
        close(name, b[name], v, l + (v.abs() + l) * HALF[b[name].dtype])
    # each by itself, into strided rows
    for name in b:
        given = {name: torch.empty((b[name].shape[0], K + 3), dtype=BF16, device="cuda")[:, :K]} if name != "dbias" else {}
        only = gdn.linear_cross_entropy_backward(dloss, x, w, t, r["lse"], **how, **given,
                                                 **{"want_" + n: n == name for n in ("dx", "dw", "dbias")})
        assert list(only) == [name] and torch.equal(only[name], b[name]), name


@pytest.mark.parametrize("M, V, K", [(2048, 16500, 64), (4096, 20011, 40), (1000, 140003, 24), (70, 33000, 72), (700, 3000, 1032),
                                     (9000, 9000, 16)])
def test_large(M, V, K):
    """Tiles of each size, several pieces of the vocabulary, dx in parts; the
    reference on the device in 64 bits."""
    g, x, w, t = data(M, V, K, M)
    bias = torch.randn(V, generator=g, device="cuda")
    r = gdn.linear_cross_entropy(x, w, t, bias=bias, label_smoothing=0.05, z_loss=1e-4)
    loss, lse, e, e_lse, *_ = loss64(x, w, bias, t, 0.05, 1e-4)
    close("loss", r["loss"], loss.cpu(), e.cpu())
    close("lse", r["lse"], lse.cpu(), e_lse.cpu())
    dloss = torch.rand(M, generator=g, device="cuda")
    del loss, lse, e, e_lse, _
    b = gdn.linear_cross_entropy_backward(dloss, x, w, t, r["lse"], bias=bias, label_smoothing=0.05, z_loss=1e-4)
    want, lim = loss_backward64(dloss, x, w, bias, t, r["lse"], 0.05, 1e-4)
    for name, v, l in zip(("dx", "dw", "dbias"), want, lim):
        close(name, b[name], v.cpu(), (l + (v.abs() + l) * HALF[b[name].dtype]).cpu())
    again = gdn.linear_cross_entropy_backward(dloss, x, w, t, r["lse"], bias=bias, label_smoothing=0.05, z_loss=1e-4)
    assert all(torch.equal(again[n], b[n]) for n in b)


@pytest.mark.parametrize("M", [7, 90])
def test_targets(M):
    """Ignored rows, all of them, another ignore index, and targets outside."""
    V, K = 300, 64
    g, x, w, t = data(M, V, K, 60, ignored=False)
    plain = gdn.linear_cross_entropy(x, w, t)
    odd = t.clone()
    odd[0], odd[1], odd[2], odd[3] = -100, -1, V, 1 << 40
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = gdn.linear_cross_entropy(x, w, odd, status=status)
    assert int(status) == gdn.GDN_STATUS_BAD_INDEX
    assert float(r["loss"][0]) == 0 and bool(r["loss"][1:4].isnan().all()) and torch.equal(r["loss"][4:], plain["loss"][4:])
    assert torch.equal(r["lse"], plain["lse"])
    one = torch.ones(1, device="cuda")
    b = gdn.linear_cross_entropy_backward(one, x, w, odd, r["lse"])
    assert bool((b["dx"][:4] == 0).all()) and bool(b["dx"].isfinite().all()) and bool(b["dw"].isfinite().all())
    keep = gdn.linear_cross_entropy_backward(one, x, w, t, plain["lse"])
    assert torch.equal(b["dx"][4:], keep["dx"][4:])
    # the index of the padding token instead
    status.zero_()
    r5 = gdn.linear_cross_entropy(x, w, torch.full_like(t, 5), ignore_index=5, status=status)
    assert int(status) == 0 and bool((r5["loss"] == 0).all())
    b5 = gdn.linear_cross_entropy_backward(one, x, w, torch.full_like(t, 5), r5["lse"], ignore_index=5, want_dbias=True)
    assert all(bool((b5[n] == 0).all()) for n in b5)


@pytest.mark.parametrize("share", [0.0, 0.03, 0.5, 0.97, 1.0])
@pytest.mark.parametrize("one", [True, False])
def test_rows_brought_together(share, one):
    """Calls large enough to bring the rows that count together: none of them,
    a few at odd places, half, nearly all and all; a bad target among the rest."""
    M, V, K = 2055, 60001, 1032
    g, x, w, t = data(M, V, K, 67, ignored=False)
    if share < 1:
        t[torch.rand(M, generator=g, device="cuda") >= share] = -100
    if share == 0.5:
        t[17], t[2054] = V, 5
    bias = torch.randn(V, generator=g, device="cuda")
    r = gdn.linear_cross_entropy(x, w, t, bias=bias, label_smoothing=0.05)
    dloss = torch.randn(1 if one else M, generator=g, device="cuda")
    b = gdn.linear_cross_entropy_backward(dloss, x, w, t, r["lse"], bias=bias, label_smoothing=0.05)
    want, lim = loss_backward64(dloss, x, w, bias, t, r["lse"], 0.05, 0.0)
    for name, v, l in zip(("dx", "dw", "dbias"), want, lim):
        close(name, b[name], v.cpu(), (l + (v.abs() + l) * HALF[b[name].dtype]).cpu())
    if share == 0.0:
        assert all(bool((b[n] == 0).all()) for n in b)
    for name in b:
        only = gdn.linear_cross_entropy_backward(dloss, x, w, t, r["lse"], bias=bias, label_smoothing=0.05,
                                                 **{"want_" + n: n == name for n in ("dx", "dw", "dbias")})
        assert torch.equal(only[name], b[name]), name


@pytest.mark.parametrize("M", [5, 70])
def test_masked_vocabulary(M):
    """A bias of -inf takes an entry out of the softmax; a bias of the type's
    lowest value does the same."""
    V, K = 500, 40
    g, x, w, t = data(M, V, K, 61, ignored=False)
    bias = torch.zeros(V, device="cuda")
    bias[::3] = float("-inf")
    bias[1::3] = torch.finfo(torch.float32).min
    t = t // 3 * 3 + 2
    t.clamp_(max=497)
    r = gdn.linear_cross_entropy(x, w, t, bias=bias)
    keep = torch.arange(2, V, 3, device="cuda")
    loss, lse, e, e_lse = loss64(x.cpu(), w[keep].cpu(), None, (t.cpu() - 2) // 3, 0.0, 0.0)[:4]
    close("loss", r["loss"], loss, e)
    close("lse", r["lse"], lse, e_lse)
    b = gdn.linear_cross_entropy_backward(torch.ones(1, device="cuda"), x, w, t, r["lse"], bias=bias)
    assert bool(b["dx"].isfinite().all()) and bool((b["dw"][::3] == 0).all()) and bool((b["dw"][1::3] == 0).all())


def test_infinite_rows():
    """Infinities and NaN in an ignored row reach nothing but its lse; in a row
    that counts its own loss and dx and what it adds to dw."""
    for M in (12, 100):
        V, K = 400, 64
        g, x, w, t = data(M, V, K, 62, ignored=False)
        t[2] = -100
        clean = gdn.linear_cross_entropy(x, w, t)
        one = torch.full((1,), 0.5, device="cuda")
        want = gdn.linear_cross_entropy_backward(one, x, w, t, clean["lse"], want_dbias=True)
        x2 = x.clone()
        x2[2, 5], x2[2, 9] = float("inf"), float("nan")
        r = gdn.linear_cross_entropy(x2, w, t)
        assert torch.equal(r["loss"], clean["loss"]) and bool(r["lse"][2].isnan())
        b = gdn.linear_cross_entropy_backward(one, x2, w, t, r["lse"], want_dbias=True)
        assert torch.equal(b["dx"], want["dx"]) and torch.equal(b["dbias"], want["dbias"])
        x2[7, 1] = float("nan")
        r = gdn.linear_cross_entropy(x2, w, t)
        others = torch.arange(M, device="cuda") != 7
        assert bool(r["loss"][7].isnan()) and torch.equal(r["loss"][others], clean["loss"][others])
        b = gdn.linear_cross_entropy_backward(one, x2, w, t, r["lse"])
        assert bool(b["dx"][7].isnan().any()) and torch.equal(b["dx"][others], want["dx"][others])


@pytest.mark.parametrize("M,V,K,stride", [(5, 300, 64, 64), (130, 700, 72, 72), (130, 700, 72, 80), (700, 1000, 1032, 1032), (600, 50001, 1000, 1008), (1300, 60001, 1032, 1032)])
def test_unset_rows(M, V, K, stride):
    """Rows without a target hold anything (the padding of a batch that nobody
    wrote): no gradient sees it, in small calls and in large ones, nor with one
    target of the vocabulary's end."""
    g, x, w, t = data(M, V, K, 68, ignored=False)
    t[1::3] = -100
    t[0] = V - 1
    t[M - 1] = V                                # not an index: its loss is NaN, and it adds nothing either
    out = t == -100
    out[M - 1] = True
    held = torch.zeros(M, stride, dtype=x.dtype, device="cuda")[:, :K]
    held.copy_(x)
    held[out] = 0
    any_ = held.clone() if stride == K else torch.zeros(M, stride, dtype=x.dtype, device="cuda")[:, :K].copy_(held)
    rows = out.nonzero()[:, 0]
    for i, v in enumerate((float("nan"), float("inf"), -float("inf"), 3e38)):
        any_[rows[i::4]] = v
    lse = gdn.linear_cross_entropy(held, w, t)["lse"]
    r = gdn.linear_cross_entropy(any_, w, t)
    assert torch.equal(r["lse"][~out], lse[~out])
    for dloss in (torch.full((1,), 0.5, device="cuda"), torch.randn(M, generator=g, device="cuda")):
        want = gdn.linear_cross_entropy_backward(dloss, held, w, t, lse, want_dbias=True)
        b = gdn.linear_cross_entropy_backward(dloss, any_, w, t, r["lse"], want_dbias=True)
        assert all(torch.equal(b[n], want[n]) and bool(b[n].isfinite().all()) for n in want)
        assert bool((b["dx"][out] == 0).all())
        only = gdn.linear_cross_entropy_backward(dloss, any_, w, t, r["lse"], want_dx=False)
        assert torch.equal(only["dw"], want["dw"])


def test_nothing_outside():
    """Guards around every written buffer, and around the workspaces."""
    for M, V, K in ((3, 77, 40), (67, 301, 72)):
        g, x, w, t = data(M, V, K, 63, ignored=False)
        dx, dw = torch.full((M + 2, K + 8), 7.0, dtype=BF16, device="cuda"), torch.full((V + 2, K + 8), 7.0, dtype=BF16, device="cuda")
        db = torch.full((V + 64,), 7.0, device="cuda")
        n = gdn.linear_cross_entropy_workspace_bytes(M, V, K)
        ws = torch.full((n + 512,), 7, dtype=torch.uint8, device="cuda")
        r = gdn.linear_cross_entropy(x, w, t, label_smoothing=0.1, workspace=ws[256:-256])
        assert bool((ws[:256] == 7).all()) and bool((ws[-256:] == 7).all())
        n = gdn.linear_cross_entropy_backward_workspace_bytes(M, V, K)
        ws = torch.full((n + 512,), 7, dtype=torch.uint8, device="cuda")
        one = torch.ones(1, device="cuda")
        b = gdn.linear_cross_entropy_backward(one, x, w, t, r["lse"], label_smoothing=0.1, dx=dx[1:-1, :K], dw=dw[1:-1, :K],
                                              dbias=db[32:-32], workspace=ws[256:-256])
        torch.cuda.synchronize()
        assert bool((ws[:256] == 7).all()) and bool((ws[-256:] == 7).all())
        for f in (dx, dw):
            assert bool((f[0] == 7).all()) and bool((f[-1] == 7).all()) and bool((f[:, K:] == 7).all())
        assert bool((db[:32] == 7).all()) and bool((db[-32:] == 7).all())
        # a workspace's contents do not matter
        ws.fill_(255)
        again = gdn.linear_cross_entropy_backward(one, x, w, t, r["lse"], label_smoothing=0.1, want_dbias=True, workspace=ws[256:-256])
        assert all(torch.equal(again[k], b[k]) for k in b)


def test_no_rows():
    w = torch.randn((70, 16), device="cuda").to(BF16)
    x, t = torch.empty((0, 16), dtype=BF16, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    r = gdn.linear_cross_entropy(x, w, t)
    assert r["loss"].shape == (0,)
    b = gdn.linear_cross_entropy_backward(torch.ones(1, device="cuda"), x, w, t, r["lse"], want_dbias=True)
    assert b["dx"].shape == (0, 16) and bool((b["dw"] == 0).all()) and bool((b["dbias"] == 0).all())


def test_rows_of_many_calls():
    """A row's loss and lse within a range of rows do not depend on the others (tiles: of the same size)."""
    V, K = 5000, 136
    g, x, w, t = data(16, V, K, 64, ignored=False)
    whole = gdn.linear_cross_entropy(x, w, t)
    part = gdn.linear_cross_entropy(x[3:9], w, t[3:9])
    assert torch.equal(part["loss"], whole["loss"][3:9]) and torch.equal(part["lse"], whole["lse"][3:9])


def test_binding_refuses():
    g, x, w, t = data(6, 30, 16, 65)
    lse, one = torch.zeros(6, device="cuda"), torch.ones(1, device="cuda")
    for call in (lambda: gdn.linear_cross_entropy(x.float(), w, t), lambda: gdn.linear_cross_entropy(x, w[:, :8], t),
                 lambda: gdn.linear_cross_entropy(x, w, t[:5]), lambda: gdn.linear_cross_entropy(x, w, t.float()),
                 lambda: gdn.linear_cross_entropy(x, w, t.cpu()), lambda: gdn.linear_cross_entropy(x[0], w, t),
                 lambda: gdn.linear_cross_entropy(x, w, t, bias=torch.zeros(29, device="cuda")),
                 lambda: gdn.linear_cross_entropy_backward(lse[:3], x, w, t, lse),
                 lambda: gdn.linear_cross_entropy_backward(one, x, w, t, lse[:5]),
                 lambda: gdn.linear_cross_entropy_backward(one, x, w, t, lse, dx=torch.zeros((6, 16), device="cuda")),
                 lambda: gdn.linear_cross_entropy_backward(one, x, w, t, lse, dw=torch.zeros((29, 16), device="cuda", dtype=BF16))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: gdn.linear_cross_entropy(x, w, t, label_smoothing=1.0), lambda: gdn.linear_cross_entropy(x, w, t, z_loss=-1.0),
                 lambda: gdn.linear_cross_entropy(x[:, :12].contiguous(), w[:, :12].contiguous(), t),
                 lambda: gdn.linear_cross_entropy(x, w, t, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(gdn.GdnError):
            call()


@pytest.mark.parametrize("M", [9, 200])
def test_stream_and_graph(M):
    """On a stream of its own, and both passes captured, replayed on new inputs
    with eager calls in between."""
    V, K = 3000, 72
    g, x, w, t = data(M, V, K, 66)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    dloss = torch.ones(1, device="cuda") / M
    ref = gdn.linear_cross_entropy(x, w, t, z_loss=1e-4)
    side = gdn.linear_cross_entropy(x, w, t, z_loss=1e-4, stream=s)
    gs = gdn.linear_cross_entropy_backward(dloss, x, w, t, side["lse"], z_loss=1e-4, want_dbias=True, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(side["loss"], ref["loss"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = gdn.linear_cross_entropy(x, w, t, z_loss=1e-4)
        b = gdn.linear_cross_entropy_backward(dloss, x, w, t, r["lse"], z_loss=1e-4, want_dbias=True)
    for seed in range(3):
        _, x2, w2, t2 = data(M, V, K, 70 + seed)
        x.copy_(x2), w.copy_(w2), t.copy_(t2)
        graph.replay()
        torch.cuda.synchronize()
        eager = gdn.linear_cross_entropy(x, w, t, z_loss=1e-4)
        assert torch.equal(eager["loss"], r["loss"]) and torch.equal(eager["lse"], r["lse"])
        eb = gdn.linear_cross_entropy_backward(dloss, x, w, t, eager["lse"], z_loss=1e-4, want_dbias=True)
        assert all(torch.equal(eb[n], b[n]) for n in b)
    del gs


@pytest.mark.parametrize("one", [True, False])
def test_graph_of_a_large_call(one):
    """Captured with all rows counting, replayed with half of them, none, one
    and all: the tiles follow the targets that a replay finds."""
    M, V, K = 1300, 60001, 1032
    g, x, w, t = data(M, V, K, 69, ignored=False)
    t0 = t.clone()
    dloss = torch.randn(1 if one else M, generator=g, device="cuda")
    lse = gdn.linear_cross_entropy(x, w, t)["lse"]
    warm = gdn.linear_cross_entropy_backward(dloss, x, w, t, lse, want_dbias=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b = gdn.linear_cross_entropy_backward(dloss, x, w, t, lse, want_dbias=True)
    for share in (0.5, 0.0, 1.0, 0.9):
        t.copy_(torch.where(torch.rand(M, generator=g, device="cuda") < share, t0, -100))
        if share == 0.0:
            t[M - 1] = 3
        graph.replay()
        torch.cuda.synchronize()
        eager = gdn.linear_cross_entropy_backward(dloss, x, w, t, lse, want_dbias=True)
        assert all(torch.equal(eager[n], b[n]) for n in b), share
        if share == 1.0:
            assert all(torch.equal(warm[n], b[n]) for n in b)


@pytest.mark.parametrize("M, V, K", [(12, 400, 64), (130, 700, 72), (700, 3000, 1032), (500, 200000, 8), (1300, 60001, 1032)])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_dloss_not_finite(M, V, K, value):
    """The mean over no rows is 1 / 0 of nothing: a dloss that is not finite
    reaches the rows that count and no others, in calls of one piece, of several,
    with dx in parts, and in those that bring rows together."""
    g, x, w, t0 = data(M, V, K, 80, ignored=False)
    none, row = torch.full_like(t0, -100), M // 2
    for smooth in (0.0, 0.1):
        # no row counts: every gradient is zero
        lse = gdn.linear_cross_entropy(x, w, none, label_smoothing=smooth)["lse"]
        for dloss in (torch.full((1,), value, device="cuda"), torch.full((M,), value, device="cuda")):
            b = gdn.linear_cross_entropy_backward(dloss, x, w, none, lse, label_smoothing=smooth, want_dbias=True)
            assert all(bool((b[n] == 0).all()) for n in b)
        # one row: dl is `value` times what it is otherwise, column by column
        t = none.clone()
        t[row] = t0[row]
        lse = gdn.linear_cross_entropy(x, w, t, label_smoothing=smooth)["lse"]
        l = x[row:row + 1].double() @ w.double().t().contiguous()
        p = torch.exp(l - lse[row].double())[0]
        p[t[row]] -= 1 - smooth
        sure = (p - smooth / V).abs() > 1e-3 * smooth / V + 1e-30          # (its sign is known in 32 bits)
        dl = (p - smooth / V) * value
        dw = dl[:, None] * x[row].double()
        for dloss in (torch.full((1,), value, device="cuda"), torch.full((M,), value, device="cuda")):
            b = gdn.linear_cross_entropy_backward(dloss, x, w, t, lse, label_smoothing=smooth, want_dbias=True)
            assert int(sure.sum()) > V // 2
            assert bool(torch.isclose(b["dbias"].double()[sure], dl[sure], equal_nan=True).all())
            some = sure.nonzero()[:, 0]
            some = torch.cat([some[:500], t[row:row + 1]])
            assert bool(torch.isclose(b["dw"][some].double(), dw[some], equal_nan=True).all())
            others = torch.arange(M, device="cuda") != row
            assert bool((b["dx"][others] == 0).all()) and bool(b["dx"][row].isnan().all())


@pytest.mark.parametrize("M, V, K", [(12, 400, 64), (700, 3000, 1032), (1300, 60001, 1032)])
def test_dloss_of_one_row_not_finite(M, V, K):
    """The other rows' dx keep their bits, an ignored row's dloss is not looked at."""
    g, x, w, t = data(M, V, K, 81, ignored=False)
    t[3], t[M - 1] = -100, -100
    lse = gdn.linear_cross_entropy(x, w, t)["lse"]
    dloss = torch.randn(M, generator=g, device="cuda").clamp(-1, 1)
    dloss[0], dloss[5] = 1.0, 0.5
    want = gdn.linear_cross_entropy_backward(dloss, x, w, t, lse, want_dbias=True)
    dloss[3], dloss[M - 1] = float("nan"), float("inf")
    b = gdn.linear_cross_entropy_backward(dloss, x, w, t, lse, want_dbias=True)
    assert all(torch.equal(b[n], want[n]) for n in b)
    dloss[5] = float("inf")
    b = gdn.linear_cross_entropy_backward(dloss, x, w, t, lse, want_dbias=True)
    others = torch.arange(M, device="cuda") != 5
    assert torch.equal(b["dx"][others], want["dx"][others]) and bool(b["dx"][5].isnan().all())
    p = torch.exp(x[5:6].double() @ w.double().t().contiguous() - lse[5].double())[0]
    p[t[5]] -= 1
    assert bool(torch.isclose(b["dbias"].double(), p * float("inf")).all())


@pytest.mark.parametrize("M", [16, 200, 1300])
@pytest.mark.parametrize("smooth", [0.0, 0.1])
def test_no_loss_below_zero(M, smooth):
    """Rows that are sure of their target, and a vocabulary of one entry: the
    loss may round to zero and not below; a NaN stays one."""
    V, K = 900, 1032
    g, x, w, t = data(M, V, K, 82, scale=1.0, ignored=False)
    x = (w[t].float() * 60).to(BF16)
    r = gdn.linear_cross_entropy(x, w, t, label_smoothing=smooth)
    loss, lse, e, e_lse = loss64(x.cpu(), w.cpu(), None, t.cpu(), smooth, 0.0)[:4]
    close("loss", r["loss"], loss, e)
    assert bool((r["loss"] >= 0).all())
    one = gdn.linear_cross_entropy(x, w[:1].contiguous(), torch.zeros_like(t), label_smoothing=smooth)
    loss, _, e = loss64(x.cpu(), w[:1].cpu(), None, torch.zeros(M, dtype=torch.int64), smooth, 0.0)[:3]
    close("loss of one entry", one["loss"], loss, e)
    assert bool((one["loss"] >= 0).all())
    x[3, 5] = float("nan")
    assert bool(gdn.linear_cross_entropy(x, w, t, label_smoothing=smooth)["loss"][3].isnan())


@pytest.mark.parametrize("M", [9, 200])
def test_status_without_loss(M):
    """A call for lse alone reports a target outside the vocabulary too, and its
    lse has the bits of a call for both."""
    V, K = 300, 64
    g, x, w, t = data(M, V, K, 83, ignored=False)
    t[4] = -100
    want = gdn.linear_cross_entropy(x, w, t)["lse"]
    ws = torch.empty(gdn.linear_cross_entropy_workspace_bytes(M, V, K), dtype=torch.uint8, device="cuda")
    for bad in (None, V, -7):
        if bad is not None:
            t[5] = bad
        lse, status = torch.zeros(M, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        io = gdn.CLossIO(M, V, K, x.data_ptr(), K, w.data_ptr(), K, None, t.data_ptr(), 8, -100, 0.0, 0.0, None, lse.data_ptr(),
                         status.data_ptr())
        assert gdn.lib().gdn_linear_cross_entropy(ctypes.byref(io), ws.data_ptr(), ws.numel(),
                                                  torch.cuda.current_stream().cuda_stream) == gdn.GDN_OK
        assert int(status) == (0 if bad is None else gdn.GDN_STATUS_BAD_INDEX) and torch.equal(lse, want)


@pytest.mark.parametrize("M, V, K", [(451, 16323, 1120), (1183, 6517, 1256), (1921, 3970, 1232), (1267, 6485, 752), (1983, 8167, 400),
                                     (660, 13763, 568), (1922, 16144, 168)])
def test_wide_tiles(M, V, K):
    """Sizes that go to tiles of 256 x 128 on 256 compute units: the first four in
    the forward pass, the first three for dl, the last three for the products (in
    parts); the reference on the device in 64 bits."""
    g, x, w, t = data(M, V, K, M + 1)
    bias = torch.randn(V, generator=g, device="cuda")
    how = dict(bias=bias, label_smoothing=0.05, z_loss=1e-4)
    r = gdn.linear_cross_entropy(x, w, t, **how)
    loss, lse, e, e_lse = loss64(x, w, bias, t, 0.05, 1e-4)[:4]
    close("loss", r["loss"], loss.cpu(), e.cpu())
    close("lse", r["lse"], lse.cpu(), e_lse.cpu())
    for dloss in (torch.randn(M, generator=g, device="cuda"), torch.full((1,), 1 / M, device="cuda")):
        b = gdn.linear_cross_entropy_backward(dloss, x, w, t, r["lse"], **how)
        want, lim = loss_backward64(dloss, x, w, bias, t, r["lse"], 0.05, 1e-4)
        for name, v, l in zip(("dx", "dw", "dbias"), want, lim):
            close(name, b[name], v.cpu(), (l + (v.abs() + l) * HALF[b[name].dtype]).cpu())
        only = gdn.linear_cross_entropy_backward(dloss, x, w, t, r["lse"], want_dx=False, want_dbias=False, **how)
        assert torch.equal(only["dw"], b["dw"])


@pytest.mark.parametrize("M, V, K", [(199, 179, 23184), (1090, 5, 25200), (131, 1412, 14376), (4304, 197, 9456)])
def test_direct_products(M, V, K):
    """One piece without parts, whose dx its product writes: on tiles of 256 x 256
    (the first two) and of 256 x 128."""
    g, x, w, t = data(M, V, K, M + 2)
    r = gdn.linear_cross_entropy(x, w, t)
    loss, lse, e, e_lse = loss64(x, w, None, t, 0.0, 0.0)[:4]
    close("loss", r["loss"], loss.cpu(), e.cpu())
    close("lse", r["lse"], lse.cpu(), e_lse.cpu())
    for dloss in (torch.randn(M, generator=g, device="cuda"), torch.full((1,), 1 / M, device="cuda")):
        b = gdn.linear_cross_entropy_backward(dloss, x, w, t, r["lse"])
        want, lim = loss_backward64(dloss, x, w, None, t, r["lse"], 0.0, 0.0)
        for name, v, l in zip(("dx", "dw"), want, lim):
            close(name, b[name], v.cpu(), (l + (v.abs() + l) * HALF[BF16]).cpu())
        for name in b:
            only = gdn.linear_cross_entropy_backward(dloss, x, w, t, r["lse"], **{"want_" + n: n == name for n in b})
            assert torch.equal(only[name], b[name]), name
