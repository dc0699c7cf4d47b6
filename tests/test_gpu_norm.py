"""The norms on the device against their definition in 64 bits: rows of every
kernel's sizes and of one value, odd widths, strides and addresses, both types
of either side; nothing written outside; the same bits from call to call."""
import pytest
import torch

import gated_deltanet_linear_03_amd as gdn
from train_helpers import HALF, U, close, norm64, norm_backward64, norm_bounds

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
KIND = {True: gdn.GDN_NORM_LAYER, False: gdn.GDN_NORM_RMS}


def rows(g, M, D, dtype, pad, first, scale=1.0, offset=0.0):
    """[M, D] with rows `pad` elements apart that begin at element `first`."""
    flat = torch.full((M * (D + pad) + first + 8,), float("nan"), device="cuda", dtype=dtype)
    t = flat[first:first + M * (D + pad)].view(M, D + pad)[:, :D] if M else flat[:0].view(0, D)
    t.copy_((torch.randn((M, D), generator=g, device="cuda") * scale + offset).to(dtype))
    return t


DIMS = [1, 2, 3, 4, 7, 8, 9, 15, 16, 63, 64, 65, 100, 128, 129, 250, 256, 257, 500, 512, 513, 1000, 1023, 1024, 1025, 1500,
        2047, 2048, 2049, 4096, 4099, 8192, 8200, 12345, 16384, 16385, 32768, 33000, 70001]


@pytest.mark.parametrize("i", range(len(DIMS)), ids=[str(d) for d in DIMS])
@pytest.mark.parametrize("turn", range(4))
def test_norm(i, turn):
    D, k = DIMS[i], i + turn
    M = (1, 2, 5, 33, 300)[(i + 3 * turn) % 5] if D < 8000 else (1, 3, 7)[k % 3]
    xt, yt = (BF16, FP32)[turn % 2], (BF16, FP32)[turn // 2]
    layer = (i + turn // 2) % 2 == 0
    g = torch.Generator(device="cuda").manual_seed(1000 + 7 * i + turn)
    x = rows(g, M, D, xt, k % 3, k % 2, scale=1 + k % 4, offset=k % 5 - 2)
    w = torch.randn(D, generator=g, device="cuda") if k % 4 != 3 else None
    b = torch.randn(D, generator=g, device="cuda") if k % 3 != 2 else None
    out = rows(g, M, D, yt, 3 * (k % 2), (k + 1) % 2)
    stats = torch.empty((2, M), device="cuda")
    eps = (1e-5, 1e-3)[k % 2]
    y = gdn.norm(x, w, b, kind=KIND[layer], eps=eps, out=out, stats=stats)
    assert y is out
    cpu = [None if t is None else t.cpu() for t in (x, w, b)]
    want, mean, rstd = norm64(*cpu, layer, eps)
    e, e_mean, e_rstd = norm_bounds(*cpu, layer, eps)
    close("y", y, want, e + (want.abs() + e) * HALF[yt])
    close("mean", stats[0], mean, e_mean)
    close("rstd", stats[1], rstd, e_rstd)
    # the same bits in a dense call
    assert torch.equal(gdn.norm(x.contiguous(), w, b, kind=KIND[layer], eps=eps, out_dtype=yt), y)


@pytest.mark.parametrize("i", range(len(DIMS)), ids=[str(d) for d in DIMS])
@pytest.mark.parametrize("turn", range(4))
def test_backward(i, turn):
    D, k = DIMS[i], i + turn
    M = (1, 2, 5, 33, 300)[(i + 2 * turn) % 5] if D < 8000 else (1, 3, 7)[k % 3]
    xt, yt = (BF16, FP32)[turn % 2], (BF16, FP32)[turn // 2]
    layer = (i + turn // 2) % 2 == 1
    g = torch.Generator(device="cuda").manual_seed(2000 + 7 * i + turn)
    x = rows(g, M, D, xt, k % 3, k % 2, scale=1 + k % 4, offset=k % 5 - 2)
    dy = rows(g, M, D, yt, (k + 1) % 3, (k + 1) % 2)
    w = torch.randn(D, generator=g, device="cuda") if k % 4 != 3 else None
    skip = rows(g, M, D, xt, k % 2, 0) if k % 3 else None
    stats = torch.empty((2, M), device="cuda")
    gdn.norm(x, w, None, kind=KIND[layer], stats=stats)
    (dx, dw, db), (e, ew, eb) = norm_backward64(dy.cpu(), x.cpu(), None if w is None else w.cpu(), stats[0].cpu(), stats[1].cpu(),
                                                layer, None if skip is None else skip.cpu())
    r = gdn.norm_backward(dy, x, w, stats, kind=KIND[layer], d_residual=skip, want_dbias=True)
    assert set(r) == {"dx", "dweight", "dbias"} and r["dx"].dtype is xt
    close("dx", r["dx"], dx, e + (dx.abs() + e) * HALF[xt])
    close("dweight", r["dweight"], dw, ew)
    close("dbias", r["dbias"], db, eb)
    # each by itself, and dx over the skip connection's gradient
    for name in r:
        one = gdn.norm_backward(dy, x, w, stats, kind=KIND[layer], d_residual=skip,
                                **{"want_" + n: n == name for n in ("dx", "dweight", "dbias")})
        assert list(one) == [name] and torch.equal(one[name], r[name]), name
    if skip is not None:
        gdn.norm_backward(dy, x, w, stats, kind=KIND[layer], d_residual=skip, dx=skip, want_dweight=False)
        assert torch.equal(skip, r["dx"])


@pytest.mark.parametrize("M, D", [(5000, 64), (20011, 100), (3001, 2048), (4097, 1023), (2100, 4096), (40000, 8)])
@pytest.mark.parametrize("types", [(BF16, BF16), (FP32, BF16)])
def test_many_rows(M, D, types):
    """More rows than work-groups: each goes round several times."""
    g = torch.Generator(device="cuda").manual_seed(M)
    x, dy = rows(g, M, D, types[0], 0, 0, scale=2, offset=1), rows(g, M, D, types[1], 0, 0)
    w = torch.randn(D, generator=g, device="cuda")
    stats = torch.empty((2, M), device="cuda")
    y = gdn.norm(x, w, None, out_dtype=types[1], stats=stats)
    want, _, _ = norm64(x.cpu(), w.cpu(), None, True, 1e-5)
    e, _, _ = norm_bounds(x.cpu(), w.cpu(), None, True, 1e-5)
    close("y", y, want, e + (want.abs() + e) * HALF[types[1]])
    r = gdn.norm_backward(dy, x, w, stats, want_dbias=True)
    ref, lim = norm_backward64(dy.cpu(), x.cpu(), w.cpu(), stats[0].cpu(), stats[1].cpu(), True, None)
    for name, a, b in zip(("dx", "dweight", "dbias"), ref, lim):
        close(name, r[name], a, b + (a.abs() + b) * HALF[r[name].dtype])
    again = gdn.norm_backward(dy, x, w, stats, want_dbias=True)
    assert all(torch.equal(again[n], r[n]) for n in r)


def test_nothing_outside():
    """Guards around every written buffer, rows apart from each other."""
    M, D = 37, 1001
    g = torch.Generator(device="cuda").manual_seed(5)
    x, dy = rows(g, M, D, BF16, 0, 0), rows(g, M, D, BF16, 0, 0)
    w = torch.randn(D, generator=g, device="cuda")

    def guarded(n, dtype):
        return torch.full((n + 64,), 7.0, device="cuda", dtype=dtype)

    fy, fx, fs, fw, fb = guarded(M * (D + 3), BF16), guarded(M * (D + 3), BF16), guarded(2 * M, FP32), guarded(D, FP32), guarded(D, FP32)
    y, dx = (f[32:32 + M * (D + 3)].view(M, D + 3)[:, :D] for f in (fy, fx))
    stats, dw, db = fs[32:32 + 2 * M].view(2, M), fw[32:32 + D], fb[32:32 + D]
    fill = torch.full((gdn.norm_backward_workspace_bytes(M, D) + 512,), 7, device="cuda", dtype=torch.uint8)
    gdn.norm(x, w, None, out=y, stats=stats)
    gdn.norm_backward(dy, x, w, stats, dx=dx, dweight=dw, dbias=db, workspace=fill[256:-256])
    torch.cuda.synchronize()
    for f, n, width in ((fy, M, D), (fx, M, D)):
        assert bool((f[:32] == 7).all()) and bool((f[-32:] == 7).all())
        assert bool((f[32:-32].view(M, D + 3)[:, D:] == 7).all())
    for f in (fs, fw, fb):
        assert bool((f[:32] == 7).all()) and bool((f[-32:] == 7).all())
    assert bool((fill[:256] == 7).all()) and bool((fill[-256:] == 7).all())
    assert torch.equal(y, gdn.norm(x, w, None))


def test_rows_are_their_own():
    """Rows of zeros, a constant, infinities and NaN, and of tiny values: the
    others keep their bits."""
    M, D = 9, 300
    g = torch.Generator(device="cuda").manual_seed(6)
    x, dy = rows(g, M, D, FP32, 0, 0), rows(g, M, D, FP32, 0, 0)
    w = torch.randn(D, generator=g, device="cuda")
    plain = gdn.norm(x, w, None)
    odd = x.clone()
    odd[1], odd[3], odd[5, 7], odd[7, 2] = 0.0, 4.0, float("inf"), float("nan")
    odd[8] *= 1e-30
    y = gdn.norm(odd, w, None)
    assert torch.equal(y[[0, 2, 4, 6]], plain[[0, 2, 4, 6]])
    assert bool((y[1] == 0).all()) and bool((y[3] == 0).all()) and bool(y[5].isnan().any()) and bool(y[7].isnan().all())
    assert bool(y[8].isfinite().all()) and float(y[8].abs().max()) < 1e-20
    assert torch.equal(gdn.norm(x[2:3], w, None), plain[2:3])


@pytest.mark.parametrize("M,D", [(8191, 4096), (4097, 8190), (40000, 1024), (3, 2050)])
def test_bits_of_some_rows(M, D):
    """A row alone, among a few and among many (fewer than 2^25 values in all,
    or rows of up to 1024): the same bits."""
    g = torch.Generator(device="cuda").manual_seed(12)
    x = torch.randn(M, D, generator=g, device="cuda").to(BF16)
    w = torch.randn(D, generator=g, device="cuda")
    y = gdn.norm(x, w, w)
    for a, b in ((0, 1), (M - 1, M), (M // 2, M // 2 + 2), (1, min(M, 700))):
        assert torch.equal(gdn.norm(x[a:b], w, w), y[a:b])


def test_no_rows():
    x = torch.empty((0, 16), device="cuda")
    assert gdn.norm(x).shape == (0, 16)
    r = gdn.norm_backward(x, x, None, torch.empty((2, 0), device="cuda"), want_dbias=True)
    assert bool((r["dweight"] == 0).all()) and bool((r["dbias"] == 0).all()) and r["dx"].shape == (0, 16)


def test_binding_refuses():
    x = torch.zeros((4, 16), device="cuda")
    stats = torch.zeros((2, 4), device="cuda")
    for call in (lambda: gdn.norm(x[0]), lambda: gdn.norm(x.half()), lambda: gdn.norm(x.t()), lambda: gdn.norm(x.cpu()),
                 lambda: gdn.norm(x, torch.zeros(15, device="cuda")), lambda: gdn.norm(x, x[0].bfloat16()),
                 lambda: gdn.norm(x, out=torch.zeros((4, 15), device="cuda")),
                 lambda: gdn.norm(x, stats=torch.zeros((4, 2), device="cuda")), lambda: gdn.norm(x, out_dtype=torch.float16),
                 lambda: gdn.norm_backward(x, x, None, None), lambda: gdn.norm_backward(x[:, :8], x, None, stats),
                 lambda: gdn.norm_backward(x, x, None, stats, d_residual=x.bfloat16()),
                 lambda: gdn.norm_backward(x, x, None, stats, dweight=torch.zeros(16, device="cuda", dtype=BF16))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(gdn.GdnError):
        gdn.norm(x, kind=7)


def test_stream_and_graph():
    """On a stream of its own, and captured there and replayed on new inputs."""
    M, D = 130, 2048
    g = torch.Generator(device="cuda").manual_seed(8)
    x, dy, w = rows(g, M, D, BF16, 0, 0), rows(g, M, D, BF16, 0, 0), torch.randn(D, generator=g, device="cuda")
    stats = torch.empty((2, M), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(gdn.norm_backward_workspace_bytes(M, D), dtype=torch.uint8, device="cuda")
    y = gdn.norm(x, w, None, stats=stats, stream=s)
    r = gdn.norm_backward(dy, x, w, stats, want_dbias=True, workspace=ws, stream=s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.norm(x, w, None, out=y, stats=stats)
        gdn.norm_backward(dy, x, w, stats, workspace=ws, **r)
    for seed in (1, 2, 3):
        x.copy_(rows(torch.Generator(device="cuda").manual_seed(seed), M, D, BF16, 0, 0))
        graph.replay()
        torch.cuda.synchronize()
        st = torch.empty((2, M), device="cuda")
        assert torch.equal(gdn.norm(x, w, None, stats=st), y) and torch.equal(st, stats)
        eager = gdn.norm_backward(dy, x, w, st, want_dbias=True)
        assert all(torch.equal(eager[n], r[n]) for n in r)


@pytest.mark.parametrize("D", [1, 2, 3, 4, 5, 6, 7])
@pytest.mark.parametrize("M", [255, 2049, 20000, 100003])
def test_many_narrow_rows(M, D):
    """Rows of fewer than eight values, in one and in many work-groups, each of
    which goes round several times; strided, and dx over d_residual."""
    k = D + M
    xt, yt = (BF16, FP32)[k % 2], (BF16, FP32)[k // 2 % 2]
    layer = D % 2 == 0 or M == 2049
    g = torch.Generator(device="cuda").manual_seed(k)
    x, dy, skip = rows(g, M, D, xt, k % 3, k % 2, scale=2, offset=1), rows(g, M, D, yt, (k + 1) % 3, 1), rows(g, M, D, xt, 1, 0)
    w, b = torch.randn(D, generator=g, device="cuda"), torch.randn(D, generator=g, device="cuda") if M % 2 else None
    stats, out = torch.empty((2, M), device="cuda"), rows(g, M, D, yt, k % 2, 1)
    y = gdn.norm(x, w, b, kind=KIND[layer], out=out, stats=stats)
    cpu = [None if t is None else t.cpu() for t in (x, w, b)]
    want, mean, rstd = norm64(*cpu, layer, 1e-5)
    e, e_mean, e_rstd = norm_bounds(*cpu, layer, 1e-5)
    close("y", y, want, e + (want.abs() + e) * HALF[yt])
    close("mean", stats[0], mean, e_mean)
    close("rstd", stats[1], rstd, e_rstd)
    assert torch.equal(gdn.norm(x[:100], w, b, kind=KIND[layer], out_dtype=yt), y[:100])
    r = gdn.norm_backward(dy, x, w, stats, kind=KIND[layer], d_residual=skip, want_dbias=True)
    ref, lim = norm_backward64(dy.cpu(), x.cpu(), w.cpu(), stats[0].cpu(), stats[1].cpu(), layer, skip.cpu())
    for name, a, l in zip(("dx", "dweight", "dbias"), ref, lim):
        close(name, r[name], a, l + (a.abs() + l) * HALF[r[name].dtype])
    only = gdn.norm_backward(dy, x, w, stats, kind=KIND[layer], want_dx=False, want_dweight=False, want_dbias=True)
    assert list(only) == ["dbias"] and torch.equal(only["dbias"], r["dbias"])
    gdn.norm_backward(dy, x, w, stats, kind=KIND[layer], d_residual=skip, dx=skip, want_dweight=False)
    assert torch.equal(skip, r["dx"])


@pytest.mark.parametrize("D", [1, 4, 7, 8, 300])
def test_sums_over_many_rows(D):
    """The parameters' gradients of rows whose terms all have one sign: a value
    goes through at most 2^21 / 2^18 additions of its thread (rows of up to seven;
    the others' work-groups hold fewer rows: 2^21 / (4 x 1024)), 10 of the
    work-group's and 64 of the work-groups'."""
    M = (1 << 21) if D < 8 else (1 << 23) // D
    x = torch.zeros((M, D), device="cuda")
    x[:, 0] = 1.0
    stats = torch.zeros((2, M), device="cuda")
    stats[1] = 0.3
    dy = torch.full((M, D), 0.1, device="cuda")
    r = gdn.norm_backward(dy, x, None, stats, kind=gdn.GDN_NORM_RMS, want_dbias=True)
    steps = 10 + 64 + (8 if D < 8 else M // 4096 + 1)
    one, hat = float(dy[0, 0]), float(dy[0, 0]) * float(stats[1, 0])
    assert float((r["dbias"].double() / (M * one) - 1).abs().max()) <= steps * U
    assert abs(float(r["dweight"][0]) / (M * hat) - 1) <= (steps + 2) * U and bool((r["dweight"][1:] == 0).all())


MANY = [(1 << 25) // D + 1 for D in (1025, 2048, 2052, 4096, 4099, 8192, 8193, 12345, 16384)] + [150, 70]
WIDTHS = [1025, 2048, 2052, 4096, 4099, 8192, 8193, 12345, 16384, 16385, 40001]


@pytest.mark.parametrize("i", range(len(WIDTHS)), ids=[str(d) for d in WIDTHS])
@pytest.mark.parametrize("types", [(BF16, BF16), (BF16, FP32), (FP32, BF16), (FP32, FP32)])
@pytest.mark.parametrize("layer", [True, False])
def test_many_long_rows(i, types, layer):
    """From 2^25 values on rows of more than 1024 go to work-groups that stay, of
    128 to 1024 threads; in the backward pass each has several rows at every width,
    and in rows of more than 16384 the parameters' threads have.  The reference on
    the device in 64 bits."""
    M, D = MANY[i], WIDTHS[i]
    xt, yt = types
    k = i + layer
    g = torch.Generator(device="cuda").manual_seed(3000 + 8 * i + 2 * layer)
    x, dy = rows(g, M, D, xt, k % 3, k % 2, scale=2, offset=1), rows(g, M, D, yt, (k + 1) % 3, 0)
    skip = rows(g, M, D, xt, 0, 0) if k % 2 else None
    w, b = torch.randn(D, generator=g, device="cuda"), torch.randn(D, generator=g, device="cuda") if k % 3 else None
    stats = torch.empty((2, M), device="cuda")
    y = gdn.norm(x, w, b, kind=KIND[layer], out_dtype=yt, stats=stats)
    with torch.device("cuda"):
        want, mean, rstd = norm64(x, w, b, layer, 1e-5)
        e, e_mean, e_rstd = norm_bounds(x, w, b, layer, 1e-5)
    assert bool(((y.double() - want).abs() <= e + (want.abs() + e) * HALF[yt]).all())
    assert bool(((stats[0].double() - mean).abs() <= e_mean).all()) and bool(((stats[1].double() - rstd).abs() <= e_rstd).all())
    del want, e
    r = gdn.norm_backward(dy, x, w, stats, kind=KIND[layer], d_residual=skip, want_dbias=True)
    ref, lim = norm_backward64(dy, x, w, stats[0], stats[1], layer, skip)
    for name, a, l in zip(("dx", "dweight", "dbias"), ref, lim):
        assert bool(((r[name].double() - a).abs() <= l + (a.abs() + l) * HALF[r[name].dtype]).all()), name
    again = gdn.norm_backward(dy, x, w, stats, kind=KIND[layer], d_residual=skip, want_dbias=True)
    assert all(torch.equal(again[n], r[n]) for n in r)


@pytest.mark.parametrize("types", [(BF16, BF16), (BF16, FP32), (FP32, BF16), (FP32, FP32)])
@pytest.mark.parametrize("D", [32, 64, 128])
def test_whole_narrow_rows(types, D):
    """Rows that fill eight, sixteen or thirty-two threads to the last column."""
    xt, yt = types
    for M, layer in ((5, True), (3001, False)):
        g = torch.Generator(device="cuda").manual_seed(D + M)
        x, dy = rows(g, M, D, xt, 0, 0, scale=2, offset=1), rows(g, M, D, yt, 0, 0)
        w, b, stats = torch.randn(D, generator=g, device="cuda"), torch.randn(D, generator=g, device="cuda"), torch.empty((2, M), device="cuda")
        y = gdn.norm(x, w, b, kind=KIND[layer], out_dtype=yt, stats=stats)
        cpu = [t.cpu() for t in (x, w, b)]
        want = norm64(*cpu, layer, 1e-5)[0]
        e = norm_bounds(*cpu, layer, 1e-5)[0]
        close("y", y, want, e + (want.abs() + e) * HALF[yt])
        r = gdn.norm_backward(dy, x, w, stats, kind=KIND[layer], want_dbias=True)
        ref, lim = norm_backward64(dy.cpu(), x.cpu(), w.cpu(), stats[0].cpu(), stats[1].cpu(), layer, None)
        for name, a, l in zip(("dx", "dweight", "dbias"), ref, lim):
            close(name, r[name], a, l + (a.abs() + l) * HALF[r[name].dtype])
