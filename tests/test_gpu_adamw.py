"""The AdamW step on the device against its definition in 64 bits, states in
32 and in 8 bits: tensors of one element, that end inside a block, that begin
anywhere, more of them than a launch holds; what is left alone; graphs."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_03_amd as gdn
from train_helpers import U, adamw64, close, random_halves, up_or_down

pytestmark = pytest.mark.gpu

BF16, FP32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HALF16 = 2.0 ** -8


def tensors(sizes, seed, bits, grad, copy, first=0):
    """Parameters, gradients and states of a few steps' age, each tensor's
    buffers beginning `first` elements into theirs."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(n, scale, dtype=FP32):
        flat = torch.randn(n + first, generator=g, device="cuda") * scale
        return flat.to(dtype)[first:]

    p = [normal(n, 0.02) for n in sizes]
    grads = [normal(n, 1e-3, grad) for n in sizes]
    copies = [torch.zeros(n + first, device="cuda", dtype=BF16)[first:] for n in sizes] if copy else None
    m = [normal(n, 3e-4) for n in sizes]
    v = [(normal(n, 0.5).exp() * 1e-3) ** 2 for n in sizes]
    if bits == 32:
        return p, grads, dict(m=m, v=v, copies=copies)
    states = {k: [] for k in ("m", "v", "m_scale", "v_scale")}
    for i, n in enumerate(sizes):
        for name, value in (("m", m[i]), ("v", v[i].sqrt())):
            full = torch.zeros(-(-n // 256) * 256, device="cuda")
            full[:n] = value
            scale = full.view(-1, 256).abs().amax(1) / 448
            q = (full.view(-1, 256) / scale[:, None]).clamp(-448, 448).to(E4M3).view(-1)
            buf = torch.zeros(n + first, device="cuda", dtype=torch.uint8)
            buf[first:] = q[:n].view(torch.uint8)
            states[name].append(buf[first:].view(E4M3))
            states[name + "_scale"].append(scale)
    return p, grads, dict(states, copies=copies)


def f64(t):
    return t.float().double().cpu().numpy()


def check(before, opt, grads, lr, k, decay, factor=1.0):
    """opt's tensors after a step against `before`, copies of them before it."""
    p0, states = before
    for i, p in enumerate(opt.params):
        n = p.numel()
        if n == 0:
            continue
        g = f64(grads[i]) * factor
        m, v = f64(states["m"][i]), f64(states["v"][i])
        if opt.bits == 8:
            block = np.arange(n) // 256
            m, v = m * f64(states["m_scale"][i])[block], (v * f64(states["v_scale"][i])[block]) ** 2
        (p1, m1, v1), (ep, em, ev) = adamw64(f64(p0[i]), g, m, v, lr, opt.beta1, opt.beta2, opt.eps, decay[i], k)
        T = torch.from_numpy
        close(f"p {i}", p, T(p1), T(ep))
        if opt.copies[i] is not None:
            close(f"copy {i}", opt.copies[i], T(p1), T(ep + HALF16 * (np.abs(p1) + ep)))
        if opt.bits == 32:
            close(f"m {i}", opt.m[i], T(m1), T(em))
            close(f"v {i}", opt.v[i], T(v1), T(ev))
            continue
        lo, hi = random_halves(opt.seed, k, i, n)
        for name, value, e, u in (("m", m1, em, lo), ("v", np.sqrt(v1), 6 * U * np.sqrt(v1), hi)):
            full = np.zeros(-(-n // 256) * 256)
            full[:n] = np.abs(value)
            fe = np.zeros_like(full)
            fe[:n] = e
            scale = full.reshape(-1, 256).max(1) / 448
            close(f"{name} scale {i}", getattr(opt, name + "_scale")[i], T(scale),
                  T(fe.reshape(-1, 256).max(1) / 448 + 3 * U * scale + 1e-37))
            with np.errstate(invalid="ignore", divide="ignore"):
                ratio = np.where(scale[block] > 0, value / scale[block], 0.0)
            want, near = up_or_down(np.clip(ratio, -448, 448), u)
            if name == "v":
                want = np.where((want == 0) & (value > 0), 2.0 ** -9, want)
            # m' is a difference that may have lost more than its own last bits
            near |= e > 16 * U * np.abs(value)
            got = f64(getattr(opt, name)[i])
            off = got != want
            assert not (off & ~near).any(), f"{name} {i}: {int((off & ~near).sum())} codes, first at {np.nonzero(off & ~near)[0][:3]}"
            step = np.exp2(np.floor(np.log2(np.maximum(np.abs(ratio), 2.0 ** -6))) - 3)
            assert bool((np.abs(got - ratio) <= step * (1 + 1e-5)).all() | (near.any())), f"{name} {i}: not a neighbour"
            assert off.mean() < 1e-3


def copy_of(p, states):
    return [t.clone() for t in p], {k: [t.clone() for t in v] for k, v in states.items() if k != "copies" and v is not None}


SIZES = [[1], [255], [256], [257], [4095, 4096, 4097], [1, 2, 3, 5, 1023, 70000], [0, 300, 0, 12], [262147, 33]]


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("i", range(len(SIZES)), ids=["+".join(map(str, s)) for s in SIZES])
def test_step(i, bits):
    sizes = SIZES[i]
    grad = (BF16, FP32)[(i + bits // 8) % 2]
    p, grads, states = tensors(sizes, 50 + i, bits, grad, i % 3 != 1, first=i % 3)
    decay = [0.1 * (k % 2) for k in range(len(sizes))]
    opt = gdn.AdamW(p, **states, beta1=0.9, beta2=(0.999, 0.95)[i % 2], eps=1e-8, weight_decay=decay, seed=77 + i)
    for k in (1, 2, 1000):
        before = copy_of(p, states)
        gdn.adamw_step(opt, grads, lr=3e-3, step=k)
        check(before, opt, grads, 3e-3, k, decay)


@pytest.mark.parametrize("bits", [8, 32])
def test_more_tensors_than_a_launch_holds(bits):
    sizes = [(37 * i) % 700 + 1 for i in range(101)]
    p, grads, states = tensors(sizes, 9, bits, FP32, True)
    opt = gdn.AdamW(p, **states, weight_decay=0.01, seed=3)
    before = copy_of(p, states)
    gdn.adamw_step(opt, grads, lr=1e-3, step=5)
    check(before, opt, grads, 1e-3, 5, [0.01] * len(sizes))


@pytest.mark.parametrize("bits", [8, 32])
def test_from_zero_states(bits):
    """The first step moves every parameter with a gradient by lr (eps apart),
    the others decay only."""
    p = [torch.randn(1000, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4))]
    grads = [torch.randn(1000, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))]
    grads[0][::3] = 0
    opt = gdn.AdamW(p, **gdn.adamw_states(p, bits), weight_decay=0.5)
    old = p[0].double().cpu()
    gdn.adamw_step(opt, grads, lr=1e-2, step=1)
    g = grads[0].double().cpu()
    want = old * (1 - 0.5e-2) - 1e-2 * g / (g.abs() + 1e-8)
    close("p", p[0], want, 4 * U * old.abs() + 1e-2 * 30 * U)
    if bits == 8:
        zero = g == 0
        assert bool((opt.m[0].float().cpu()[zero] == 0).all()) and bool((opt.v[0].float().cpu()[zero] == 0).all())
        # no positive r has gone to zero
        assert bool((opt.v[0].float().cpu()[~zero] > 0).all())


def test_rounding_keeps_the_mean():
    """A state of 2^20 elements over 16 steps with nothing but decay in sight:
    the sum of m falls as beta1 says.  Each rounding is off by less than a step,
    with a mean of 0 and at most half a step's deviation: 6 deviations."""
    n = 1 << 20
    p, g = [torch.zeros(n, device="cuda")], [torch.zeros(n, device="cuda")]
    value = torch.rand(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) * 0.9 + 0.1
    st = gdn.adamw_states(p, 8)
    st["m_scale"][0].fill_(1.0 / 448)
    st["m"][0].copy_((value * 448).to(E4M3))
    opt = gdn.AdamW(p, **st, seed=9)
    total = float((st["m"][0].double() / 448).sum())
    for k in range(1, 17):
        gdn.adamw_step(opt, g, lr=0.0, step=k)
    now = (st["m"][0].double() * st["m_scale"][0].double().repeat_interleave(256)).sum()
    # a step of e4m3 is at most an eighth of its value, here at most 1/8; 16 of them, sqrt(n) each
    assert abs(float(now) - total * 0.9 ** 16) < 6 * (n * 16) ** 0.5 / 16
    # the same rounding to the nearest would have moved it by far more than that
    assert 6 * (n * 16) ** 0.5 / 16 < 0.02 * total * 0.9 ** 16


def test_extremes():
    """Gradients of the largest and the smallest sizes, infinities and NaN: a
    block's neighbours are untouched, a finite state stays finite."""
    n = 1024
    p, grads, states = tensors([n], 12, 8, FP32, True)
    q, _, other = tensors([n], 12, 8, FP32, True)
    plain = [grads[0].clone()]
    grads[0][300:303] = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda")
    grads[0][600] = 1e-30
    grads[0][900] = 1e15
    a, b = gdn.AdamW(p, **states, seed=1), gdn.AdamW(q, **other, seed=1)
    gdn.adamw_step(a, grads, lr=1e-3, step=3)
    gdn.adamw_step(b, plain, lr=1e-3, step=3)
    for x, y in ((p, q), (states["m"], other["m"]), (states["v"], other["v"])):
        assert torch.equal(x[0][:256].float(), y[0][:256].float())
    assert bool(p[0][300].isnan()) and bool(states["m"][0][300].float().isnan()) and bool(states["v"][0][300].float().isnan())
    far = torch.ones(n, dtype=torch.bool)
    far[300:303] = False
    assert bool(p[0].cpu()[far].isfinite().all()) and bool(states["m_scale"][0][2:].isfinite().all())
    assert float(states["m"][0][900].float()) == 448 and float(states["v"][0][900].float()) == 448
    # next to such a neighbour all others are at the format's least, none at zero
    assert bool((states["v"][0][768:1024].float() > 0).all())


def test_grad_scale_and_device_numbers():
    sizes = [1000, 333]
    for bits in (8, 32):
        p, grads, states = tensors(sizes, 21, bits, BF16, True)
        opt = gdn.AdamW(p, **states, weight_decay=0.1, seed=2)
        lr, step, factor = torch.tensor([2e-3], device="cuda"), torch.tensor([7], dtype=torch.int32, device="cuda"), torch.tensor([0.25], device="cuda")
        before = copy_of(p, states)
        gdn.adamw_step(opt, grads, lr=lr, step=step, grad_scale=factor)
        check(before, opt, grads, float(lr), 7, [0.1, 0.1], factor=0.25)
        for bad in (float("nan"), float("inf")):
            before = copy_of(p, states)
            factor.fill_(bad)
            gdn.adamw_step(opt, grads, lr=lr, step=step, grad_scale=factor)
            assert all(torch.equal(a, b) for a, b in zip(before[0], p))
            assert all(torch.equal(a.float(), b.float()) for k in before[1] for a, b in zip(before[1][k], states[k]))


@pytest.mark.parametrize("bits", [8, 32])
def test_captured_steps(bits):
    """A captured step follows the learning rate and the step number on the device."""
    sizes = [5000, 77, 256]
    p, grads, states = tensors(sizes, 31, bits, BF16, False)
    q, _, other = tensors(sizes, 31, bits, BF16, False)
    opt, eager = gdn.AdamW(p, **states, seed=4), gdn.AdamW(q, **other, seed=4)
    lr, step = torch.tensor([1e-3], device="cuda"), torch.tensor([0], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step += 1
        gdn.adamw_step(opt, grads, lr=lr, step=step)
    for k in range(1, 5):
        rate = 1e-3 / k
        lr.fill_(rate)
        graph.replay()
        torch.cuda.synchronize()
        gdn.adamw_step(eager, grads, lr=float(torch.tensor(rate, dtype=FP32)), step=k)
        assert all(torch.equal(a, b) for a, b in zip(p, q))
        for name in ("m", "v"):
            assert all(torch.equal(a.float(), b.float()) for a, b in zip(states[name], other[name]))


def test_nothing_outside():
    """Guards around every buffer of an odd-sized tensor."""
    n = 1000
    for bits in (8, 32):
        p, grads, states = tensors([n + 64], 41, bits, FP32, True)
        all_of = [p[0], states["m"][0], states["v"][0], states["copies"][0]]
        inner = [t[32:32 + n] for t in all_of]
        scales = {}
        if bits == 8:
            sm, sv = torch.full((6,), 0.5, device="cuda"), torch.full((6,), 0.5, device="cuda")
            scales = dict(m_scale=[sm[1:5]], v_scale=[sv[1:5]])
        old = [t.clone() for t in all_of]
        opt = gdn.AdamW([inner[0]], [inner[1]], [inner[2]], copies=[inner[3]], **scales)
        gdn.adamw_step(opt, [grads[0][32:32 + n]], lr=1e-3, step=2)
        for a, b in zip(all_of, old):
            assert torch.equal(a[:32].float(), b[:32].float()) and torch.equal(a[32 + n:].float(), b[32 + n:].float())
        assert not torch.equal(all_of[0], old[0])
        if bits == 8:
            assert float(sm[0]) == float(sm[5]) == float(sv[0]) == float(sv[5]) == 0.5


def test_tensors_without_a_gradient():
    """They are left as they are, and the others' random bits do not move."""
    sizes = [300, 5, 1000]
    p, grads, states = tensors(sizes, 51, 8, FP32, True)
    opt = gdn.AdamW(p, **states, weight_decay=0.1, seed=6)
    before = copy_of(p, states)
    gdn.adamw_step(opt, [grads[0], None, grads[2]], lr=1e-3, step=4)
    assert torch.equal(p[1], before[0][1]) and all(torch.equal(states[k][1].float(), before[1][k][1].float()) for k in before[1])
    q, _, other = tensors(sizes, 51, 8, FP32, True)
    full = gdn.AdamW(q, **other, weight_decay=0.1, seed=6)
    gdn.adamw_step(full, grads, lr=1e-3, step=4)
    for i in (0, 2):
        assert torch.equal(p[i], q[i]) and all(torch.equal(states[k][i].float(), other[k][i].float()) for k in before[1])


def test_shared_memory_is_refused():
    """The same tensor twice, and a state inside another's."""
    a, b = torch.zeros(100, device="cuda"), torch.zeros(100, device="cuda")
    st = gdn.adamw_states([a, b])
    with pytest.raises(ValueError, match="share memory"):
        gdn.AdamW([a, a], **st)
    with pytest.raises(ValueError, match="share memory"):
        gdn.AdamW([a, b], m=[st["m"][0], st["m"][0]], v=st["v"])
    flat = torch.zeros(150, device="cuda")
    with pytest.raises(ValueError, match="share memory"):
        gdn.AdamW([flat[:100], flat[50:]], **st)
    gdn.AdamW([flat[:100], flat[100:]], **gdn.adamw_states([flat[:100], flat[100:]]))


def test_binding_refuses():
    p = [torch.zeros(10, device="cuda")]
    st = gdn.adamw_states(p)
    opt = gdn.AdamW(p, **st)
    g = [torch.zeros(10, device="cuda")]
    for call in (lambda: gdn.AdamW(p, st["m"], []), lambda: gdn.AdamW([p[0].bfloat16()], **st), lambda: gdn.AdamW([p[0].cpu()], **st),
                 lambda: gdn.AdamW(p, **st, m_scale=[g[0]]), lambda: gdn.AdamW(p, **st, weight_decay=[0.1, 0.2]),
                 lambda: gdn.AdamW(p, **st, copies=[g[0]]), lambda: gdn.AdamW([torch.zeros(10, 2, device="cuda")[:, 0]], **st),
                 lambda: gdn.AdamW(p, **dict(gdn.adamw_states(p, 8), m_scale=[torch.zeros(2, device="cuda")])),
                 lambda: gdn.adamw_states(p, 4), lambda: gdn.adamw_step(opt, [], lr=1e-3, step=1),
                 lambda: gdn.adamw_step(opt, [g[0][:9]], lr=1e-3, step=1), lambda: gdn.adamw_step(opt, [g[0].half()], lr=1e-3, step=1),
                 lambda: gdn.adamw_step(opt, g, lr=torch.zeros(2, device="cuda"), step=1),
                 lambda: gdn.adamw_step(opt, g, lr=1e-3, step=torch.ones(1, device="cuda")),
                 lambda: gdn.adamw_step(opt, g, lr=1e-3, step=1, grad_scale=torch.ones(1))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(gdn.GdnError):
        gdn.adamw_step(opt, g, lr=1e-3, step=0)
    assert float(p[0].abs().max()) == 0


@pytest.mark.parametrize("bits", [8, 32])
def test_moved_memory(bits):
    """A parameter with other memory than at the start is refused; states that
    the caller lets go of stay alive."""
    p = [torch.ones(300, device="cuda"), torch.ones(70, device="cuda")]
    st = gdn.adamw_states(p, bits)
    opt = gdn.AdamW(p, **st)
    was = opt._held[0]
    p[0].data = torch.full((300,), 2.0, device="cuda")
    g = [torch.ones_like(x) for x in p]
    with pytest.raises(ValueError, match="memory"):
        gdn.adamw_step(opt, g, lr=1e-2, step=1)
    assert float((was - 1).abs().max()) == 0 and float((p[0] - 2).abs().max()) == 0 and float((p[1] - 1).abs().max()) == 0
    opt = gdn.AdamW(p, **st)
    for t in st["m"] + st["v"]:
        t.data = torch.empty(0, dtype=t.dtype, device="cuda")
    gdn.adamw_step(opt, g, lr=1e-2, step=1)
    assert float((p[0] - 1.99).abs().max()) < 1e-5 and float((p[1] - 0.99).abs().max()) < 1e-5


@pytest.mark.parametrize("grad", [BF16, FP32])
def test_codes_to_the_last(grad):
    """Scales and codes of 8-bit states are the formula's, none but by a border:
    in 64 bits from the states as they stand in 32, over scales in 32."""
    rng = np.random.RandomState(19)
    sizes = [int(n) for n in rng.randint(1, 700, 200)] + [70001]
    p, grads, states = tensors(sizes, 91, 8, grad, False, first=1)
    opt = gdn.AdamW(p, **states, beta1=0.9, beta2=0.95, seed=4)
    old = {k: [f64(t) for t in states[k]] for k in ("m", "v", "m_scale", "v_scale")}
    gdn.adamw_step(opt, grads, lr=1e-3, step=33)
    for i, n in enumerate(sizes):
        block = np.arange(n) // 256
        m, r = ((old[k][i] * old[k + "_scale"][i][block]).astype(np.float32) for k in ("m", "v"))
        g, v = f64(grads[i]), (r * r).astype(np.float64)
        lo, hi = random_halves(4, 33, i, n)
        for name, value, u in (("m", opt.beta1 * m.astype(np.float64) + (1 - opt.beta1) * g, lo),
                               ("v", np.sqrt(opt.beta2 * v + (1 - opt.beta2) * g * g), hi)):
            full = np.zeros(-(-n // 256) * 256)
            full[:n] = np.abs(value)
            scale = f64(getattr(opt, name + "_scale")[i])
            assert (scale == (full.reshape(-1, 256).max(1) / 448).astype(np.float32)).all(), (name, i)
            want = up_or_down(np.clip(value / scale[block], -448, 448), u)[0]
            if name == "v":
                want = np.where((want == 0) & (value > 0), 2.0 ** -9, want)
            assert (f64(getattr(opt, name)[i]) == want).all(), (name, i)


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("how", ["data", "entry"])
def test_moved_states_and_copies(bits, how):
    """A bf16 copy or a state with other memory than at the start, by its data
    or as another tensor in its list, is refused and nothing is written; the
    step goes on once it is back, and where copies were let go."""
    p = [torch.ones(n, device="cuda") for n in (300, 70, 0)]
    g = [torch.ones_like(x) for x in p]
    st = gdn.adamw_states(p, bits)
    copies = [torch.ones(300, device="cuda", dtype=BF16), None, torch.ones(0, device="cuda", dtype=BF16)]
    opt = gdn.AdamW(p, **st, copies=copies)
    for name in ["m", "v", "copies"] + ["m_scale", "v_scale"] * (bits == 8):
        t = getattr(opt, name)[0]
        other, was = t.clone(), t.data
        if how == "data":
            t.data = other
        else:
            getattr(opt, name)[0] = other
        with pytest.raises(ValueError, match=rf"opt\.{name}\[0\].*memory"):
            gdn.adamw_step(opt, g, lr=1e-2, step=1)
        assert all(float((x - 1).abs().sum()) == 0 for x in p) and float((was.float() - other.float()).abs().max()) == 0
        if how == "data":
            t.data = was
        else:
            getattr(opt, name)[0] = t
    opt.copies[1] = torch.ones(70, device="cuda", dtype=BF16)
    with pytest.raises(ValueError, match=r"opt\.copies\[1\]"):
        gdn.adamw_step(opt, g, lr=1e-2, step=1)
    opt.copies[1] = None
    opt.m.append(opt.m[0])
    with pytest.raises(ValueError, match=r"opt\.m: 3 entries"):
        gdn.adamw_step(opt, g, lr=1e-2, step=1)
    opt.m.pop()
    gdn.adamw_step(opt, g, lr=1e-2, step=1)
    assert float((copies[0].float() - 0.99).abs().max()) < 2.0 ** -8 and float((p[0] - 0.99).abs().max()) < 1e-5
    copies[0].data = torch.empty(0, device="cuda", dtype=BF16)
    gdn.adamw_step(opt, g, lr=1e-2, step=2)
    opt.copies = [None] * 3
    gdn.adamw_step(opt, g, lr=1e-2, step=3)
    assert float((p[0] - 0.97).abs().max()) < 1e-5
    # a list that had none
    bare = gdn.AdamW([torch.ones(5, device="cuda")], **gdn.adamw_states([torch.ones(5, device="cuda")], bits))
    bare.copies = [torch.ones(5, device="cuda", dtype=BF16)]
    with pytest.raises(ValueError, match=r"opt\.copies\[0\]"):
        gdn.adamw_step(bare, [torch.ones(5, device="cuda")], lr=1e-2, step=1)


@pytest.mark.parametrize("bits", [8, 32])
def test_changed_weight_decay(bits):
    """A weight decay that was changed since, one of the list or all of them,
    holds from the next step on, as the other numbers of the object do."""
    p = [torch.ones(300, device="cuda"), torch.ones(70, device="cuda")]
    g = [torch.zeros_like(x) for x in p]
    opt = gdn.AdamW(p, **gdn.adamw_states(p, bits), weight_decay=0.0)
    want = [1.0, 1.0]
    for new in (0.0, [0.5, 0.0], 0.25, "entry", (0.0, 0.125)):
        if new == "entry":
            opt.weight_decay = [0.25, 0.25]
            gdn.adamw_step(opt, g, lr=0.0, step=1)
            opt.weight_decay[1] = 0.5
        else:
            opt.weight_decay = new
        gdn.adamw_step(opt, g, lr=0.5, step=1)
        each = [0.25, 0.5] if new == "entry" else list(new) if isinstance(new, (list, tuple)) else [new] * 2
        want = [w * (1 - 0.5 * d) for w, d in zip(want, each)]            # (exact: few bits)
        assert [float(x.min()) for x in p] == [float(x.max()) for x in p] == want
    opt.weight_decay = [0.1]
    with pytest.raises(ValueError, match="weight_decay: 2 entries"):
        gdn.adamw_step(opt, g, lr=0.5, step=1)
    opt.weight_decay = -1.0
    with pytest.raises(gdn.GdnError, match="weight_decay"):
        gdn.adamw_step(opt, g, lr=0.5, step=1)
    opt.weight_decay = 0.0
    gdn.adamw_step(opt, g, lr=0.5, step=1)
    assert [float(x.max()) for x in p] == want


@pytest.mark.parametrize("grad", [BF16, FP32])
def test_ties(grad):
    """Blocks with many largest values: all of one size, of both signs, from two
    pairs of a state and a gradient that differ by less than 32 bits tell, and of
    one value among zeros: scales and codes to the last, as of any other block."""
    rng = np.random.RandomState(23)
    n = 256 * 12 + 100
    p, grads, states = tensors([n], 92, 8, grad, False)
    m, v, g = (np.zeros(n, dtype=np.float32) for _ in range(3))
    block = np.arange(n) // 256
    sign = np.where(rng.rand(n) < 0.5, -1, 1)
    half = rng.rand(n) < 0.5
    ulp = np.float32(2.0 ** -24)
    g[block < 4] = 1e-3                                     # one value
    g[(block >= 2) & (block < 4)] *= sign[(block >= 2) & (block < 4)]
    m[block == 3] = 448 * sign[block == 3]                  # a state of the same or the other sign
    for b in (4, 5, 6, 7):                                  # m' = 0.9 m + 0.1 g: 0.9 * 448 s or 0.1 g, nearly as large
        here = block == b
        m[here & half] = 448
        g[here & ~half] = np.float32(0.9 * 448 / 0.1 * 2.0 ** -12) * (1 + (b - 5) * ulp * 2)
        v[here & half] = 448
    g[256 * 8 + 77] = -1e-3
    m[256 * 9] = v[256 * 9 + 255] = 448
    m[block == 10], v[block == 10] = 416 * sign[block == 10], 3.5
    g[block == 12] = rng.choice([1e-3, -1e-3, 0.0], 100)
    scale = np.float32(2.0 ** -12)
    states["m"][0].copy_(torch.from_numpy(m)), states["v"][0].copy_(torch.from_numpy(v))
    for k in ("m_scale", "v_scale"):
        states[k][0].fill_(float(scale))
    grads[0].copy_(torch.from_numpy(g))
    opt = gdn.AdamW(p, **states, beta1=0.9, beta2=0.95, seed=6)
    g64 = f64(grads[0])
    gdn.adamw_step(opt, grads, lr=1e-3, step=3)
    lo, hi = random_halves(6, 3, 0, n)
    r = (v * scale).astype(np.float32)
    for name, value, u in (("m", 0.9 * (m * scale).astype(np.float64) + (1 - 0.9) * g64, lo),
                           ("v", np.sqrt(0.95 * (r * r).astype(np.float64) + (1 - 0.95) * g64 * g64), hi)):
        full = np.zeros(-(-n // 256) * 256)
        full[:n] = np.abs(value)
        got = f64(getattr(opt, name + "_scale")[0])
        assert (got == (full.reshape(-1, 256).max(1) / 448).astype(np.float32)).all(), name
        with np.errstate(invalid="ignore", divide="ignore"):
            ratio = np.where(got[block] > 0, value / got[block], 0.0)
        want = up_or_down(np.clip(ratio, -448, 448), u)[0]
        if name == "v":
            want = np.where((want == 0) & (value > 0), 2.0 ** -9, want)
        assert (f64(getattr(opt, name)[0]) == want).all(), name


@pytest.mark.parametrize("first", [False, True])
def test_small_gradients(first):
    """8-bit states where v' leaves the range of 32 bits: gradients of 1e-17 to
    1e-28, alone in their blocks and beside ordinary ones, from zero states and
    from states as small: codes and scales to the last (a scale is 0 where the
    largest magnitude is below 2^-100, and no positive r is rounded to 0)."""
    rng = np.random.RandomState(29)
    sizes = [10 ** -k for k in range(17, 29)]
    n = 256 * 2 * len(sizes) + 50
    g = np.zeros(n, dtype=np.float32)
    for k, size in enumerate(sizes):
        g[512 * k:512 * k + 512] = rng.randn(512) * size
        g[512 * k + 256 + 5 * k] = 1e-3                     # the second block of each: beside this one
    g[-50:] = 1e-24
    g[::7] = 0
    p = [torch.zeros(n, device="cuda")]
    st = gdn.adamw_states(p, 8)
    if not first:                                           # the states that a few steps of other gradients leave
        opt = gdn.AdamW(p, **st, beta1=0.9, beta2=0.95, seed=8)
        for k in range(1, 4):
            gdn.adamw_step(opt, [torch.from_numpy(np.roll(g, k)).cuda()], lr=0.0, step=k)
    old = {k: f64(st[k][0]) for k in st}
    opt = gdn.AdamW(p, **st, beta1=0.9, beta2=0.95, seed=9, eps=1e-8)
    gdn.adamw_step(opt, [torch.from_numpy(g).cuda()], lr=1e-3, step=4)
    block = np.arange(n) // 256
    m, r = ((old[k] * old[k + "_scale"][block]).astype(np.float32) for k in ("m", "v"))
    g64, square = g.astype(np.float64), (r * r).astype(np.float64)
    v = np.where(square < 2.0 ** -96, r.astype(np.float64) ** 2, square)
    lo, hi = random_halves(9, 4, 0, n)
    for name, value, u in (("m", 0.9 * m.astype(np.float64) + (1 - 0.9) * g64, lo),
                           ("v", np.sqrt(0.95 * v + (1 - 0.95) * g64 * g64), hi)):
        full = np.zeros(-(-n // 256) * 256)
        full[:n] = np.abs(value)
        top = full.reshape(-1, 256).max(1)
        got = f64(getattr(opt, name + "_scale")[0])
        assert (got == np.where(top < 2.0 ** -100, 0.0, top / 448).astype(np.float32)).all(), name
        assert first is False or name == "m" or int((got > 0).sum()) >= 2 * len(sizes)       # 1e-28 has an r above 2^-100
        with np.errstate(invalid="ignore", divide="ignore"):
            ratio = np.where(got[block] > 0, value / got[block], 0.0)
        want = up_or_down(np.clip(ratio, -448, 448), u)[0]
        if name == "v":
            want = np.where((want == 0) & (value > 0) & (got[block] > 0), 2.0 ** -9, want)
        assert (f64(getattr(opt, name)[0]) == want).all(), name


@pytest.mark.parametrize("bits", [8, 32])
def test_no_eps(bits):
    """A first step without eps is lr long whatever the gradient's size, as long
    as 32 bits hold v' (8 bits: r): in 32 bits below 2^-126 with what they lose
    of it, half of 2^-149."""
    size = torch.tensor([10.0 ** -k for k in range(0, 21)], dtype=torch.float64)
    g = size.float().repeat(20).cuda()
    p = [torch.zeros(g.numel(), device="cuda")]
    opt = gdn.AdamW(p, **gdn.adamw_states(p, bits), eps=0.0)
    gdn.adamw_step(opt, [g], lr=1.0, step=1)
    v = (1 - 0.999) * g.double().cpu() ** 2
    # v' and its root, c1 and c2, the reciprocal: adamw64's count; v' may lose two halves of its least bit (product, sum)
    lost = 2 * 2.0 ** -150 / v if bits == 32 else torch.zeros_like(v)
    close("p", p[0], -torch.ones_like(v), 30 * U + lost)


@pytest.mark.parametrize("grad", [BF16, FP32])
def test_every_code_is_a_neighbour(grad):
    """Every element's new code, those next to a border and those whose m' is a
    difference too, is one of the two values of the format around its ratio to
    the scale (in 64 bits, over the scale in 32): within a step of it, and on its
    side of zero."""
    rng = np.random.RandomState(31)
    sizes = [int(n) for n in rng.randint(1, 900, 100)] + [200003]
    p, grads, states = tensors(sizes, 93, 8, grad, False)
    for i in range(0, len(sizes), 2):                       # m' next to nothing of either term
        m = states["m"][i].float() * states["m_scale"][i].repeat_interleave(256)[:sizes[i]]
        grads[i].copy_(-9 * m * (1 + 1e-6 * torch.randn(sizes[i], device="cuda", generator=torch.Generator(device="cuda").manual_seed(i))))
    opt = gdn.AdamW(p, **states, beta1=0.9, beta2=0.999, seed=5)
    for k in (1, 2):
        old = {n: [f64(t) for t in getattr(opt, n)] for n in ("m", "v", "m_scale", "v_scale")}
        gdn.adamw_step(opt, grads, lr=1e-3, step=k)
        for i, n in enumerate(sizes):
            block = np.arange(n) // 256
            m, r = ((old[q][i] * old[q + "_scale"][i][block]).astype(np.float32) for q in ("m", "v"))
            g = f64(grads[i])
            for name, value in (("m", 0.9 * m.astype(np.float64) + (1 - 0.9) * g),
                                ("v", np.sqrt(0.999 * (r * r).astype(np.float64) + (1 - 0.999) * g * g))):
                scale = f64(getattr(opt, name + "_scale")[i])[block]
                ratio = np.where(scale > 0, value / np.where(scale > 0, scale, 1), 0.0)
                got = f64(getattr(opt, name)[i])
                unit = np.exp2(np.floor(np.log2(np.maximum(np.abs(ratio), 2.0 ** -6))) - 3)
                # (64 bits are exact to 2^-50 of the terms, which are at most 10 times the block's largest where m' cancels)
                assert bool((np.abs(got - ratio) <= unit * (1 + 1e-9)).all()) and bool((got * ratio >= 0).all()), (name, i, k)


@pytest.mark.parametrize("bits", [8, 32])
def test_freed_memory(bits):
    """A state or a copy whose storage itself was resized to nothing is refused
    (its memory is gone); copies that the object's list no longer has are not."""
    p = [torch.ones(300, device="cuda")]
    g = [torch.ones(300, device="cuda")]
    for name in ["m", "v", "copies"] + ["m_scale", "v_scale"] * (bits == 8):
        opt = gdn.AdamW(p, **gdn.adamw_states(p, bits), copies=[torch.ones(300, device="cuda", dtype=BF16)])
        getattr(opt, name)[0].untyped_storage().resize_(0)
        with pytest.raises(ValueError, match=rf"opt\.{name}\[0\].*memory"):
            gdn.adamw_step(opt, g, lr=1e-2, step=1)
        assert float((p[0] - 1).abs().max()) == 0
    opt = gdn.AdamW(p, **gdn.adamw_states(p, bits), copies=[torch.ones(300, device="cuda", dtype=BF16)])
    opt.copies = None
    gdn.adamw_step(opt, g, lr=1e-2, step=1)
    assert float((p[0] - 0.99).abs().max()) < 1e-5
