"""A training step as it is used: a recurrent block between two norms, the
vocabulary's cross entropy behind it, the backward passes of all of them and
the update of every weight; eager, with a captured step, and with two steps
under way on two streams."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_03_amd as gdn
from train_helpers import adamw64, close

pytestmark = pytest.mark.gpu

LENS, H, D, V = [130, 0, 300, 7], 64, 96, 1003
T = sum(LENS)
BF16 = torch.bfloat16
MATRICES, VECTORS = ("w_in", "w_out", "w_vocab"), ("n1", "n2", "n2_bias", "in_bias", "A_log", "dt_bias")


class Model:
    """fp32 parameters, bf16 copies of the matrices, and a step over them."""

    def __init__(self, seed, bits):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.p = {"w_in": rn(4 * D, H) / 8, "w_out": rn(H, D) / 10, "w_vocab": rn(V, H) / 8, "n1": 1 + 0.1 * rn(H),
                  "n2": 1 + 0.1 * rn(H), "n2_bias": 0.1 * rn(H), "in_bias": 0.1 * rn(4 * D), "A_log": 0.5 * rn(D), "dt_bias": rn(D) - 2}
        self.w = {n: self.p[n].to(BF16) for n in MATRICES}
        self.x = rn(T, H)
        self.targets = torch.randint(0, V, (T,), generator=g, device="cuda")
        self.targets[::5] = -100
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(LENS)]), dtype=torch.int32, device="cuda")
        self.dloss = (1 / (self.targets >= 0).sum().float()).reshape(1)
        self.names = MATRICES + VECTORS
        params = [self.p[n] for n in self.names]
        self.states = gdn.adamw_states(params, bits)
        self.opt = gdn.AdamW(params, **self.states, copies=[self.w.get(n) for n in self.names],
                             weight_decay=[0.1 if n in MATRICES else 0.0 for n in self.names], seed=3)

    def gradients(self):
        p, w = self.p, self.w
        rec = gdn.Recur(D=D, A_log=p["A_log"], dt_bias=p["dt_bias"])
        st1, st2 = torch.empty((2, T), device="cuda"), torch.empty((2, T), device="cuda")
        h1 = gdn.norm(self.x, p["n1"], kind=gdn.GDN_NORM_RMS, eps=1e-6, out_dtype=BF16, stats=st1)
        proj = gdn.linear(h1, w["w_in"], bias=p["in_bias"])
        xs, a, b, z = (proj[:, i * D:(i + 1) * D] for i in range(4))
        f = gdn.recur_forward(rec, xs, a, b, z, self.cu, want_saved=True)
        stream = gdn.linear(f["out"], w["w_out"], residual=self.x)
        h2 = gdn.norm(stream, p["n2"], p["n2_bias"], out_dtype=BF16, stats=st2)
        out = gdn.linear_cross_entropy(h2, w["w_vocab"], self.targets, z_loss=1e-3)

        gv = gdn.linear_cross_entropy_backward(self.dloss, h2, w["w_vocab"], self.targets, out["lse"], z_loss=1e-3)
        g2 = gdn.norm_backward(gv["dx"], stream, p["n2"], st2, want_dbias=True)
        go = gdn.linear_backward(g2["dx"], f["out"], w["w_out"])
        dp = torch.empty((T, 4 * D), dtype=BF16, device="cuda")
        dA, dd = torch.empty_like(p["A_log"]), torch.empty_like(p["dt_bias"])
        ws = torch.empty(gdn.recur_backward_workspace_bytes(rec, len(LENS), T), dtype=torch.uint8, device="cuda")
        gdn.recur_backward_raw(rec, N=len(LENS), T_total=T, cu_seqlens=self.cu, x=xs, a=a, b=b, z=z, dy=go["dx"], saved=f["saved"],
                               dA_log=dA, ddt_bias=dd, workspace=ws,
                               **{n: dp[:, i * D:(i + 1) * D] for i, n in enumerate(("dx", "da", "db", "dz"))})
        gi = gdn.linear_backward(dp, h1, w["w_in"], want_dbias=True)
        g1 = gdn.norm_backward(gi["dx"], self.x, p["n1"], st1, kind=gdn.GDN_NORM_RMS, d_residual=g2["dx"])
        grads = {"w_in": gi["dw"], "w_out": go["dw"], "w_vocab": gv["dw"], "n1": g1["dweight"], "n2": g2["dweight"],
                 "n2_bias": g2["dbias"], "in_bias": gi["dbias"], "A_log": dA, "dt_bias": dd}
        return out["loss"], grads, g1["dx"]

    def step(self, lr, step):
        loss, grads, dx = self.gradients()
        gdn.adamw_step(self.opt, [grads[n] for n in self.names], lr=lr, step=step)
        return loss, grads, dx


def reference(model):
    """The same in 64 bits by automatic differentiation, from the matrices as they are in bf16."""
    leaf = {n: model.w.get(n, model.p[n]).double().cpu().requires_grad_() for n in model.names}
    x = model.x.double().cpu().requires_grad_()
    h1 = x * (x.square().mean(1, keepdim=True) + 1e-6) ** -0.5 * leaf["n1"]
    P = h1 @ leaf["w_in"].t() + leaf["in_bias"]
    X, A, B, Z = (P[:, i * D:(i + 1) * D] for i in range(4))
    gl = -torch.exp(leaf["A_log"]) * torch.nn.functional.softplus(A + leaf["dt_bias"])
    al, u = torch.exp(gl), torch.sqrt(-torch.expm1(2 * gl)) * torch.sigmoid(B) * X
    rows, at = [], 0
    for L in LENS:
        h = torch.zeros(D, dtype=torch.float64)
        for t in range(at, at + L):
            h = al[t] * h + u[t]
            rows.append(h)
        at += L
    s = x + (torch.stack(rows) * Z * torch.sigmoid(Z)) @ leaf["w_out"].t()
    d = s - s.mean(1, keepdim=True)
    h2 = d * (d.square().mean(1, keepdim=True) + 1e-5) ** -0.5 * leaf["n2"] + leaf["n2_bias"]
    logits = h2 @ leaf["w_vocab"].t()
    lse = torch.logsumexp(logits, 1)
    t = model.targets.cpu()
    loss = torch.where(t >= 0, lse - logits.gather(1, t.clamp(min=0)[:, None])[:, 0] + 1e-3 * lse * lse, 0.0)
    (loss.sum() * float(model.dloss)).backward()
    return loss.detach(), {n: v.grad for n, v in leaf.items()}, x.grad


def test_gradients_of_a_step():
    """What separates the two is rounding to bf16 between the steps: each tensor
    handed over is rounded once (2^-9 relative, root mean square below 2^-9);
    no gradient passes through more than eleven of them, each of which it can
    meet twice, in a value and in a slope."""
    model = Model(5, 32)
    loss, grads, dx = model.gradients()
    want, ref, ref_dx = reference(model)
    rel = lambda p, q: float((p.double().cpu() - q).norm() / q.norm())  # noqa: E731
    bound = 22 * 2.0 ** -9
    assert rel(loss, want) < bound and rel(dx, ref_dx) < bound
    for n in model.names:
        assert rel(grads[n], ref[n]) < bound, n


@pytest.mark.parametrize("bits", [8, 32])
def test_steps(bits):
    """Three steps: each updates every weight by the gradients it computed, and
    the copies that the next one multiplies with."""
    model = Model(6, bits)
    for k in (1, 2, 3):
        old = {n: v.clone() for n, v in model.p.items()}
        m = [t.float().double().cpu().numpy() for t in model.states["m"]]
        v = [t.float().double().cpu().numpy() for t in model.states["v"]]
        if bits == 8:
            scale = lambda name, i, shape: np.repeat(model.states[name][i].double().cpu().numpy(), 256)[:int(np.prod(shape))].reshape(shape)  # noqa: E731
            m = [t * scale("m_scale", i, t.shape) for i, t in enumerate(m)]
            v = [(t * scale("v_scale", i, t.shape)) ** 2 for i, t in enumerate(v)]
        loss, grads, _ = model.step(1e-3, k)
        assert bool(loss.isfinite().all())
        for i, n in enumerate(model.names):
            (p, _, _), (e, _, _) = adamw64(old[n].double().cpu().numpy(), grads[n].double().cpu().numpy(), m[i], v[i], 1e-3, 0.9, 0.999,
                                           1e-8, 0.1 if n in MATRICES else 0.0, k)
            close(n, model.p[n], torch.from_numpy(p), torch.from_numpy(e))
            if n in MATRICES:
                assert torch.equal(model.w[n], model.p[n].to(BF16))


@pytest.mark.parametrize("bits", [8, 32])
def test_captured_step(bits):
    """A whole step in a graph, the learning rate and the step's number on the
    device: the same bits as eager steps, with eager work in between."""
    eager, model = Model(7, bits), Model(7, bits)
    lr, step = torch.tensor([1e-3], device="cuda"), torch.tensor([1], dtype=torch.int32, device="cuda")
    Model(8, bits).step(lr, step)                     # everything loaded
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, grads, dx = model.step(lr, step)
    for k in range(1, 4):
        lr.fill_(1e-3 / k)
        step.fill_(k)
        graph.replay()
        torch.cuda.synchronize()
        want, eg, edx = eager.step(float(torch.tensor(1e-3 / k)), k)
        assert torch.equal(want, loss) and torch.equal(edx, dx)
        for n in model.names:
            assert torch.equal(eg[n], grads[n]), n
            assert torch.equal(eager.p[n], model.p[n]), n
        assert all(torch.equal(a.float(), b.float()) for k2 in model.states for a, b in zip(eager.states[k2], model.states[k2]))


def test_two_steps_at_once():
    """Two models' steps on two streams, each with its own buffers."""
    a, b, c, d = Model(9, 32), Model(10, 8), Model(9, 32), Model(10, 8)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for k in (1, 2):
        with torch.cuda.stream(s1):
            r1 = a.step(1e-3, k)
        with torch.cuda.stream(s2):
            r2 = b.step(1e-3, k)
    torch.cuda.synchronize()
    for k in (1, 2):
        e1, e2 = c.step(1e-3, k), d.step(1e-3, k)
    assert torch.equal(r1[0], e1[0]) and torch.equal(r2[0], e2[0])
    for n in a.names:
        assert torch.equal(a.p[n], c.p[n]) and torch.equal(b.p[n], d.p[n]), n
