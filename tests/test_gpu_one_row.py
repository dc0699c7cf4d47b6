"""A single row's stride means nothing: the last token of a long prompt, as it
is sliced, through the linear layer and the recurrence."""
import pytest
import torch

import gated_deltanet_linear_03_amd as gdn

pytestmark = pytest.mark.gpu


def _apart(t, stride):
    """The row t [1, n] inside a buffer of two rows `stride` elements apart."""
    buf = torch.zeros((2, stride), dtype=t.dtype, device="cuda")
    row = buf[1:, 8:8 + t.shape[1]]
    row.copy_(t)
    assert row.stride(0) == stride
    return row


@pytest.mark.parametrize("stride", [4096 * 2048 + 8, 1036])
def test_linear(stride):
    g = torch.Generator(device="cuda").manual_seed(1)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    x, w, r, dy, pre = rn(1, 512), rn(72, 512) / 20, rn(1, 72), rn(1, 72), rn(1, 72)
    # (whole 16-byte runs are what an operand needs, of its rows' starts)
    wide = torch.zeros((1, 4096, 2048), dtype=torch.bfloat16, device="cuda")
    wide[:, -1, :512] = x
    xs = wide[:, -1, :512] if stride > 2048 else torch.zeros(2 * stride, dtype=torch.bfloat16, device="cuda")[:512][None]
    xs = xs.as_strided((1, 512), (stride, 1))
    xs.copy_(x)
    rs, dys, pres = (_apart(t, stride) for t in (r, dy, pre))
    y, q = _apart(torch.zeros_like(r), stride), _apart(torch.zeros_like(r), stride)
    gdn.linear(xs, w, act=gdn.GDN_ACT_SILU, residual=rs, out=y, preact=q)
    p = torch.zeros_like(r)
    assert torch.equal(y, gdn.linear(x, w, act=gdn.GDN_ACT_SILU, residual=r, preact=p)) and torch.equal(q, p)
    want = gdn.linear_backward(dy, x, w, preact=pre, act=gdn.GDN_ACT_SILU, want_dbias=True)
    got = gdn.linear_backward(dys, xs, w, preact=pres, act=gdn.GDN_ACT_SILU, want_dbias=True, dx=_apart(torch.zeros_like(x), stride))
    for n in want:
        assert torch.equal(got[n], want[n]), n
    # one row of weights
    w1 = w[:1].as_strided((1, 512), (stride + 4, 1)) if stride > 2048 else w[:1].as_strided((1, 512), (516, 1))
    many = rn(40, 512)
    assert torch.equal(gdn.linear(many, w1), gdn.linear(many, w[:1].clone()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_recurrence(dtype):
    D, stride = 100, (1 << 22) + 5
    g = torch.Generator(device="cuda").manual_seed(2)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    rec = gdn.Recur(D=D, A_log=rn(D), dt_bias=rn(D) - 2, act_dtype=gdn.GDN_DTYPE_BF16 if dtype == torch.bfloat16 else gdn.GDN_DTYPE_FP32)
    rows = [rn(1, D).to(dtype) for _ in range(5)]
    far = [_apart(t, stride) for t in rows]
    state = rn(1, D)
    one, two = state.clone(), state.clone()
    y = _apart(torch.zeros_like(rows[0]), stride)
    gdn.recur_decode(rec, *far[:4], one, out=y)
    assert torch.equal(y, gdn.recur_decode(rec, *rows[:4], two)["out"]) and torch.equal(one, two)
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    a = gdn.recur_forward(rec, *far[:4], cu, initial_state=state, want_saved=True)
    b = gdn.recur_forward(rec, *rows[:4], cu, initial_state=state, want_saved=True)
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["final_state"], b["final_state"])
    ga = gdn.recur_backward(rec, *far, a["saved"], cu, want_d_initial=True)
    gb = gdn.recur_backward(rec, *rows, b["saved"], cu, want_d_initial=True)
    for n in gb:
        assert torch.equal(ga[n], gb[n]), n
