"""A stream of another device than the current one is refused before anything
is allocated for it or launched on it."""
import types

import pytest
import torch

import gated_deltanet_linear_03_amd as gdn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("given", [False, True], ids=["new", "given"])
def test_a_stream_of_another_device_is_refused(given):
    other = types.SimpleNamespace(device=torch.device("cuda", torch.cuda.current_device() + 1), cuda_stream=0)
    T, D = 6, 16
    t = [torch.randn((T, D), device="cuda").to(torch.bfloat16) for _ in range(5)]
    rec = gdn.Recur(D=D, A_log=torch.zeros(D, device="cuda"), dt_bias=torch.zeros(D, device="cuda"))
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    state = torch.zeros((1, D), device="cuda")
    out = torch.full((T, D), 3.0, dtype=torch.bfloat16, device="cuda") if given else None
    saved = gdn.recur_forward(rec, *t[:4], cu, want_saved=True)["saved"]
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda") if given else None
    w = torch.randn((D, D), device="cuda").to(torch.bfloat16)
    with pytest.raises(ValueError, match="stream"):
        gdn.recur_forward(rec, *t[:4], cu, initial_state=state, in_place=True, out=out, stream=other)
    with pytest.raises(ValueError, match="stream"):
        gdn.recur_decode(rec, *t[:4], torch.zeros((T, D), device="cuda"), out=out, stream=other)
    with pytest.raises(ValueError, match="stream"):
        gdn.recur_backward(rec, *t, saved, cu, workspace=ws, stream=other)
    with pytest.raises(ValueError, match="stream"):
        gdn.linear(t[0], w, out=out, stream=other)
    with pytest.raises(ValueError, match="stream"):
        gdn.linear_backward(t[1], t[0], w, dx=out, dw=w.clone(), workspace=ws, stream=other)
    torch.cuda.synchronize()
    if given:
        assert (out == 3.0).all()
    assert (state == 0).all()


def test_a_bare_handle_is_taken_as_it_is():
    D = 16
    t = [torch.randn((3, D), device="cuda").to(torch.bfloat16) for _ in range(4)]
    rec = gdn.Recur(D=D, A_log=torch.zeros(D, device="cuda"), dt_bias=torch.zeros(D, device="cuda"))
    side = torch.cuda.Stream()
    out, a, b = torch.empty_like(t[0]), torch.zeros((3, D), device="cuda"), torch.zeros((3, D), device="cuda")
    want = gdn.recur_decode(rec, *t, a)["out"]
    torch.cuda.synchronize()
    gdn.recur_decode(rec, *t, b, out=out, stream=types.SimpleNamespace(cuda_stream=side.cuda_stream))
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(a, b)
