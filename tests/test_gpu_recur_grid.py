"""The recurrence with so many sequences that its tiles (or tokens) need more
work-items than one grid dimension holds (2^32): the bits of the same
sequences in small calls."""
import pytest
import torch

import gated_deltanet_linear_03_amd as gdn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _give_back():
    yield
    torch.cuda.empty_cache()


def _rows(T, D, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((T, D), generator=g, device="cuda", dtype=torch.bfloat16)


def _recur(D):
    g = torch.Generator(device="cuda").manual_seed(1)
    return gdn.Recur(D=D, A_log=torch.rand(D, generator=g, device="cuda"), dt_bias=torch.randn(D, generator=g, device="cuda") - 2)


def _room(gib):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib * 2 ** 30:
        pytest.skip(f"needs {gib} GiB of device memory")


def test_forward():
    """262144 one-token sequences x 4096 channels: 16.9 M tiles of 256 threads."""
    _room(32)
    N, D = 262144, 4096
    rec, x, a = _recur(D), _rows(N, D, 2), _rows(N, D, 3)
    cu = torch.arange(N + 1, dtype=torch.int32, device="cuda")
    status = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    f = gdn.recur_forward(rec, x, a, x, None, cu, status=status)
    assert status.item() == 0
    for lo in (0, 131000, N - 600):
        s = slice(lo, lo + 600)
        one = gdn.recur_forward(rec, x[s], a[s], x[s], None, cu[:601])
        assert torch.equal(f["out"][s], one["out"]) and torch.equal(f["final_state"][s], one["final_state"]), lo


def test_short_calls():
    """300 one-token sequences x 2^22 channels, without a workspace: 19.7 M work-groups."""
    _room(32)
    N, D = 300, 1 << 22
    rec, x, a = _recur(D), _rows(N, D, 7), _rows(N, D, 8)
    cu = torch.arange(N + 1, dtype=torch.int32, device="cuda")
    status = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    f = gdn.recur_forward(rec, x, a, x, None, cu, status=status)
    assert status.item() == 0
    for lo in (0, 1 << 21, D - 4096):
        c = slice(lo, lo + 4096)
        part = gdn.Recur(D=4096, A_log=rec.A_log[c], dt_bias=rec.dt_bias[c])
        one = gdn.recur_forward(part, x[:, c], a[:, c], x[:, c], None, cu)
        assert torch.equal(f["out"][:, c], one["out"]) and torch.equal(f["final_state"][:, c], one["final_state"]), lo


def test_backward():
    """131072 one-token sequences x 4096 channels: as many tiles, two for each."""
    _room(64)
    N, D = 131072, 4096
    rec, x, a = _recur(D), _rows(N, D, 4), _rows(N, D, 5)
    cu = torch.arange(N + 1, dtype=torch.int32, device="cuda")
    f = gdn.recur_forward(rec, x, a, x, None, cu, want_saved=True)
    status = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    g = gdn.recur_backward(rec, x, a, x, None, a, f["saved"], cu, want_d_initial=True, status=status)
    assert status.item() == 0
    for lo in (0, 65000, N - 600):
        s = slice(lo, lo + 600)
        one = gdn.recur_forward(rec, x[s], a[s], x[s], None, cu[:601], want_saved=True)
        og = gdn.recur_backward(rec, x[s], a[s], x[s], None, a[s], one["saved"], cu[:601], want_d_initial=True)
        for n in ("dx", "da", "db"):
            assert torch.equal(g[n][s], og[n]), (n, lo)
        assert torch.equal(g["d_initial_state"][s], og["d_initial_state"]), lo


def test_decode():
    """2^34 channels in all, four to a lane; the output in the input's place."""
    _room(110)
    N, D = 4096 * 1024 + 3, 4096
    rec = _recur(D)
    x = torch.empty((N, D), dtype=torch.bfloat16, device="cuda")
    part = _rows(1024, D, 6)
    spots = (0, 2000000, N - 1024)
    x.zero_()
    for lo in spots:
        x[lo:lo + 1024] = part
    state = torch.zeros((N, D), device="cuda")
    want = gdn.recur_decode(rec, part, part, part, None, torch.zeros((1024, D), device="cuda"))
    gdn.recur_decode(rec, x, x, x, None, state, out=x)
    for lo in spots:
        assert torch.equal(x[lo:lo + 1024], want["out"]) and torch.equal(state[lo:lo + 1024], want["final_state"]), lo


@pytest.mark.parametrize("N", [3, 600])
def test_only_empty_sequences(N):
    """Without a token anywhere the states and their gradients pass through."""
    D = 70
    rec, none = _recur(D), torch.empty((0, D), dtype=torch.bfloat16, device="cuda")
    cu = torch.zeros(N + 1, dtype=torch.int32, device="cuda")
    status = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    state, grad = torch.randn((N, D), device="cuda"), torch.randn((N, D), device="cuda")
    f = gdn.recur_forward(rec, none, none, none, none, cu, initial_state=state, want_saved=True, status=status)
    assert status.item() == 0 and torch.equal(f["final_state"], state)
    g = gdn.recur_backward(rec, none, none, none, none, none, f["saved"], cu, d_final_state=grad, want_d_initial=True, status=status)
    assert status.item() == 0 and torch.equal(g["d_initial_state"], grad)
    assert (g["dA_log"] == 0).all() and (g["ddt_bias"] == 0).all()
