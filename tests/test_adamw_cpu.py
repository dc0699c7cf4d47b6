"""The AdamW step on the host: calls that are refused before anything is
enqueued, and the reference's rounding of 8-bit states."""
import ctypes

import numpy as np
import pytest
import torch

import gated_deltanet_linear_03_amd as gdn
from train_helpers import mix, random_halves, up_or_down

FAKE = 0x10000            # never dereferenced
FAR = 1 << 36


def _call(n=1, change=None, **kw):
    a = gdn.CAdamW(8, 0.9, 0.999, 1e-3, 1e-8, 1, 5, None, None, None)
    for k, v in kw.items():
        setattr(a, k, v)
    t = (gdn.CAdamWTensor * max(n, 1))()
    for i in range(n):
        t[i].n = 1000
        for k, f in enumerate(("param", "grad", "copy", "m", "v", "m_scale", "v_scale")):
            setattr(t[i], f, FAKE + (8 * i + k) * FAR)
    for k, v in (change or {}).items():
        setattr(t[n - 1], k, v)
    return gdn.lib().gdn_adamw_step(ctypes.byref(a), t, n, None), gdn.lib().gdn_last_error().decode()


@pytest.mark.parametrize("kw, word", [
    (dict(state_bits=16), "state_bits"), (dict(beta1=1.0), "beta1"), (dict(beta2=-0.1), "beta2"), (dict(beta2=float("nan")), "beta"),
    (dict(eps=-1.0), "eps"), (dict(lr=float("inf")), "lr"), (dict(step=0), "step"), (dict(lr_ptr=FAKE + 2), "lr_ptr"),
    (dict(step_ptr=FAKE + 1), "step_ptr"), (dict(grad_scale=FAKE + 3), "grad_scale"), (dict(grad_scale=FAKE), "overlap"),
])
def test_step_refuses(kw, word):
    st, err = _call(**kw)
    assert st == gdn.GDN_ERR_INVALID_ARGUMENT and word in err


@pytest.mark.parametrize("change, word", [
    (dict(n=-1), "n (-1)"), (dict(n=1 << 41), "too large"), (dict(grad_dtype=2), "grad_dtype"), (dict(param=None), "NULL"),
    (dict(grad=None), "NULL"), (dict(m=None), "NULL"), (dict(v=None), "NULL"), (dict(m_scale=None), "NULL"),
    (dict(v_scale=None), "NULL"), (dict(param=FAKE + 9 * FAR + 2), "aligned"), (dict(grad=FAKE + 9 * FAR + 2), "aligned"),
    (dict(copy=FAKE + 9 * FAR + 1), "aligned"), (dict(m_scale=FAKE + 9 * FAR + 2), "aligned"),
    (dict(weight_decay=-0.1), "weight_decay"), (dict(weight_decay=float("inf")), "weight_decay"),
    (dict(grad=FAKE + 8 * FAR + 3996), "overlap"), (dict(copy=FAKE + 8 * FAR), "overlap"), (dict(v=FAKE + 11 * FAR + 999), "overlap"),
    (dict(v_scale=FAKE + 13 * FAR + 12), "overlap"),
])
def test_tensor_refuses(change, word):
    """The second of two tensors is wrong."""
    st, err = _call(2, change)
    assert st == gdn.GDN_ERR_INVALID_ARGUMENT and "tensor 1" in err and word in err


def test_nothing_to_do():
    assert _call(0)[0] == gdn.GDN_OK
    assert _call(1, dict(n=0, param=None))[0] == gdn.GDN_OK
    assert gdn.lib().gdn_adamw_step(None, None, 0, None) == gdn.GDN_ERR_INVALID_ARGUMENT
    a = gdn.CAdamW(32, 0.9, 0.999, 1e-3, 1e-8, 1, 5, None, None, None)
    assert gdn.lib().gdn_adamw_step(ctypes.byref(a), None, 1, None) == gdn.GDN_ERR_INVALID_ARGUMENT
    assert gdn.lib().gdn_adamw_step(ctypes.byref(a), None, -1, None) == gdn.GDN_ERR_INVALID_ARGUMENT


def test_reference_hash():
    """The finaliser on words whose images are known (0 stays 0, and it is a
    permutation: no two of 2^16 words meet)."""
    assert int(mix(0)) == 0 and int(mix(1)) == 0x514E28B7
    assert len(np.unique(mix(np.arange(1 << 16, dtype=np.uint32)))) == 1 << 16
    lo, hi = random_halves(3, 7, 2, 100000)
    # uniform on 0 .. 65535: the mean of 1e5 is within 6 of its deviations, 65536 / sqrt(12e5)
    assert abs(lo.mean() - 32767.5) < 6 * 60 and abs(hi.mean() - 32767.5) < 6 * 60
    a, b = random_halves(3, 7, 2, 10, first=(1 << 32) + 5), random_halves(3, 7, 2, 10, first=5)
    assert not np.array_equal(a[0], b[0])


def test_reference_rounding():
    """Values of the format stay, others go to a neighbour of theirs, on
    average where they are."""
    every = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    for u in (0, 30000, 65535):
        v, _ = up_or_down(np.concatenate([every, -every]), u)
        assert np.array_equal(np.abs(v), np.concatenate([every, every]))
    x = np.random.RandomState(1).uniform(0, 448, 500)
    x[:200] *= 2.0 ** -np.random.RandomState(2).randint(0, 16, 200)
    lo, hi = (np.array([every[every <= a].max() for a in x]), np.array([every[every >= a].min() for a in x]))
    mean = np.zeros_like(x)
    for u in range(0, 65536, 64):
        v, _ = up_or_down(x, u)
        assert bool(((v == lo) | (v == hi)).all())
        mean += v / 1024
    # 1024 evenly spread u: off by a 1024th of a step at the most
    assert bool((np.abs(mean - x) <= (hi - lo) / 1000).all())
