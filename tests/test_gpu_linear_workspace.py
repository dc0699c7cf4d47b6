"""Which calls of the linear layer need a workspace is the library's to say."""
import pytest
import torch

import gated_deltanet_linear_03_amd as gdn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 16, 17, 256, 257, 400])
def test_the_binding_asks_the_library(M, monkeypatch):
    real, seen = gdn.lib(), []

    class Lib:
        def __getattr__(self, name):
            return getattr(real, name)

        def gdn_linear_workspace_bytes(self, m, n, k):
            seen.append((m, n, k))
            return max(real.gdn_linear_workspace_bytes(m, n, k), 512)

        def gdn_linear(self, io, ws, nbytes, stream):
            seen.append((ws is not None, nbytes))
            return real.gdn_linear(io, ws, nbytes, stream)

    x = torch.randn((M, 1032), device="cuda").to(torch.bfloat16)
    w = torch.randn((70, 1032), device="cuda").to(torch.bfloat16)
    want = gdn.linear(x, w)
    monkeypatch.setattr(gdn, "_lib", Lib())
    assert torch.equal(gdn.linear(x, w), want)
    need = max(real.gdn_linear_workspace_bytes(M, 70, 1032), 512)
    assert seen == [(M, 70, 1032), (True, need)]
