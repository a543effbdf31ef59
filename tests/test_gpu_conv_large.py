"""Convolutions whose x fills the last-level cache, with rows of whole cache lines (which
are loaded another way) and without: the same bits as a third of the rows."""
import pytest
import torch

import kalman_delta_rule_amd as kda

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a HIP GPU")


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("activation", [None, "silu"])
@pytest.mark.parametrize("io,T,D,fused", [("bf16", 3650, 2048, 1), ("f32", 1825, 2048, 1), ("bf16", 3650, 2048, 2),
                                          ("bf16", 3680, 2040, 1), ("f32", 58400, 64, 1)])
def test_the_bits_of_a_third(io, T, D, fused, activation, W):
    B, dt = 18, DT[io]
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.empty(B, T, fused * D, device="cuda").normal_(generator=g).to(dt)[..., (fused - 1) * D:]
    dy = torch.empty(B, T, D, device="cuda").normal_(generator=g).to(dt)
    w, b = torch.randn(W, D, device="cuda"), torch.randn(D, device="cuda")
    s0 = torch.randn(B, W - 1, D, device="cuda").to(dt)
    assert x.numel() * x.element_size() > 256 << 20

    def calls(p):
        kw = dict(bias=b, state0=s0[p], activation=activation)
        y, s_T = kda.kdn_conv_fwd(x[p], w, want_state=True, **kw)
        c = kda.kdn_conv_bwd(dy[p], x[p], w, **kw)
        return [y, s_T, c["dx"], c["dstate0"]]
    whole = calls(slice(0, B))
    for k in range(0, B, B // 3):
        p = slice(k, k + B // 3)
        for i, (v, t) in enumerate(zip(whole, calls(p))):
            assert torch.equal(v[p], t), (i, k)
