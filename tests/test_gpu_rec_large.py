"""Recurrences whose x fills the last-level cache, with rows of whole cache lines (which
are loaded another way) and without: the same bits as a third of the rows."""
import pytest
import torch

import kalman_delta_rule_amd as kda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a HIP GPU")


@pytest.mark.parametrize("gate", ["preact", "alpha"])
@pytest.mark.parametrize("io,T,D", [("bf16", 3700, 2048), ("bf16", 3700, 2047), ("f32", 1850, 2048), ("f32", 1850, 2049)])
def test_the_bits_of_a_third(io, T, D, gate):
    B, dt = 18, torch.bfloat16 if io == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(5)
    x, dy = (torch.empty(B, T, D, device="cuda").normal_(generator=g).to(dt) for _ in range(2))
    a = torch.empty(B, T, D, device="cuda").normal_(generator=g).add_(2)
    a = torch.sigmoid(a) if gate == "alpha" else a.to(dt)
    h0, dh_T = (torch.empty(B, D, device="cuda").normal_(generator=g) for _ in range(2))
    assert x.numel() * x.element_size() > 256 << 20

    def calls(p):
        h, h_T, chk = kda.kdn_rec_fwd(x[p], a[p], h0=h0[p], gate=gate, blend=True, want_checkpoints=True)
        r = kda.kdn_rec_bwd(dy[p], x[p], a[p], chk, h0=h0[p], dh_T=dh_T[p], gate=gate, blend=True)
        return [h, h_T, chk, r["dx"], r["da"], r["dh0"]]
    whole = calls(slice(0, B))
    for k in range(0, B, B // 3):
        p = slice(k, k + B // 3)
        for i, (v, t) in enumerate(zip(whole, calls(p))):
            assert torch.equal(v[p], t), (i, k)
