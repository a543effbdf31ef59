"""Packed linear attention at the ends: offsets that are none, and what a caller's
tensors hold behind the last sequence."""
import pytest
import torch

import kalman_delta_rule_amd as kda
from test_gpu_block import offsets
from test_gpu_linattn import backward, data

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a HIP GPU")


@pytest.mark.parametrize("cu", [[0, 900, 100, 5000, 1400], [-5, 3, -1, 70000, 2], [0, 5, 9, 1400, 2000]])
def test_the_last_segment_hands_nothing_on(cu):
    # 1500 tokens are eight segments of 192, the last one short: no state of it is formed,
    # whatever the offsets claim to follow it
    T, H, dk, S = 1500, 2, 32, 8
    d = data(1, T, H, H, dk, dk, "bf16", 5, cu)
    states = S * H * dk * dk  # fp32, and 16 bytes a segment
    L = kda._lib.lib()
    assert L.kdn_linattn_fwd_workspace_size(1, T, H, dk, dk) == 4 * states + 16 * S
    assert L.kdn_linattn_bwd_workspace_size(1, T, H, H, dk, dk) == 2 * (4 * states + 16 * S)
    ws = torch.full((2 * (states + 4 * S),), 7.0, device="cuda")
    raw = ws.view(torch.uint8)
    one = H * dk * dk
    kda.kdn_linattn_fwd(d["q"][0], d["k"][0], d["v"][0], d["g"][0], S0=d["S0"][0], cu_seqlens=offsets(cu),
                        want_state=True, workspace=raw)
    assert (ws[states - one:states] == 7).all() and not (ws[:states - one] == 7).all()
    ws.fill_(7.0)
    backward(d, None, cu, workspace=raw)
    # the forward's states, and behind them the backward's, whose walk ends at the first segment
    assert (ws[states - one:states] == 7).all()
    back = ws[states + 4 * S:]
    assert (back[:one] == 7).all() and not (back[one:states] == 7).all()


@pytest.mark.parametrize("H,dk,dv", [(300, 256, 256), (4096, 64, 72)])
def test_states_of_many_heads(H, dk, dv):
    """A sequence's states are more than 2^24 values: as rows of 256 more than 65536 of them."""
    assert H * dk * dv > 1 << 24
    q = torch.randn(1, 3, 1, dk, device="cuda")
    v = torch.randn(1, 3, H, dv, device="cuda")
    S0 = torch.randn(3, H, dk, dv, device="cuda")
    g = torch.full((H,), 0.5, device="cuda")
    o, S_T = kda.kdn_linattn_fwd(q, q, v, g, S0=S0, cu_seqlens=offsets([0, 0, 2, 2]), want_state=True)
    assert torch.equal(S_T[0], S0[0]) and torch.equal(S_T[2], S0[2])
    # the state of one element of each head, token by token in 64 bits: a dozen roundings
    k, w, at = q[0, :2, 0, -1].double(), v[0, :2, :, -1].double(), S0[1, :, -1, -1].double()
    want = 0.25 * at + 0.5 * k[0] * w[0] + k[1] * w[1]
    size = 0.25 * at.abs() + (0.5 * k[0] * w[0]).abs() + (k[1] * w[1]).abs()
    assert ((S_T[1, :, -1, -1].double() - want).abs() <= 16 * 2.0 ** -24 * size).all()
    r = kda.kdn_linattn_bwd(v, q, q, v, g, S0=S0, dS_T=S0, cu_seqlens=offsets([0, 0, 2, 2]))
    assert torch.equal(r["dS0"][0], S0[0]) and torch.equal(r["dS0"][2], S0[2])
    none = kda.kdn_linattn_fwd(q[:, :0], q[:, :0], v[:, :0], g, want_state=True)[1]
    assert none.shape == (1, H, dk, dv) and (none == 0).all()
