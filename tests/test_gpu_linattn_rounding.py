"""Linear attention's roundings: outputs by token in bf16 are off by their own
rounding and by terms of 16 bits, not of 8; what is infinite stays so; states are
rounded once a chunk."""
import numpy as np
import pytest
import torch

import linattn_reference as R
from test_gpu_block import dev, host
from test_gpu_linattn import CUTS, backward, data, forward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a HIP GPU")


# A term of an output by token is q_i k_j v_j with its decay, or q_i X.  Its first two factors'
# product, or X, is an operand of two bf16 parts, which loses at most 2^-8 2^-8 of it, and X
# was summed from terms of two such parts: 2^-15 in all, beside the fp32 arithmetic.
TERM = 2.0 ** -15


def check(got, ref, name, d, T):
    value, loose = ref
    a = R._bounds("f32", T, d)[0]
    G = 8  # heads that share a key, at most: the sum of their terms
    bound = loose * (TERM + a + G * R.U) / R._bounds("bf16", T, d)[0]
    # half a step at the value: bf16 holds 8 bits
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(value), 2.0 ** -120))) - 7)
    off, tol = np.abs(host(got) - value), step / 2 + 1.01 * bound
    worst = np.argmax(off - tol)
    assert (off <= tol).all(), "%s: off by %.3g where %.3g is allowed (value %.6g), %d of %d" % (
        name, off.flat[worst], tol.flat[worst], value.flat[worst], (off > tol).sum(), off.size)


def tokens(d, scale, cu=None):
    S0, dS = (d[n][1] if n in d else None for n in ("S0", "dS"))
    T, dk, dv = d["q"][1].shape[1], d["q"][1].shape[3], d["v"][1].shape[3]
    ref = R.forward(d["q"][1], d["k"][1], d["v"][1], d["g"][1], scale, S0, cu, "bf16")
    check(forward(d, scale, cu)[0], ref["o"], "o", dk, T)
    ref = R.backward(d["do"][1], d["q"][1], d["k"][1], d["v"][1], d["g"][1], scale, S0, dS, cu, "bf16")
    g = backward(d, scale, cu)
    for n, size in (("dq", dv), ("dk", dv), ("dv", dk)):
        check(g[n], ref[n], n, size, T)


@pytest.mark.parametrize("dk,dv", [(1, 1), (8, 24), (33, 31), (64, 64), (63, 65), (128, 64), (128, 128), (100, 200),
                                   (255, 129), (256, 256)])
def test_head_sizes(dk, dv):
    tokens(data(2, 83, 2, 1, dk, dv, "bf16", dk * 5 + dv), 0.25)


@pytest.mark.parametrize("T,H,Hk", [(1, 2, 2), (16, 2, 1), (17, 1, 1), (33, 2, 2), (49, 8, 1), (64, 2, 2), (128, 4, 1),
                                    (200, 2, 2), (1500, 2, 2), (2048, 2, 1)])
def test_lengths(T, H, Hk):
    tokens(data(1, T, H, Hk, 40, 48, "bf16", T, state=T % 2 == 0), 0.3)


@pytest.mark.parametrize("name", ["mixed", "tail", "empty", "segments"])
def test_packed(name):
    T, cu = CUTS[name]
    tokens(data(1, T, 2, 1, 24, 72, "bf16", T, cu), 1.0, cu)


@pytest.mark.parametrize("T", [40, 90])
@pytest.mark.parametrize("dk", [32, 128, 256])
def test_infinities_of_states_and_products(T, dk):
    """An infinite element of a state, or of a key, in one direction of q: the output is infinite
    with the sign that its q gives, as the definition has it, and other heads do not change."""
    d = data(1, T, 2, 2, dk, 64, "bf16", T, state=True)
    d["g"] = dev(np.array([1.0, 0.5]))
    q = torch.where(d["q"][0] < 0, -1.0, 1.0).to(torch.bfloat16)
    d["q"] = (q,)
    o, _ = forward(d, 1.0)
    S0 = d["S0"][0].clone()
    S0[0, 0, 3, 5] = float("inf")
    S0[0, 0, 7, 6] = float("-inf")
    e = dict(d, S0=(S0,))
    got, S_T = forward(e, 1.0)
    # the first chunk reads the state as it came
    first = min(T, 32)
    assert (got[0, :first, 0, 5] == q[0, :first, 0, 3].float() * float("inf")).all()
    assert (got[0, :first, 0, 6] == q[0, :first, 0, 7].float() * float("-inf")).all()
    assert not torch.isfinite(got[0, :, 0, 5:7]).any()
    assert torch.equal(got[0, :, 1], o[0, :, 1]) and torch.equal(got[0, :, 0, :5], o[0, :, 0, :5])
    # an infinite key: every product with it is infinite, and with a v of ones so is the output
    k, v = d["k"][0].clone(), torch.ones_like(d["v"][0])
    k[0, 9, 0, 2] = float("inf")
    got, _ = forward(dict(d, k=(k,), v=(v,)), 1.0)
    assert (got[0, 9, 0] == (q[0, 9, 0, 2].float() * float("inf"))).all()
    assert torch.isfinite(got[0, :9]).all() and not torch.isfinite(got[0, 9:, 0]).any()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T,dk", [(32, 64), (64, 128), (320, 64), (320, 256), (2560, 32)])
def test_small_terms_reach_a_large_state(T, dk, io):
    """A state of 2^24, where floats are 2 apart, and terms of 3/4 without decay: their sum over
    a chunk is exact, and adding it rounds by 1 at most.  A chunk is 32 tokens at least; the
    segments of 2560 tokens start from states of their own, whose sums are joined alike."""
    one = lambda *s: dev(np.ones(s), io)
    d = {"q": one(1, T, 2, dk), "k": one(1, T, 2, dk), "v": dev(np.full((1, T, 2, 32), 0.75), io),
         "do": dev(np.full((1, T, 2, 32), 0.75), io), "g": dev(np.ones(2)),
         "S0": dev(np.full((1, 2, dk, 32), 2.0 ** 24)), "dS": dev(np.full((1, 2, dk, 32), 2.0 ** 24))}
    want = 2.0 ** 24 + 0.75 * T
    for got in (forward(d, 1.0)[1], backward(d, 1.0)["dS0"]):
        assert np.abs(host(got) - want).max() <= T / 32
