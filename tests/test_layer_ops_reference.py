"""The 64-bit references of group norm and dropout: gradients against
differences, the generator against its published vectors.  CPU only."""
import numpy as np
import pytest

import layer_ops_reference as R
from test_block_reference import agree


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("S,C,G", [(1, 6, 2), (5, 4, 1), (3, 6, 6)])
def test_group_norm_gradients(S, C, G, silu):
    rng = np.random.default_rng(S)
    x, dy = rng.standard_normal((3, S, C)) + 1, rng.standard_normal((3, S, C))
    w, b = rng.standard_normal(C), rng.standard_normal(C)
    eps = 1e-2
    f = R.group_norm(x, G, w, b, eps, silu)
    g = R.group_norm_bwd(dy, x, f["mean"][0], f["rstd"][0], w, b, silu)
    loss = lambda x, w, b: float((R.group_norm(x, G, w, b, eps, silu)["y"][0] * dy).sum())
    agree(loss, dict(x=x, w=w, b=b), dict(x=g["dx"][0], w=g["dweight"][0], b=g["dbias"][0]), rng)


@pytest.mark.parametrize("counter,key,words", [
    ([0] * 4, [0] * 2, [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]),
    ([0xffffffff] * 4, [0xffffffff] * 2, [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]),
    ([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344], [0xa4093822, 0x299f31d0],
     [0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1])])
def test_generator(counter, key, words):
    assert R.philox(np.array([counter], np.uint64), key)[0].tolist() == words


def test_shares():
    # a share of n independent bits is off by more than 6 standard deviations in one of 5e8
    n = 1 << 20
    for p in (0.0, 0.1, 0.5, 1.0):
        keep, share = R.kept(n, p, 12345, 7)
        assert abs(keep.mean() - share) <= 6 * (share * (1 - share) / n) ** 0.5
    a, b = R.kept(n, 0.5, 1, 0)[0], R.kept(n, 0.5, 1, 1)[0]
    assert abs((a == b).mean() - 0.5) <= 6 * 0.5 / n ** 0.5
