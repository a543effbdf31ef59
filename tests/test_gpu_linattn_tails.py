"""Packed linear attention's gradients behind the last sequence, with keys of every
head's own and shared ones: a caller's tensors keep what they held, new ones hold
zeros, and either may stand beside the other."""
import pytest
import torch

from test_gpu_block import same
from test_gpu_linattn import CUTS, backward, data

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a HIP GPU")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("name", CUTS)
@pytest.mark.parametrize("Hk", [1, 2])
def test_gradients_given_and_new(name, io, Hk):
    T, cu = CUTS[name]
    d = data(1, T, 2, Hk, 24, 20, io, T, cu)
    end = cu[-1]
    g = backward(d, None, cu)
    names = ("dq", "dk", "dv")
    assert all((g[n][:, end:] == 0).all() for n in names)
    for given in (names, ("dq",), ("dk",), ("dv",), ("dq", "dv")):
        mine = {n: torch.full_like(g[n], 7.0) for n in given}
        h = backward(d, None, cu, **mine)
        for n in names:
            assert (h[n] is mine.get(n)) == (n in given)
            assert same(h[n][:, :end], g[n][:, :end]), n
            assert (h[n][:, end:] == (7 if n in given else 0)).all(), n
        assert same(h["dS0"], g["dS0"])
