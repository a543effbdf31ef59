"""Group norm's statistics where single values lie far from the others."""
import numpy as np
import pytest
import torch

import block_reference as BR
import kalman_delta_rule_amd as kda
import layer_ops_reference as R
from test_gpu_block import dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a HIP GPU")


def tolerance(S, C, io):
    """Relative, of rstd: half the variance's.  Only squares are added, each with a few
    roundings, and none cancels: a thread of a channel joins S / 4 of its share of the
    positions one after another, then threads and tiles pairwise and in turns of 256."""
    V = 8 if io == "bf16" else 4
    lanes = min(64, 1 << (-(-C // V) - 1).bit_length())
    joins = S * lanes / 256 / 4 + C * 1024 / 256
    return 0.5 * (joins + 64) * BR.U + 4 * BR.U


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("N,S,C,G", [(1, 100000, 16, 1), (1, 20000, 8, 1), (2, 70000, 24, 3), (1030, 4200, 8, 1),
                                     (1100, 260, 136, 8), (3, 3000, 5, 1), (130, 1000, 32, 8)])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
def test_one_position_far_from_the_others(N, S, C, G, io, where):
    rng = np.random.default_rng(S + C)
    base = torch.from_numpy(rng.standard_normal((S, C))).cuda()
    at = {"first": 0, "middle": S // 2, "last": S - 1}[where]
    for far in (30.0, 1000.0, 1e5):
        x = base.repeat(N, 1, 1)
        x[:, at, :] = far
        x[:, at, C - 1] = -far
        x = x.to(torch.bfloat16 if io == "bf16" else torch.float32)
        y, mean, rstd = kda.kdn_group_norm_fwd(x, G, eps=1e-5, want_stats=True)
        one = host(x[:1])
        ref = R.group_norm(one, G, None, None, float(np.float32(1e-5)), False)
        want = np.broadcast_to(ref["rstd"][0], (N, G))
        off = np.abs(host(rstd) / want - 1).max()
        assert off <= tolerance(S, C, io), (far, off)
        for n in {0, N - 1}:
            BR.check(host(y[n:n + 1]), ref["y"], io, "y")
            BR.check(host(mean[n:n + 1]), ref["mean"], "f32", "mean")
