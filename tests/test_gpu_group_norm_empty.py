"""Group norm of samples without positions."""
import pytest
import torch

import kalman_delta_rule_amd as kda
from kalman_delta_rule_amd.api import _launch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a HIP GPU")


@pytest.mark.parametrize("N,C,G", [(1, 8, 2), (300, 96, 96)])
def test_statistics_of_no_positions_are_written(N, C, G):
    x = torch.empty(N, 0, C, device="cuda")
    y, mean, rstd = kda.kdn_group_norm_fwd(x, G, want_stats=True)
    assert y.shape == x.shape and mean.shape == rstd.shape == (N, G)
    assert (mean == 0).all() and (rstd == 0).all()
    L = kda._lib.lib()
    stats = torch.full((2, N * G + 1), 7.0, device="cuda")
    for given in ((0, 1), (0,), (1,)):
        stats.fill_(7.0)
        m, r = (stats[i].data_ptr() if i in given else None for i in (0, 1))
        _launch(x.device, L.kdn_group_norm_fwd, N, 0, C, G, 0, 0, 1e-5, None, C, None, None, None, m, r, None, 0)
        for i in (0, 1):
            assert (stats[i, :N * G] == (0 if i in given else 7)).all() and stats[i, N * G] == 7
    g = kda.kdn_group_norm_bwd(x, x, mean, rstd)
    assert g["dx"].shape == x.shape and (g["dweight"] == 0).all() and (g["dbias"] == 0).all()
