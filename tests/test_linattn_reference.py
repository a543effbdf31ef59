"""The 64-bit reference of linear attention against differences: every gradient
as (L(v + e d) - L(v - e d)) / 2e along random directions.  CPU only."""
import numpy as np
import pytest

import linattn_reference as R
from test_block_reference import agree


@pytest.mark.parametrize("Hk,H", [(2, 2), (1, 3)])
@pytest.mark.parametrize("cu", [None, [0, 1, 1, 7, 9]])
def test_gradients(cu, Hk, H):
    rng = np.random.default_rng(H)
    B, T, dk, dv = (2 if cu is None else 1), 9, 3, 4
    N = B if cu is None else len(cu) - 1
    x = dict(q=rng.standard_normal((B, T, Hk, dk)), k=rng.standard_normal((B, T, Hk, dk)),
             v=rng.standard_normal((B, T, H, dv)), S0=rng.standard_normal((N, H, dk, dv)))
    g, scale = rng.uniform(0, 1, H), 0.7
    do, dS = rng.standard_normal((B, T, H, dv)), rng.standard_normal((N, H, dk, dv))

    def loss(q, k, v, S0):
        f = R.forward(q, k, v, g, scale, S0, cu, "f32")
        return float((f["o"][0] * do).sum() + (f["S_T"][0] * dS).sum())
    b = R.backward(do, x["q"], x["k"], x["v"], g, scale, x["S0"], dS, cu, "f32")
    agree(loss, x, dict(q=b["dq"][0], k=b["dk"][0], v=b["dv"][0], S0=b["dS0"][0]), rng)


def test_forward_is_the_sum_over_pairs():
    rng = np.random.default_rng(3)
    T, dk, dv, g, scale = 11, 3, 2, 0.8, 0.5
    q, k, v = (rng.standard_normal((1, T, 1, d)) for d in (dk, dk, dv))
    S0 = rng.standard_normal((1, 1, dk, dv))
    f = R.forward(q, k, v, np.array([g]), scale, S0, None, "f32")
    o = np.zeros((T, dv))
    for i in range(T):
        o[i] = scale * g ** (i + 1) * q[0, i, 0] @ S0[0, 0]
        for j in range(i + 1):
            o[i] += scale * g ** (i - j) * (q[0, i, 0] @ k[0, j, 0]) * v[0, j, 0]
    assert np.allclose(f["o"][0][0, :, 0], o, atol=1e-13)
