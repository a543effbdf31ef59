"""The 64-bit references of the block operators against differences: every
gradient formula as (L(v + e d) - L(v - e d)) / 2e along random directions.
CPU only."""
import numpy as np
import pytest

import block_reference as R


def slope(loss, values, name, direction, e=1e-5):
    up, down = dict(values), dict(values)
    up[name] = values[name] + e * direction
    down[name] = values[name] - e * direction
    return (loss(**up) - loss(**down)) / (2 * e)


def agree(loss, values, grads, rng):
    for name, g in grads.items():
        d = rng.standard_normal(g.shape)
        num, ana = slope(loss, values, name, d), float((g * d).sum())
        # third derivatives of order one: e^2 = 1e-10, and cancellation 1e-16 / 1e-5
        assert abs(num - ana) <= 1e-6 * max(1.0, np.abs(g * d).sum()), name


@pytest.mark.parametrize("D", [1, 7, 64])
def test_layer_norm_gradients(D):
    rng = np.random.default_rng(D)
    x, dy = rng.standard_normal((5, D)) + 2, rng.standard_normal((5, D))
    w, b = rng.standard_normal(D), rng.standard_normal(D)
    eps = 1e-2
    f = R.layer_norm(x, w, b, eps)
    g = R.layer_norm_bwd(dy, x, f["mean"][0], f["rstd"][0], w)
    loss = lambda x, w, b: float((R.layer_norm(x, w, b, eps)["y"][0] * dy).sum())
    agree(loss, dict(x=x, w=w, b=b), dict(x=g["dx"][0], w=g["dweight"][0], b=g["dbias"][0]), rng)


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("cu", [None, [0, 1, 1, 9, 12], [0, 5]])
def test_conv_gradients(W, silu, cu):
    rng = np.random.default_rng(W)
    B, T, D = (2 if cu is None else 1), 12, 3
    N = B if cu is None else len(cu) - 1
    v = dict(x=rng.standard_normal((B, T, D)), weight=rng.standard_normal((W, D)),
             bias=rng.standard_normal(D), state0=rng.standard_normal((N, W - 1, D)))
    dy, ds = rng.standard_normal((B, T, D)), rng.standard_normal((N, W - 1, D))

    def loss(**v):
        f = R.conv(v["x"], v["weight"], v["bias"], v["state0"], cu, silu)
        end = T if cu is None else cu[-1]
        return float((f["y"][0] * dy)[:, :end].sum() + (f["state_T"][0] * ds).sum())
    g = R.conv(v["x"], v["weight"], v["bias"], v["state0"], cu, silu, dy, ds)
    agree(loss, v, dict(x=g["dx"][0], weight=g["dweight"][0], bias=g["dbias"][0],
                        state0=g["dstate0"][0]), rng)


@pytest.mark.parametrize("preact", [False, True])
@pytest.mark.parametrize("blend", [False, True])
@pytest.mark.parametrize("cu", [None, [0, 1, 1, 9, 12], [0, 5]])
def test_rec_gradients(preact, blend, cu):
    rng = np.random.default_rng(3)
    B, T, D = (2 if cu is None else 1), 12, 3
    N = B if cu is None else len(cu) - 1
    v = dict(x=rng.standard_normal((B, T, D)), a=rng.uniform(0.2, 0.9, (B, T, D)),
             h0=rng.standard_normal((N, D)))
    dh, dT = rng.standard_normal((B, T, D)), rng.standard_normal((N, D))

    def loss(**v):
        f = R.rec(v["x"], v["a"], v["h0"], cu, preact, blend)
        return float((f["h"][0] * dh).sum() + (f["h_T"][0] * dT).sum())
    g = R.rec(v["x"], v["a"], v["h0"], cu, preact, blend, dh, dT)
    agree(loss, v, dict(x=g["dx"][0], a=g["da"][0], h0=g["dh0"][0]), rng)


def test_rec_is_the_closed_form():
    # constant decay: h_T = a^T h0 + sum a^(T-1-t) x_t
    rng = np.random.default_rng(4)
    x, a = rng.standard_normal((1, 20, 2)), np.full((1, 20, 2), 0.75)
    f = R.rec(x, a, np.ones((1, 2)), None, False, False)
    want = 0.75 ** 20 + (0.75 ** np.arange(19, -1, -1)[:, None] * x[0]).sum(0)
    assert np.allclose(f["h_T"][0][0], want, rtol=1e-14)


def test_check_refuses_a_wrong_value():
    value = np.ones(4)
    R.check(value * (1 + 2.0 ** -9), (value, np.zeros(4)), "bf16", "fine")
    with pytest.raises(AssertionError):
        R.check(value * (1 + 2.0 ** -7), (value, np.zeros(4)), "bf16", "too far")
    with pytest.raises(AssertionError):
        R.check(np.array([1, 1, 1, np.nan]), (value, np.zeros(4)), "bf16", "NaN")
