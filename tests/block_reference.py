"""64-bit references of the operators around the mixer (layer norm, short
convolution, gated recurrence), written from their definitions in numpy, and
the error that fp32 arithmetic with one final rounding may leave.

Every reference returns {name: (value, bound)}: ``bound`` is the fp32 part of
the tolerance, propagated through the definition with U = 2^-24 per operation.
``check`` adds the rounding of the stored value: half a step, 2^-8 of the
value in bf16 and 2^-24 in fp32, and the smallest normal fp32 number times the
terms, since denormal results may be flushed.
"""
import numpy as np

U = 2.0 ** -24
STORE = {"bf16": 2.0 ** -8, "f32": U}
TINY = 2.0 ** -120


def check(got, ref, io, name):
    """got: the stored tensor as float64; ref: (value, bound)."""
    value, bound = ref
    got = np.asarray(got, np.float64)
    assert got.shape == value.shape, (name, got.shape, value.shape)
    if not value.size:
        return
    assert np.array_equal(np.isnan(got), np.isnan(value)), name + ": NaN in other places"
    fine = np.isfinite(value)
    assert np.array_equal(got[~fine & ~np.isnan(value)], value[~fine & ~np.isnan(value)]), name
    # 1.01: products of the small terms, left out of the bounds
    tol = STORE[io] * np.abs(value) + 1.01 * bound * (1 + STORE[io]) + TINY
    off = np.abs(got - value)[fine]
    worst = np.argmax(off - tol[fine])
    assert (off <= tol[fine]).all(), "%s: off by %.3g where %.3g is allowed (value %.6g), %d of %d" % (
        name, off[worst], tol[fine][worst], value[fine][worst], (off > tol[fine]).sum(), off.size)


# ---- layer norm -----------------------------------------------------------

def chain(n):
    """Additions in the longest chain of a sum of n terms as the kernels form
    it: at most max(64, n / 256) terms one after another, then pairwise."""
    return max(64, n / 256) + 12


def layer_norm(x, weight, bias, eps):
    D = x.shape[-1]
    w = np.ones(D) if weight is None else weight
    b = np.zeros(D) if bias is None else bias
    K = chain(D)
    mean = x.mean(-1, keepdims=True)
    e_mean = K * U * np.abs(x).mean(-1, keepdims=True)
    d = x - mean
    var = np.square(d).mean(-1, keepdims=True)
    e_var = (K + 4) * U * var + np.square(e_mean)
    with np.errstate(divide="ignore", invalid="ignore"):
        rstd = 1 / np.sqrt(var + eps)
        r_rstd = 0.5 * e_var / (var + eps) + 4 * U
        xh = d * rstd
        y = xh * w + b
        e_y = np.abs(w) * rstd * (e_mean + U * np.abs(d)) + np.abs(xh * w) * (r_rstd + 4 * U) + 2 * U * np.abs(b)
    return {"y": (y, e_y), "mean": (mean[..., 0], e_mean[..., 0]),
            "rstd": (rstd[..., 0], (rstd * r_rstd)[..., 0])}


def layer_norm_bwd(dy, x, mean, rstd, weight):
    """For the statistics as given (fp32 values)."""
    rows, D = x.shape
    w = np.ones(D) if weight is None else weight
    K = chain(D)
    m, r = mean[:, None], rstd[:, None]
    xh = (x - m) * r
    e_xh = 2 * U * np.abs(xh)
    g = dy * w
    s1, s2 = g.mean(-1, keepdims=True), (g * xh).mean(-1, keepdims=True)
    e1 = (K + 2) * U * np.abs(g).mean(-1, keepdims=True)
    e2 = (K + 6) * U * np.abs(g * xh).mean(-1, keepdims=True)
    dx = r * (g - s1 - xh * s2)
    e_dx = r * (e1 + np.abs(xh) * e2 + e_xh * np.abs(s2) + 4 * U * (np.abs(g) + np.abs(s1) + np.abs(xh * s2)))
    Kr = chain(rows) + rows / 512 + 520
    return {"dx": (dx, e_dx),
            "dweight": ((dy * xh).sum(0), (Kr + 4) * U * np.abs(dy * xh).sum(0)),
            "dbias": (dy.sum(0), Kr * U * np.abs(dy).sum(0))}


# ---- sequences ------------------------------------------------------------

def spans(B, T, cu):
    """(row, first token, behind the last) of every sequence."""
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    return [(0, int(p), int(q)) for p, q in zip(cu[:-1], cu[1:])]


def sigmoid(z):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-z))


def gate_error(a):
    """Relative error of sigmoid(a) from base-2 hardware operations: the
    exponent a log2(e) is off by 2 roundings of |a|, exp2 and the reciprocal
    by one unit in the last place (2 U) each, the sum by a rounding."""
    return (2 * np.abs(a) + 6) * U


# ---- short convolution ------------------------------------------------------

def conv(x, weight, bias, state0, cu, silu, dy=None, dstate_T=None):
    """Forward, and with dy the gradients too."""
    B, T, D = x.shape
    W = weight.shape[0]
    seqs = spans(B, T, cu)
    N = len(seqs)
    b = np.zeros(D) if bias is None else bias
    y, e_y = np.zeros_like(x), np.zeros_like(x)
    state = np.zeros((N, W - 1, D))
    dx, e_dx = np.zeros_like(x), np.zeros_like(x)
    ds0, e_ds0 = np.zeros((N, W - 1, D)), np.zeros((N, W - 1, D))
    dw, db, m_dw, m_db = np.zeros((W, D)), np.zeros(D), np.zeros((W, D)), np.zeros(D)
    for n, (row, p, q) in enumerate(seqs):
        first = np.zeros((W - 1, D)) if state0 is None else state0[n]
        wide = np.concatenate([first, x[row, p:q]])
        L = q - p
        state[n] = wide[L:]
        z, m = np.tile(b, (L, 1)), np.tile(np.abs(b), (L, 1))
        for j in range(W):  # tap j of token t is row t + W - 1 - j of wide
            z = z + weight[W - 1 - j] * wide[W - 1 - j:W - 1 - j + L]
            m = m + np.abs(weight[W - 1 - j] * wide[W - 1 - j:W - 1 - j + L])
        e_z = (W + 1) * U * m
        s = sigmoid(z)
        r_s = gate_error(z)
        if silu:
            y[row, p:q] = z * s
            slope = s * (1 + z * (1 - s))
            e_y[row, p:q] = e_z * 1.1 + np.abs(z * s) * (r_s + 2 * U)
            # |silu''| <= 1/2; the slope's own operations: each term's error
            e_slope = 0.5 * e_z + np.abs(s) * (r_s + 3 * U) * (1 + 2 * np.abs(z)) + 3 * U
        else:
            y[row, p:q], e_y[row, p:q] = z, e_z
            slope, e_slope = np.ones_like(z), np.zeros_like(z)
        if dy is None:
            continue
        d = dy[row, p:q]
        g, e_g = d * slope, np.abs(d) * e_slope + U * np.abs(d * slope)
        dwide, e_dwide = np.zeros_like(wide), np.zeros_like(wide)
        if dstate_T is not None:
            dwide[L:] += dstate_T[n]
        for j in range(W):
            at = slice(W - 1 - j, W - 1 - j + L)
            dwide[at] += weight[W - 1 - j] * g
            e_dwide[at] += np.abs(weight[W - 1 - j]) * (e_g + (W + 2) * U * np.abs(g))
            dw[W - 1 - j] += (g * wide[at]).sum(0)
            m_dw[W - 1 - j] += (e_g * np.abs(wide[at])).sum(0)
        db += g.sum(0)
        m_db += e_g.sum(0)
        if dstate_T is not None:
            e_dwide[L:] += (W + 1) * U * np.abs(dstate_T[n])
        dx[row, p:q], e_dx[row, p:q] = dwide[W - 1:], e_dwide[W - 1:]
        ds0[n], e_ds0[n] = dwide[:W - 1], e_dwide[:W - 1]
    out = {"y": (y, e_y), "state_T": (state, np.zeros_like(state))}
    if dy is not None:
        # the sums over tokens: their longest chain, times the magnitudes
        K = chain(B * T) + B * T / 512 + 520
        mg = np.abs(dy) * 1.1
        big = np.abs(x).max(initial=0) if state0 is None else max(np.abs(x).max(initial=0), np.abs(state0).max(initial=0))
        out.update({"dx": (dx, e_dx), "dstate0": (ds0, e_ds0),
                    "dweight": (dw, m_dw + K * U * mg.sum((0, 1)) * big),
                    "dbias": (db, m_db + K * U * mg.sum((0, 1)))})
    return out


# ---- gated recurrence -----------------------------------------------------------

def rec(x, a, h0, cu, preact, blend, dh=None, dh_T=None, interval=64):
    B, T, D = x.shape
    seqs = spans(B, T, cu)
    N = len(seqs)
    alpha = sigmoid(a) if preact else a
    rest = sigmoid(-a) if preact else 1 - a
    r_g = gate_error(a) if preact else np.full_like(a, U)
    u = rest * x if blend else x
    e_u = np.abs(u) * ((r_g + U) if blend else 0)
    h, e_h = np.zeros_like(x), np.zeros_like(x)
    prev, e_prev = np.zeros_like(x), np.zeros_like(x)
    h_T, e_T = np.zeros((N, D)), np.zeros((N, D))
    chk = np.full((B, -(-T // interval), D), np.nan)
    e_chk = np.zeros_like(chk)
    for n, (row, p, q) in enumerate(seqs):
        now = np.zeros(D) if h0 is None else h0[n]
        e = np.zeros(D)
        m = np.abs(now)  # the sum of the magnitudes behind `now`
        for t in range(p, q):
            if t % interval == 0:
                chk[row, t // interval], e_chk[row, t // interval] = now, e
            prev[row, t], e_prev[row, t] = now, e
            al = alpha[row, t]
            m = al * m + np.abs(u[row, t])
            # a step, or a factor of the products that join spans: alpha's
            # error, and 3 roundings
            e = al * e + (r_g[row, t] + 3 * U) * m + e_u[row, t]
            now = al * now + u[row, t]
            h[row, t], e_h[row, t] = now, e
        h_T[n], e_T[n] = now, e
    out = {"h": (h, e_h), "h_T": (h_T, e_T), "checkpoints": (chk, e_chk)}
    if dh is None:
        return out
    lam, e_lam = np.zeros_like(x), np.zeros_like(x)
    dh0, e_dh0 = np.zeros((N, D)), np.zeros((N, D))
    for n, (row, p, q) in enumerate(seqs):
        g = np.zeros(D) if dh_T is None else dh_T[n]
        e, m = np.zeros(D), np.abs(g)
        for t in range(q - 1, p - 1, -1):
            al = alpha[row, t]
            lam[row, t] = dh[row, t] + g
            m = m + np.abs(dh[row, t])
            e = e + 3 * U * m
            e_lam[row, t] = e
            g = al * lam[row, t]
            m = al * m
            e = al * e + (r_g[row, t] + 3 * U) * m
        dh0[n], e_dh0[n] = g, e
    part = prev - x if blend else prev
    e_part = e_prev + (U * np.abs(part) if blend else 0)
    slope = alpha * rest if preact else np.ones_like(alpha)
    da = lam * part * slope
    e_da = slope * (e_lam * np.abs(part) + np.abs(lam) * e_part) + np.abs(da) * (2 * r_g + 4 * U)
    dx = lam * rest if blend else lam
    e_dx = (rest * e_lam + np.abs(dx) * (r_g + 2 * U)) if blend else e_lam
    out.update({"dx": (dx, e_dx), "da": (da, e_da), "dh0": (dh0, e_dh0)})
    return out
