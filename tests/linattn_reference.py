"""64-bit reference of linear attention with a decay for each head, token by
token from its definition in numpy, with the bounds of the kernels' rounding.

``forward`` and ``backward`` return {name: (value, bound)} as block_reference
does; ``bound`` is the sum of the terms' magnitudes times what a term may lose:
- fp32 arithmetic, U = 2^-24 an operation: a product q k of dk terms, 64 terms
  of a chunk, 8 operations for each further 32 tokens of the state, and a power
  g^n = exp(n log g), off by (|n log g| + 4) U, which is at most 110 U where it
  does not vanish (two of them in a term);
- bf16 io: a term of y is rounded to bf16 as an operand once (half a step,
  2^-8), a term of a state is held as two bf16 parts (2^-16).
"""
import numpy as np

from block_reference import U


def walk(q, k, v, g, X0, late):
    """q, k [L,H,d], v [L,H,e] -> y [L,H,e] and the last state [H,d,e]: the
    state meets q behind a token (late = 0), or before its last decay does (1)."""
    X = X0.copy()
    y = np.empty(v.shape)
    for t in range(len(v)):
        if not late:
            X = g * X
        X = X + k[t][:, :, None] * v[t][:, None, :]
        y[t] = (X * q[t][:, :, None]).sum(1)
        if late:
            X = g * X
    return y, X


def spans(B, T, cu):
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    return [(0, p, e) for p, e in zip(cu[:-1], cu[1:])]


def _bounds(io, T, d):
    arithmetic = (d + 64 + 8 * (T // 32 + 1) + 220) * U
    return ((2.0 ** -8 + 2.0 ** -16 + arithmetic, 2.0 ** -16 + arithmetic) if io == "bf16"
            else (arithmetic, arithmetic))


def _over(B, T, cu, q, k, v, g, X0, late, back):
    """The walk over every sequence: y [B,T,H,e] (zeros behind the last one), X."""
    y, X = np.zeros(v.shape), X0.copy()
    for n, (row, p, e) in enumerate(spans(B, T, cu)):
        cut = lambda x: x[row, p:e][::-1] if back else x[row, p:e]
        if e > p:
            out, X[n] = walk(cut(q), cut(k), cut(v), g, X0[n], late)
            y[row, p:e] = out[::-1] if back else out
    return y, X


def _both(make):
    return make(lambda x: x), make(np.abs)


def forward(q, k, v, g, scale, S0, cu, io):
    B, T, H, dv = v.shape
    G, dk = H // q.shape[2], q.shape[3]
    N = len(spans(B, T, cu))
    q, k = (np.repeat(x, G, 2) for x in (q, k))
    g = g[:, None, None]
    S0 = np.zeros((N, H, dk, dv)) if S0 is None else S0
    (o, S), (oa, Sa) = _both(lambda f: _over(B, T, cu, f(q), f(k), f(v), g, f(S0), 0, False))
    ey, es = _bounds(io, T, dk)
    return {"o": (scale * o, abs(scale) * oa * ey), "S_T": (S, Sa * es)}


def backward(do, q, k, v, g, scale, S0, dS, cu, io):
    B, T, H, dv_ = v.shape
    Hk, dk_ = q.shape[2:]
    G = H // Hk
    N = len(spans(B, T, cu))
    q, k = (np.repeat(x, G, 2) for x in (q, k))
    g = g[:, None, None]
    S0 = np.zeros((N, H, dk_, dv_)) if S0 is None else S0
    dS = np.zeros((N, H, dk_, dv_)) if dS is None else dS
    turn = lambda x: x.swapaxes(-1, -2)
    shared = lambda x: x.reshape(B, T, Hk, G, dk_).sum(3)
    out = {}

    def put(name, both, bound, finish=lambda x: x):
        out[name] = (finish(both[0]), finish(both[1]) * bound + U * G * finish(np.abs(both[0])))
    dq = _both(lambda f: _over(B, T, cu, f(do), f(v), f(k), g, f(turn(S0)), 0, False)[0] * f(scale))
    dk = _both(lambda f: _over(B, T, cu, f(v), f(do) * f(scale), f(q), g, f(turn(dS)), 1, True)[0])
    (dv, dS0), (dva, dS0a) = _both(lambda f: _over(B, T, cu, f(k), f(q) * f(scale), f(do), g, f(dS), 1, True))
    ey, _ = _bounds(io, T, dv_)
    put("dq", dq, ey, shared)
    put("dk", dk, ey, shared)
    ey, es = _bounds(io, T, dk_)
    put("dv", (dv, dva), ey)
    out["dS0"] = (dS0, dS0a * es)
    return out
