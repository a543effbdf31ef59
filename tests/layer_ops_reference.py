"""64-bit references of group norm with an activation and of dropout, from their
definitions in numpy, with the bounds of fp32 arithmetic (block_reference)."""
import numpy as np

from block_reference import U, chain, layer_norm, sigmoid


def _units(x, G):
    """x [N,S,C] as rows [N G, S C / G]."""
    N, S, C = x.shape
    return x.reshape(N, S, G, C // G).transpose(0, 2, 1, 3).reshape(N * G, S * (C // G))


def _back(u, shape, G):
    N, S, C = shape
    return u.reshape(N, G, S, C // G).transpose(0, 2, 1, 3).reshape(shape)


def _param(p, shape, G, other):
    """[C] at every element of the units."""
    return _units(np.broadcast_to(np.full(shape[2], other) if p is None else p, shape), G)


def silu_error(z):
    """Of z sigmoid(z) and of its slope: the sigmoid is off by 3 |z| U (the
    exponent's rounding) and 4 U (base 2 exponential, reciprocal, their sum)."""
    return (3 * np.abs(z) + 8) * U


def group_norm(x, G, weight, bias, eps, silu):
    shape = x.shape
    u, w, b = _units(x, G), _param(weight, shape, G, 1.0), _param(bias, shape, G, 0.0)
    r = layer_norm(u, w, b, eps)
    z, e_z = r["y"]
    if silu:
        y = z * sigmoid(z)
        e_y = 1.1 * e_z + np.abs(y) * silu_error(z)
    else:
        y, e_y = z, e_z
    stats = {n: tuple(v.reshape(shape[0], G) for v in r[n]) for n in ("mean", "rstd")}
    return dict(stats, y=(_back(y, shape, G), _back(e_y, shape, G)))


def group_norm_bwd(dy, x, mean, rstd, weight, bias, silu):
    """For the statistics as given (fp32 values)."""
    shape, G = x.shape, mean.shape[1]
    u, d, w, b = _units(x, G), _units(dy, G), _param(weight, shape, G, 1.0), _param(bias, shape, G, 0.0)
    m, r = mean.reshape(-1, 1), rstd.reshape(-1, 1)
    K = chain(u.shape[1])
    xh = (u - m) * r
    e_xh = 2 * U * np.abs(xh)
    g, e_g = d, 0.0 * np.abs(d)
    if silu:
        z = xh * w + b
        p = sigmoid(z)
        g = d * p * (1 + z * (1 - p))
        # slope: terms p and p z (1 - p); its own slope is at most 1/2
        e_z = np.abs(w) * e_xh + 2 * U * (np.abs(xh * w) + np.abs(b))
        e_g = np.abs(d) * (0.5 * e_z + (p + p * np.abs(z) * (1 - p) + np.abs(p * z) * p) * silu_error(z) + 2 * U)
    q = g * w
    s1, s2 = q.mean(-1, keepdims=True), (q * xh).mean(-1, keepdims=True)
    e1 = (K + 2) * U * np.abs(q).mean(-1, keepdims=True) + (e_g * np.abs(w)).mean(-1, keepdims=True)
    e2 = (K + 6) * U * np.abs(q * xh).mean(-1, keepdims=True) + (e_g * np.abs(w * xh)).mean(-1, keepdims=True)
    dx = r * (q - s1 - xh * s2)
    e_dx = r * (e_g * np.abs(w) + e1 + np.abs(xh) * e2 + e_xh * np.abs(s2)
                + 4 * U * (np.abs(q) + np.abs(s1) + np.abs(xh * s2)))
    rows = shape[0] * shape[1]
    Kr = chain(rows) + rows / 512 + 520
    over = lambda t: _back(t, shape, G).sum((0, 1))
    return {"dx": (_back(dx, shape, G), _back(e_dx, shape, G)),
            "dweight": (over(g * xh), (Kr + 4) * U * over(np.abs(g * xh)) + over(e_g * np.abs(xh))),
            "dbias": (over(g), Kr * U * over(np.abs(g)) + over(e_g))}


# ---- dropout ----------------------------------------------------------------

def philox(counter, key):
    """Philox4x32-10 of counters [n,4] (32-bit words, low first) and a key of two words."""
    c = [np.asarray(counter[:, i], np.uint64) for i in range(4)]
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    k = [int(key[0]), int(key[1])]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> half) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> half) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, 1).astype(np.uint32)


def kept(n, p, seed, offset):
    """Which of n elements stay, and the share that does."""
    blocks = np.arange((n + 7) // 8, dtype=np.uint64)
    counter = np.empty((len(blocks), 4), np.uint64)
    counter[:, 0], counter[:, 1] = blocks & np.uint64(0xFFFFFFFF), blocks >> np.uint64(32)
    counter[:, 2], counter[:, 3] = offset & 0xFFFFFFFF, offset >> 32
    words = philox(counter, (seed & 0xFFFFFFFF, seed >> 32))
    bits = np.stack([words & np.uint32(0xFFFF), words >> np.uint32(16)], 2).reshape(-1)[:n]
    least = round(p * 65536)
    return bits >= least, (65536 - least) / 65536
