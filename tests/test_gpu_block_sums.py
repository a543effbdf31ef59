"""Sums over rows and tokens -- layer norm's dweight and dbias, the convolution's -- with
bounds that a lost or doubled row would break: sizes whose workgroups walk many sets of
rows and whose runs have borders everywhere, and calls larger than the last-level
cache, against 64 bits."""
import numpy as np
import pytest
import torch

import kalman_delta_rule_amd as kda

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a HIP GPU")


def close(got, want, bound, magnitude, count, name):
    """Within the bound; for up to 10000 rows that is less than half of what the average
    one adds, so that a row too many or too few shows (of more rows the count is
    tested, in whole numbers, below)."""
    assert count > 10000 or (bound <= 0.5 * magnitude / count).all(), name
    off = (got.double() - want).abs()
    bad = off > bound
    assert not bad.any(), "%s: %d of %d off, worst %.3g of the bound" % (
        name, int(bad.sum()), bad.numel(), float((off / bound).max()))


def layer_norm_sums(x, dy, mean, rstd):
    """In 64 bits, of the statistics as given: sums, and sums of magnitudes."""
    xh = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    t = dy.double() * xh
    return (t.sum(0), dy.double().sum(0)), (t.abs().sum(0), dy.double().abs().sum(0))


# every number of threads and vectors a row, with workgroups of several sets of rows
SHAPES = [(70000, 60), (70000, 64), (40000, 100), (20000, 250), (9000, 500), (9000, 1000), (5000, 2048),
          (3001, 3000), (1500, 6001), (1500, 8192), (1500, 16384), (700, 16385), (300, 40000)]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D", SHAPES)
def test_layer_norm_sums(rows, D, io):
    g = torch.Generator(device="cuda").manual_seed(rows + D)
    x, dy = (torch.randn(rows, D, generator=g, device="cuda").to(DT[io]) for _ in range(2))
    w = torch.randn(D, generator=g, device="cuda")
    _, mean, rstd = kda.kdn_layer_norm_fwd(x, w, want_stats=True)
    q = kda.kdn_layer_norm_bwd(dy, x, mean, rstd, w)
    (dw, db), (mw, mb) = layer_norm_sums(x, dy, mean, rstd)
    # a thread adds one row of each of its workgroup's sets (at least 16 rows a workgroup,
    # at most 512 workgroups), the lanes and sets of a workgroup are joined (22 at
    # most), then 512 / 16 partial sums and 16 shares; 4 roundings of a term
    terms = max(rows / 256, 16) + 22 + 32 + 16 + 4
    close(q["dweight"], dw, terms * U * mw, mw, rows, "dweight")
    close(q["dbias"], db, terms * U * mb, mb, rows, "dbias")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [60, 250, 1000, 2050, 6144, 16384])
def test_layer_norm_sums_larger_than_the_last_level_cache(D, io):
    dt = DT[io]
    rows = ((256 << 20) // (D * dt.itemsize) // 3 + 1) * 3
    g = torch.Generator(device="cuda").manual_seed(7)
    x, dy = (torch.empty(rows, D, device="cuda").normal_(generator=g).to(dt) for _ in range(2))
    assert x.numel() * x.element_size() >= 256 << 20
    _, mean, rstd = kda.kdn_layer_norm_fwd(x, want_stats=True)
    q = kda.kdn_layer_norm_bwd(dy, x, mean, rstd)
    want, size = [0, 0], [0, 0]
    for p in torch.arange(rows, device="cuda").tensor_split(8):
        p = slice(int(p[0]), int(p[-1]) + 1)
        a, m = layer_norm_sums(x[p], dy[p], mean[p], rstd[p])
        want, size = [u + v for u, v in zip(want, a)], [u + v for u, v in zip(size, m)]
    # a workgroup's threads of a column: (sets of) 1024 * 16 / (D bytes) rows at a time,
    # 512 workgroups, so rows / 512 / that many terms one after another, then as above
    sets = max(1024 * 16 // (2 * D * dt.itemsize), 1)
    terms = rows / (256 * sets) + 22 + 32 + 16 + 4
    for k, v, m in zip(("dweight", "dbias"), want, size):
        close(q[k], v, terms * U * m, m, rows, k)
    n = kda.kdn_layer_norm_bwd(torch.ones_like(dy), x, mean, rstd)["dbias"]
    assert (n == rows).all()  # every row once


# runs of 8 to 128 tokens, one to 32 of them a workgroup, one and several tiles; borders
# in runs, at their ends, in the tokens before them; rows of one token
SEQ = [(40, 100, 5, None), (64, 37, 40, None), (700, 1, 66, None), (1, 5000, 130, None), (1, 3000, 1, None),
       (3, 1021, 333, None), (2, 4100, 520, None),
       (1, 2000, 70, [0, 1, 2, 3, 4, 7, 8, 15, 16, 17, 63, 64, 65, 128, 300, 301, 512, 1024, 1900]),
       (1, 4000, 260, [0, 8, 1000, 1000, 2040, 3990]), (1, 1200, 33, list(range(0, 1201, 5)))]


def conv_sums(x, dy, w, b, s0, cu):
    """dweight and dbias in 64 bits, the sums of the magnitudes |g x| and |g|, and those of
    their terms' own errors: z is off by (W + 1) U of its terms' magnitudes, the sigmoid s by
    (2 |z| + 6) U of itself, so the slope s (1 + z (1 - s)), with |slope'| <= 1/2, by
    what is added up below, and g by a rounding more."""
    B, T, D = x.shape
    W = w.shape[0]
    spans = [(n, 0, T) for n in range(B)] if cu is None else [(0, p, q) for p, q in zip(cu[:-1], cu[1:])]
    dw, mw, ew = (torch.zeros(W, D).double() for _ in range(3))
    db, mb, eb = (torch.zeros(D).double() for _ in range(3))
    for n, (row, p, q) in enumerate(spans):
        wide = torch.cat((s0[n], x[row, p:q])).double()
        taps = [wide[k:k + q - p] for k in range(W)]
        z = b + sum(w[k] * taps[k] for k in range(W))
        e_z = (W + 1) * U * (b.abs() + sum((w[k] * taps[k]).abs() for k in range(W)))
        s = torch.sigmoid(z)
        d = dy[row, p:q].double()
        g = d * s * (1 + z * (1 - s))
        e = d.abs() * (0.5 * e_z + s * (2 * z.abs() + 9) * U * (1 + 2 * z.abs()) + 3 * U) + U * g.abs()
        for k in range(W):
            dw[k] += (g * taps[k]).sum(0)
            mw[k] += (g * taps[k]).abs().sum(0)
            ew[k] += (e * taps[k].abs()).sum(0)
        db += g.sum(0)
        mb += g.abs().sum(0)
        eb += e.sum(0)
    return (dw, db), (mw, mb), (ew, eb)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("case", SEQ, ids=lambda c: "B%dT%dD%d%s" % (c[:3] + ("" if c[3] is None else "N",)))
def test_conv_sums(case, W, io):
    B, T, D, cu = case
    N = B if cu is None else len(cu) - 1
    g = torch.Generator().manual_seed(T + D + W)
    new = lambda *s: torch.randn(*s, generator=g)
    x, dy, s0 = (t.to(DT[io]) for t in (new(B, T, D), new(B, T, D), new(N, W - 1, D)))
    w, b = new(W, D) * 0.5, new(D)
    want, size, own = conv_sums(x, dy, w.double(), b.double(), s0, cu)
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    q = kda.kdn_conv_bwd(dy.cuda(), x.cuda(), w.cuda(), bias=b.cuda(), state0=s0.cuda(), cu_seqlens=c, activation="silu")
    # a run adds its tokens (128 at most) one after another, the runs of a wave are
    # joined in 3 steps and the waves in 2, the tiles' sums in tiles / 16 and 16 steps
    # (a tile has at least 32 tokens)
    terms = 128 + 5 + B * T / 32 / 16 + 16
    for k, v, m, e in zip(("dweight", "dbias"), want, size, own):
        close(q[k].cpu(), v, terms * U * m + 1.01 * e, m, B * T, k)


def test_conv_counts_every_token_once():
    # whole numbers: no activation, inputs and gradients of one, so the sums are exact
    for B, T, D, W in ((1, 100000, 64, 4), (7, 4099, 260, 3), (333, 65, 9, 2), (1, 40000, 2048, 4), (5, 9000, 6, 4)):
        for dt in DT.values():
            one = torch.ones(B, T, D, dtype=dt, device="cuda")
            q = kda.kdn_conv_bwd(one, one, torch.ones(W, D, device="cuda"), bias=torch.ones(D, device="cuda"))
            assert (q["dbias"] == B * T).all()
            for j in range(W):  # j tokens of every row have none so far behind them
                assert (q["dweight"][W - 1 - j] == B * max(T - j, 0)).all()


def test_layer_norm_counts_every_row_once():
    # xh = +-1 and dy = 1: whole numbers
    for rows, D in ((100000, 64), (70001, 250), (9000, 2048), (3001, 6144), (800, 16384), (257, 20000)):
        for dt in DT.values():
            x = torch.ones(rows, D, dtype=dt, device="cuda")
            mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
            q = kda.kdn_layer_norm_bwd(x, x, mean, rstd)
            assert (q["dbias"] == rows).all() and (q["dweight"] == rows).all()
