"""The operators around the mixer (layer norm, short convolution, gated
recurrence) on the GPU against their 64-bit references, value by value, with
the bounds of block_reference: sizes from one token to several tiles, odd
channel counts, packed sequences with empty ones, slices of wider rows, tokens
behind the last sequence, values that must not cross into another sequence,
captured and replayed calls, other streams."""
import numpy as np
import pytest
import torch

import block_reference as R
import kalman_delta_rule_amd as kda

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a HIP GPU")


def host(t):
    return t.detach().cpu().double().numpy()


def dev(a, io="f32"):
    """A float64 array on the GPU, and what it holds there as float64."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DT[io])
    return t.cuda(), t.double().numpy()


def sliced(t, width):
    """The same values as a slice of rows `width` times as wide."""
    wide = torch.full(t.shape[:-1] + (width * t.shape[-1] + 1,), float("nan"), dtype=t.dtype,
                      device=t.device)
    part = wide[..., 1:1 + t.shape[-1]]
    part.copy_(t)
    return part


def offsets(cu):
    return None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")


def same(a, b):
    """Equal bit for bit, NaN included."""
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ---- layer norm -----------------------------------------------------------

LN_SHAPES = [(0, 8), (1, 1), (3, 1), (5, 2), (7, 63), (64, 64), (33, 100), (130, 128), (9, 257),
             (17, 512), (21, 777), (12, 1024), (40, 1537), (19, 2048), (11, 2049), (6, 4096),
             (5, 6001), (4, 8192), (3, 10007), (3, 16384), (2, 16385), (2, 40000), (5000, 64),
             (3001, 100), (1200, 2048)]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D", LN_SHAPES)
def test_layer_norm(rows, D, io):
    rng = np.random.default_rng(rows * 31 + D)
    x, xr = dev(rng.standard_normal((rows, D)) * 2 + 0.5, io)
    dy, dyr = dev(rng.standard_normal((rows, D)), io)
    w, wr = dev(rng.standard_normal(D))
    b, br = dev(rng.standard_normal(D))
    if (rows + D) % 3 == 1:
        x = sliced(x, 2)
    if (rows + D) % 4 == 1:
        w = b = wr = br = None
    eps = 1e-5
    ref = R.layer_norm(xr, wr, br, float(np.float32(eps)))
    y, mean, rstd = kda.kdn_layer_norm_fwd(x, w, b, eps=eps, want_stats=True)
    y2, none, _ = kda.kdn_layer_norm_fwd(x, w, b, eps=eps)
    assert none is None and same(y, y2)
    R.check(host(y), ref["y"], io, "y")
    R.check(host(mean), ref["mean"], "f32", "mean")
    R.check(host(rstd), ref["rstd"], "f32", "rstd")
    g = kda.kdn_layer_norm_bwd(dy, x, mean, rstd, w)
    ref = R.layer_norm_bwd(dyr, xr, host(mean), host(rstd), wr)
    R.check(host(g["dx"]), ref["dx"], io, "dx")
    R.check(host(g["dweight"]), ref["dweight"], "f32", "dweight")
    R.check(host(g["dbias"]), ref["dbias"], "f32", "dbias")
    only = kda.kdn_layer_norm_bwd(dy, x, mean, rstd, w, want_param_grads=False)
    assert set(only) == {"dx"} and same(only["dx"], g["dx"])


def test_layer_norm_far_from_zero():
    # a spread of one around 20000: the variance has to be taken around the mean
    rng = np.random.default_rng(5)
    x, xr = dev(rng.standard_normal((64, 2048)) + 20000.0)
    y, mean, rstd = kda.kdn_layer_norm_fwd(x, eps=0.0, want_stats=True)
    ref = R.layer_norm(xr, None, None, 0.0)
    for got, name in ((y, "y"), (mean, "mean"), (rstd, "rstd")):
        R.check(host(got), ref[name], "f32", name)


def test_layer_norm_constant_rows_and_bad_rows():
    x = torch.full((8, 384), 3.0, device="cuda")
    x[3, 7] = float("nan")
    x[5, 9] = float("inf")
    y, mean, rstd = kda.kdn_layer_norm_fwd(x, eps=1e-6, want_stats=True)
    good = [0, 1, 2, 4, 6, 7]
    assert (y[good] == 0).all() and (mean[good] == 3).all()
    assert torch.isnan(y[3]).all() and torch.isnan(y[5]).all()
    # a bad row spoils its own dx and the parameter gradients, no other row
    g = kda.kdn_layer_norm_bwd(torch.ones_like(x), x, mean, rstd)
    assert torch.isfinite(g["dx"][good]).all() and torch.isnan(g["dx"][[3, 5]]).all()


def test_layer_norm_over_heads_is_rows():
    # o [B,T,H,dv] normalised over dv, and a slice along T of a longer buffer
    x = torch.randn(2, 6, 3, 64, device="cuda").to(torch.bfloat16)
    y, mean, _ = kda.kdn_layer_norm_fwd(x, want_stats=True)
    assert y.shape == x.shape and mean.shape == (2, 6, 3)
    flat, _, _ = kda.kdn_layer_norm_fwd(x.view(36, 64))
    assert same(y.view(36, 64), flat)
    with pytest.raises(ValueError, match="evenly spaced"):
        kda.kdn_layer_norm_fwd(x[:, 1:4])
    with pytest.raises(ValueError, match="side by side"):
        kda.kdn_layer_norm_fwd(x.transpose(-1, -2))


# ---- sequences --------------------------------------------------------------

def layouts(T):
    """Packings of a row of T tokens: one token, empty sequences at both ends
    and in the middle, borders on and around the tiles' edges, tokens left
    behind the last sequence."""
    cuts = sorted({min(c, T) for c in (0, 1, 1, 2, 5, 63, 64, 65, 127, 128, 255, 256, 257, 300, 512, 1000)})
    return [[0, T], [0, 0, T, T], [0] + cuts + [T], [0, T // 3, T // 3, T - T // 4]]


SEQ_CASES = [(2, 0, 5, None), (3, 1, 4, None), (2, 2, 1, None), (1, 3, 3, None), (4, 5, 7, None),
             (2, 16, 64, None), (1, 17, 130, None), (2, 64, 8, None), (3, 65, 33, None),
             (1, 200, 100, None), (2, 256, 66, None), (1, 257, 129, None), (2, 700, 72, None),
             (1, 1500, 31, None), (1, 0, 6, [0, 0, 0]), (1, 1, 6, [0, 0, 1])]
# more sequences than a workgroup has threads; many rows (the recurrence's short tiles);
# a single channel; several tiles of channels
SEQ_CASES += [(1, 2000, 6, [0] + sorted(np.random.default_rng(8).integers(0, 1990, 1500).tolist()) + [1995]),
              (200, 300, 5, None), (193, 1, 3, None), (1, 300, 1, None), (1, 300, 1, [0, 0, 7, 290]),
              (1, 150, 12300, None), (1, 90, 520, [0, 33, 90])]
SEQ_CASES += [(1, T, D, cu) for T, D in ((7, 9), (64, 16), (259, 40), (600, 70), (1301, 12)) for cu in layouts(T)]


def ids(case):
    B, T, D, cu = case
    return "B%dT%dD%d%s" % (B, T, D, "" if cu is None else "N%d" % (len(cu) - 1))


def check_rows(got, ref, io, name, T, cu):
    """Per-token outputs: values up to the last sequence, the sentinel behind."""
    end = T if cu is None else cu[-1]
    R.check(host(got)[:, :end], (ref[0][:, :end], ref[1][:, :end]), io, name)
    assert (host(got)[:, end:] == 77).all(), name + ": written behind the last sequence"


def poison(shape, dtype):
    return torch.full(shape, 77.0, dtype=dtype, device="cuda")


# ---- short convolution ---------------------------------------------------------

@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("W,silu", [(2, True), (3, False), (4, True)])
@pytest.mark.parametrize("case", SEQ_CASES, ids=ids)
def test_conv(case, W, silu, io):
    B, T, D, cu = case
    N = B if cu is None else len(cu) - 1
    rng = np.random.default_rng(T * 7 + D + W)
    x, xr = dev(rng.standard_normal((B, T, D)), io)
    dy, dyr = dev(rng.standard_normal((B, T, D)), io)
    w, wr = dev(rng.standard_normal((W, D)))
    b, br = dev(rng.standard_normal(D))
    s0, s0r = dev(rng.standard_normal((N, W - 1, D)), io)
    ds, dsr = dev(rng.standard_normal((N, W - 1, D)), io)
    if (T + D) % 3 == 1:
        x = sliced(x, 3)
    if (T + W) % 4 == 1:
        b = br = s0 = s0r = ds = dsr = None
    act = "silu" if silu else None
    ref = R.conv(xr, wr, br, s0r, cu, silu, dyr, dsr)
    y, state = kda.kdn_conv_fwd(x, w, bias=b, state0=s0, cu_seqlens=offsets(cu), activation=act,
                                want_state=True, y=poison((B, T, D), DT[io]))
    check_rows(y, ref["y"], io, "y", T, cu)
    R.check(host(state), ref["state_T"], io, "state_T")
    _, none = kda.kdn_conv_fwd(x, w, bias=b, state0=s0, cu_seqlens=offsets(cu), activation=act)
    assert none is None
    g = kda.kdn_conv_bwd(dy, x, w, bias=b, state0=s0, cu_seqlens=offsets(cu), activation=act,
                         dstate_T=ds, dx=poison((B, T, D), DT[io]))
    check_rows(g["dx"], ref["dx"], io, "dx", T, cu)
    R.check(host(g["dweight"]), ref["dweight"], "f32", "dweight")
    assert ("dbias" in g) == (b is not None) and ("dstate0" in g) == (s0 is not None)
    if b is not None:
        R.check(host(g["dbias"]), ref["dbias"], "f32", "dbias")
        R.check(host(g["dstate0"]), ref["dstate0"], io, "dstate0")


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_conv_long_runs_are_the_short_ones(io):
    """A call large enough for runs of many tokens against calls on pieces of it,
    which have the shortest: the same operations for every y and dx, so the
    same bits; the sums to their rounding."""
    g = torch.Generator(device="cuda").manual_seed(6)
    T, D, W = 40000, 2048, 4
    x = torch.randn(1, T, D, generator=g, device="cuda").to(DT[io])
    dy = torch.randn(1, T, D, generator=g, device="cuda").to(DT[io])
    w, b = torch.randn(W, D, generator=g, device="cuda"), torch.randn(D, generator=g, device="cuda")
    cut = 17001
    cu = offsets([0, cut, T])
    y, _ = kda.kdn_conv_fwd(x, w, bias=b, cu_seqlens=cu, activation="silu")
    q = kda.kdn_conv_bwd(dy, x, w, bias=b, cu_seqlens=cu, activation="silu")
    for p in (0, 5000, 16900, cut, 39000):
        end = min(p + 1000, cut if p < cut else T)
        reach = min(end + W - 1, cut if p < cut else T)  # dx takes what follows in the sequence
        piece = x[:, p:reach].contiguous()
        kw = dict(bias=b, activation="silu")
        if p not in (0, cut):
            kw["state0"] = x[:, p - W + 1:p].contiguous()
        s, _ = kda.kdn_conv_fwd(piece, w, **kw)
        assert same(y[:, p:end], s[:, :end - p]), p
        d = kda.kdn_conv_bwd(dy[:, p:reach].contiguous(), piece, w, **kw)["dx"]
        # (a piece's first tokens lack nothing: dx looks ahead only)
        assert same(q["dx"][:, p:end], d[:, :end - p]), p
    halves = [kda.kdn_conv_bwd(dy[:, p:e].contiguous(), x[:, p:e].contiguous(), w, bias=b, activation="silu")
              for p, e in ((0, cut), (cut, T))]
    for k in ("dweight", "dbias"):
        # each side is off by at most its longest chain of additions times the sum of
        # magnitudes; a chain has under 128 + 16 + 400 / 16 + 20 terms
        size = (dy.float().abs() * 1.1).sum((0, 1)) * (x.float().abs().max() if k == "dweight" else 1)
        off = (q[k].double() - halves[0][k].double() - halves[1][k].double()).abs()
        assert (off <= 2 * 200 * R.U * size.double()).all(), k


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,D,W", [(1, 1, 2), (3, 5, 3), (2, 64, 4), (300, 33, 4), (5, 6144, 4),
                                   (1, 2050, 3)])
def test_conv_steps_are_the_forward(B, D, W, io):
    rng = np.random.default_rng(B + D)
    T = 6
    x, xr = dev(rng.standard_normal((B, T, D)), io)
    w, wr = dev(rng.standard_normal((W, D)))
    b, br = dev(rng.standard_normal(D))
    s0, s0r = dev(rng.standard_normal((B, W - 1, D)), io)
    ref = R.conv(xr, wr, br, s0r, None, True)
    state = s0.clone()
    for t in range(T):
        y = kda.kdn_conv_step(x[:, t], w, state, bias=b, activation="silu")
        R.check(host(y), (ref["y"][0][:, t], ref["y"][1][:, t]), io, "token %d" % t)
    assert np.array_equal(host(state), ref["state_T"][0])


# ---- gated recurrence ---------------------------------------------------------------

def rec_data(case, io, preact, seed):
    B, T, D, cu = case
    N = B if cu is None else len(cu) - 1
    rng = np.random.default_rng(seed)
    x, xr = dev(rng.standard_normal((B, T, D)), io)
    a = rng.standard_normal((B, T, D)) * 0.5 + rng.uniform(-2, 7, D)
    a, ar = dev(a if preact else R.sigmoid(a), io if preact else "f32")
    if not preact and T > 3:
        a[:, T // 2], ar[:, T // 2] = 0.0, 0.0
        a[:, 1], ar[:, 1] = 1.0, 1.0
    dh, dhr = dev(rng.standard_normal((B, T, D)), io)
    h0, h0r = dev(rng.standard_normal((N, D)))
    dT, dTr = dev(rng.standard_normal((N, D)))
    return (x, a, dh, h0, dT), (xr, ar, dhr, h0r, dTr)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("gate,blend", [("preact", True), ("preact", False), ("alpha", True),
                                        ("alpha", False)])
@pytest.mark.parametrize("case", SEQ_CASES, ids=ids)
def test_rec(case, gate, blend, io):
    B, T, D, cu = case
    preact = gate == "preact"
    (x, a, dh, h0, dT), (xr, ar, dhr, h0r, dTr) = rec_data(case, io, preact, T * 5 + D)
    if (T + D) % 3 == 1:
        x, a = sliced(x, 3), sliced(a, 2)
    if (T + D) % 4 == 1:
        h0 = h0r = dT = dTr = None
    ref = R.rec(xr, ar, h0r, cu, preact, blend, dhr, dTr)
    kw = dict(cu_seqlens=offsets(cu), gate=gate, blend=blend)
    h, h_T, chk = kda.kdn_rec_fwd(x, a, h0=h0, want_checkpoints=True, h=poison((B, T, D), DT[io]), **kw)
    check_rows(h, ref["h"], io, "h", T, cu)
    R.check(host(h_T), ref["h_T"], "f32", "h_T")
    end = T if cu is None else cu[-1]
    k = -(-end // 64)  # later ones belong to no sequence
    R.check(host(chk)[:, :k], (ref["checkpoints"][0][:, :k], ref["checkpoints"][1][:, :k]), "f32", "checkpoints")
    h2, h2_T, none = kda.kdn_rec_fwd(x, a, h0=h0, h=poison((B, T, D), DT[io]), **kw)
    assert none is None and same(h, h2) and same(h_T, h2_T)
    g = kda.kdn_rec_bwd(dh, x, a, chk, h0=h0, dh_T=dT, dx=poison((B, T, D), DT[io]), **kw)
    check_rows(g["dx"], ref["dx"], io, "dx", T, cu)
    R.check(host(g["da"])[:, :end], (ref["da"][0][:, :end], ref["da"][1][:, :end]),
            io if preact else "f32", "da")
    R.check(host(g["dh0"]), ref["dh0"], "f32", "dh0")


@pytest.mark.parametrize("T", [4096, 5000, 20000])
def test_rec_long(T):
    # many tiles, groups and (beyond 64 tiles) blocks of them; decays close to one
    # carry across all of them
    D = 64 if T < 10000 else 3
    for case, io in (((1, T, D, None), "f32"), ((1, T, 10, [0, 3, 900, 900, 2500, T - 7]), "bf16")):
        (x, a, dh, h0, dT), (xr, ar, dhr, h0r, dTr) = rec_data(case, io, True, T)
        ref = R.rec(xr, ar, h0r, case[3], True, True, dhr, dTr)
        kw = dict(cu_seqlens=offsets(case[3]), blend=True)
        h, h_T, chk = kda.kdn_rec_fwd(x, a, h0=h0, want_checkpoints=True, h=poison(x.shape, x.dtype), **kw)
        g = kda.kdn_rec_bwd(dh, x, a, chk, h0=h0, dh_T=dT, dx=poison(x.shape, x.dtype), **kw)
        check_rows(h, ref["h"], io, "h", T, case[3])
        check_rows(g["dx"], ref["dx"], io, "dx", T, case[3])
        R.check(host(h_T), ref["h_T"], "f32", "h_T")
        R.check(host(g["dh0"]), ref["dh0"], "f32", "dh0")
        end = T if case[3] is None else case[3][-1]
        R.check(host(g["da"])[:, :end], (ref["da"][0][:, :end], ref["da"][1][:, :end]), io, "da")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("gate,blend", [("preact", True), ("alpha", False)])
@pytest.mark.parametrize("B,D", [(1, 1), (3, 5), (2, 64), (300, 33), (1, 2050)])
def test_rec_steps_are_the_forward(B, D, gate, blend, io):
    case, T = (B, 5, D, None), 5
    (x, a, _, h0, _), (xr, ar, _, h0r, _) = rec_data(case, io, gate == "preact", B + D)
    ref = R.rec(xr, ar, h0r, None, gate == "preact", blend)
    state = h0.clone()
    for t in range(T):
        h = kda.kdn_rec_step(x[:, t], a[:, t], state, gate=gate, blend=blend)
        R.check(host(h), (ref["h"][0][:, t], ref["h"][1][:, t]), io, "token %d" % t)
    R.check(host(state), ref["h_T"], "f32", "state")


def test_steps_read_one_token_of_a_long_buffer():
    # rows 6.3 million elements apart: beyond the recurrence's own limit for whole rows
    B, T, D = 3, 3001, 2100
    x = torch.randn(B, T, D, device="cuda")
    t = 1234
    cut, w = x[:, t].contiguous(), torch.randn(4, D, device="cuda")
    s1, s2 = torch.zeros(B, 3, D, device="cuda"), torch.zeros(B, 3, D, device="cuda")
    assert same(kda.kdn_conv_step(x[:, t], w, s1), kda.kdn_conv_step(cut, w, s2)) and same(s1, s2)
    r1, r2 = torch.ones(B, D, device="cuda"), torch.ones(B, D, device="cuda")
    assert same(kda.kdn_rec_step(x[:, t], x[:, t], r1), kda.kdn_rec_step(cut, cut, r2)) and same(r1, r2)
    assert same(kda.kdn_layer_norm_fwd(x[:, t])[0], kda.kdn_layer_norm_fwd(cut)[0])
    y, _ = kda.kdn_conv_fwd(x[:, t:t + 1], w)
    assert same(y[:, 0], kda.kdn_conv_step(cut, w, torch.zeros(B, 3, D, device="cuda")))
    with pytest.raises(kda.KdnError, match="x_stride is at most"):
        kda.kdn_rec_fwd(x[:, t:t + 1], x[:, t:t + 1])


# ---- values that must stay in their sequence -------------------------------------

@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_sequences_do_not_leak(bad):
    T, D, cu = 700, 40, [0, 130, 131, 400, 400, 700]
    g = torch.Generator(device="cuda").manual_seed(1)
    new = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, a, dy, w = new(1, T, D), new(1, T, D), new(1, T, D), new(4, D)
    h0, dT, s0, ds = new(5, D), new(5, D), new(5, 3, D), new(5, 3, D)
    c = offsets(cu)

    def calls(x, a, dy, h0, s0):
        y, st = kda.kdn_conv_fwd(x, w, state0=s0, cu_seqlens=c, activation="silu", want_state=True)
        gc = kda.kdn_conv_bwd(dy, x, w, state0=s0, cu_seqlens=c, activation="silu", dstate_T=ds)
        h, h_T, chk = kda.kdn_rec_fwd(x, a, h0=h0, cu_seqlens=c, want_checkpoints=True)
        gr = kda.kdn_rec_bwd(dy, x, a, chk, h0=h0, dh_T=dT, cu_seqlens=c)
        rows = [y[0], gc["dx"][0], h[0], gr["dx"][0], gr["da"][0]]
        return rows, [st, h_T, gc["dstate0"], gr["dh0"]]
    clean = calls(x, a, dy, h0, s0)
    spoiled = [t.clone() for t in (x, a, dy, h0, s0)]
    for t in spoiled[:3]:
        t[0, 131:400] = bad
    for t in spoiled[3:]:
        t[2] = bad
    rows, states = calls(*spoiled)
    for i, (r, q) in enumerate(zip(rows, clean[0])):
        assert same(r[:131], q[:131]) and same(r[400:], q[400:]), i
    for i, (r, q) in enumerate(zip(states, clean[1])):
        keep = [0, 1, 3, 4]
        assert same(r[keep], q[keep]), i


def test_padding_tokens_add_nothing():
    # tokens behind the last sequence hold NaN: no gradient takes them up
    T, D, cu = 300, 24, [0, 100, 210]
    x, dy, w = torch.randn(1, T, D, device="cuda"), torch.randn(1, T, D, device="cuda"), torch.randn(4, D, device="cuda")
    b = torch.randn(D, device="cuda")
    a = torch.randn(1, T, D, device="cuda")
    short = [t[:, :210].contiguous() for t in (x, dy, a)]
    for t in (x, dy, a):
        t[:, 210:] = float("nan")
    c = offsets(cu)
    g = kda.kdn_conv_bwd(dy, x, w, bias=b, cu_seqlens=c, activation="silu")
    assert torch.isfinite(g["dweight"]).all() and torch.isfinite(g["dbias"]).all()
    q = kda.kdn_conv_bwd(short[1], short[0], w, bias=b, cu_seqlens=c, activation="silu")
    assert torch.allclose(g["dweight"], q["dweight"], rtol=1e-4, atol=1e-4)
    _, h_T, chk = kda.kdn_rec_fwd(x, a, cu_seqlens=c, want_checkpoints=True)
    _, q_T, _ = kda.kdn_rec_fwd(short[0], short[2], cu_seqlens=c)
    assert torch.isfinite(h_T).all() and torch.allclose(h_T, q_T, rtol=1e-5, atol=1e-5)
    gr = kda.kdn_rec_bwd(dy, x, a, chk, cu_seqlens=c)
    assert torch.isfinite(gr["dx"][:, :210]).all() and torch.isfinite(gr["da"][:, :210]).all()


# ---- a block of them together ----------------------------------------------------

def test_block_forward_backward_and_decode():
    """norm -> conv (SiLU) -> recurrence -> norm per head, in fp32 against
    autograd in 64 bits, and the same tokens one at a time."""
    B, T, H, dv, W = 2, 150, 3, 32, 4
    D = H * dv
    g = torch.Generator().manual_seed(3)
    new = lambda *s: torch.randn(*s, generator=g)
    p = dict(x=new(B, T, D), w1=new(D), b1=new(D), wc=new(W, D) * 0.5, bc=new(D), a=new(B, T, D) + 1,
             w2=new(dv), b2=new(dv))
    dy = new(B, T, H, dv)
    q = {k: v.double().requires_grad_() for k, v in p.items()}
    n = torch.nn.functional.layer_norm(q["x"], (D,), q["w1"], q["b1"], 1e-5)
    wide = torch.nn.functional.pad(n, (0, 0, W - 1, 0))
    z = q["bc"] + sum(wide[:, j:j + T] * q["wc"][j] for j in range(W))
    u = z * torch.sigmoid(z)
    al = torch.sigmoid(q["a"])
    hs, h = [], torch.zeros(B, D, dtype=torch.float64)
    for t in range(T):
        h = al[:, t] * h + (1 - al[:, t]) * u[:, t]
        hs.append(h)
    y = torch.nn.functional.layer_norm(torch.stack(hs, 1).view(B, T, H, dv), (dv,), q["w2"], q["b2"], 1e-5)
    y.backward(dy.double())

    d = {k: v.cuda() for k, v in p.items()}
    n1, m1, r1 = kda.kdn_layer_norm_fwd(d["x"], d["w1"], d["b1"], want_stats=True)
    c, _ = kda.kdn_conv_fwd(n1, d["wc"], bias=d["bc"], activation="silu")
    hh, _, chk = kda.kdn_rec_fwd(c, d["a"], blend=True, want_checkpoints=True)
    out, m2, r2 = kda.kdn_layer_norm_fwd(hh.view(B, T, H, dv), d["w2"], d["b2"], want_stats=True)
    # errors of 1e-7 grow by the norms' 1 / spread (h's spread is above 0.05)
    assert (out.cpu().double() - y).abs().max() < 1e-4
    g2 = kda.kdn_layer_norm_bwd(dy.cuda(), hh.view(B, T, H, dv), m2, r2, d["w2"])
    gr = kda.kdn_rec_bwd(g2["dx"].view(B, T, D), c, d["a"], chk, blend=True)
    gc = kda.kdn_conv_bwd(gr["dx"], n1, d["wc"], bias=d["bc"], activation="silu")
    g1 = kda.kdn_layer_norm_bwd(gc["dx"], d["x"], m1, r1, d["w1"])
    for got, name in ((g1["dx"], "x"), (g1["dweight"], "w1"), (g1["dbias"], "b1"),
                      (gc["dweight"], "wc"), (gc["dbias"], "bc"), (gr["da"], "a"),
                      (g2["dweight"], "w2"), (g2["dbias"], "b2")):
        want = q[name].grad
        off = (got.cpu().double() - want).norm() / want.norm()
        assert off < 1e-5, (name, float(off))

    cs, rs = torch.zeros(B, W - 1, D, device="cuda"), torch.zeros(B, D, device="cuda")
    for t in range(T):
        s1, _, _ = kda.kdn_layer_norm_fwd(d["x"][:, t].contiguous(), d["w1"], d["b1"])
        s2 = kda.kdn_conv_step(s1, d["wc"], cs, bias=d["bc"], activation="silu")
        s3 = kda.kdn_rec_step(s2, d["a"][:, t], rs, blend=True)
        s4, _, _ = kda.kdn_layer_norm_fwd(s3.view(B, H, dv), d["w2"], d["b2"])
        assert (s4.cpu().double() - y[:, t]).abs().max() < 1e-4, t


def test_conv_and_norm_around_the_mixer():
    """x -> norm -> one convolution over a fused q, k, v -> the KDN forward ->
    norm per head, whole and as a prefix continued from its states."""
    B, T, H, dk, W = 1, 96, 2, 64, 4
    D, f = H * dk, torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(9)
    new = lambda *s: torch.randn(*s, generator=g, device="cuda")
    qkv = new(B, T, 3 * D).to(f)
    w, b = new(W, 3 * D) * 0.5, new(3 * D) * 0.1
    alpha = torch.sigmoid(new(B, T, H, dk) + 2)
    omega, r = torch.nn.functional.softplus(new(B, T, H, dk)), torch.nn.functional.softplus(new(B, T, H)) + 0.1

    def run(t0, t1, conv=None, S=None, p=None):
        y, st = kda.kdn_conv_fwd(qkv[:, t0:t1], w, bias=b, state0=conv, activation="silu", want_state=True)
        heads = [y[..., i * D:(i + 1) * D].reshape(B, t1 - t0, H, dk).contiguous() for i in range(3)]
        q, k = (torch.nn.functional.normalize(h.float(), dim=-1).to(f) for h in heads[:2])
        cut = lambda z: z[:, t0:t1].contiguous()
        o, S, p = kda.kdn_diag_fwd(q, k, heads[2], cut(alpha), cut(omega), cut(r), S0=S, p0=p)
        return kda.kdn_layer_norm_fwd(o)[0], st, S, p
    whole, st, S, p = run(0, T)
    first, st1, S1, p1 = run(0, 64)
    second, st2, S2, p2 = run(64, T, st1, S1, p1)
    assert same(st, st2)
    assert torch.isfinite(whole).all()
    # the mixer's own chunks start elsewhere: its results agree to its rounding
    both = torch.cat((first, second), 1).float()
    assert (both - whole.float()).norm() / whole.float().norm() < 2e-2


# ---- streams, graphs, workspaces, far offsets ----------------------------------------

def all_calls(seed, T=700, D=96, io=torch.bfloat16):
    """Every operator once on inputs of a seed; returns run() and its buffers."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda *s, dtype=io: torch.randn(*s, generator=g, device="cuda").to(dtype)
    f32 = torch.float32
    x, a, dy = new(2, T, D), new(2, T, D), new(2, T, D)
    w, b, wc = new(D, dtype=f32), new(D, dtype=f32), new(4, D, dtype=f32)
    h0, dT, s0 = new(2, D, dtype=f32), new(2, D, dtype=f32), new(2, 3, D)
    sx, sa = new(7, D), new(7, D)
    cs, rs = new(7, 3, D), new(7, D, dtype=f32)

    def run():
        y, m, r = kda.kdn_layer_norm_fwd(x, w, b, want_stats=True)
        gn = kda.kdn_layer_norm_bwd(dy, x, m, r, w)
        c, st = kda.kdn_conv_fwd(x, wc, bias=b, state0=s0, activation="silu", want_state=True)
        gc = kda.kdn_conv_bwd(dy, x, wc, bias=b, state0=s0, activation="silu")
        h, h_T, chk = kda.kdn_rec_fwd(x, a, h0=h0, blend=True, want_checkpoints=True)
        gr = kda.kdn_rec_bwd(dy, x, a, chk, h0=h0, dh_T=dT, blend=True)
        cs1, rs1 = cs.clone(), rs.clone()
        z = kda.kdn_conv_step(sx, wc, cs1, bias=b)
        hs = kda.kdn_rec_step(sx, sa, rs1)
        return [y, m, r, c, st, h, h_T, chk, z, hs, cs1, rs1] + [
            g[k] for g in (gn, gc, gr) for k in sorted(g)]
    return run, (x, a, dy, sx, sa)


@pytest.mark.parametrize("T", [1, 100, 3000])
def test_captured_and_replayed(T):
    run, inputs = all_calls(11, T)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    for k in range(4):
        for t in inputs:
            t.mul_(-1.0 if k % 2 else 0.5)
        want = run()
        torch.cuda.synchronize()
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for i, (o, q) in enumerate(zip(outs, want)):
            assert same(o, q), (k, i)


def test_two_streams_at_once():
    runs = [all_calls(s, 2500)[0] for s in (21, 22)]
    want = [r() for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    got = [None, None]
    for _ in range(3):
        for i, (r, s) in enumerate(zip(runs, streams)):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got[i] = r()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(same(p, q) for p, q in zip(a, b))


def test_runs_are_identical_and_workspaces_carry_nothing():
    run, _ = all_calls(31, 3000)
    first = run()
    for _ in range(3):
        assert all(same(a, b) for a, b in zip(first, run()))
    # a workspace full of NaN, and one that a call of another shape used
    x, a = torch.randn(1, 4000, 70, device="cuda"), torch.randn(1, 4000, 70, device="cuda")
    L = kda.api._lib.lib()
    n = max(L.kdn_rec_fwd_workspace_size(1, 4000, 70), L.kdn_rec_bwd_workspace_size(1, 4000, 70))
    ws = torch.full((n + 64,), 255, dtype=torch.uint8, device="cuda")
    h, h_T, chk = kda.kdn_rec_fwd(x, a, want_checkpoints=True)
    for fill in (255, 0, None):
        if fill is not None:
            ws.fill_(fill)
        h2, h2_T, _ = kda.kdn_rec_fwd(x, a, workspace=ws)
        assert same(h, h2) and same(h_T, h2_T)
        g = kda.kdn_rec_bwd(x, x, a, chk, workspace=ws)
        q = kda.kdn_rec_bwd(x, x, a, chk)
        assert all(same(g[k], q[k]) for k in q)


def test_offsets_beyond_32_bits():
    """Tensors of 5.4 GB each: the last channels, and the last rows, against a
    small call on the same values."""
    T, D = 65600, 20480
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty(1, T, D, device="cuda").normal_(generator=g)
    a = torch.empty(1, T, D, device="cuda").normal_(generator=g).add_(1)
    assert x.numel() * 4 > 1 << 32
    cols = slice(D - 64, D)
    xs, as_ = x[..., cols].contiguous(), a[..., cols].contiguous()
    h, h_T, chk = kda.kdn_rec_fwd(x, a, want_checkpoints=True)
    q, q_T, qchk = kda.kdn_rec_fwd(xs, as_, want_checkpoints=True)
    # few channels go in longer tiles, so the spans are joined in another order:
    # each side is within e_t = alpha e_{t-1} + c U m_t, m_t = alpha m_{t-1} + |x_t|,
    # c = 2 |a| + 6 for the decay and 3 roundings (block_reference.rec); both
    # recurrences are the call's own, on values that are not negative
    c = (2 * as_.abs().max().item() + 9) * 2.0 ** -24
    m, m_T, _ = kda.kdn_rec_fwd(xs.abs(), as_)
    e, e_T, _ = kda.kdn_rec_fwd(c * m, as_)
    assert ((h[..., cols] - q).abs() <= 2.02 * e).all() and ((h_T[:, cols] - q_T).abs() <= 2.02 * e_T).all()
    assert ((chk[:, 1:, cols] - qchk[:, 1:]).abs() <= 2.02 * e[:, 63:-1:64]).all()
    del h
    gr, qr = kda.kdn_rec_bwd(x, x, a, chk), kda.kdn_rec_bwd(xs, xs, as_, qchk)
    ml = kda.kdn_rec_bwd(xs.abs(), xs, as_, qchk)["dx"]
    el = kda.kdn_rec_bwd(c * ml, xs, as_, qchk)["dx"]
    assert ((gr["dx"][..., cols] - qr["dx"]).abs() <= 2.02 * el).all()
    # da = lam h_{t-1} alpha (1 - alpha): both factors' errors, and the slope's
    prev, ep, mp = (torch.nn.functional.pad(t, (0, 0, 1, 0))[:, :-1] for t in (q.abs(), e, m))
    al = torch.sigmoid(as_)
    ed = al * (1 - al) * (el * prev + qr["dx"].abs() * ep) + 2 * c * qr["da"].abs()
    assert ((gr["da"][..., cols] - qr["da"]).abs() <= 2.02 * ed).all()
    del gr, a
    w = torch.randn(4, D, device="cuda")
    y, _ = kda.kdn_conv_fwd(x, w, activation="silu")
    z, _ = kda.kdn_conv_fwd(xs, w[:, cols].contiguous(), activation="silu")
    assert torch.equal(y[..., cols], z)
    gc = kda.kdn_conv_bwd(y, x, w, activation="silu")
    qc = kda.kdn_conv_bwd(z, xs, w[:, cols].contiguous(), activation="silu")
    assert torch.equal(gc["dx"][..., cols], qc["dx"])
    del gc, y
    n, m, r = kda.kdn_layer_norm_fwd(x, want_stats=True)
    last, _, _ = kda.kdn_layer_norm_fwd(x[:, -3:].contiguous())
    assert torch.equal(n[:, -3:], last)
    gn = kda.kdn_layer_norm_bwd(n, x, m, r)
    qn = kda.kdn_layer_norm_bwd(last, x[:, -3:].contiguous(), m[:, -3:].contiguous(), r[:, -3:].contiguous())
    assert torch.equal(gn["dx"][:, -3:], qn["dx"])


def in_thirds(B, calls):
    """The whole call gives what a third of the rows gives: the same bits, since the
    thirds are cut into the same tiles."""
    whole = calls(slice(0, B))
    for k in range(0, B, B // 3):
        p = slice(k, k + B // 3)
        for i, (v, t) in enumerate(zip(whole, calls(p))):
            assert torch.equal(v[p], t), (i, k)


@pytest.mark.parametrize("io,gate,T", [("bf16", "preact", 1900), ("bf16", "alpha", 1500), ("f32", "preact", 950),
                                       ("f32", "alpha", 950)])
def test_rec_larger_than_the_last_level_cache(io, gate, T):
    B, D = 18, 2050
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(5)
    x, dy = (torch.empty(B, T, D, device="cuda").normal_(generator=g).to(dt) for _ in range(2))
    a = torch.empty(B, T, D, device="cuda").normal_(generator=g).add_(2)
    a = torch.sigmoid(a) if gate == "alpha" else a.to(dt)
    h0, dh_T = (torch.empty(B, D, device="cuda").normal_(generator=g) for _ in range(2))
    assert x.numel() * (2 * x.element_size() + a.element_size()) > 256 << 20

    def calls(p):
        h, h_T, chk = kda.kdn_rec_fwd(x[p], a[p], h0=h0[p], gate=gate, blend=True, want_checkpoints=True)
        r = kda.kdn_rec_bwd(dy[p], x[p], a[p], chk, h0=h0[p], dh_T=dh_T[p], gate=gate, blend=True)
        return [h, h_T, chk, r["dx"], r["da"], r["dh0"]]
    in_thirds(B, calls)


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("io,T", [("bf16", 3650), ("f32", 1825)])
def test_conv_larger_than_the_last_level_cache(io, T, W):
    B, D = 18, 2050
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(6)
    x, dy = (torch.empty(B, T, D, device="cuda").normal_(generator=g).to(dt) for _ in range(2))
    w, b = torch.randn(W, D, device="cuda"), torch.randn(D, device="cuda")
    s0 = torch.randn(B, W - 1, D, device="cuda").to(dt)
    assert x.numel() * x.element_size() > 256 << 20

    def calls(p):
        kw = dict(bias=b, state0=s0[p], activation="silu")
        y, s_T = kda.kdn_conv_fwd(x[p], w, want_state=True, **kw)
        c = kda.kdn_conv_bwd(dy[p], x[p], w, **kw)
        return [y, s_T, c["dx"], c["dstate0"]]
    in_thirds(B, calls)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [60, 128, 250, 500, 1000, 2050, 6144, 8200, 16384])
def test_layer_norm_larger_than_the_last_level_cache(D, io):
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    rows = ((256 << 20) // (D * dt.itemsize) // 3 + 1) * 3
    g = torch.Generator(device="cuda").manual_seed(7)
    x, dy = (torch.empty(rows, D, device="cuda").normal_(generator=g).to(dt) for _ in range(2))
    w, b = torch.randn(D, device="cuda"), torch.randn(D, device="cuda")
    assert x.numel() * x.element_size() >= 256 << 20

    def calls(p):
        y, m, r = kda.kdn_layer_norm_fwd(x[p], w, b, want_stats=True)
        return [y, m, r, kda.kdn_layer_norm_bwd(dy[p], x[p], m, r, w)["dx"]]
    in_thirds(rows, calls)
