"""Infinities and NaN in the gated recurrence: they stay in their sequence to its
end, as the definition has it, however far the decays shrink and wherever the tiles
and runs lie, and they enter no other sequence.  Against the 64-bit reference, whose
NaN and infinities have to be at the same places."""
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
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DT[io])
    return t.cuda(), t.double().numpy()


def check(got, ref, io, name):
    if np.isfinite(ref[0]).any():
        R.check(got, ref, io, name)
    else:
        assert np.array_equal(got, ref[0], equal_nan=True), name


def spoil(rng, a, axis_tokens, bad):
    """A third of the channels get one bad value, each at a token of its own."""
    B, T, D = a.shape
    for b in range(B):
        for c in rng.choice(D, max(D // 3, 1), replace=False):
            a[b, axis_tokens(rng), c] = bad


# one row in tiles of 256 and (64 rows) of 128 tokens; packed sequences with borders in
# and around runs, empty ones among them
CASES = [(1, 2000, 70, None), (64, 140, 130, None), (2, 700, 66, None), (1, 300, 1, None),
         (1, 2600, 40, [0, 3, 900, 900, 901, 2500, 2600]), (1, 700, 40, [0, 130, 131, 400, 400, 650]),
         (1, 17000, 6, None)]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("gate,blend", [("preact", True), ("preact", False), ("alpha", True), ("alpha", False)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "B%dT%dD%d%s" % (c[:3] + ("" if c[3] is None else "N",)))
def test_bad_values_stay_to_the_end(case, bad, gate, blend, io):
    B, T, D, cu = case
    N = B if cu is None else len(cu) - 1
    end = T if cu is None else cu[-1]
    rng = np.random.default_rng(T + D)
    preact = gate == "preact"
    token = lambda r: r.integers(0, end)
    x, dh = rng.standard_normal((B, T, D)), rng.standard_normal((B, T, D))
    h0, dT = rng.standard_normal((N, D)), rng.standard_normal((N, D))
    spoil(rng, x, token, bad)
    spoil(rng, dh, token, bad)
    h0[rng.integers(0, N), ::5] = bad
    dT[rng.integers(0, N), 1::5] = bad
    # decays about 0.4: over 256 tokens their product is far below the smallest number
    # (in some channels about 2^-10: below it within 16 tokens)
    a = rng.standard_normal((B, T, D)) - 0.4
    a[..., 2::7] -= 6.5
    if not preact:
        a = R.sigmoid(a)
        for c in range(0, D, 4):  # and zeros, at a token of a channel's own
            a[:, token(rng), c] = 0.0
            a[:, token(rng), c] = -0.0
    (x, xr), (dh, dhr), (a, ar) = dev(x, io), dev(dh, io), dev(a, io if preact else "f32")
    (h0, h0r), (dT, dTr) = dev(h0), dev(dT)
    with np.errstate(invalid="ignore", over="ignore"):
        ref = R.rec(xr, ar, h0r, cu, preact, blend, dhr, dTr)
    kw = dict(h0=h0, cu_seqlens=None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda"),
              gate=gate, blend=blend)
    h, h_T, chk = kda.kdn_rec_fwd(x, a, want_checkpoints=True, **kw)
    g = kda.kdn_rec_bwd(dh, x, a, chk, dh_T=dT, **kw)
    part = lambda v: tuple(q[:, :end] for q in v)
    with np.errstate(invalid="ignore", over="ignore"):
        check(host(h)[:, :end], part(ref["h"]), io, "h")
        check(host(h_T), ref["h_T"], "f32", "h_T")
        k = -(-end // 64)
        check(host(chk)[:, :k], tuple(q[:, :k] for q in ref["checkpoints"]), "f32", "checkpoints")
        check(host(g["dx"])[:, :end], part(ref["dx"]), io, "dx")
        check(host(g["dh0"]), ref["dh0"], "f32", "dh0")
        # (the order of da's factors is free: an infinite one times one that is zero
        # in fp32 or infinite may be NaN for one order only)
        fine = np.isfinite(ref["da"][0][:, :end])
        got = host(g["da"])[:, :end]
        assert np.isfinite(got[fine]).all() and not np.isfinite(got[~fine]).any()


@pytest.mark.parametrize("T,D", [(2000, 70), (300, 1)])
def test_negative_decays_keep_their_sign(T, D):
    """A decay given below zero is outside what the call promises, and is computed all the
    same; its errors are at most those of its magnitude."""
    rng = np.random.default_rng(7)
    (x, xr), (dh, dhr) = (dev(rng.standard_normal((1, T, D))) for _ in range(2))
    a, ar = dev(rng.uniform(-1, 1, (1, T, D)))
    ref = R.rec(xr, ar, None, None, False, False, dhr)
    size = R.rec(np.abs(xr), np.abs(ar), None, None, False, False, np.abs(dhr))
    h, h_T, chk = kda.kdn_rec_fwd(x, a, gate="alpha", want_checkpoints=True)
    g = kda.kdn_rec_bwd(dh, x, a, chk, gate="alpha")
    for got, k in ((h, "h"), (h_T, "h_T"), (g["dx"], "dx"), (g["da"], "da"), (g["dh0"], "dh0")):
        check(host(got), (ref[k][0], size[k][1]), "f32", k)
