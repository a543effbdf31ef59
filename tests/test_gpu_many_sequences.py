"""Many packed sequences, more than a workgroup has threads many times over, most of
them empty or all of them: values against the 64-bit references, and the time that a
call takes with them against the time without."""
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


def cuts(T, N, seed, end=None):
    """N sequences in T tokens: random borders, many of them equal."""
    end = T if end is None else end
    inner = np.sort(np.random.default_rng(seed).integers(0, end + 1, N - 1))
    return [0] + inner.tolist() + [end]


def crowd(T, N, at):
    """All but two sequences empty, at one token."""
    return [0] + [at] * (N - 1) + [T]


# (around 20 a run: 4 to 32 runs of the convolution, 8 and 16 of the recurrence)
CASES = [(1000, 6, cuts(1000, n, n)) for n in (80, 81, 160, 161, 320, 321, 640, 641)]
CASES += [(1500, 300, cuts(1500, 81, 3)), (1500, 300, cuts(1500, 321, 4)),
          (5000, 6, cuts(5000, 4500, 5)), (5000, 6, cuts(5000, 9000, 6, 4990)), (300, 3, cuts(300, 20000, 7)),
          (700, 5, crowd(700, 5000, 300)), (700, 5, crowd(700, 5000, 0)), (700, 5, crowd(700, 5000, 700)),
          (1, 2, cuts(1, 3000, 8)), (0, 4, [0] * 3001), (40, 4, [0] * 5001), (2600, 1, cuts(2600, 2500, 9))]
IDS = ["T%dD%dN%d-%d" % (t, d, len(c) - 1, i) for i, (t, d, c) in enumerate(CASES)]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("T,D,cu", CASES, ids=IDS)
def test_values(T, D, cu, given, io):
    N, W, end = len(cu) - 1, 4, cu[-1]
    rng = np.random.default_rng(N)
    (x, xr), (dy, dyr), (a, ar) = (dev(rng.standard_normal((1, T, D)), io) for _ in range(3))
    w, wr = dev(rng.standard_normal((W, D)))
    (s0, s0r), (ds, dsr) = (dev(rng.standard_normal((N, W - 1, D)), io) for _ in range(2))
    (h0, h0r), (dT, dTr) = (dev(rng.standard_normal((N, D))) for _ in range(2))
    if not given:
        s0 = s0r = ds = dsr = h0 = h0r = dT = dTr = None
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    part = lambda v: tuple(q[:, :end] for q in v)

    ref = R.conv(xr, wr, None, s0r, cu, True, dyr, dsr)
    kw = dict(state0=s0, cu_seqlens=c, activation="silu")
    nan = torch.full((N, W - 1, D), float("nan"), dtype=DT[io], device="cuda")
    y, state = kda.kdn_conv_fwd(x, w, state_T=nan, **kw)
    R.check(host(y)[:, :end], part(ref["y"]), io, "y")
    assert np.array_equal(host(state), ref["state_T"][0])
    g = kda.kdn_conv_bwd(dy, x, w, dstate_T=ds, **kw)
    R.check(host(g["dx"])[:, :end], part(ref["dx"]), io, "conv dx")
    R.check(host(g["dweight"]), ref["dweight"], "f32", "dweight")
    if given:
        R.check(host(g["dstate0"]), ref["dstate0"], io, "dstate0")

    ref = R.rec(xr, ar, h0r, cu, True, True, dyr, dTr)
    kw = dict(h0=h0, cu_seqlens=c, blend=True)
    h, h_T, chk = kda.kdn_rec_fwd(x, a, want_checkpoints=True, h_T=nan.float()[:, 0].contiguous(), **kw)
    R.check(host(h)[:, :end], part(ref["h"]), io, "h")
    R.check(host(h_T), ref["h_T"], "f32", "h_T")
    g = kda.kdn_rec_bwd(dy, x, a, chk, dh_T=dT, **kw)
    R.check(host(g["dx"])[:, :end], part(ref["dx"]), io, "rec dx")
    R.check(host(g["da"])[:, :end], part(ref["da"]), io, "da")
    R.check(host(g["dh0"]), ref["dh0"], "f32", "dh0")


def test_rows_without_tokens():
    # not packed: every row is an empty sequence
    for B in (3, 100, 5000):
        x, w = torch.empty(B, 0, 20, device="cuda"), torch.ones(3, 20, device="cuda")
        s0, h0 = torch.randn(B, 2, 20, device="cuda"), torch.randn(B, 20, device="cuda")
        assert torch.equal(kda.kdn_conv_fwd(x, w, state0=s0, want_state=True)[1], s0)
        g = kda.kdn_conv_bwd(x, x, w, state0=s0, dstate_T=s0 + 1)
        assert torch.equal(g["dstate0"], s0 + 1) and (g["dweight"] == 0).all()
        _, h_T, chk = kda.kdn_rec_fwd(x, x, h0=h0, want_checkpoints=True)
        assert torch.equal(h_T, h0)
        assert torch.equal(kda.kdn_rec_bwd(x, x, x, chk, h0=h0, dh_T=h0 + 1)["dh0"], h0 + 1)


def timed(f):
    """Milliseconds of a call, the best of a few."""
    for _ in range(2):
        f()
    best = float("inf")
    for _ in range(5):
        e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        e[0].record()
        for _ in range(4):
            f()
        e[1].record()
        torch.cuda.synchronize()
        best = min(best, e[0].elapsed_time(e[1]) / 4)
    return best


def calls(T, D, N, states):
    g = torch.Generator(device="cuda").manual_seed(1)
    new = lambda *s, dtype=torch.bfloat16: torch.randn(*s, generator=g, device="cuda").to(dtype)
    x, a, dy, w = new(1, T, D), new(1, T, D), new(1, T, D), new(4, D, dtype=torch.float32)
    c = torch.tensor(cuts(T, N, 1), dtype=torch.int32, device="cuda")
    s0, h0 = (new(N, 3, D), new(N, D, dtype=torch.float32)) if states else (None, None)
    chk = kda.kdn_rec_fwd(x, a, h0=h0, cu_seqlens=c, want_checkpoints=True)[2]
    return {"conv forward": lambda: kda.kdn_conv_fwd(x, w, state0=s0, cu_seqlens=c, want_state=states),
            "conv backward": lambda: kda.kdn_conv_bwd(dy, x, w, state0=s0, cu_seqlens=c),
            "rec forward": lambda: kda.kdn_rec_fwd(x, a, h0=h0, cu_seqlens=c),
            "rec backward": lambda: kda.kdn_rec_bwd(dy, x, a, chk, h0=h0, cu_seqlens=c)}


def test_borders_of_many_sequences_take_little_time():
    """A workgroup finds the borders in its tile without a look at every offset: of 2^20
    sequences without states in 65536 tokens of 512 channels.  Measured 2 times (looking
    at every offset, 230 times)."""
    many, one = calls(65536, 512, 1 << 20, False), calls(65536, 512, 2, False)
    for k in ("conv forward", "conv backward"):
        t, t1 = timed(many[k]), timed(one[k])
        print("%s: %.3f ms, with two sequences %.3f ms" % (k, t, t1))
        assert t < 20 * t1, (k, t, t1)


def test_states_of_many_sequences_take_little_time():
    """65536 sequences in as many tokens, 512 channels: their states are as many bytes as x
    four times over, and no run of the first tile may go through them one by one (100 times
    the time of the call with one sequence, and more).  Measured 2 to 7 times."""
    many, one = calls(65536, 512, 65536, True), calls(65536, 512, 2, True)
    for k in many:
        t, t1 = timed(many[k]), timed(one[k])
        print("%s: %.3f ms, with two sequences %.3f ms" % (k, t, t1))
        assert t < 20 * t1, (k, t, t1)
