"""Linear attention with a decay for each head on the GPU against its 64-bit
reference (linattn_reference's bounds, value by value): head sizes, shared keys,
one token to several segments, packed sequences, strides, exact whole numbers,
what is not finite, single tokens, graphs, streams, refusals."""
import numpy as np
import pytest
import torch

import block_reference as BR
import kalman_delta_rule_amd as kda
import linattn_reference as R
from test_gpu_block import DT, dev, host, offsets, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a HIP GPU")


def data(B, T, H, Hk, dk, dv, io, seed, cu=None, state=True):
    rng = np.random.default_rng(seed)
    n = lambda *s: rng.standard_normal(s)
    N = B if cu is None else len(cu) - 1
    d = {"q": dev(n(B, T, Hk, dk), io), "k": dev(n(B, T, Hk, dk), io), "v": dev(n(B, T, H, dv), io),
         "do": dev(n(B, T, H, dv), io), "g": dev(1 - 2.0 ** -rng.uniform(0.5, 9, H))}
    if state:
        d.update(S0=dev(n(N, H, dk, dv)), dS=dev(n(N, H, dk, dv)))
    return d


def forward(d, scale=None, cu=None, **kw):
    S0 = d["S0"][0] if "S0" in d else None
    return kda.kdn_linattn_fwd(d["q"][0], d["k"][0], d["v"][0], d["g"][0], scale=scale, S0=S0,
                               cu_seqlens=offsets(cu), want_state=True, **kw)


def backward(d, scale=None, cu=None, **kw):
    S0, dS = (d[n][0] if n in d else None for n in ("S0", "dS"))
    return kda.kdn_linattn_bwd(d["do"][0], d["q"][0], d["k"][0], d["v"][0], d["g"][0], scale=scale,
                               S0=S0, dS_T=dS, cu_seqlens=offsets(cu), **kw)


# relative 2-norms: three roundings of independent terms for values in bf16 (2^-8 each at
# most), 2^-16 for states of bf16 terms, some tens of roundings for fp32
NORM = {"bf16": 2.0 ** -7, "f32": 2.0 ** -18}


def close(got, ref, io, name, state=False, cu=None):
    got, (value, bound) = host(got), ref
    BR.check(got, ref, "f32" if state else io, name)
    if np.linalg.norm(value):
        off = np.linalg.norm(got - value) / np.linalg.norm(value)
        assert off <= (2.0 ** -16 if state and io == "bf16" else NORM[io]), (name, off)


def both(d, io, scale, cu=None):
    """The calls and their references."""
    S0, dS = (d[n][1] if n in d else None for n in ("S0", "dS"))
    s = d["q"][1].shape[-1] ** -0.5 if scale is None else scale
    o, S_T = forward(d, scale, cu)
    ref = R.forward(d["q"][1], d["k"][1], d["v"][1], d["g"][1], s, S0, cu, io)
    close(o, ref["o"], io, "o")
    close(S_T, ref["S_T"], io, "S_T", True)
    g = backward(d, scale, cu)
    ref = R.backward(d["do"][1], d["q"][1], d["k"][1], d["v"][1], d["g"][1], s, S0, dS, cu, io)
    for n in ("dq", "dk", "dv"):
        close(g[n], ref[n], io, n)
    assert ("dS0" in g) == (S0 is not None)
    if S0 is not None:
        close(g["dS0"], ref["dS0"], io, "dS0", True)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(1, 1), (8, 64), (16, 5), (33, 31), (64, 64), (63, 65), (72, 101), (128, 64),
                                   (128, 128), (100, 200), (256, 32), (255, 129), (256, 256)])
def test_head_sizes(dk, dv, io):
    both(data(2, 83, 2, 1, dk, dv, io, dk * 7 + dv), io, None)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T", [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 128, 130, 1000])
def test_lengths(T, io):
    both(data(1, T, 3, 3, 48, 40, io, T, state=T % 2 == 0), io, 0.3)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1024, 1500, 4099])
def test_segments(T, io):
    # few heads: the walk is split over time
    L = kda._lib.lib()
    assert L.kdn_linattn_fwd_workspace_size(1, T, 2, 16, 16) > 0
    both(data(1, T, 2, 2, 16, 16, io, T), io, None)


CUTS = {"mixed": (150, [0, 1, 1, 64, 65, 130, 150]), "tail": (100, [0, 30, 70]), "empty": (9, [0, 0, 0, 9, 9]),
        "none": (40, [0, 0]), "one": (70, [0, 70]), "all empty": (5, [0, 0, 0, 0]),
        "segments": (2100, [0, 3, 600, 600, 1031, 1100, 2048]), "long": (3000, [0, 2999]),
        "borders": (2048, [0, 512, 1024, 1024, 1088, 1536, 2048]),
        "many": (1300, [0] + sorted(np.random.default_rng(8).integers(0, 1300, 700).tolist()))}


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("name", CUTS)
def test_packed(name, io):
    T, cu = CUTS[name]
    d = data(1, T, 2, 1, 24, 20, io, T, cu)
    both(d, io, None, cu)
    # rows behind the last sequence: zeros of new tensors, a caller's as they were
    end = cu[-1]
    o, _ = forward(d, None, cu)
    assert (o[:, end:] == 0).all()
    mine = torch.full_like(o, 7.0)
    forward(d, None, cu, o=mine)
    assert (mine[:, end:] == 7).all() and same(mine[:, :end], o[:, :end])
    g = backward(d, None, cu)
    for G in (1, 2):
        given = {n: torch.full_like(g[n], 7.0) for n in ("dq", "dk", "dv")}
        backward(d, None, cu, **given)
        for n, t in given.items():
            assert (g[n][:, end:] == 0).all() and (t[:, end:] == 7).all() and same(t[:, :end], g[n][:, :end])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T,N,tail,H", [(90, 30, 0, 6), (41, 269, 0, 2), (700, 40, 13, 2), (1700, 23, 5, 1), (64, 64, 0, 40),
                                        (5, 1, 2, 1)])
def test_many_short_sequences(T, N, tail, H, io):
    # several workgroups share a segment's sequences: cuts anywhere, empty ones, long ones
    rng = np.random.default_rng(T + N)
    cu = [0] + sorted(rng.integers(0, T - tail + 1, N - 1).tolist()) + [T - tail]
    both(data(1, T, H, H, 49, 32, io, seed=T, cu=cu), io, None, cu)
    one_by_one = list(range(T - tail + 1))
    both(data(1, T, 1, 1, 16, 70, io, seed=N, cu=one_by_one), io, None, one_by_one)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hk", [(4, 4), (4, 2), (6, 2), (8, 1)])
def test_shared_keys(H, Hk, io):
    both(data(2, 70, H, Hk, 32, 48, io, H + Hk), io, None)


def whole_numbers(B, T, H, Hk, dk, dv, io, seed, cu=None, spread=1):
    """Values of -1, 0, 1, few of them: with decays of one and none every sum is a
    whole number that bf16 holds (at most 256), so results are exact to the last
    rounding."""
    rng = np.random.default_rng(seed)
    n = lambda *s: rng.integers(-1, 2, s) * (rng.random(s) < spread)
    N = B if cu is None else len(cu) - 1
    d = {"q": dev(n(B, T, Hk, dk), io), "k": dev(n(B, T, Hk, dk), io), "v": dev(n(B, T, H, dv), io),
         "do": dev(n(B, T, H, dv), io), "g": dev(np.arange(H) % 2 * 1.0), "S0": dev(n(N, H, dk, dv)),
         "dS": dev(n(N, H, dk, dv))}
    return d


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,H,Hk,dk,dv,cu", [
    (2, 100, 4, 2, 64, 64, None), (1, 2100, 2, 2, 64, 64, None), (1, 3000, 2, 1, 40, 24, [0, 5, 700, 700, 2900]),
    (3, 333, 2, 2, 128, 96, None), (1, 1500, 2, 2, 256, 256, None)])
def test_whole_numbers_are_exact(B, T, H, Hk, dk, dv, cu, io):
    d = whole_numbers(B, T, H, Hk, dk, dv, io, T, cu, 0.5)
    S0, dS = d["S0"][1], d["dS"][1]
    ref = R.forward(d["q"][1], d["k"][1], d["v"][1], d["g"][1], 0.5, S0, cu, io)
    ref.update(R.backward(d["do"][1], d["q"][1], d["k"][1], d["v"][1], d["g"][1], 0.5, S0, dS, cu, io))
    assert np.abs(ref["S_T"][0]).max() <= 256 and np.abs(ref["dS0"][0]).max() <= 128  # halves
    o, S_T = forward(d, 0.5, cu)
    got = dict(backward(d, 0.5, cu), o=o, S_T=S_T)
    for n, t in got.items():
        want = torch.from_numpy(ref[n][0]).to(t.dtype)
        assert torch.equal(t.cpu(), want), n


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_slices_of_wider_rows(io):
    B, T, H, Hk, dk, dv = 2, 90, 4, 2, 40, 24
    d = data(B, T, H, Hk, dk, dv, io, 4)
    o, S_T = forward(d)
    g = backward(d)
    wide = torch.full((B, T, 3 + H * (dv + 5) + 2 * Hk * dk), float("nan"), dtype=DT[io], device="cuda")
    q = wide[..., 3:3 + Hk * dk].unflatten(-1, (Hk, dk))
    k = wide[..., 3 + Hk * dk:3 + 2 * Hk * dk].unflatten(-1, (Hk, dk))
    v = wide[..., 3 + 2 * Hk * dk:].unflatten(-1, (H, dv + 5))[..., 2:2 + dv]
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        t.copy_(d[n][0])
    e = dict(d, q=(q,), k=(k,), v=(v,))
    o2, S2 = forward(e)
    assert same(o, o2) and same(S_T, S2)
    h = backward(e)
    assert all(same(g[n], h[n]) for n in g)
    # the tokens of a row may be part of a longer one; rows may not then be several
    with pytest.raises(ValueError, match="evenly spaced"):
        kda.kdn_linattn_fwd(q[:, 1:], k[:, 1:], v[:, 1:], d["g"][0])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,Hk,dk,dv", [(1, 1, 1, 1, 1), (3, 4, 2, 33, 5), (2, 2, 2, 128, 128), (70, 3, 3, 64, 96),
                                          (2, 2, 1, 256, 255)])
def test_steps_are_the_forward(B, H, Hk, dk, dv, io):
    T = 5
    d = data(B, T, H, Hk, dk, dv, io, B + dk)
    ref = R.forward(d["q"][1], d["k"][1], d["v"][1], d["g"][1], dk ** -0.5, d["S0"][1], None, "f32")
    state = d["S0"][0].clone()
    out = [kda.kdn_linattn_step(d["q"][0][:, t], d["k"][0][:, t], d["v"][0][:, t], d["g"][0], state) for t in range(T)]
    BR.check(host(torch.stack(out, 1)), ref["o"], io, "o")
    BR.check(host(state), ref["S_T"], "f32", "state")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_what_is_not_finite_reaches_no_earlier_token(io, bad):
    B, T, H, dk, dv, at = 2, 200, 2, 32, 40, 85
    d = data(B, T, H, H, dk, dv, io, 6)
    o, S_T = forward(d)
    g = backward(d)
    for name, spoils in (("v", "column"), ("k", "later"), ("q", "token")):
        e = dict(d)
        t = d[name][0].clone()
        t[0, at, 1, 3] = bad
        e[name] = (t,)
        o2, S2 = forward(e)
        assert same(o2[1], o[1]) and same(o2[:, :, 0], o[:, :, 0]) and same(o2[0, :at], o[0, :at])
        assert same(S2[1], S_T[1]) and same(S2[:, 0], S_T[:, 0])
        if spoils == "column":
            clean = [c for c in range(dv) if c != 3]
            assert torch.equal(o2[0, :, 1, clean], o[0, :, 1, clean]) and not torch.isfinite(o2[0, at:, 1, 3]).any()
            assert not torch.isfinite(S2[0, 1, :, 3]).any() and torch.isfinite(S2[0, 1, :, clean]).all()
        elif spoils == "later":
            assert not torch.isfinite(o2[0, at:, 1]).any()
            assert not torch.isfinite(S2[0, 1, 3]).any() and same(S2[0, 1, 4:], S_T[0, 1, 4:])
        else:
            assert not torch.isfinite(o2[0, at, 1]).any() and same(o2[0, at + 1:], o[0, at + 1:]) and same(S2, S_T)
        h = backward(e)
        for n in h:
            assert same(h[n][1], g[n][1])
        # dq reads what lies before, dk and dv what lies behind
        assert same(h["dq"][0, :at], g["dq"][0, :at])
        for n in ("dk", "dv"):
            assert same(h[n][0, at + 1:], g[n][0, at + 1:]), (name, n)


@pytest.mark.parametrize("T,shift,bound", [(128, 11, 2.0 ** -20), (128, 7, 2.0 ** -20), (1024, 6, 2.0 ** -19),
                                           (1500, 5, 2.0 ** -19)])
def test_states_of_bf16_are_as_exact_as_fp32_sums(T, shift, bound):
    # Relative 2-norm of a state's error.  128 tokens are two chunks of a decay's product and
    # six matrix products: 14 roundings of 2^-24 at most, under 2^-20.  Longer: what is summed
    # last weighs most, and of the tokens that have decayed to an eighth the terms are rounded
    # to 2^-16 (2^-18 in the 2-norm): 2^-21 and the 14 roundings together are under 2^-19.
    # Terms of two bf16 parts alone are 2^-18.4 off.
    d = data(2, T, 2, 2, 64, 64, "bf16", seed=T + shift)
    d["g"] = dev(np.full(2, 1 - 2.0 ** -shift), "f32")
    want = R.forward(d["q"][1], d["k"][1], d["v"][1], d["g"][1], 0.125, d["S0"][1], None, "bf16")["S_T"][0]
    off = host(forward(d, 0.125)[1]) - want
    assert np.linalg.norm(off) <= bound * np.linalg.norm(want)
    g = backward(d, 0.125)
    want = R.backward(d["do"][1], d["q"][1], d["k"][1], d["v"][1], d["g"][1], 0.125, d["S0"][1], d["dS"][1], None,
                      "bf16")["dS0"][0]
    assert np.linalg.norm(host(g["dS0"]) - want) <= bound * np.linalg.norm(want)


def test_sequences_do_not_leak():
    cu = [0, 40, 100, 100, 130]
    d = data(1, 130, 2, 2, 32, 32, "bf16", 9, cu)
    o, S_T = forward(d, None, cu)
    g = backward(d, None, cu)
    e = dict(d)
    for n in ("q", "k", "v", "do"):
        t = d[n][0].clone()
        t[:, 40:100] = float("nan")
        e[n] = (t,)
    o2, S2 = forward(e, None, cu)
    h = backward(e, None, cu)
    for a, b in ((o, o2), (g["dq"], h["dq"]), (g["dk"], h["dk"]), (g["dv"], h["dv"])):
        assert same(a[:, :40], b[:, :40]) and same(a[:, 100:], b[:, 100:]) and torch.isnan(b[:, 41:99]).any()
    for n in (0, 2, 3):
        assert same(S_T[n], S2[n]) and same(g["dS0"][n], h["dS0"][n])


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_decays_of_zero_and_one(io):
    d = data(1, 150, 4, 4, 16, 16, io, 11)
    d["g"] = dev(np.array([0.0, 1.0, 1e-30, 1 - 2.0 ** -24]))
    both(d, io, None)


def test_prompt_in_pieces_then_single_tokens():
    B, T, H, dk, dv = 2, 130, 3, 32, 64
    d = data(B, T, H, H, dk, dv, "f32", 13)
    q, k, v, g, S0 = (d[n][0] for n in ("q", "k", "v", "g", "S0"))
    ref = R.forward(*(d[n][1] for n in ("q", "k", "v", "g")), dk ** -0.5, d["S0"][1], None, "f32")
    cut = lambda p, e: [t[:, p:e].contiguous() for t in (q, k, v)]
    out, S = [], S0
    for p, e in ((0, 50), (50, 51), (51, 120)):
        o, S = kda.kdn_linattn_fwd(*cut(p, e), g, S0=S, want_state=True)
        out.append(o)
    for t in range(120, T):
        out.append(kda.kdn_linattn_step(q[:, t], k[:, t], v[:, t], g, S)[:, None])
    BR.check(host(torch.cat(out, 1)), ref["o"], "f32", "o")
    BR.check(host(S), ref["S_T"], "f32", "S")


@pytest.mark.parametrize("T,Hk", [(100, 2), (2000, 1)])
def test_captured_and_replayed(T, Hk):
    cu = [0, T // 3, T // 3, T - 5]
    d = data(1, T, 2, Hk, 64, 64, "bf16", T, cu)
    q1, k1, v1 = (d[n][0][0, :1].contiguous() for n in ("q", "k", "v"))
    state = d["S0"][0][:1].clone()
    cu_t = offsets(cu)

    def run():
        args = (d["q"][0], d["k"][0], d["v"][0], d["g"][0])
        o, S_T = kda.kdn_linattn_fwd(*args, S0=d["S0"][0], cu_seqlens=cu_t, want_state=True)
        g = kda.kdn_linattn_bwd(d["do"][0], *args, S0=d["S0"][0], dS_T=d["dS"][0], cu_seqlens=cu_t)
        return [o, S_T, kda.kdn_linattn_step(q1, k1, v1, d["g"][0], state)] + [g[n] for n in sorted(g)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        static = run()
    for i in range(4):
        for n in ("q", "v", "do"):
            d[n][0].normal_()
        state.normal_()
        before = state.clone()
        for t in static:
            t.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in static]
        state.copy_(before)
        assert all(same(a, b) for a, b in zip(got, run())), i


def test_two_streams_at_once():
    calls = [data(1, 3000, 2, 2, 64, 64, "bf16", s) for s in (1, 2)]
    want = [(forward(d), backward(d)) for d in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = []
    for d, s in zip(calls, streams):
        with torch.cuda.stream(s):
            got.append((forward(d), backward(d)))
    torch.cuda.synchronize()
    for (a, b), (c, e) in zip(want, got):
        assert same(a[0], c[0]) and same(a[1], c[1]) and all(same(b[n], e[n]) for n in b)


def test_workspaces_carry_nothing():
    d = data(1, 2500, 4, 2, 64, 64, "bf16", 3)
    o, S_T = forward(d)
    g = backward(d)
    L = kda._lib.lib()
    n = max(L.kdn_linattn_fwd_workspace_size(1, 2500, 4, 64, 64),
            L.kdn_linattn_bwd_workspace_size(1, 2500, 4, 2, 64, 64))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for fill in (255, 0, None):
        if fill is not None:
            ws.fill_(fill)
        o2, S2 = forward(d, workspace=ws)
        assert same(o, o2) and same(S_T, S2)
        h = backward(d, workspace=ws)
        assert all(same(g[n], h[n]) for n in g)
    with pytest.raises(kda.KdnError, match="workspace"):
        forward(d, workspace=ws[:16])


def test_bad_offsets_stay_inside():
    d = data(1, 1500, 2, 2, 32, 32, "bf16", 5, [0, 1, 2, 3, 4])
    o = torch.full((1, 1502, 2, 32), 9.0, dtype=torch.bfloat16, device="cuda")
    for cu in ([0, 900, 100, 5000, 1400], [-5, 3, -1, 70000, 2], [1500, 0, 1500, 0, 1500], [7, 7, 7, 7, 9]):
        inner = o[:, 1:-1]
        kda.kdn_linattn_fwd(d["q"][0], d["k"][0], d["v"][0], d["g"][0], S0=d["S0"][0], cu_seqlens=offsets(cu),
                            o=inner, want_state=True)
        backward(d, None, cu)
        torch.cuda.synchronize()
        assert (o[:, 0] == 9).all() and (o[:, -1] == 9).all()


def test_long_offsets():
    # tensors of over 2^31 bytes: the last rows against a call on those rows alone
    B, T, H, dk = 17, 66000, 4, 256
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k, v = (torch.empty(B, T, H, dk, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(3))
    decay = torch.full((H,), 0.9, device="cuda")
    assert q.numel() * 2 > 1 << 31
    o, S_T = kda.kdn_linattn_fwd(q, k, v, decay, want_state=True)
    r = kda.kdn_linattn_bwd(v, q, k, v, decay)
    last = [t[-1:].contiguous() for t in (q, k, v)]
    o1, S1 = kda.kdn_linattn_fwd(*last, decay, want_state=True)
    r1 = kda.kdn_linattn_bwd(last[2], *last, decay)
    # other segments: states joined elsewhere (2^-16 a term), y within its bf16 roundings
    norm = lambda a, b: ((a.float() - b.float()).norm() / b.float().norm()).item()
    assert norm(S_T[-1:], S1) <= 2.0 ** -15 and norm(o[-1:], o1) <= 2.0 ** -7
    assert all(norm(r[n][-1:], r1[n]) <= 2.0 ** -7 for n in r)
