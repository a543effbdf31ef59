"""Group norm with an activation and dropout on the GPU against their 64-bit
references, value by value, and a block of linear attention, group norm and
dropout against autograd: sizes from one value to several workgroups a group,
odd ones, slices of wider rows, what is not finite, graphs, streams."""
import numpy as np
import pytest
import torch

import block_reference as BR
import kalman_delta_rule_amd as kda
import layer_ops_reference as R
from test_gpu_block import DT, dev, host, same, sliced

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a HIP GPU")


# ---- group norm -----------------------------------------------------------

SHAPES = [(0, 1, 8, 2), (3, 0, 8, 2), (1, 1, 1, 1), (1, 1, 5, 5), (3, 1, 6, 3), (7, 1, 64, 4), (33, 1, 2048, 16),
          (130, 1, 333, 9), (9, 1, 700, 7), (5, 1, 8192, 1), (3, 1, 16384, 2), (2, 1, 40000, 1), (2, 1, 40000, 2),
          (2000, 1, 256, 8), (40000, 1, 128, 2), (30000, 1, 72, 9), (2, 5, 12, 3), (3, 64, 64, 4), (2, 100, 333, 9),
          (4, 1000, 32, 32), (16, 257, 48, 3), (1, 4096, 512, 32), (5, 1021, 333, 9), (130, 33, 16, 2),
          (2, 3, 20000, 2), (300, 64, 128, 4), (1, 20000, 8, 1), (9000, 32, 8, 1), (4100, 64, 8, 1),
          (2100, 128, 8, 1), (1030, 256, 8, 1), (260, 1024, 8, 1), (130, 4096, 8, 1), (130, 8192, 8, 1),
          (20, 4096, 240, 30), (2, 2, 4096, 4096), (1, 3000, 3, 1), (70, 50, 24, 2)]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("N,S,C,G", SHAPES)
def test_group_norm(N, S, C, G, io):
    rng = np.random.default_rng(N * 31 + S * 7 + C)
    silu = (N + S + C) % 3 != 0
    x, xr = dev(rng.standard_normal((N, S, C)) * 2 + 0.5, io)
    dy, dyr = dev(rng.standard_normal((N, S, C)), io)
    w, wr = dev(rng.standard_normal(C))
    b, br = dev(rng.standard_normal(C))
    if (N + C) % 3 == 1:
        x = sliced(x, 2)
    if (S + C) % 4 == 1:
        w = b = wr = br = None
    act = "silu" if silu else None
    eps = 1e-5
    y, mean, rstd = kda.kdn_group_norm_fwd(x, G, w, b, eps=eps, activation=act, want_stats=True)
    y2, none, _ = kda.kdn_group_norm_fwd(x, G, w, b, eps=eps, activation=act)
    assert none is None and same(y, y2)
    if N and S:
        ref = R.group_norm(xr, G, wr, br, float(np.float32(eps)), silu)
        BR.check(host(y), ref["y"], io, "y")
        BR.check(host(mean), ref["mean"], "f32", "mean")
        BR.check(host(rstd), ref["rstd"], "f32", "rstd")
    g = kda.kdn_group_norm_bwd(dy, x, mean, rstd, w, b, activation=act)
    if N and S:
        ref = R.group_norm_bwd(dyr, xr, host(mean), host(rstd), wr, br, silu)
        BR.check(host(g["dx"]), ref["dx"], io, "dx")
        BR.check(host(g["dweight"]), ref["dweight"], "f32", "dweight")
        BR.check(host(g["dbias"]), ref["dbias"], "f32", "dbias")
    else:
        assert (g["dweight"] == 0).all() and (g["dbias"] == 0).all()
    only = kda.kdn_group_norm_bwd(dy, x, mean, rstd, w, b, activation=act, want_param_grads=False)
    assert set(only) == {"dx"} and same(only["dx"], g["dx"])


# groups whose last vector holds one to all but one of its values; large calls of such
# groups, whose sums go by channel
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("N,S,C,G", [(50, 3, 3 * n, 3) for n in range(5, 24)] + [(2, 9000, 2 * n, 2) for n in (5, 9, 14, 23)] +
                         [(1, 9000, n, 1) for n in (3, 5, 7, 9, 13)] + [(64, 260, 1029, 7), (300, 70, 900, 36)])
def test_group_norm_of_uneven_groups(N, S, C, G, io):
    test_group_norm(N, S, C, G, io)


def test_one_group_of_a_row_is_layer_norm():
    x = torch.randn(300, 1000, device="cuda")
    w, b = torch.randn(1000, device="cuda"), torch.randn(1000, device="cuda")
    y, mean, rstd = kda.kdn_group_norm_fwd(x, 1, w, b, want_stats=True)
    z, m, r = kda.kdn_layer_norm_fwd(x, w, b, want_stats=True)
    # each within its bound of the same value: e_y of block_reference.layer_norm, twice
    ref = BR.layer_norm(host(x), host(w), host(b), float(np.float32(1e-5)))
    assert (np.abs(host(y) - host(z)) <= 2.1 * ref["y"][1] + 2.1 * BR.U * np.abs(host(y)) + BR.TINY).all()


@pytest.mark.parametrize("shape,G", [((64, 1, 2048), 1), ((3, 4096, 64), 4), ((2, 70000, 16), 1)])
def test_group_norm_far_from_zero(shape, G):
    # a spread of one around 20000: the variance has to be taken around the mean
    rng = np.random.default_rng(5)
    x, xr = dev(rng.standard_normal(shape) + 20000.0)
    y, mean, rstd = kda.kdn_group_norm_fwd(x, G, eps=0.0, want_stats=True)
    ref = R.group_norm(xr, G, None, None, 0.0, False)
    for got, name in ((y, "y"), (mean, "mean"), (rstd, "rstd")):
        BR.check(host(got), ref[name], "f32", name)


@pytest.mark.parametrize("S,C,G", [(1, 384, 3), (700, 24, 3), (40000, 24, 3)])
def test_group_norm_constant_groups_and_bad_ones(S, C, G):
    x = torch.full((8, S, C), 3.0, device="cuda")
    x[3, S // 2, 7] = float("nan")          # group 0 of sample 3
    x[5, S // 2, C - 1] = float("inf")      # the last group of sample 5
    y, mean, rstd = kda.kdn_group_norm_fwd(x, G, eps=1e-6, want_stats=True)
    bad = torch.zeros(8, G, dtype=torch.bool, device="cuda")
    bad[3, 0] = bad[5, G - 1] = True
    assert (mean[~bad] == 3).all() and torch.isnan(rstd[bad]).all()
    parts = y.view(8, S, G, C // G).transpose(1, 2)
    assert (parts[~bad] == 0).all() and torch.isnan(parts[bad]).all()
    g = kda.kdn_group_norm_bwd(torch.ones_like(x), x, mean, rstd)
    parts = g["dx"].view(8, S, G, C // G).transpose(1, 2)
    assert torch.isfinite(parts[~bad]).all() and torch.isnan(parts[bad]).all()
    one = C // G
    assert torch.isnan(g["dweight"][:one]).all() and torch.isfinite(g["dweight"][one:2 * one]).all()


def test_group_norm_of_heads_and_many_axes():
    o = torch.randn(2, 6, 3, 64, device="cuda").to(torch.bfloat16)
    y, mean, _ = kda.kdn_group_norm_fwd(o.view(12, 192), 3, want_stats=True)
    n, m, _ = kda.kdn_layer_norm_fwd(o, want_stats=True)
    assert torch.allclose(mean.view(2, 6, 3), m, rtol=0, atol=80 * 2.0 ** -24)  # 64 values of size one
    x = torch.randn(2, 5, 7, 24, device="cuda")
    y, mean, _ = kda.kdn_group_norm_fwd(x, 4, want_stats=True)
    z, _, _ = kda.kdn_group_norm_fwd(x.view(2, 35, 24), 4)
    assert y.shape == x.shape and mean.shape == (2, 4) and same(y.view(2, 35, 24), z)


# ---- dropout ----------------------------------------------------------------

@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D", [(0, 8), (1, 1), (1, 7), (3, 8), (5, 33), (64, 64), (31, 1000), (300, 2049)])
def test_dropout(rows, D, io):
    rng = np.random.default_rng(rows + D)
    x, xr = dev(rng.standard_normal((rows, D)), io)
    dy, dyr = dev(rng.standard_normal((rows, D)), io)
    res, resr = dev(rng.standard_normal((rows, D)), io)
    for p, seed, offset in ((0.0, 0, 0), (0.1, 5, 1), (0.5, (1 << 64) - 1, (1 << 64) - 2), (0.9, 1 << 40, 1 << 33),
                            (1.0, 3, 4)):
        keep, share = R.kept(rows * D, p, seed, offset)
        keep = keep.reshape(rows, D)
        scaled = lambda t: np.where(keep, t / max(share, 1e-9), 0.0)
        for t in (x, sliced(x, 2)):
            y = kda.kdn_dropout_fwd(t, p, seed, offset)
            BR.check(host(y), (scaled(xr), 3 * BR.U * np.abs(scaled(xr))), io, "y")
            y = kda.kdn_dropout_fwd(t, p, seed, offset, residual=res)
            BR.check(host(y), (scaled(xr) + resr, 4 * BR.U * (np.abs(scaled(xr)) + np.abs(resr))), io, "y + residual")
        dx = kda.kdn_dropout_bwd(dy, p, seed, offset)
        BR.check(host(dx), (scaled(dyr), 3 * BR.U * np.abs(scaled(dyr))), io, "dx")
        assert ((host(dx) == 0) == (~keep | (dyr == 0))).all()
        state = torch.tensor([v - (1 << 64) if v >= 1 << 63 else v for v in (seed, offset)], device="cuda")
        assert same(dx, kda.kdn_dropout_bwd(dy, p, state))
        assert same(y, kda.kdn_dropout_fwd(x, p, state, residual=res))


def test_what_is_dropped_leaves_no_trace():
    x = torch.randn(100, 100, device="cuda")
    keep = torch.from_numpy(R.kept(10000, 0.5, 9, 0)[0].reshape(100, 100)).cuda()
    bad = x.clone()
    bad[~keep] = float("nan")
    assert same(kda.kdn_dropout_fwd(x, 0.5, 9), kda.kdn_dropout_fwd(bad, 0.5, 9))
    assert (kda.kdn_dropout_fwd(torch.full_like(x, float("inf")), 1.0, 9) == 0).all()


# ---- both, and linear attention before them -----------------------------------------

def block(x, qkv, g, w, b, seed, H, dk, dv, d_out=None):
    """A mixer block behind its projection: heads' attention, group norm with silu,
    dropout, the residual stream.  With d_out its gradients by qkv, w and b."""
    B, T = x.shape[:2]
    q, k, v = (t.unflatten(-1, (H, -1)) for t in qkv.split([H * dk, H * dk, H * dv], -1))
    o, _ = kda.kdn_linattn_fwd(q, k, v, g)
    flat = o.view(B * T, H * dv)
    n, mean, rstd = kda.kdn_group_norm_fwd(flat, H, w, b, activation="silu", want_stats=True)
    y = kda.kdn_dropout_fwd(n.view(B, T, -1), 0.25, seed, residual=x)
    if d_out is None:
        return [y]
    dn = kda.kdn_dropout_bwd(d_out, 0.25, seed)
    gn = kda.kdn_group_norm_bwd(dn.view(B * T, -1), flat, mean, rstd, w, b, activation="silu")
    r = kda.kdn_linattn_bwd(gn["dx"].view(B, T, H, dv), q, k, v, g)
    return [y, r["dq"], r["dk"], r["dv"], gn["dweight"], gn["dbias"]]


def test_block_against_autograd():
    B, T, H, dk, dv = 2, 70, 3, 16, 24
    gen = torch.Generator().manual_seed(5)
    n = lambda *s: torch.randn(*s, generator=gen)
    x, d_out, qkv = n(B, T, H * dv), n(B, T, H * dv), n(B, T, H * (2 * dk + dv))
    w, b, g = n(H * dv), n(H * dv), torch.tensor([0.5, 0.9, 0.99])
    got = block(*(t.cuda() for t in (x, qkv, g, w, b)), 77, H, dk, dv, d_out.cuda())
    lead = [t.double().requires_grad_() for t in (qkv, w, b)]
    q, k, v = (t.unflatten(-1, (H, -1)) for t in lead[0].split([H * dk, H * dk, H * dv], -1))
    S, os = torch.zeros(B, H, dk, dv, dtype=torch.float64), []
    for t in range(T):
        S = g.double()[:, None, None] * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        os.append((S * q[:, t, :, :, None]).sum(2) * dk ** -0.5)
    o = torch.stack(os, 1)
    xh = (o - o.mean(-1, keepdim=True)) / torch.sqrt(o.var(-1, correction=0, keepdim=True) + 1e-5)
    z = xh.flatten(2) * lead[1] + lead[2]
    keep, share = R.kept(B * T * H * dv, 0.25, 77, 0)
    y = x.double() + torch.nn.functional.silu(z) * torch.from_numpy(keep.reshape(B, T, -1)) / share
    grads = torch.autograd.grad(y, lead, d_out.double())
    want = [y.detach()] + [t.unflatten(-1, (H, -1)) for t in grads[0].split([H * dk, H * dk, H * dv], -1)] + list(grads[1:])
    for a, r in zip(got, want):
        # three operators of a few hundred roundings of 2^-24 each at most
        assert (a.cpu().double() - r).norm() <= 1000 * 2.0 ** -24 * r.norm()


def all_calls(io=torch.bfloat16, T=300):
    B, H, dk, dv = 2, 4, 32, 64
    x = torch.randn(B, T, H * dv, device="cuda").to(io)
    d_out = torch.randn(B, T, H * dv, device="cuda").to(io)
    qkv = torch.randn(B, T, H * (2 * dk + dv), device="cuda").to(io)
    w, b = torch.randn(H * dv, device="cuda"), torch.randn(H * dv, device="cuda")
    g = torch.tensor([0.5, 0.9, 0.99, 0.999], device="cuda")
    seed = torch.tensor([3, 4], device="cuda")
    wide = torch.randn(1, 5000, 64, device="cuda").to(io)  # large groups: several launches

    def run():
        y, mean, rstd = kda.kdn_group_norm_fwd(wide, 2, activation="silu", want_stats=True)
        n = kda.kdn_group_norm_bwd(wide, wide, mean, rstd, activation="silu")
        return block(x, qkv, g, w, b, seed, H, dk, dv, d_out) + [y] + [n[k] for k in sorted(n)]
    return [x, d_out, qkv, wide, seed], run


@pytest.mark.parametrize("T", [1, 300, 1100])
def test_captured_and_replayed(T):
    inputs, run = all_calls(T=T)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        static = run()
    for i in range(4):
        for t in inputs[:-1]:
            t.normal_()
        inputs[-1].add_(1)
        for t in static:
            t.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in static]
        assert all(same(a, b) for a, b in zip(got, run())), i


def test_two_streams_at_once():
    calls = [all_calls()[1] for _ in range(2)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    got = []
    for c in calls:
        with torch.cuda.stream(torch.cuda.Stream()):
            got.append(c())
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(same(x, y) for x, y in zip(a, b))


def test_group_norm_workspaces_carry_nothing():
    x = torch.randn(1, 6000, 96, device="cuda")
    y, mean, rstd = kda.kdn_group_norm_fwd(x, 3, want_stats=True)
    g = kda.kdn_group_norm_bwd(x, x, mean, rstd)
    L = kda._lib.lib()
    n = max(L.kdn_group_norm_fwd_workspace_size(1, 6000, 96, 3), L.kdn_group_norm_bwd_workspace_size(1, 6000, 96, 3))
    assert L.kdn_group_norm_fwd_workspace_size(1, 6000, 96, 3) > 0
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for fill in (255, 0):
        ws.fill_(fill)
        assert same(y, kda.kdn_group_norm_fwd(x, 3, workspace=ws)[0])
        h = kda.kdn_group_norm_bwd(x, x, mean, rstd, workspace=ws)
        assert all(same(g[k], h[k]) for k in g)
    with pytest.raises(kda.KdnError, match="workspace"):
        kda.kdn_group_norm_fwd(x, 3, workspace=ws[:16])


def test_offsets_beyond_32_bits():
    """Tensors of over 4 GiB: the last samples, and elements, against small calls."""
    N, S, C = 70000, 1, 16384
    x = torch.empty(N, S, C, device="cuda").normal_()
    assert x.numel() * 4 > 1 << 32
    y, mean, rstd = kda.kdn_group_norm_fwd(x, 128, activation="silu", want_stats=True)
    last, _, _ = kda.kdn_group_norm_fwd(x[-3:].contiguous(), 128, activation="silu")
    # (few samples go in other shapes: the same values within their bounds, some tens of roundings)
    assert (y[-3:] - last).abs().max() <= 200 * 2.0 ** -24 * last.abs().max()
    g = kda.kdn_group_norm_bwd(x, x, mean, rstd, activation="silu")["dx"][-3:]
    h = kda.kdn_group_norm_bwd(x[-3:].contiguous(), x[-3:].contiguous(), mean[-3:].contiguous(),
                               rstd[-3:].contiguous(), activation="silu")["dx"]
    assert (g - h).abs().max() <= 200 * 2.0 ** -24 * h.abs().max()
    del y, g
    z = kda.kdn_dropout_bwd(x, 0.5, 11)
    n = N * S * C
    tail = 1 << 16
    counter = np.zeros((tail // 8, 4), np.uint64)
    counter[:, 0] = np.arange((n - tail) // 8, n // 8)
    words = R.philox(counter, (11, 0))
    bits = np.stack([words & np.uint32(0xFFFF), words >> np.uint32(16)], 2).reshape(-1)
    assert np.array_equal(host(z.view(-1)[-tail:]) != 0, bits >= 32768)
