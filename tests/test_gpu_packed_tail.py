"""Rows behind the last packed sequence: zeros in what the binding allocates itself, left
as they were in what the caller passes in, and nothing for the operators that take
all rows of them."""
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


def poison_allocator(nbytes):
    """The memory that torch hands out next holds NaN (bytes of ones)."""
    torch.cuda.synchronize()
    blocks = [torch.full((max(nbytes // k, 1),), 255, dtype=torch.uint8, device="cuda")
              for k in (1, 2, 32, 64, 128) for _ in range(6)]
    torch.cuda.synchronize()
    del blocks


def offsets(cu):
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


# no token in a sequence; borders inside runs and tiles; a tail of several tiles; a single channel
CASES = [(40, 6, [0, 0, 0]), (40, 6, [0, 7, 40]), (130, 33, [0, 1, 129]), (700, 64, [0, 100, 100, 257]),
         (3000, 70, [0, 900, 1003]), (3000, 1, [0, 5]), (1500, 520, [0, 1024]), (9000, 16, [0, 64, 4096])]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["preact", "alpha"])
@pytest.mark.parametrize("T,D,cu", CASES, ids=lambda v: str(v) if isinstance(v, int) else "N%d" % (len(v) - 1))
def test_new_outputs_hold_zeros(T, D, cu, gate, io):
    g = torch.Generator(device="cuda").manual_seed(T + D)
    new = lambda *s, dtype=DT[io]: torch.randn(*s, generator=g, device="cuda").to(dtype)
    x, dy, w = new(1, T, D), new(1, T, D), new(3, D, dtype=torch.float32)
    a = new(1, T, D) if gate == "preact" else torch.rand(1, T, D, generator=g, device="cuda")
    for t in (x, dy, a):
        t[:, cu[-1]:] = float("nan")
    c, size = offsets(cu), x.numel() * 4
    outs = {}
    poison_allocator(size)
    outs["y"], _ = kda.kdn_conv_fwd(x, w, cu_seqlens=c, activation="silu")
    poison_allocator(size)
    gc = kda.kdn_conv_bwd(dy, x, w, cu_seqlens=c, activation="silu")
    poison_allocator(size)
    outs["h"], _, chk = kda.kdn_rec_fwd(x, a, cu_seqlens=c, gate=gate, want_checkpoints=True)
    poison_allocator(size)
    gr = kda.kdn_rec_bwd(dy, x, a, chk, cu_seqlens=c, gate=gate)
    outs.update(conv_dx=gc["dx"], dx=gr["dx"], da=gr["da"])
    for name, t in outs.items():
        assert (t[:, cu[-1]:] == 0).all(), name
        assert torch.isfinite(t).all(), name
    assert (chk[:, -(-cu[-1] // 64):] == 0).all() and torch.isfinite(chk).all()
    assert torch.isfinite(gc["dweight"]).all()

    # the caller's keep what they hold, and the rest is the same
    mine = lambda like: torch.full_like(like, 77.0)
    y, _ = kda.kdn_conv_fwd(x, w, cu_seqlens=c, activation="silu", y=mine(x))
    dx = kda.kdn_conv_bwd(dy, x, w, cu_seqlens=c, activation="silu", dx=mine(x))["dx"]
    h, _, chk2 = kda.kdn_rec_fwd(x, a, cu_seqlens=c, gate=gate, want_checkpoints=True, h=mine(x))
    both = kda.kdn_rec_bwd(dy, x, a, chk2, cu_seqlens=c, gate=gate, dx=mine(x), da=mine(a))
    for t, q in ((y, outs["y"]), (dx, outs["conv_dx"]), (h, outs["h"]), (both["dx"], outs["dx"]), (both["da"], outs["da"])):
        assert torch.equal(t[:, :cu[-1]], q[:, :cu[-1]]) and (t[:, cu[-1]:] == 77).all()
    # one of two
    poison_allocator(size)
    one = kda.kdn_rec_bwd(dy, x, a, chk, cu_seqlens=c, gate=gate, dx=mine(x))
    assert (one["dx"][:, cu[-1]:] == 77).all() and torch.equal(one["da"], outs["da"])
    poison_allocator(size)
    one = kda.kdn_rec_bwd(dy, x, a, chk, cu_seqlens=c, gate=gate, da=mine(a))
    assert (one["da"][:, cu[-1]:] == 77).all() and torch.equal(one["dx"], outs["dx"])


def test_a_padded_row_trains_like_its_sequences():
    """recurrence -> convolution -> layer norm, backward: parameter gradients summed
    over all rows of a padded packing are those of the sequences alone."""
    T, D, cu = 1000, 96, [0, 300, 300, 900]  # (both rows are eight tiles of the recurrence)
    g = torch.Generator(device="cuda").manual_seed(12)
    new = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, a, dh, w, wn = new(1, T, D), new(1, T, D), new(1, T, D), new(4, D), new(D)
    c, end = offsets(cu), cu[-1]

    def run(x, a, dh):
        poison_allocator(T * D * 4)
        n, mean, rstd = kda.kdn_layer_norm_fwd(x, wn, want_stats=True)
        y, _ = kda.kdn_conv_fwd(n, w, cu_seqlens=c, activation="silu")
        h, _, chk = kda.kdn_rec_fwd(y, a, cu_seqlens=c, blend=True, want_checkpoints=True)
        gr = kda.kdn_rec_bwd(dh, y, a, chk, cu_seqlens=c, blend=True)
        gc = kda.kdn_conv_bwd(gr["dx"], n, w, cu_seqlens=c, activation="silu")
        gn = kda.kdn_layer_norm_bwd(gc["dx"], x, mean, rstd, wn)
        return gc, gn, (gc["dx"], (x - mean[..., None]) * rstd[..., None], gr["dx"], n)
    whole = run(x, a, dh)
    short = run(*(t[:, :end].contiguous() for t in (x, a, dh)))
    # up to the convolution's dx it is the same operations
    for p, q in zip(whole[2], short[2]):
        assert torch.equal(p[:, :end], q)
    dy, xh, dz, n = (t.abs().double() for t in short[2])
    # each side is off by its longest chain of additions (under 128 + 16 + 20 terms for either
    # operator's 1000 rows) and a few roundings of a term, times the sum of the magnitudes; |silu'| < 1.1
    size = {"dweight": (dy * xh).sum((0, 1)), "dbias": dy.sum((0, 1))}
    for k, m in size.items():
        assert torch.isfinite(whole[1][k]).all()
        assert ((whole[1][k] - short[1][k]).abs() <= 2 * 180 * U * m).all(), k
    m = 1.1 * dz.sum((0, 1)) * n.amax((0, 1))
    assert ((whole[0]["dweight"] - short[0]["dweight"]).abs() <= 2 * 180 * U * m).all()


def test_captured_with_a_tail():
    T, D, cu = 900, 40, [0, 100, 500]
    x, a, w = (torch.randn(*s, device="cuda") for s in ((1, T, D), (1, T, D), (4, D)))
    c = offsets(cu)

    def run():
        y, _ = kda.kdn_conv_fwd(x, w, cu_seqlens=c)
        h, _, chk = kda.kdn_rec_fwd(y, a, cu_seqlens=c, want_checkpoints=True)
        g = kda.kdn_rec_bwd(h, y, a, chk, cu_seqlens=c)
        return [y, h, chk, g["dx"], g["da"], kda.kdn_conv_bwd(g["dx"], x, w, cu_seqlens=c)["dx"]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    for end in (500, 700, 100, 900):  # the offsets are read on the device
        c.copy_(offsets([0, min(100, end), end]))
        want = run()
        for o in outs:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for o, q in zip(outs, want):
            assert torch.equal(o, q)
            assert o.shape[1] != T or (o[:, end:] == 0).all()
