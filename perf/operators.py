"""The block operators around the mixer, as cases to measure: layer norm, the
short causal convolution and the gated recurrence, forward, backward and as
single-token steps.

``own`` false computes a case in plain torch operations (fp32, rounded once at
the end), true makes the library's calls.  ``exact`` computes it in 64 bits from
the definition: a token loop, or autograd over it.  A step's state moves on by
one token each pass, as in decoding.

  layer norm  y = (x - mean) rstd weight + bias over rows of D
  conv        z_t = bias + sum_j weight[W-1-j] x_{t-j}, y = z or z sigmoid(z);
              inputs before a sequence's first token come from its state
  recurrence  h_t = alpha_t h_{t-1} + u_t, u = x, or (1 - alpha) x with "blend";
              alpha = sigmoid(a) ("preact") or given ("alpha", fp32)
"""
import math

import torch

own = False

EPS = 1e-5
MOST = 1 << 27  # elements [B, T, D] of the largest training case


def listed():
    return [
        # decode: 256 sequences, one token each, the residual stream of 16 heads of 128
        dict(name="ln decode", op="ln", train=False, rows=256, D=2048, io="bf16"),
        # the mixer's output normalised per head: B8 T4096 H16, rows of dv = 128
        dict(name="ln per head", op="ln", train=False, rows=8 * 4096 * 16, D=128, io="bf16"),
        # pre-norm of the residual stream in training: B8 T4096, forward and backward
        dict(name="ln train", op="ln", train=True, rows=8 * 4096, D=2048, io="bf16"),
        # odd width and row count in fp32: nothing is a multiple of a vector or a tile
        dict(name="ln train odd fp32", op="ln", train=True, rows=4099, D=1537, io="f32"),
        # decode: the q, k and v channels of 256 sequences through their short filters
        dict(name="conv step", op="conv_step", B=256, D=6144, W=4, io="bf16", silu=True),
        # prompts of 4096 tokens, x one third of a fused q, k, v projection
        dict(name="conv prompt", op="conv", train=False, B=8, T=4096, D=2048, W=4, io="bf16",
             silu=True, seqs=0, fused=3),
        # training on documents packed into one row
        dict(name="conv train packed", op="conv", train=True, B=1, T=32768, D=2048, W=4, io="bf16",
             silu=True, seqs=37, fused=1),
        # odd channels and lengths, three taps, no activation, fp32
        dict(name="conv train odd fp32", op="conv", train=True, B=3, T=1021, D=333, W=3, io="f32",
             silu=False, seqs=0, fused=1),
        # decode: one token of 256 sequences
        dict(name="rec step", op="rec_step", B=256, D=2048, io="bf16", gate="preact", blend=True),
        # prompts of 4096 tokens
        dict(name="rec prompt", op="rec", train=False, B=8, T=4096, D=2048, io="bf16",
             gate="preact", blend=True, seqs=0),
        # training on one long sequence: few channels, the scan has to be split over time
        dict(name="rec train long", op="rec", train=True, B=1, T=65536, D=2048, io="bf16",
             gate="preact", blend=True, seqs=0),
        # packed documents, odd channels, decay given in fp32
        dict(name="rec train packed fp32", op="rec", train=True, B=1, T=5003, D=771, io="f32",
             gate="alpha", blend=False, seqs=23),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm spread evenly."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999))))))


def _width(rng, lo, hi):
    D = _spread(rng, lo, hi)
    kind = rng.random()
    return max(lo, D // 64 * 64) if kind < 0.5 else max(lo, D // 2 * 2) if kind < 0.7 else D


def draw(rng):
    op = rng.choice(["ln", "ln", "conv_step", "conv", "conv", "rec_step", "rec", "rec", "rec"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op == "ln":
        D = _width(rng, 64, 16384)
        return dict(op=op, train=rng.random() < 0.6, rows=_spread(rng, 1, MOST // 2 // D), D=D, io=io)
    if op == "conv_step":
        return dict(op=op, B=_spread(rng, 1, 1024), D=_width(rng, 64, 8192), W=rng.randint(2, 4), io=io,
                    silu=rng.random() < 0.7)
    if op == "rec_step":
        return dict(op=op, B=_spread(rng, 1, 1024), D=_width(rng, 64, 8192), io=io,
                    gate=rng.choice(["preact", "alpha"]), blend=rng.random() < 0.5)
    train = rng.random() < 0.6
    D = _width(rng, 64, 8192)
    most = MOST // 2 if io == "bf16" else MOST // 4
    T = _spread(rng, 1, min(65536, most // D))
    seqs = _spread(rng, 1, 300) if rng.random() < 0.4 else 0
    B = 1 if seqs else _spread(rng, 1, max(1, min(16, most // D // T)))
    if op == "conv":
        return dict(op=op, train=train, B=B, T=T, D=D, W=rng.randint(2, 4), io=io,
                    silu=rng.random() < 0.7, seqs=seqs, fused=rng.choice([1, 1, 3]))
    return dict(op=op, train=train, B=B, T=T, D=D, io=io, gate=rng.choice(["preact", "preact", "alpha"]),
                blend=rng.random() < 0.5, seqs=seqs)


def _dtype(case):
    return torch.bfloat16 if case["io"] == "bf16" else torch.float32


def _seqlens(case, g):
    """Offsets [N+1] of the packed sequences: N random cuts of [0, T], so that
    lengths run from zero to long; None where each row is one sequence."""
    if not case.get("seqs"):
        return None
    cuts = torch.randint(0, case["T"] + 1, (case["seqs"] - 1,), generator=g, device="cuda").sort().values
    ends = torch.tensor([0, case["T"]], device="cuda")
    return torch.cat((ends[:1], cuts, ends[1:])).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _dtype(case)

    def normal(*shape, dtype=torch.float32, scale=1.0, mean=0.0):
        return torch.randn(*shape, generator=g, device="cuda").mul_(scale).add_(mean).to(dtype)

    op, D = case["op"], case["D"]
    s = dict(case=dict(case))
    if op == "ln":
        # a residual stream: channels of unequal scale around a mean that is not zero
        scale = torch.exp(normal(D, scale=0.5))
        s["x"] = normal(case["rows"], D).mul_(scale).add_(0.3).to(dt)
        s["weight"] = normal(D, scale=0.2, mean=1.0)
        s["bias"] = normal(D, scale=0.2)
        if case["train"]:
            s["dy"] = normal(case["rows"], D, dtype=dt)
        return s
    if op == "conv_step":
        B, W = case["B"], case["W"]
        s["x"] = normal(B, D, dtype=dt)
        s["state"] = normal(B, W - 1, D, dtype=dt)
        s["weight"] = normal(W, D, scale=W ** -0.5)
        s["bias"] = normal(D, scale=0.1)
        return s
    # decays from tens to about a thousand tokens, by channel
    middle = torch.rand(D, generator=g, device="cuda") * 6 + 1
    if op == "rec_step":
        B = case["B"]
        s["x"] = normal(B, D, dtype=dt)
        a = normal(B, D, scale=0.5).add_(middle)
        s["a"] = a.to(dt) if case["gate"] == "preact" else torch.sigmoid(a)
        s["state"] = normal(B, D)
        return s
    B, T = case["B"], case["T"]
    s["cu"] = _seqlens(case, g)
    N = case["seqs"] or B
    if op == "conv":
        W = case["W"]
        wide = normal(B, T, case["fused"] * D, dtype=dt)
        s["x"] = wide[..., :D] if case["fused"] == 1 else wide[..., D:2 * D]
        s["weight"] = normal(W, D, scale=W ** -0.5)
        s["bias"] = normal(D, scale=0.1)
        s["state0"] = normal(N, W - 1, D, dtype=dt)
        if case["train"]:
            s["dy"] = normal(B, T, D, dtype=dt)
            s["dstate"] = normal(N, W - 1, D, dtype=dt)
        return s
    s["x"] = normal(B, T, D, dtype=dt)
    a = normal(B, T, D, scale=0.5).add_(middle)
    s["a"] = a.to(dt) if case["gate"] == "preact" else torch.sigmoid(a)
    s["h0"] = normal(N, D)
    if case["train"]:
        s["dh"] = normal(B, T, D, dtype=dt)
        s["dhT"] = normal(N, D)
    return s


# ---- the library's calls ------------------------------------------------

def _own(s):
    import kalman_delta_rule_amd as kda
    case = s["case"]
    op = case["op"]
    if op == "ln":
        y, mean, rstd = kda.kdn_layer_norm_fwd(s["x"], s["weight"], s["bias"], eps=EPS,
                                               want_stats=case["train"])
        if not case["train"]:
            return dict(y=y)
        g = kda.kdn_layer_norm_bwd(s["dy"], s["x"], mean, rstd, s["weight"])
        return dict(y=y, mean=mean, rstd=rstd, **g)
    act = "silu" if case.get("silu") else None
    if op == "conv_step":
        y = kda.kdn_conv_step(s["x"], s["weight"], s["state"], bias=s["bias"], activation=act)
        return dict(y=y, state=s["state"])
    if op == "conv":
        y, state = kda.kdn_conv_fwd(s["x"], s["weight"], bias=s["bias"], state0=s["state0"],
                                    cu_seqlens=s["cu"], activation=act, want_state=True)
        if not case["train"]:
            return dict(y=y, state=state)
        g = kda.kdn_conv_bwd(s["dy"], s["x"], s["weight"], bias=s["bias"], state0=s["state0"],
                             cu_seqlens=s["cu"], activation=act, dstate_T=s["dstate"])
        return dict(y=y, state=state, **g)
    if op == "rec_step":
        h = kda.kdn_rec_step(s["x"], s["a"], s["state"], gate=case["gate"], blend=case["blend"])
        return dict(h=h, state=s["state"])
    h, h_T, chk = kda.kdn_rec_fwd(s["x"], s["a"], h0=s["h0"], cu_seqlens=s["cu"], gate=case["gate"],
                                  blend=case["blend"], want_checkpoints=case["train"])
    if not case["train"]:
        return dict(h=h, h_T=h_T)
    g = kda.kdn_rec_bwd(s["dh"], s["x"], s["a"], chk, h0=s["h0"], dh_T=s["dhT"], cu_seqlens=s["cu"],
                        gate=case["gate"], blend=case["blend"])
    return dict(h=h, h_T=h_T, **g)


# ---- the plain form ------------------------------------------------------

def _plain_ln(s, dt):
    x = s["x"].float()
    mean = x.mean(-1, keepdim=True)
    rstd = torch.rsqrt((x - mean).square().mean(-1, keepdim=True) + EPS)
    xh = (x - mean) * rstd
    y = (xh * s["weight"] + s["bias"]).to(dt)
    if "dy" not in s:
        return dict(y=y)
    dy = s["dy"].float()
    g = dy * s["weight"]
    dx = (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True)) * rstd
    return dict(y=y, mean=mean[..., 0], rstd=rstd[..., 0], dx=dx.to(dt), dweight=(dy * xh).sum(0),
                dbias=dy.sum(0))


def _places(s, B, T):
    """Of the tokens of [B, T] in one row: the sequence of each; of the
    sequences: their first token and the one behind their last."""
    if s["cu"] is None:
        first = torch.arange(B, device="cuda") * T
        return torch.arange(B, device="cuda").repeat_interleave(T), first, first + T
    cu = s["cu"].long()
    return torch.searchsorted(cu, torch.arange(T, device="cuda"), right=True) - 1, cu[:-1], cu[1:]


def _silu_slope(z):
    p = torch.sigmoid(z)
    return p * (1 + z * (1 - p))


def _plain_conv(s, dt):
    case = s["case"]
    B, T, D = s["x"].shape
    W = s["weight"].shape[0]
    seq, first, end = _places(s, B, T)
    # each sequence behind its W - 1 state rows: every tap is a row of `wide`
    at = torch.arange(B * T, device="cuda") + (seq + 1) * (W - 1)
    before = (first + torch.arange(first.numel(), device="cuda") * (W - 1))[:, None] + torch.arange(W - 1, device="cuda")
    last = (end + torch.arange(first.numel(), device="cuda") * (W - 1))[:, None] + torch.arange(W - 1, device="cuda")
    wide = s["x"].new_empty(B * T + before.numel(), D, dtype=torch.float32)
    wide[at] = s["x"].reshape(B * T, D).float()
    wide[before] = s["state0"].float()
    w = s["weight"]
    z = s["bias"] + sum(wide[at - j] * w[W - 1 - j] for j in range(W))
    y = z * torch.sigmoid(z) if case["silu"] else z
    out = dict(y=y.to(dt).view(B, T, D), state=wide[last].to(dt))
    if "dy" not in s:
        return out
    g = s["dy"].reshape(B * T, D).float()
    if case["silu"]:
        g = g * _silu_slope(z)
    dwide = torch.zeros_like(wide)
    dwide[last] = s["dstate"].float()
    dw = torch.empty_like(w)
    for j in range(W):
        dwide[at - j] += g * w[W - 1 - j]
        dw[W - 1 - j] = (g * wide[at - j]).sum(0)
    return dict(out, dx=dwide[at].to(dt).view(B, T, D), dweight=dw, dbias=g.sum(0), dstate0=dwide[before].to(dt))


def _plain_scan(A, u):
    """h_t = A_t h_{t-1} + u_t along the first axis, h before it zero: spans
    doubled log2(T) times."""
    A, u, step = A.clone(), u.clone(), 1
    while step < u.shape[0]:
        u[step:] = u[step:] + A[step:] * u[:-step]
        A[step:] = A[step:] * A[:-step]
        step *= 2
    return u


def _plain_rec(s, dt):
    case = s["case"]
    B, T, D = s["x"].shape
    seq, first, end = _places(s, B, T)
    some = end > first
    x, a = s["x"].reshape(B * T, D).float(), s["a"].reshape(B * T, D).float()
    alpha, rest = (torch.sigmoid(a), torch.sigmoid(-a)) if case["gate"] == "preact" else (a, 1 - a)
    u = rest * x if case["blend"] else x
    starts = torch.arange(B * T, device="cuda") == first[seq]
    ends = torch.arange(B * T, device="cuda") == end[seq] - 1
    zero = torch.zeros((), device="cuda")
    inside = torch.where(starts[:, None], zero, alpha)
    h = _plain_scan(inside, torch.where(starts[:, None], u + alpha * s["h0"][seq], u))
    h_T = torch.where(some[:, None], h[(end - 1).clamp(min=0)], s["h0"])
    out = dict(h=h.to(dt).view(B, T, D), h_T=h_T)
    if "dh" not in s:
        return out
    dh = s["dh"].reshape(B * T, D).float()
    dh = torch.where(ends[:, None], dh + s["dhT"][seq], dh)
    later = torch.where(ends[:, None], zero, alpha.roll(-1, 0))
    lam = _plain_scan(later.flip(0), dh.flip(0)).flip(0)
    prev = torch.where(starts[:, None], s["h0"][seq], h.roll(1, 0))
    da = lam * (prev - x) if case["blend"] else lam * prev
    if case["gate"] == "preact":
        da = da * alpha * rest
    dx = lam * rest if case["blend"] else lam
    at = first.clamp(max=B * T - 1)
    dh0 = torch.where(some[:, None], (alpha * lam)[at], s["dhT"])
    return dict(out, dx=dx.to(dt).view(B, T, D), da=da.to(s["a"].dtype).view(B, T, D), dh0=dh0)


def _plain(s):
    case = s["case"]
    dt = _dtype(case)
    op = case["op"]
    if op == "ln":
        return _plain_ln(s, dt)
    if op == "conv":
        return _plain_conv(s, dt)
    if op == "rec":
        return _plain_rec(s, dt)
    if op == "conv_step":
        wide = torch.cat((s["state"], s["x"][:, None]), 1)
        z = (wide.float() * s["weight"]).sum(1) + s["bias"]
        s["state"] = wide[:, 1:].contiguous()
        return dict(y=(z * torch.sigmoid(z) if case["silu"] else z).to(dt), state=s["state"])
    a, x = s["a"].float(), s["x"].float()
    alpha, rest = (torch.sigmoid(a), torch.sigmoid(-a)) if case["gate"] == "preact" else (a, 1 - a)
    s["state"] = alpha * s["state"] + (rest * x if case["blend"] else x)
    return dict(h=s["state"].to(dt), state=s["state"])


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    e = 2 if case["io"] == "bf16" else 4
    op, D = case["op"], case["D"]
    ea = e if case.get("gate") == "preact" else 4
    if op == "ln":
        n, rows = case["rows"] * D, case["rows"]
        fwd = 2 * e * n + 8 * D + (8 * rows if case["train"] else 0)
        bwd = 3 * e * n + 8 * rows + 12 * D if case["train"] else 0
        return dict(bytes=fwd + bwd, flops=(8 + (14 if case["train"] else 0)) * n)
    if op == "conv_step":
        W, n = case["W"], case["B"] * D
        return dict(bytes=e * n * 2 * W + 4 * D * (W + 1), flops=(2 * W + 4) * n)
    if op == "rec_step":
        n = case["B"] * D
        return dict(bytes=(ea + 2 * e + 8) * n, flops=8 * n)
    n, N = case["B"] * case["T"] * D, case["seqs"] or case["B"]
    if op == "conv":
        W = case["W"]
        fwd = 2 * e * n + 4 * D * (W + 1) + 2 * e * N * (W - 1) * D
        bwd = 3 * e * n + 8 * D * (W + 1) + 3 * e * N * (W - 1) * D if case["train"] else 0
        return dict(bytes=fwd + bwd, flops=(2 * W + 4 + (6 * W + 10 if case["train"] else 0)) * n)
    fwd = (ea + 2 * e) * n + 8 * N * D
    bwd = (2 * ea + 3 * e) * n + 12 * N * D if case["train"] else 0
    return dict(bytes=fwd + bwd, flops=(8 + (20 if case["train"] else 0)) * n)


# ---- 64 bits, from the definitions ---------------------------------------

def _exact_ln(s):
    x = s["x"].double().requires_grad_("dy" in s)
    w, b = (s[k].double().requires_grad_("dy" in s) for k in ("weight", "bias"))
    var, mean = torch.var_mean(x, dim=-1, correction=0, keepdim=True)
    rstd = (var + EPS) ** -0.5
    y = w * ((x - mean) * rstd) + b
    if "dy" not in s:
        return dict(y=y)
    dx, dw, db = torch.autograd.grad(y, (x, w, b), s["dy"].double())
    return dict(y=y.detach(), mean=mean[..., 0].detach(), rstd=rstd[..., 0].detach(), dx=dx, dweight=dw, dbias=db)


def _spans(s):
    """(row, first token, behind the last) of every sequence, on the host."""
    if s["cu"] is None:
        return [(b, 0, s["x"].shape[1]) for b in range(s["x"].shape[0])]
    cu = s["cu"].tolist()
    return [(0, p, q) for p, q in zip(cu[:-1], cu[1:])]


def _exact_conv(s):
    case = s["case"]
    train = "dy" in s
    w, b = (s[k].double().requires_grad_(train) for k in ("weight", "bias"))
    W = w.shape[0]
    y = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
    dx = torch.empty_like(y)
    states, dstates, dw, db = [], [], torch.zeros_like(w), torch.zeros_like(b)
    for n, (row, p, q) in enumerate(_spans(s)):
        wide = torch.cat((s["state0"][n], s["x"][row, p:q])).double().requires_grad_(train)
        z = (wide.unfold(0, W, 1) * w.t()).sum(-1) + b
        out = z / (1 + torch.exp(-z)) if case["silu"] else z
        last = wide[q - p:]
        y[row, p:q] = out.detach()
        states.append(last.detach())
        if train:
            cot = (s["dy"][row, p:q].double(), s["dstate"][n].double())
            gw, gww, gwb = torch.autograd.grad((out, last), (wide, w, b), cot)
            dstates.append(gw[:W - 1])
            dx[row, p:q] = gw[W - 1:]
            dw, db = dw + gww, db + gwb
    res = dict(y=y, state=torch.stack(states))
    return dict(res, dx=dx, dweight=dw.detach(), dbias=db.detach(), dstate0=torch.stack(dstates)) if train else res


def _exact_rec(s):
    case = s["case"]
    x, a = s["x"].double(), s["a"].double()
    alpha = 1 / (1 + torch.exp(-a)) if case["gate"] == "preact" else a
    rest = 1 / (1 + torch.exp(a)) if case["gate"] == "preact" else 1 - a
    u = rest * x if case["blend"] else x
    B, T, _ = x.shape
    h = torch.empty_like(x)
    prev = torch.empty_like(x)
    h_T = s["h0"].double()
    first, last = {}, {}
    spans = _spans(s)
    if s["cu"] is None:
        first[0], last[T - 1] = slice(None), slice(None)
    for n, (_, p, q) in enumerate(spans if s["cu"] is not None else []):
        if q > p:
            first[p], last[q - 1] = slice(n, n + 1), slice(n, n + 1)
    now = None
    for t in range(T):
        if t in first:
            now = s["h0"][first[t]].double()
        prev[:, t] = now
        now = torch.addcmul(u[:, t], alpha[:, t], now)
        h[:, t] = now
        if t in last:
            h_T[last[t]] = now
    out = dict(h=h, h_T=h_T)
    if "dh" not in s:
        return out
    lam = torch.empty_like(x)
    dh0 = s["dhT"].double()
    dh = s["dh"].double()
    for t in reversed(range(T)):
        if t in last:
            now = s["dhT"][last[t]].double()
        torch.add(dh[:, t], now, out=lam[:, t])
        now = alpha[:, t] * lam[:, t]
        if t in first:
            dh0[first[t]] = now
    da = lam * (prev - x if case["blend"] else prev)
    if case["gate"] == "preact":
        da = da * alpha * rest
    return dict(out, dx=lam * rest if case["blend"] else lam, da=da, dh0=dh0)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "ln":
        return _exact_ln(s)
    if op == "conv":
        return _exact_conv(s)
    if op == "rec":
        return _exact_rec(s)
    if op == "conv_step":
        wide = torch.cat((s["state"], s["x"][:, None]), 1).double()
        z = torch.einsum("bwd,wd->bd", wide, s["weight"].double()) + s["bias"].double()
        return dict(y=z / (1 + torch.exp(-z)) if case["silu"] else z, state=wide[:, 1:])
    a, x, h = s["a"].double(), s["x"].double(), s["state"].double()
    alpha = 1 / (1 + torch.exp(-a)) if case["gate"] == "preact" else a
    rest = 1 / (1 + torch.exp(a)) if case["gate"] == "preact" else 1 - a
    h = h * alpha + (x * rest if case["blend"] else x)
    return dict(h=h, state=h.clone())
