"""More operators around the mixer, as cases to measure: linear attention with a
decay for each head, group norm with an activation (channels last), and dropout
from a counter-based generator, forward, backward and, for the attention, as
single-token steps.

``own`` false computes a case in plain torch operations (fp32, rounded once at
the end), true makes the library's calls.  ``exact`` computes it in 64 bits from
the definition.  A step's state moves on by one token each pass, as in decoding.

  linear attention  S_t = g S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t, with g the
                    head's decay; a group of adjacent heads shares one q and k
  group norm        x [N, S, C]: (x - mean) rstd weight + bias over each sample's
                    positions and the channels of a group, then z or z sigmoid(z)
  dropout           element i is kept where its 16 random bits are at least
                    round(p 65536); what is kept is divided by the share kept.
                    The bits are word (i % 8) / 2, half i % 2, of Philox4x32-10
                    (Salmon, Moraes, Dror, Shaw 2011) at counter i / 8 (low words)
                    and offset (high words) under the key seed
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
MOST = 1 << 26  # elements of a drawn case's largest tensor
CHUNK = 64      # of the plain form


def listed():
    return [
        # decode: one token of 256 sequences
        dict(name="la step", op="la_step", B=256, H=16, Hk=16, dk=128, dv=128, io="bf16"),
        # the next 100 tokens of four running conversations: latency counts
        dict(name="la short prompt", op="la", train=False, B=4, T=100, H=16, Hk=16, dk=128, dv=128, io="bf16",
             state=True, seqs=0, end=0, fused=True),
        # prompts of 4096 tokens, q, k and v slices of one projection
        dict(name="la prompt", op="la", train=False, B=8, T=4096, H=16, Hk=16, dk=128, dv=128, io="bf16",
             state=False, seqs=0, end=0, fused=True),
        # training on one long sequence: few heads, the walk has to be split over time
        dict(name="la train long", op="la", train=True, B=1, T=65536, H=16, Hk=16, dk=128, dv=128, io="bf16",
             state=False, seqs=0, end=0, fused=False),
        # training on packed documents, four heads to a query and key
        dict(name="la train packed", op="la", train=True, B=1, T=32768, H=16, Hk=4, dk=64, dv=128, io="bf16",
             state=True, seqs=37, end=0, fused=False),
        # odd lengths and head sizes in fp32, nothing a multiple of a tile
        dict(name="la train odd fp32", op="la", train=True, B=2, T=2047, H=6, Hk=3, dk=72, dv=101, io="f32",
             state=True, seqs=0, end=0, fused=False),
        # decode: the heads of 256 tokens normalised
        dict(name="gn decode", op="gn", train=False, N=256, S=1, C=2048, G=16, io="bf16", silu=True),
        # training: the mixer's output normalised per head, B8 T4096
        dict(name="gn heads train", op="gn", train=True, N=8 * 4096, S=1, C=2048, G=16, io="bf16", silu=True),
        # training: frames or patches, statistics over 4096 positions
        dict(name="gn positions train", op="gn", train=True, N=16, S=4096, C=512, G=32, io="bf16", silu=True),
        # odd channels, groups and positions, fp32
        dict(name="gn odd fp32 train", op="gn", train=True, N=5, S=1021, C=333, G=9, io="f32", silu=False),
        # training: a block's output dropped and added to the residual stream, B8 T4096
        dict(name="dropout train", op="drop", train=True, rows=8 * 4096, D=2048, io="bf16", p=0.1, residual=True,
             fused=1),
        # odd width, fp32, no residual
        dict(name="dropout odd fp32", op="drop", train=True, rows=1021, D=1537, io="f32", p=0.5, residual=False,
             fused=1),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm spread evenly."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999))))))


def _width(rng, lo, hi):
    D = _spread(rng, lo, hi)
    kind = rng.random()
    return max(lo, D // 64 * 64) if kind < 0.5 else max(lo, D // 2 * 2) if kind < 0.7 else D


def _head(rng):
    """Channels of a head: a power of two, a multiple of 8, or any number."""
    kind = rng.random()
    return rng.choice([32, 64, 128, 256]) if kind < 0.6 else 8 * rng.randint(2, 32) if kind < 0.8 else rng.randint(8, 256)


def draw(rng):
    op = rng.choice(["la_step", "la", "la", "la", "gn", "gn", "drop"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op == "drop":
        D = _width(rng, 64, 16384)
        return dict(op=op, train=rng.random() < 0.5, rows=_spread(rng, 1, MOST // D), D=D, io=io,
                    p=rng.choice([0.0, 0.1, 0.25, 0.5, 0.9]), residual=rng.random() < 0.5, fused=rng.choice([1, 1, 2]))
    if op == "gn":
        G = rng.choice([1, 4, 8, 9, 16, 32])
        C = G * _spread(rng, 2, 4096 // G)
        S = 1 if rng.random() < 0.4 else _spread(rng, 2, min(16384, MOST // C))
        N = _spread(rng, 1, max(1, min(32768, MOST // C // S)))
        return dict(op=op, train=rng.random() < 0.6, N=N, S=S, C=C, G=G, io=io, silu=rng.random() < 0.6)
    Hk = _spread(rng, 1, 16)
    H = Hk * rng.choice([1, 1, 1, 2, 4])
    dk, dv = _head(rng), _head(rng)
    if rng.random() < 0.5:
        dv = dk
    if op == "la_step":
        return dict(op=op, B=_spread(rng, 1, max(1, min(1024, MOST // (H * dk * dv)))), H=H, Hk=Hk, dk=dk, dv=dv, io=io)
    train = rng.random() < 0.6
    most = MOST if io == "bf16" else MOST // 4
    T = _spread(rng, 1, min(65536, most // (H * max(dk, dv))))
    seqs = _spread(rng, 1, max(1, min(300, MOST // (H * dk * dv)))) if rng.random() < 0.4 else 0
    B = 1 if seqs else _spread(rng, 1, max(1, min(16, most // (H * max(dk, dv)) // T)))
    return dict(op=op, train=train, B=B, T=T, H=H, Hk=Hk, dk=dk, dv=dv, io=io, state=rng.random() < 0.5, seqs=seqs,
                end=rng.randint(0, T // 4) if seqs and rng.random() < 0.3 else 0, fused=rng.random() < 0.3)


def _dtype(case):
    return torch.bfloat16 if case["io"] == "bf16" else torch.float32


def _seqlens(case, g):
    """Offsets [N+1] of the packed sequences: N random cuts of all tokens but the
    last `end`, so that lengths run from zero to long; None where each row is one
    sequence."""
    if not case["seqs"]:
        return None
    T = case["T"] - case["end"]
    cuts = torch.randint(0, T + 1, (case["seqs"] - 1,), generator=g, device="cuda").sort().values
    ends = torch.tensor([0, T], device="cuda")
    return torch.cat((ends[:1], cuts, ends[1:])).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _dtype(case)

    def normal(*shape, dtype=torch.float32, scale=1.0, mean=0.0):
        return torch.randn(*shape, generator=g, device="cuda").mul_(scale).add_(mean).to(dtype)

    op = case["op"]
    s = dict(case=dict(case))
    if op == "drop":
        rows, D = case["rows"], case["D"]
        s["x"] = normal(rows, case["fused"] * D, dtype=dt)[:, (case["fused"] - 1) * D:]
        s["seed"] = int(seed) * 0x9E3779B97F4A7C15 % (1 << 64)
        s["offset"] = int(seed) % 1000
        if case["residual"]:
            s["residual"] = normal(rows, D, dtype=dt)
        if case["train"]:
            s["dy"] = normal(rows, D, dtype=dt)
        return s
    if op == "gn":
        N, S, C = case["N"], case["S"], case["C"]
        # channels of unequal scale around a mean that is not zero
        scale = torch.exp(normal(C, scale=0.5))
        s["x"] = normal(N, S, C).mul_(scale).add_(0.3).to(dt)
        s["weight"] = normal(C, scale=0.2, mean=1.0)
        s["bias"] = normal(C, scale=0.2)
        if case["train"]:
            s["dy"] = normal(N, S, C, dtype=dt)
        return s
    B, H, Hk, dk, dv = (case[n] for n in ("B", "H", "Hk", "dk", "dv"))
    # memories from a few tokens to some thousand, by head
    power = 1 + torch.arange(H, device="cuda") * (9.0 / max(H - 1, 1)) + torch.rand(H, generator=g, device="cuda")
    s["decay"] = 1 - torch.exp2(-power)
    if op == "la_step":
        s["q"], s["k"] = normal(B, Hk, dk, dtype=dt), normal(B, Hk, dk, dtype=dt)
        s["v"] = normal(B, H, dv, dtype=dt)
        s["state"] = normal(B, H, dk, dv)
        return s
    T = case["T"]
    N = case["seqs"] or B
    s["cu"] = _seqlens(case, g)
    if case["fused"]:
        wide = normal(B, T, 2 * Hk * dk + H * dv, dtype=dt)
        q, k, v = wide.split([Hk * dk, Hk * dk, H * dv], -1)
        s["q"], s["k"], s["v"] = q.unflatten(-1, (Hk, dk)), k.unflatten(-1, (Hk, dk)), v.unflatten(-1, (H, dv))
    else:
        s["q"], s["k"] = normal(B, T, Hk, dk, dtype=dt), normal(B, T, Hk, dk, dtype=dt)
        s["v"] = normal(B, T, H, dv, dtype=dt)
    s["S0"] = normal(N, H, dk, dv) if case["state"] else None
    if case["train"]:
        s["do"] = normal(B, T, H, dv, dtype=dt)
        s["dS"] = normal(N, H, dk, dv) if case["state"] else None
    return s


# ---- the library's calls ------------------------------------------------

def _own(s):
    import kalman_delta_rule_amd as kda
    case = s["case"]
    op = case["op"]
    if op == "drop":
        y = kda.kdn_dropout_fwd(s["x"], case["p"], s["seed"], s["offset"], residual=s.get("residual"))
        if not case["train"]:
            return dict(y=y)
        return dict(y=y, dx=kda.kdn_dropout_bwd(s["dy"], case["p"], s["seed"], s["offset"]))
    if op == "gn":
        act = "silu" if case["silu"] else None
        y, mean, rstd = kda.kdn_group_norm_fwd(s["x"], case["G"], s["weight"], s["bias"], eps=EPS, activation=act,
                                               want_stats=case["train"])
        if not case["train"]:
            return dict(y=y)
        g = kda.kdn_group_norm_bwd(s["dy"], s["x"], mean, rstd, s["weight"], s["bias"], activation=act)
        return dict(y=y, mean=mean, rstd=rstd, **g)
    if op == "la_step":
        o = kda.kdn_linattn_step(s["q"], s["k"], s["v"], s["decay"], s["state"])
        return dict(o=o, state=s["state"])
    o, S_T = kda.kdn_linattn_fwd(s["q"], s["k"], s["v"], s["decay"], S0=s["S0"], cu_seqlens=s["cu"], want_state=True)
    if not case["train"]:
        return dict(o=o, S_T=S_T)
    g = kda.kdn_linattn_bwd(s["do"], s["q"], s["k"], s["v"], s["decay"], S0=s["S0"], dS_T=s["dS"], cu_seqlens=s["cu"])
    return dict(o=o, S_T=S_T, **g)


# ---- the plain form ------------------------------------------------------

def _keep(n, p, seed, offset):
    """Which of n elements dropout keeps: bool [n]."""
    c0 = torch.arange(-(-n // 8), device="cuda")
    c1, c2, c3 = torch.zeros_like(c0), torch.full_like(c0, offset & 0xFFFFFFFF), torch.full_like(c0, offset >> 32)
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # 64-bit products: the wrapped sign does no harm
        c0, c1, c2, c3 = (((b >> 32) & 0xFFFFFFFF) ^ c1 ^ k0, b & 0xFFFFFFFF,
                          ((a >> 32) & 0xFFFFFFFF) ^ c3 ^ k1, a & 0xFFFFFFFF)
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    words = torch.stack((c0, c1, c2, c3), 1)
    bits = torch.stack((words & 0xFFFF, words >> 16), 2).reshape(-1)[:n]
    return bits >= round(p * 65536)


def _plain_drop(s, dt):
    case = s["case"]
    rows, D, p = case["rows"], case["D"], case["p"]
    keep = _keep(rows * D, p, s["seed"], s["offset"]).view(rows, D)
    scale = 65536 / max(65536 - round(p * 65536), 1)
    zero = torch.zeros((), device="cuda")
    y = torch.where(keep, s["x"].float() * scale, zero)
    if case["residual"]:
        y = y + s["residual"].float()
    out = dict(y=y.to(dt))
    if case["train"]:
        out["dx"] = torch.where(keep, s["dy"].float() * scale, zero).to(dt)
    return out


def _plain_gn(s, dt):
    case = s["case"]
    N, S, C = s["x"].shape
    shape = (N, S, case["G"], C // case["G"])
    x = s["x"].float().view(shape)
    mean = x.mean((1, 3), keepdim=True)
    rstd = torch.rsqrt((x - mean).square().mean((1, 3), keepdim=True) + EPS)
    xh = (x - mean) * rstd
    w, b = s["weight"].view(shape[2:]), s["bias"].view(shape[2:])
    z = xh * w + b
    y = (z * torch.sigmoid(z) if case["silu"] else z).to(dt).view(N, S, C)
    if not case["train"]:
        return dict(y=y)
    g = s["dy"].float().view(shape)
    if case["silu"]:
        p = torch.sigmoid(z)
        g = g * p * (1 + z * (1 - p))
    gw = g * w
    dx = (gw - gw.mean((1, 3), keepdim=True) - xh * (gw * xh).mean((1, 3), keepdim=True)) * rstd
    return dict(y=y, mean=mean.view(N, -1), rstd=rstd.view(N, -1), dx=dx.to(dt).view(N, S, C),
                dweight=(g * xh).sum((0, 1)).view(C), dbias=g.sum((0, 1)).view(C))


class _Chunks:
    """Every sequence cut into chunks of its own: where its tokens lie among the
    chunks, counted from its front or (back) from its end."""

    def __init__(self, case, cu, back):
        B, T, dev = case["B"], case["T"], "cuda"
        if cu is None:
            first = torch.arange(B, device=dev) * T
            end = first + T
            self.count = B * -(-T // CHUNK)  # a bound on the chunks that needs no look at the offsets
        else:
            first, end = cu[:-1].long(), cu[1:].long()
            self.count = -(-T // CHUNK) + first.numel()
        token = torch.arange(B * T, device=dev)
        seq = (torch.searchsorted(end, token, right=True)).clamp(max=first.numel() - 1)
        self.tokens = token < end[-1]
        pos = (end[seq] - 1 - token) if back else (token - first[seq])
        length = end - first
        chunks = (length + CHUNK - 1) // CHUNK
        base = chunks.cumsum(0) - chunks
        self.slot = torch.where(self.tokens, (base[seq] + pos // CHUNK) * CHUNK + pos % CHUNK, self.count * CHUNK)
        n = torch.arange(self.count, device=dev)
        self.seq = (torch.searchsorted(base + chunks, n, right=True)).clamp(max=first.numel() - 1)
        self.index = n - base[self.seq]
        self.live = n < chunks.sum()
        self.held = (length[self.seq] - self.index * CHUNK).clamp(0, CHUNK)
        self.length, self.N = length, first.numel()

    def lay(self, x):
        """[B,T,H,d] as [count, H, CHUNK, d] in fp32, zeros where no token is"""
        flat = x.flatten(0, 1).float()
        wide = flat.new_zeros(self.count * CHUNK + 1, *flat.shape[1:])
        wide[self.slot] = flat
        return wide[:-1].unflatten(0, (self.count, CHUNK)).transpose(1, 2)

    def back(self, y, shape):
        flat = y.transpose(1, 2).flatten(0, 1)
        flat = torch.cat((flat, flat.new_zeros(1, *flat.shape[1:])))
        return flat[self.slot].view(shape)


def _power(decay, n):
    """decay^n [H, ...] of the heads' decays and whole numbers n >= 0"""
    n = n.clamp(min=0)
    d = decay.double().view(-1, *[1] * n.dim())
    return torch.pow(d, n.double()).float()


def _plain_walk(c, q, k, v, decay, X0, late, of_p, of_x, of_u):
    """With X the state X0 at a sequence's front: y_i = of_x g^(i + 1 - late) X^T q_i
    + of_p sum_{j <= i} g^(i - j) (q_i k_j) v_j, and the state behind the sequence,
    of_u g^(L - 1 - j + late) k_j v_j^T summed and g^L X0 added."""
    Q, K, V = c.lay(q), c.lay(k), c.lay(v)
    i = torch.arange(CHUNK, device="cuda")
    D = _power(decay, i[:, None] - i) * (i[:, None] >= i)
    y = (Q @ K.transpose(-1, -2)) * (D * of_p) @ V
    w = _power(decay, c.held[:, None] - 1 - i + late).transpose(0, 1) * of_u
    U = (K * w[..., None]).transpose(-1, -2) @ V
    flat = U.transpose(0, 1).flatten(2)
    n = torch.arange(c.count, device="cuda")
    before = (c.seq[:, None] == c.seq) & (n < n[:, None]) & c.live
    M = _power(decay, CHUNK * (n[:, None] - 1 - n)) * before
    X = M @ flat
    mine = (torch.arange(c.N, device="cuda")[:, None] == c.seq) & c.live
    left = c.length[:, None] - c.index * CHUNK - c.held
    end = (_power(decay, left) * mine) @ flat
    if X0 is not None:
        first = X0.transpose(0, 1).flatten(2)
        X = X + _power(decay, CHUNK * c.index)[..., None] * first[:, c.seq]
        end = end + _power(decay, c.length)[..., None] * first
    X = X.unflatten(2, U.shape[2:]).transpose(0, 1)
    y = y + _power(decay, i + 1 - late)[..., None] * of_x * (Q @ X)
    return y, end.unflatten(2, U.shape[2:]).transpose(0, 1)


def _plain_la(s, dt):
    case = s["case"]
    H, Hk, dk = case["H"], case["Hk"], case["dk"]
    scale = dk ** -0.5
    q, k = (s[n].repeat_interleave(H // Hk, 2) for n in ("q", "k"))
    v, decay = s["v"], s["decay"]
    c = _Chunks(case, s["cu"], False)
    o, S_T = _plain_walk(c, q, k, v, decay, s["S0"], 0, scale, scale, 1.0)
    out = dict(o=c.back(o, v.shape).to(dt), S_T=S_T)
    if not case["train"]:
        return out
    do = s["do"]
    shared = lambda y: y.unflatten(2, (Hk, H // Hk)).sum(3).to(dt)
    S0 = None if s["S0"] is None else s["S0"].transpose(-1, -2)
    dS = None if s["dS"] is None else s["dS"].transpose(-1, -2)
    dq, _ = _plain_walk(c, do, v, k, decay, S0, 0, scale, scale, 1.0)
    dq = shared(c.back(dq, q.shape))
    c = _Chunks(case, s["cu"], True)
    dv, dS0 = _plain_walk(c, k, q, do, decay, s["dS"], 1, scale, 1.0, scale)
    dk_, _ = _plain_walk(c, v, do, q, decay, dS, 1, scale, 1.0, scale)
    out.update(dq=dq, dk=shared(c.back(dk_, q.shape)), dv=c.back(dv, v.shape).to(dt))
    if s["S0"] is not None:
        out["dS0"] = dS0
    return out


def _plain(s):
    case = s["case"]
    dt = _dtype(case)
    op = case["op"]
    if op == "drop":
        return _plain_drop(s, dt)
    if op == "gn":
        return _plain_gn(s, dt)
    if op == "la":
        return _plain_la(s, dt)
    q, k = (s[n].repeat_interleave(case["H"] // case["Hk"], 1).float() for n in ("q", "k"))
    s["state"] = s["state"] * s["decay"][:, None, None] + k[..., None] * s["v"].float()[..., None, :]
    o = (q[..., None] * s["state"]).sum(2) * case["dk"] ** -0.5
    return dict(o=o.to(dt), state=s["state"])


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    e = 2 if case["io"] == "bf16" else 4
    op = case["op"]
    if op == "drop":
        n = case["rows"] * case["D"]
        tensors = 2 + case["residual"] + (2 if case["train"] else 0)
        return dict(bytes=e * n * tensors, flops=(3 + (2 if case["train"] else 0)) * n)
    if op == "gn":
        n, stats = case["N"] * case["S"] * case["C"], 8 * case["N"] * case["G"]
        fwd = 2 * e * n + 8 * case["C"] + (stats if case["train"] else 0)
        bwd = 3 * e * n + stats + 16 * case["C"] if case["train"] else 0
        return dict(bytes=fwd + bwd, flops=(12 + (24 if case["train"] else 0)) * n)
    H, Hk, dk, dv = (case[n] for n in ("H", "Hk", "dk", "dv"))
    rows, state = 2 * Hk * dk + H * dv, 4 * H * dk * dv
    if op == "la_step":
        return dict(bytes=case["B"] * (e * (rows + H * dv) + 2 * state), flops=5 * case["B"] * H * dk * dv)
    tokens, N = case["B"] * case["T"] - case["end"], case["seqs"] or case["B"]
    fwd = e * tokens * (rows + H * dv) + N * state * (2 if case["state"] else 1)
    flops = 4 * tokens * H * dk * dv
    if not case["train"]:
        return dict(bytes=fwd, flops=flops)
    bwd = e * tokens * (2 * rows + H * dv) + (3 * N * state if case["state"] else 0)
    return dict(bytes=fwd + bwd, flops=flops + 10 * tokens * H * dk * dv)


# ---- 64 bits, from the definitions ---------------------------------------

def _exact_drop(s):
    case = s["case"]
    rows, D = case["rows"], case["D"]
    n = rows * D
    low = np.uint64(0xFFFFFFFF)
    half = np.uint64(32)
    c = [np.arange((n + 7) // 8, dtype=np.uint64), np.uint64(0), np.uint64(s["offset"]) & low,
         np.uint64(s["offset"]) >> half]
    key = [s["seed"] & 0xFFFFFFFF, s["seed"] >> 32]
    for _ in range(10):
        m0, m1 = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(m1 >> half) ^ c[1] ^ np.uint64(key[0]), m1 & low, (m0 >> half) ^ c[3] ^ np.uint64(key[1]), m0 & low]
        key = [(key[0] + 0x9E3779B9) % (1 << 32), (key[1] + 0xBB67AE85) % (1 << 32)]
    u = np.empty((c[0].size, 8), dtype=np.uint16)
    for j in range(8):
        u[:, j] = c[j // 2] >> np.uint64(16 * (j % 2)) & np.uint64(0xFFFF)
    least = round(case["p"] * 65536)
    keep = torch.from_numpy((u.reshape(-1)[:n].astype(np.int32) >= least).reshape(rows, D)).cuda()
    share = (65536 - least) / 65536
    none = torch.zeros((), dtype=torch.float64, device="cuda")
    y = torch.where(keep, s["x"].double() / share, none)
    if case["residual"]:
        y = y + s["residual"].double()
    return dict(y=y, dx=torch.where(keep, s["dy"].double() / share, none)) if case["train"] else dict(y=y)


def _exact_gn(s):
    case = s["case"]
    N, S, C = s["x"].shape
    G, train = case["G"], case["train"]
    x, w, b = (s[n].double().requires_grad_(train) for n in ("x", "weight", "bias"))
    groups = x.view(N, S, G, C // G).transpose(1, 2).flatten(2)
    var, mean = torch.var_mean(groups, dim=-1, correction=0, keepdim=True)
    rstd = (var + EPS) ** -0.5
    z = ((groups - mean) * rstd).view(N, G, S, C // G).transpose(1, 2).reshape(N, S, C) * w + b
    y = z / (1 + torch.exp(-z)) if case["silu"] else z
    if not train:
        return dict(y=y)
    dx, dw, db = torch.autograd.grad(y, (x, w, b), s["dy"].double())
    return dict(y=y.detach(), mean=mean[..., 0].detach(), rstd=rstd[..., 0].detach(), dx=dx, dweight=dw, dbias=db)


def _exact_la(s):
    """The recurrence written out as sums over pairs of tokens, sequence by sequence and
    a block of readers i at a time: o_i = scale sum_{j <= i} g^(i - j) (q_i k_j) v_j and
    what the states before and behind add; its gradients likewise."""
    case = s["case"]
    H, Hk, dk, dv = (case[n] for n in ("H", "Hk", "dk", "dv"))
    G, scale = H // Hk, case["dk"] ** -0.5
    B, T = case["B"], case["T"]
    N, train = case["seqs"] or B, case["train"]
    heads = lambda x: x.double().transpose(0, 1).contiguous()  # [H, L, d]
    # g^n for n = T .. -T, zero below n = 0: row i of the decays between tokens is a piece of it
    n = torch.arange(T, -T - 1, -1, device="cuda", dtype=torch.float64)
    powers = s["decay"].double()[:, None] ** n.clamp(min=0) * (n >= 0)
    power = lambda lo, hi: powers[:, T - hi + 1:T - lo + 1].flip(1)[..., None]  # g^lo .. g^(hi - 1), [H, hi - lo, 1]
    new = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device="cuda")
    S0 = new(N, H, dk, dv) if s["S0"] is None else s["S0"].double()
    o, S_T = new(B, T, H, dv), S0.clone()
    if train:
        dS = new(N, H, dk, dv) if s["dS"] is None else s["dS"].double()
        dq, dk_, dv_, dS0 = new(B, T, H, dk), new(B, T, H, dk), new(B, T, H, dv), dS.clone()
    at = s["cu"].tolist() if s["cu"] is not None else None
    for m in range(N):
        row, p, e = (m, 0, T) if at is None else (0, at[m], at[m + 1])
        L = e - p
        if not L:
            continue
        q, k = (heads(s[x][row, p:e].repeat_interleave(G, 1)) for x in ("q", "k"))
        v = heads(s["v"][row, p:e])
        front, tail = power(1, L + 1), power(0, L).flip(1)
        gL = powers[:, T - L, None, None]
        S_T[m] = gL * S0[m] + (k * tail).transpose(1, 2) @ v
        O = scale * front * (q @ S0[m])
        if train:
            w = heads(s["do"][row, p:e])
            dS0[m] = gL * dS[m] + scale * (q * front).transpose(1, 2) @ w
            dQ = scale * front * (w @ S0[m].transpose(1, 2))
            dK, dV = tail * (v @ dS[m].transpose(1, 2)), tail * (k @ dS[m])
        for i in range(0, L, 512):
            I, J = slice(i, min(i + 512, L)), slice(0, min(i + 512, L))
            rows, cols = I.stop - i, J.stop
            # D[h, a, j] = g^(i + a - j), which stands at T - i - a + j of `powers`
            D = scale * torch.as_strided(powers, (H, rows, cols), (2 * T + 1, 1, 1), T - i - rows + 1).flip(1)
            A = q[:, I] @ k[:, J].transpose(1, 2) * D
            O[:, I] += A @ v[:, J]
            if train:
                dV[:, J] += A.transpose(1, 2) @ w[:, I]
                A = w[:, I] @ v[:, J].transpose(1, 2) * D
                dQ[:, I] += A @ k[:, J]
                dK[:, J] += A.transpose(1, 2) @ q[:, I]
        o[row, p:e] = O.transpose(0, 1)
        if train:
            for to, x in ((dq, dQ), (dk_, dK), (dv_, dV)):
                to[row, p:e] = x.transpose(0, 1)
    out = dict(o=o, S_T=S_T)
    if train:
        out.update(dq=dq.unflatten(2, (Hk, G)).sum(3), dk=dk_.unflatten(2, (Hk, G)).sum(3), dv=dv_)
        if s["S0"] is not None:
            out["dS0"] = dS0
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "drop":
        return _exact_drop(s)
    if op == "gn":
        return _exact_gn(s)
    if op == "la":
        return _exact_la(s)
    G = case["H"] // case["Hk"]
    q, k = (s[n].repeat_interleave(G, 1).double() for n in ("q", "k"))
    S = s["decay"].double()[:, None, None] * s["state"].double() + torch.einsum("bhi,bhj->bhij", k, s["v"].double())
    return dict(o=torch.einsum("bhij,bhi->bhj", S, q) * case["dk"] ** -0.5, state=S)
