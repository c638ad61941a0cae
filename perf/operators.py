"""Cases of the scalar-gated delta rule and of sliding-window attention with sink tokens.

The two mixers of a hybrid recurrent / local-attention stack, each in training (forward and
gradients), prefill (a batch or packed prompts, ending in the state that decoding starts from)
and decoding (one token per sequence, state updated in place).  `run` computes them in plain
torch operations in fp32, or, where `own` is true, through the library's entry points.

Layouts: tokens [B, T, heads, channels], or [rows, heads, channels] for sequences packed along
the token axis; recurrent state [B, H, dv, dk]; cache of the window [B, sinks + window, H, d].
"""
import math

import torch

own = False

CHUNK = 64   # tokens that the plain delta rule handles at once


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # one request decoding alone: launch latency is all there is
        dict(name="delta_step_1", op="delta", use="step", B=1, Hk=16, Hv=16, d=128, dtype="bf16", decay=False),
        # a full decoding batch of the 16-head layer: the fp32 states stream through once
        dict(name="delta_step_256", op="delta", use="step", B=256, Hk=16, Hv=16, d=128, dtype="bf16", decay=False),
        # a batch of equal prompts through the 16-head layer
        dict(name="delta_prefill_4x2048", op="delta", use="prefill", B=4, T=2048, Hk=16, Hv=16, d=128, dtype="bf16",
             decay=False, S0=False, lens=""),
        # packed prompts that continue from kept states; key heads shared by two value heads; the
        # decay with its amplitude and bias; an empty and a one-token sequence among them
        dict(name="delta_prefill_packed", op="delta", use="prefill", B=9, T=2333, Hk=8, Hv=16, d=128, dtype="bf16",
             decay=True, S0=True, lens="577,1,0,2333,64,129,1024,63,1500"),
        # the training step of the 16-head layer
        dict(name="delta_train_8x4096", op="delta", use="train", B=8, T=4096, Hk=16, Hv=16, d=128, dtype="bf16",
             decay=False, S0=False, lens=""),
        # a small fp32 model in a parity run, odd length, shared key head
        dict(name="delta_train_fp32", op="delta", use="train", B=1, T=257, Hk=1, Hv=2, d=64, dtype="fp32",
             decay=False, S0=False, lens=""),
        # one request decoding alone
        dict(name="window_step_1", op="window", use="step", B=1, Hq=16, Hkv=4, d=128, window=512, sinks=4,
             dtype="bf16", reach=3.0),
        # a full decoding batch, positions from the first token to far beyond the window
        dict(name="window_step_256", op="window", use="step", B=256, Hq=16, Hkv=4, d=128, window=1024, sinks=4,
             dtype="bf16", reach=16.0),
        # a batch of equal prompts, and the cache that decoding starts from
        dict(name="window_prefill_4x2048", op="window", use="prefill", B=4, T=2048, Hq=16, Hkv=4, d=128, window=512,
             sinks=4, dtype="bf16", lens=""),
        # packed prompts of odd lengths, an odd window, 64 channels
        dict(name="window_prefill_packed", op="window", use="prefill", B=7, T=2047, Hq=12, Hkv=4, d=64, window=301,
             sinks=7, dtype="bf16", lens="1000,1,0,2047,300,777,65"),
        # the training step of the local-attention layer beside the 16-head recurrent ones
        dict(name="window_train_8x4096", op="window", use="train", B=8, T=4096, Hq=16, Hkv=4, d=128, window=1024,
             sinks=4, dtype="bf16", lens=""),
        # a small fp32 model in a parity run, odd length and window
        dict(name="window_train_fp32", op="window", use="train", B=2, T=333, Hq=4, Hkv=2, d=64, window=100, sinks=3,
             dtype="fp32", lens=""),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["delta", "window"])
    use = rng.choice(["step", "prefill", "train"])
    d = rng.choice([64, 128, 128])
    dtype = "fp32" if rng.random() < 0.2 else "bf16"
    heads = rng.choice([1, 2, 4, 8])
    share = rng.choice([1, 2, 4])
    if use == "step":
        B = _log_int(rng, 1, 256 if heads * share <= 16 else 128)
        if op == "delta":
            return dict(op=op, use=use, B=B, Hk=heads, Hv=heads * share, d=d, dtype=dtype, decay=rng.random() < 0.5)
        return dict(op=op, use=use, B=B, Hq=heads * share, Hkv=heads, d=d, window=_log_int(rng, 16, 1024),
                    sinks=rng.choice([0, 1, 4, 7, 16]), dtype=dtype, reach=round(rng.uniform(0.3, 8.0), 2))
    # rows x heads stay below the largest listed case's; fp32 is for small models
    most = (1 << 19) if dtype == "bf16" else (1 << 13)
    if use == "train":
        most //= 4
    rows = _log_int(rng, 33, min(32768, max(64, most // (heads * share))))
    packed = use == "prefill" and rng.random() < 0.5
    lens = ""
    if packed:
        B = rng.randint(2, 12)
        cuts = sorted(rng.randint(0, rows) for _ in range(B - 1))
        ls = [b - a for a, b in zip([0] + cuts, cuts + [rows])]
        T, lens = max(ls), ",".join(map(str, ls))
    else:
        B = rng.choice([1, 1, 2, 3, 4, 8])
        T = max(1, rows // B)
    if op == "delta":
        return dict(op=op, use=use, B=B, T=T, Hk=heads, Hv=heads * share, d=d, dtype=dtype,
                    decay=use == "prefill" and rng.random() < 0.5, S0=use == "prefill" and rng.random() < 0.5,
                    lens=lens)
    return dict(op=op, use=use, B=B, T=T, Hq=heads * share, Hkv=heads, d=d, window=_log_int(rng, 16, 2048),
                sinks=rng.choice([0, 1, 4, 7, 16]), dtype=dtype, lens=lens)


def _lens(c):
    return [int(x) for x in c["lens"].split(",")] if c["lens"] else [c["T"]] * c["B"]


def _positions(c):
    """Tokens that each sequence of a decoding batch already has: spread evenly over
    0 .. reach * window."""
    top = int(c["reach"] * c["window"])
    return [top if c["B"] == 1 else top * b // (c["B"] - 1) for b in range(c["B"])]


def _pairs(T, window, sinks):
    """(query, key) pairs that a sequence of T tokens has."""
    n = min(T, window)
    near = n * (n + 1) // 2 + max(0, T - window) * window
    far = sum(max(0, min(sinks, i - window + 1)) for i in range(window, min(T, window + sinks)))
    return near + far + max(0, T - window - sinks) * sinks


def work(c):
    e = 2 if c["dtype"] == "bf16" else 4
    d = c["d"]
    if c["op"] == "delta":
        Hk, Hv = c["Hk"], c["Hv"]
        if c["use"] == "step":
            state = c["B"] * Hv * d * d
            return {"bytes": 8 * state + e * c["B"] * (2 * Hk * d + 2 * Hv * d + 2 * Hv), "flops": 7 * state}
        rows = sum(_lens(c))
        # per token and value head, chunks of L tokens in WY form: 6 d^2 for the three products
        # with the state, 5 L d for the products within the chunk, L^2 / 3 for the solve
        flops = rows * Hv * (6 * d * d + 5 * CHUNK * d + CHUNK * CHUNK // 3)
        io = e * rows * (2 * Hk * d + 2 * Hv * d + 2 * Hv)
        if c["use"] == "prefill":
            return {"bytes": io + 4 * c["B"] * Hv * d * d * (2 if c["S0"] else 1), "flops": flops}
        grads = e * rows * (2 * Hk * d + 2 * Hv * d + 2 * Hv)
        return {"bytes": io + grads, "flops": flops + rows * Hv * (14 * d * d + 14 * CHUNK * d + CHUNK * CHUNK)}
    Hq, Hkv, W, s = c["Hq"], c["Hkv"], c["window"], c["sinks"]
    if c["use"] == "step":
        keys = sum(min(p + 1, W) + min(s, max(0, p + 1 - W)) for p in _positions(c))
        return {"bytes": 2 * e * keys * Hkv * d + e * c["B"] * d * (2 * Hq + 4 * Hkv), "flops": 4 * keys * Hq * d}
    lens = _lens(c)
    rows, pairs = sum(lens), sum(_pairs(T, W, s) for T in lens)
    if c["use"] == "prefill":
        kept = sum(min(T, W + s) for T in lens)
        return {"bytes": e * d * (rows * (2 * Hq + 2 * Hkv) + 2 * kept * Hkv), "flops": 4 * pairs * Hq * d}
    # training: q, k, v, dO read, o and three gradients written; 4 + 10 flops a pair and channel
    return {"bytes": e * rows * d * (4 * Hq + 4 * Hkv), "flops": 14 * pairs * Hq * d}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _unit(x):
    return x / x.square().sum(-1, keepdim=True).sqrt()


def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32

    def normal(*shape, scale=1.0, shift=0.0):
        return torch.randn(*shape, generator=gen, device="cuda") * scale + shift

    B, d = c["B"], c["d"]
    st = dict(case=c)
    lead = (B,)
    if c["use"] != "step":
        lens = _lens(c)
        lead = (sum(lens),) if c["lens"] else (B, c["T"])
        st["cu"] = None
        if c["lens"]:
            st["cu"] = torch.tensor([sum(lens[:n]) for n in range(B + 1)], dtype=torch.int32, device="cuda")
            st["max_len"] = max(lens)
    if c["op"] == "delta":
        Hk, Hv = c["Hk"], c["Hv"]
        st["q"] = _unit(normal(*lead, Hk, d)).to(dt)
        st["k"] = _unit(normal(*lead, Hk, d)).to(dt)
        st["v"] = normal(*lead, Hv, d).to(dt)
        st["g"] = normal(*lead, Hv, scale=0.5, shift=-3.0).to(dt)
        st["w"] = normal(*lead, Hv).to(dt)
        st["A_dec"] = st["tau"] = st["S0"] = None
        if c.get("decay"):
            st["A_dec"] = (0.5 + 1.5 * torch.rand(Hv, generator=gen, device="cuda")).log()
            st["tau"] = normal(Hv, scale=0.5)
        if c["use"] == "step" or c["S0"]:
            st["S0"] = normal(B, Hv, d, d, scale=0.05)
        if c["use"] == "train":
            st["dO"] = normal(*lead, Hv, d).to(dt)
        return st
    Hq, Hkv, slots = c["Hq"], c["Hkv"], c["sinks"] + c["window"]
    st["q"] = normal(*lead, Hq, d).to(dt)
    st["k"] = normal(*lead, Hkv, d).to(dt)
    st["v"] = normal(*lead, Hkv, d).to(dt)
    if c["use"] == "step":
        st["k_cache"] = normal(B, slots, Hkv, d).to(dt)
        st["v_cache"] = normal(B, slots, Hkv, d).to(dt)
        st["pos"] = torch.tensor(_positions(c), dtype=torch.int64, device="cuda")
    elif c["use"] == "prefill":
        st["k_cache"] = torch.zeros(B, slots, Hkv, d, dtype=dt, device="cuda")
        st["v_cache"] = torch.zeros(B, slots, Hkv, d, dtype=dt, device="cuda")
    else:
        st["dO"] = normal(*lead, Hq, d).to(dt)
    return st


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------
def _log_decay(g, A_dec, tau):
    x = g if tau is None else g + tau
    soft = x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))
    return -soft if A_dec is None else -torch.exp(A_dec) * soft


def _padded(st):
    """(rows of the packed tensors [N, T], which of them are tokens) of a packed call."""
    cu = st["cu"].long()
    at = torch.arange(max(1, st["max_len"]), device="cuda")
    there = at < (cu[1:] - cu[:-1])[:, None]
    return torch.where(there, cu[:-1, None] + at, 0), there


def _delta_plain(q, k, v, g, w, S):
    """Chunked WY form in fp32: q, k, v [N, T, H, d], log decay g and write strength w [N, T, H],
    state S [N, H, dv, dk].  Returns the outputs and the last state."""
    N, T, H, d = v.shape
    C = min(CHUNK, 1 << max(0, T - 1).bit_length())
    n = -(-T // C)

    def chunks(x):   # [N, T, H, ...] -> [n, N, H, C, ...]; rows past the end are zero: inert
        x = torch.cat([x, x.new_zeros(N, n * C - T, *x.shape[2:])], 1)
        return x.unflatten(1, (n, C)).movedim(1, 0).movedim(3, 2).contiguous()

    q, k, v, g, w = (chunks(x) for x in (q, k, v, g, w))
    G = g.cumsum(-1)
    low = torch.ones(C, C, dtype=torch.bool, device="cuda").tril()
    decay = torch.where(low, G[..., :, None] - G[..., None, :], -math.inf).exp()
    X = -(w[..., None] * decay * (k @ k.transpose(-1, -2))).tril(-1)
    eye = torch.eye(C, device="cuda")
    inv, step = eye + X, 2            # (I - X)^-1 = (I + X)(I + X^2)(I + X^4) ...
    while step < C:
        X = X @ X
        inv = inv + inv @ X
        step *= 2
    eG = G.exp()[..., None]
    W, U0 = inv @ (w[..., None] * eG * k), inv @ (w[..., None] * v)
    A = decay * (q @ k.transpose(-1, -2))
    qd, kd, last = q * eG, k * (G[..., -1:] - G).exp()[..., None], G[..., -1].exp()[..., None, None]
    outs = []
    for c in range(n):
        U = U0[c] - W[c] @ S.transpose(-1, -2)
        outs.append(qd[c] @ S.transpose(-1, -2) + A[c] @ U)
        S = last[c] * S + U.transpose(-1, -2) @ kd[c]
    return torch.stack(outs).movedim(2, 3).movedim(0, 1).flatten(1, 2)[:, :T], S


def _delta_run(st):
    c = st["case"]
    Hk, Hv, d = c["Hk"], c["Hv"], c["d"]
    step, packed = c["use"] == "step", c["use"] != "step" and st["cu"] is not None
    xs = [st[x].float() for x in ("q", "k", "v", "g", "w")]
    leaves = None
    if c["use"] == "train":
        leaves = [x.detach().requires_grad_() for x in xs]
        xs = list(leaves)
    q, k, v, g, w = xs
    q, k = (x.repeat_interleave(Hv // Hk, -2) for x in (q, k))
    g, w = _log_decay(g, st["A_dec"], st["tau"]), torch.sigmoid(w)
    if step:
        S = st["S0"] * g.exp()[..., None, None]
        u = w[..., None] * (v - (S * k[..., None, :]).sum(-1))
        S = S + u[..., None] * k[..., None, :]
        st["S0"].copy_(S)
        return (S * q[..., None, :]).sum(-1).to(st["q"].dtype), st["S0"]
    if packed:
        rows, there = _padded(st)
        q, k, v, g, w = (torch.where(there.reshape(there.shape + (1,) * (x.dim() - 1)), x[rows], 0.0)
                         for x in (q, k, v, g, w))
    S = st["S0"] if st["S0"] is not None else torch.zeros(c["B"], Hv, d, d, device="cuda")
    o, S = _delta_plain(q, k, v, g, w, S)
    if c["use"] == "prefill":
        return (o[there] if packed else o).to(st["q"].dtype), S
    grads = torch.autograd.grad(o, leaves, st["dO"].float())
    return (o.detach().to(st["q"].dtype),) + tuple(x.to(st["q"].dtype) for x in grads)


def _window_plain(q, k, v, window, sinks, first, seq, scale):
    """q, k, v [N, T, H, d] fp32; row t belongs to sequence seq[N, T] whose first row is
    first[N, T].  Queries in blocks of `size` see their own and the previous blocks that the
    window reaches; sinks beyond the window are gathered."""
    N, T, H, d = q.shape
    size = 1 << (max(16, min(window, T)) - 1).bit_length()
    n, back = -(-T // size), -(-(window - 1) // size)
    pad = n * size - T

    def blocks(x, fill=0):   # [N, T, ...] -> [N, n, size, ...]
        return torch.cat([x, x.new_full((N, pad) + x.shape[2:], fill)], 1).unflatten(1, (n, size))

    def reach(x, fill=0):    # [N, n, size, ...] -> [N, n, (back + 1) size, ...]: blocks n - back .. n
        x = torch.cat([x.new_full((N, back) + x.shape[2:], fill), x], 1)
        return torch.cat([x[:, j:j + n] for j in range(back + 1)], 2)

    qb, kb, vb = blocks(q), reach(blocks(k)), reach(blocks(v))
    at = torch.arange(n * size, device="cuda").reshape(1, n, size).expand(N, n, size)
    sq, sk = blocks(seq, -1), reach(blocks(seq, -2), -2)
    gap = at[..., :, None] - reach(at)[..., None, :]
    seen = (gap >= 0) & (gap < window) & (sq[..., :, None] == sk[..., None, :])
    s = torch.einsum("nbihd,nbjhd->nbhij", qb, kb) * scale
    s = torch.where(seen[:, :, None], s, -math.inf)
    vs = None
    if sinks:
        far = first[..., None] + torch.arange(sinks, device="cuda")                     # [N, T, sinks]
        out = torch.arange(T, device="cuda")[None, :, None] - far >= window
        far = torch.where(out, far, 0)
        batch = torch.arange(N, device="cuda")[:, None, None]
        vs = blocks(v[batch, far])
        ss = torch.einsum("nbihd,nbishd->nbhis", qb, blocks(k[batch, far])) * scale
        s = torch.cat([s, torch.where(blocks(out, False)[:, :, None], ss, -math.inf)], -1)
    m = s.amax(-1, keepdim=True).detach()
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    J = (back + 1) * size
    o = torch.einsum("nbhij,nbjhd->nbihd", p[..., :J], vb)
    if sinks:
        o = o + torch.einsum("nbhis,nbishd->nbihd", p[..., J:], vs)
    return o.flatten(1, 2)[:, :T]


def _cache_rows(c, cu, lens):
    """(sequence, slot, row) of the tokens that the caches keep after a prompt."""
    W, s = c["window"], c["sinks"]
    at = torch.arange(max(1, c["T"]), device="cuda")
    keep = (at < lens[:, None]) & ((at < s) | (at >= lens[:, None] - W))
    n, t = keep.nonzero(as_tuple=True)
    return n, torch.where(t < s, t, s + (t - s) % W), cu[n] + t


def _window_run(st):
    c = st["case"]
    G, W, s, scale = c["Hq"] // c["Hkv"], c["window"], c["sinks"], c["d"] ** -0.5
    dt = st["q"].dtype
    if c["use"] == "step":
        pos = st["pos"]
        rows = torch.arange(c["B"], device="cuda")
        slot = torch.where(pos < s, pos, s + (pos - s) % W)
        st["k_cache"][rows, slot] = st["k"]
        st["v_cache"][rows, slot] = st["v"]
        at = torch.arange(s + W, device="cuda")
        token = torch.where(at < s, at, pos[:, None] - (pos[:, None] - at) % W)   # the newest token of each slot
        seen = (token <= pos[:, None]) & ((at < s) | (token >= s))
        q = st["q"].float().unflatten(1, (c["Hkv"], G))
        p = torch.einsum("bhgd,bjhd->bhgj", q, st["k_cache"].float()) * scale
        p = torch.where(seen[:, None, None], p, -math.inf)
        p = torch.exp(p - p.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
        o = torch.einsum("bhgj,bjhd->bhgd", p, st["v_cache"].float())
        return o.flatten(1, 2).to(dt), st["k_cache"], st["v_cache"]
    packed = st["cu"] is not None
    xs = [st[x].float() for x in ("q", "k", "v")]
    xs = [x[None] for x in xs] if packed else xs
    leaves = None
    if c["use"] == "train":
        leaves = [x.detach().requires_grad_() for x in xs]
        xs = list(leaves)
    q, k, v = xs
    N, T = q.shape[:2]
    if packed:
        cu = st["cu"].long()
        at = torch.arange(T, device="cuda")
        seq = torch.searchsorted(cu, at, right=True)[None] - 1
        first = cu[seq]
    else:
        cu = torch.arange(N, device="cuda") * T
        seq = first = torch.zeros(N, T, dtype=torch.int64, device="cuda")
    o = _window_plain(q, k.repeat_interleave(G, 2), v.repeat_interleave(G, 2), W, s, first, seq, scale)
    if c["use"] == "prefill":
        lens = cu[1:] - cu[:-1] if packed else torch.full((N,), T, device="cuda")
        n, slot, row = _cache_rows(c, cu, lens)
        st["k_cache"][n, slot] = st["k"].flatten(0, -3)[row]
        st["v_cache"][n, slot] = st["v"].flatten(0, -3)[row]
        return (o[0] if packed else o).to(dt), st["k_cache"], st["v_cache"]
    grads = torch.autograd.grad(o, leaves, st["dO"].float())
    return (o.detach().to(dt),) + tuple(x.to(dt) for x in grads)


# ---------------------------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------------------------
def _own(st):
    import chunk_gated_delta_b200 as carve
    c = st["case"]
    if c["op"] == "delta":
        x = (st["q"], st["k"], st["v"], st["g"], st["w"])
        more = dict(A_dec=st["A_dec"], tau=st["tau"])
        if c["use"] == "step":
            return carve.carve_gdr_step(*x, st["S0"], **more), st["S0"]
        more["cu_seqlens"] = st["cu"]
        if c["use"] == "prefill":
            out = carve.carve_gdr_fwd(*x, S0=st["S0"], save_for_bwd=False, **more)
            return out["o"], out["S_final"]
        out = carve.carve_gdr_fwd(*x, **more)
        g = carve.carve_gdr_bwd(*x, out["saved"], st["dO"], want_dS0=False, **more)
        return out["o"], g["dq"], g["dk"], g["dv"], g["dg_logit"], g["dw_logit"]
    x = (st["q"], st["k"], st["v"])
    at = dict(window=c["window"], sinks=c["sinks"])
    if c["use"] == "step":
        return carve.carve_swa_step(*x, st["k_cache"], st["v_cache"], st["pos"], **at), st["k_cache"], st["v_cache"]
    at["cu_seqlens"] = st["cu"]
    if c["use"] == "prefill":
        out = carve.carve_swa_fwd(*x, want_lse=False, **at)
        carve.carve_swa_fill(st["k"], st["v"], st["k_cache"], st["v_cache"], **at)
        return out["o"], st["k_cache"], st["v_cache"]
    out = carve.carve_swa_fwd(*x, **at)
    g = carve.carve_swa_bwd(*x, out["o"], out["lse"], st["dO"], **at)
    return out["o"], g["dq"], g["dk"], g["dv"]


def run(st):
    if own:
        return _own(st)
    return _delta_run(st) if st["case"]["op"] == "delta" else _window_run(st)


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------
def _token_by_token(q, k, v, a, w, S, dO=None):
    """The recurrence as it is written, in fp64: q, k, v [T, N, d], retention a and write
    strength w [T, N], state S [N, dv, dk].  With dO, the gradients too (states of every 64th
    token kept, those between computed again)."""
    T = len(q)
    o = torch.empty_like(v)
    kept = []

    def step(S, t):
        old = torch.einsum("nvk,nk->nv", S, k[t]) * a[t][:, None]
        u = w[t][:, None] * (v[t] - old)
        return torch.baddbmm(S * a[t][:, None, None], u[:, :, None], k[t][:, None, :]), u

    for t in range(T):
        if dO is not None and t % 64 == 0:
            kept.append(S)
        S, _ = step(S, t)
        o[t] = torch.bmm(S, q[t][:, :, None])[..., 0]
    if dO is None:
        return o, S
    dq, dk, dv, da, dw = (torch.empty_like(x) for x in (q, k, v, a, w))
    dS = torch.zeros_like(S)
    for part in reversed(range(len(kept))):
        states, us = [kept.pop()], []
        here = range(part * 64, min(T, part * 64 + 64))
        for t in here:
            S, u = step(states[-1], t)
            states.append(S)
            us.append(u)
        for t in reversed(here):
            after, before, u = states.pop(), states[-1], us.pop()
            dq[t] = torch.bmm(dO[t][:, None, :], after)[:, 0]
            dS = torch.baddbmm(dS, dO[t][:, :, None], q[t][:, None, :])
            du = torch.bmm(dS, k[t][:, :, None])[..., 0]
            kS = torch.bmm(before, k[t][:, :, None])[..., 0]
            e = w[t][:, None] * du                       # gradient of v - a S k
            dk[t] = torch.bmm(u[:, None, :], dS)[:, 0] - a[t][:, None] * torch.bmm(e[:, None, :], before)[:, 0]
            dv[t] = e
            dw[t] = (du * (v[t] - a[t][:, None] * kS)).sum(-1)
            da[t] = (dS * before).sum((-1, -2)) - (e * kS).sum(-1)
            dS = torch.baddbmm(a[t][:, None, None] * dS, (-a[t][:, None] * e)[:, :, None], k[t][:, None, :])
    return o, dq, dk, dv, da, dw


def _delta_exact(st):
    c = st["case"]
    B, Hk, Hv, d = c["B"], c["Hk"], c["Hv"], c["d"]
    q, k, v, g, w = (st[x].double() for x in ("q", "k", "v", "g", "w"))
    share = Hv // Hk
    x = g if st["tau"] is None else g + st["tau"].double()
    amp = 1.0 if st["A_dec"] is None else st["A_dec"].double().exp()
    a, ws = torch.exp(-amp * torch.logaddexp(x, torch.zeros_like(x))), 1 / (1 + torch.exp(-w))
    q, k = q.repeat_interleave(share, -2), k.repeat_interleave(share, -2)
    S = torch.zeros(B, Hv, d, d, dtype=torch.float64, device="cuda") if st["S0"] is None else st["S0"].double()
    S = S.reshape(B * Hv, d, d)
    if c["use"] == "step":
        o, S = _token_by_token(*(y.reshape((1, B * Hv) + y.shape[2:]) for y in (q, k, v, a, ws)), S)
        return o.reshape(B, Hv, d), S.reshape(B, Hv, d, d)
    if c["lens"]:
        o, last, row = torch.empty_like(v), S.reshape(B, Hv, d, d).clone(), 0
        for n, T in enumerate(_lens(c)):
            o[row:row + T], last[n] = _token_by_token(*(y[row:row + T] for y in (q, k, v, a, ws)), last[n])
            row += T
        return o, last

    def lay(y):   # [B, T, H, ...] -> [T, B H, ...]
        return y.transpose(0, 1).flatten(1, 2).contiguous()

    def back(y):
        return y.unflatten(1, (B, Hv)).transpose(0, 1)

    xs = [lay(y) for y in (q, k, v, a, ws)]
    if c["use"] == "prefill":
        o, S = _token_by_token(*xs, S)
        return back(o), S.reshape(B, Hv, d, d)
    o, dq, dk, dv, da, dw = (back(y) for y in _token_by_token(*xs, S, lay(st["dO"].double())))
    dq, dk = (y.unflatten(2, (Hk, share)).sum(3) for y in (dq, dk))
    return o, dq, dk, dv, -da * a / (1 + torch.exp(-g)), dw * ws * (1 - ws)


def _attend(q, k, v, window, sinks, scale, dO=None):
    """One head of one sequence by its definition in fp64: q, k, v [T, d]."""
    at = torch.arange(len(q), device="cuda")
    gap = at[:, None] - at
    hidden = (gap < 0) | ((gap >= window) & (at >= sinks))
    p = torch.softmax((q @ k.T * scale).masked_fill(hidden, -math.inf), -1)
    o = p @ v
    if dO is None:
        return o
    ds = p * (dO @ v.T - (dO * o).sum(-1, keepdim=True)) * scale
    return o, ds @ k, ds.T @ q, p.T @ dO


def _window_exact(st):
    c = st["case"]
    Hq, Hkv, W, s, d = c["Hq"], c["Hkv"], c["window"], c["sinks"], c["d"]
    G, scale = Hq // Hkv, 1 / math.sqrt(d)
    q, k, v = (st[x].double() for x in ("q", "k", "v"))
    if c["use"] == "step":
        o = torch.empty_like(q)
        kc, vc = st["k_cache"].double(), st["v_cache"].double()
        for b, p in enumerate(_positions(c)):
            now = p if p < s else s + (p - s) % W
            kc[b, now], vc[b, now] = k[b], v[b]
            tokens = [j for j in range(min(s, p + 1))] + [j for j in range(max(s, p - W + 1), p + 1)]
            slots = torch.tensor([j if j < s else s + (j - s) % W for j in tokens], device="cuda")
            x = torch.einsum("hgd,jhd->hgj", q[b].reshape(Hkv, G, d), kc[b, slots]) * scale
            o[b] = torch.einsum("hgj,jhd->hgd", torch.softmax(x, -1), vc[b, slots]).reshape(Hq, d)
        return o, kc, vc
    lens = _lens(c)
    q, k, v = (x.flatten(0, -3) for x in (q, k, v))
    o, dq, dk, dv = torch.empty_like(q), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    train = c["use"] == "train"
    if train:
        dO = st["dO"].double().flatten(0, -3)
    else:
        kc, vc = st["k_cache"].double(), st["v_cache"].double()
    row = 0
    for n, T in enumerate(lens):
        r = slice(row, row + T)
        for h in range(Hq if T else 0):
            j = h // G
            if train:
                o[r, h], dq[r, h], x, y = _attend(q[r, h], k[r, j], v[r, j], W, s, scale, dO[r, h])
                dk[r, j] += x
                dv[r, j] += y
            else:
                o[r, h] = _attend(q[r, h], k[r, j], v[r, j], W, s, scale)
        if not train and T:
            kept = [t for t in range(T) if t < s or t >= T - W]
            slots = torch.tensor([t if t < s else s + (t - s) % W for t in kept], device="cuda")
            kept = torch.tensor(kept, device="cuda") + row
            kc[n, slots], vc[n, slots] = k[kept], v[kept]
        row += T
    if train:
        return tuple(x.unflatten(0, (c["B"], c["T"])) for x in (o, dq, dk, dv))
    return (o if c["lens"] else o.unflatten(0, (c["B"], c["T"]))), kc, vc


def exact(c, seed):
    st = prepare(c, seed)
    return _delta_exact(st) if c["op"] == "delta" else _window_exact(st)
