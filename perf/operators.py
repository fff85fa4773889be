"""Linear attention with a decay for each head, and group norm with an activation: what is measured.

Each case is one pass through one of five entry points of ``state_space_lm_b200.m3``:

* ``linattn_chunked_fwd``  -- prompts:      S_t = gamma_h S_{t-1} + k_t v_t^T,   y_t = scale S_t^T q_t
* ``linattn_step_decode``  -- one token:    the same recurrence, the state updated in place
* ``linattn_chunked_bwd``  -- training:     gradients of q, k, v and the initial state
* ``group_norm_fwd``       -- u = (x - mean) rstd w + b per (batch, group);  y = act(u), or u act(gate)
* ``group_norm_bwd``       -- gradients of x, w, b and the gate

With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


# ---- the cases ----------------------------------------------------------------
def _lin(name, op, batch, seqlen, heads, groups, dk, dv, dtype, ragged=False, fused=False, init=False):
    c = dict(op=op, batch=batch, seqlen=seqlen, heads=heads, groups=groups, dk=dk, dv=dv, dtype=dtype, ragged=ragged,
             fused=fused, init=init)
    return dict(c, name=name) if name else c


def _norm(name, op, batch, seqlen, channels, groups, dtype, act, gated):
    c = dict(op=op, batch=batch, seqlen=seqlen, channels=channels, groups=groups, dtype=dtype, act=act, gated=gated)
    return dict(c, name=name) if name else c


def listed():
    return [
        # a training or prefill batch at the default workload's shape (8 x 2048 tokens, 16 heads of 64, state 128)
        _lin("fwd 8x2048 h16", "lin_fwd", 8, 2048, 16, 16, 128, 64, "bf16"),
        # one long prompt over few heads, continued from a state: the time axis has to be split
        _lin("fwd long 1x32768 h32", "lin_fwd", 1, 32768, 32, 32, 128, 64, "bf16", init=True),
        # a ragged batch of short prompts cut out of one fused projection, q and k shared by four heads each
        _lin("fwd ragged 13x397 h12 g3", "lin_fwd", 13, 397, 12, 3, 64, 96, "bf16", ragged=True, fused=True, init=True),
        # a small fp32 model with sizes that are multiples of nothing
        _lin("fwd f32 3x333 h5", "lin_fwd", 3, 333, 5, 5, 37, 29, "f32", init=True),
        # a serving batch of single tokens: bound by the states
        _lin("step 512 h16", "lin_step", 512, 1, 16, 16, 128, 64, "bf16"),
        # one user's next token: bound by latency
        _lin("step 1 h16", "lin_step", 1, 1, 16, 16, 128, 64, "bf16"),
        # the training step's gradients at the default workload's shape
        _lin("bwd 8x2048 h16", "lin_bwd", 8, 2048, 16, 16, 128, 64, "bf16"),
        # gradients of shared q and k heads, ragged, with an initial state and an odd length
        _lin("bwd ragged 5x777 h8 g2", "lin_bwd", 5, 777, 8, 2, 64, 64, "bf16", ragged=True, init=True),
        # the norm of each head of each token behind the attention, gated: 16384 tokens of d_model 1024, 16 heads
        _norm("norm fwd heads 16384x1024", "norm_fwd", 16384, 1, 1024, 16, "bf16", "silu", True),
        # group norm over whole sequences, channels last
        _norm("norm fwd seq 8x2048x1024", "norm_fwd", 8, 2048, 1024, 32, "bf16", "silu", False),
        # its gradients, and those of the gated form
        _norm("norm bwd seq 8x2048x1024", "norm_bwd", 8, 2048, 1024, 32, "bf16", "silu", False),
        _norm("norm bwd heads 1037x1000 f32", "norm_bwd", 1037, 1, 1000, 8, "f32", "gelu", True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    top = 550e6   # bytes: no drawn case costs more than the largest listed one
    while True:
        op = rng.choice(["lin_fwd", "lin_fwd", "lin_step", "lin_bwd", "norm_fwd", "norm_bwd"])
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        if op.startswith("lin"):
            groups = rng.choice([1, 2, 3, 4, 8, 16])
            heads = groups * rng.choice([1, 1, 2, 4, 5])
            dk, dv = (rng.choice([8 * rng.randint(2, 16), 64, 128, rng.randint(9, 128)]) for _ in range(2))
            batch = _log_int(rng, 1, 600 if op == "lin_step" else 24)
            seqlen = 1 if op == "lin_step" else _log_int(rng, 1, 20000)
            ragged = op != "lin_step" and rng.random() < 0.4
            c = _lin("", op, batch, seqlen, heads, groups, dk, dv, dtype, ragged, rng.random() < 0.3, rng.random() < 0.5)
            if c["fused"] and any(e % 8 for e in (groups * dk, heads * dv)):
                c["fused"] = False        # slices of a projection start on 16 bytes
            cost = batch * seqlen * heads * (dk + dv) * 4
            if heads > 40 or cost > (40e6 if dtype == "f32" else 160e6):
                continue
        else:
            per = rng.choice([rng.randint(1, 9), 8 * rng.randint(1, 16), 64, rng.randint(10, 130)])
            groups = rng.choice([1, 2, 4, 7, 8, 16, 32])
            seqlen = rng.choice([1, _log_int(rng, 2, 6000)])
            batch = _log_int(rng, 1, 20000 if seqlen == 1 else 16)
            c = _norm("", op, batch, seqlen, per * groups, groups, dtype, rng.choice(["silu", "gelu", "relu", "none"]),
                      rng.random() < 0.4)
        if work(c)["bytes"] <= top:
            return c


# ---- inputs --------------------------------------------------------------------
def _lengths(c, gen):
    if not c["ragged"]:
        return None
    n = torch.randint(0, c["seqlen"] + 1, (c["batch"],), generator=gen, device="cuda", dtype=torch.int32)
    n[0] = c["seqlen"]
    return n


def _decay(c):
    # gamma_h = 1 - 2^-e_h with e_h from 5 to 12 over the heads: memories of 32 to 4096 tokens
    e = torch.linspace(5.0, 12.0, c["heads"], dtype=torch.float64)
    return torch.log1p(-torch.exp2(-e)).float().cuda()


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)
    dt = DTYPES[c["dtype"]]

    def normal(*shape, dtype=dt):
        return torch.randn(*shape, generator=gen, device="cuda").to(dtype)

    if c["op"].startswith("lin"):
        B, T, H, G, dk, dv = (c[k] for k in ("batch", "seqlen", "heads", "groups", "dk", "dv"))
        lead = (B,) if c["op"] == "lin_step" else (B, T)
        if c["fused"]:
            # one projection's output, q | k | v: the user passes views of it
            flat = normal(*lead, 2 * G * dk + H * dv)
            q = flat[..., :G * dk].unflatten(-1, (G, dk))
            k = flat[..., G * dk:2 * G * dk].unflatten(-1, (G, dk))
            v = flat[..., 2 * G * dk:].unflatten(-1, (H, dv))
        else:
            q, k, v = normal(*lead, G, dk), normal(*lead, G, dk), normal(*lead, H, dv)
        s = dict(op=c["op"], q=q, k=k, v=v, log_decay=_decay(c), s0=None, lengths=None)
        if c["op"] == "lin_step":
            s["s"] = normal(B, H, dk, dv, dtype=torch.float32)
            return s
        s["lengths"] = _lengths(c, gen)
        if c["init"]:
            s["s0"] = normal(B, H, dk, dv, dtype=torch.float32)
        if c["op"] == "lin_bwd":
            s["dy"] = normal(B, T, H, dv)
            s["ds"] = normal(B, H, dk, dv, dtype=torch.float32) if c["init"] else None
        return s
    B, L, C, G = (c[k] for k in ("batch", "seqlen", "channels", "groups"))
    x = (torch.randn(B, L, C, generator=gen, device="cuda") * 1.5 + 0.25).to(dt)
    s = dict(op=c["op"], x=x, groups=G, act=c["act"], gate=normal(B, L, C) if c["gated"] else None,
             weight=1.0 + 0.1 * normal(C, dtype=torch.float32), bias=0.1 * normal(C, dtype=torch.float32))
    if c["op"] == "norm_bwd":
        s["dy"] = normal(B, L, C)
        # what the forward left: the statistics of each (batch, group)
        x64 = x.view(B, L, G, C // G).double()
        s["mean"] = x64.mean((1, 3)).float()
        s["rstd"] = torch.rsqrt(x64.var((1, 3), unbiased=False) + EPS).float()
    return s


# ---- the plain forms -------------------------------------------------------------
CHUNK = 128


def _heads(t, H):
    """(B, T, G, d) in 32 bits, one row per head: (B, H, T, d)."""
    t = t.float().transpose(1, 2)
    return t.repeat_interleave(H // t.shape[1], 1) if t.shape[1] != H else t


def _powers(log_decay, n):
    """gamma_h^n for whole numbers n (any shape), in 64 bits: (H, *n.shape), rounded once; 0 where n < 0."""
    n = n.double()
    p = torch.exp(log_decay.double().view(-1, *([1] * n.dim())) * n.clamp(min=0))
    return torch.where(n < 0, 0.0, p).float()


def _mix(q, k, v, log_decay, s0):
    """sum_{s <= t} gamma^(t-s) (q_t . k_s) v_s + gamma^(t+1) s0^T q_t over (B, H, T, d), in chunks of the time axis."""
    B, H, T, dk = q.shape
    dv, n = v.shape[-1], -(-T // CHUNK)
    C = min(CHUNK, T)
    pad = n * C - T
    if pad:
        q, k, v = (torch.nn.functional.pad(t, (0, 0, 0, pad)) for t in (q, k, v))
    q, k, v = (t.reshape(B, H, n, C, t.shape[-1]) for t in (q, k, v))
    i = torch.arange(C, device=q.device)
    mask = _powers(log_decay, i[:, None] - i[None, :]).view(1, H, 1, C, C)
    y = ((q @ k.transpose(-1, -2)) * mask) @ v
    own_state = (k * _powers(log_decay, C - 1 - i).view(1, H, 1, C, 1)).transpose(-1, -2) @ v
    # the state entering chunk c: sum over c' < c of gamma^(C (c-1-c')) own_state[c'], and s0 decayed
    j = torch.arange(n, device=q.device)
    carry = _powers(log_decay, (j[:, None] - 1 - j[None, :]) * C).view(1, H, n, n)
    state = (carry @ own_state.reshape(B, H, n, dk * dv)).view(B, H, n, dk, dv)
    if s0 is not None:
        state = state + s0[:, :, None] * _powers(log_decay, j * C).view(1, H, n, 1, 1)
    y = y + (q * _powers(log_decay, i + 1).view(1, H, 1, C, 1)) @ state
    return y.reshape(B, H, n * C, dv)[:, :, :T]


def _row_lengths(s, B, T, device):
    n = s["lengths"]
    return torch.full((B,), T, device=device) if n is None else n.long()


def _fwd_plain(s):
    B, T, H, dv = s["v"].shape
    dk = s["q"].shape[-1]
    ld, io = s["log_decay"], s["v"].dtype
    q, k, v = _heads(s["q"], H), _heads(s["k"], H), _heads(s["v"], H)
    n = _row_lengths(s, B, T, q.device)
    live = (torch.arange(T, device=q.device)[None] < n[:, None]).view(B, 1, T, 1)
    y = _mix(q, k, v, ld, s["s0"]) * dk ** -0.5
    left = _powers(ld, n[:, None] - 1 - torch.arange(T, device=q.device)[None]).transpose(0, 1)
    final = (k * left[..., None]).transpose(-1, -2) @ v
    if s["s0"] is not None:
        final = final + s["s0"] * _powers(ld, n).transpose(0, 1)[..., None, None]
    return torch.where(live, y, 0.0).transpose(1, 2).to(io).contiguous(), final


def _bwd_plain(s):
    B, T, H, dv = s["v"].shape
    G, dk = s["q"].shape[2:]
    ld, io, scale = s["log_decay"], s["v"].dtype, s["q"].shape[-1] ** -0.5
    n = _row_lengths(s, B, T, s["v"].device)
    t = torch.arange(T, device=n.device)
    live = (t[None] < n[:, None]).view(B, 1, T, 1)
    q, k, v, dy = (torch.where(live, _heads(x, H), 0.0) for x in (s["q"], s["k"], s["v"], s["dy"]))
    dq = scale * _mix(dy, v, k, ld, None if s["s0"] is None else s["s0"].transpose(-1, -2))
    dk_ = scale * _mix(v.flip(2), dy.flip(2), q.flip(2), ld, None).flip(2)
    dv_ = scale * _mix(k.flip(2), q.flip(2), dy.flip(2), ld, None).flip(2)
    ds0 = scale * ((q * _powers(ld, t + 1).view(1, H, T, 1)).transpose(-1, -2) @ dy)
    if s["ds"] is not None:
        left = _powers(ld, n[:, None] - 1 - t[None]).transpose(0, 1)[..., None]
        dk_ = dk_ + left * (v @ s["ds"].transpose(-1, -2))
        dv_ = dv_ + left * (k @ s["ds"])
        ds0 = ds0 + s["ds"] * _powers(ld, n).transpose(0, 1)[..., None, None]
    dq, dk_, dv_ = (torch.where(live, x, 0.0) for x in (dq, dk_, dv_))
    dq, dk_ = (x.view(B, G, H // G, T, dk).sum(2) for x in (dq, dk_))
    return tuple(x.transpose(1, 2).to(io).contiguous() for x in (dq, dk_, dv_)) + (ds0,)


def _step_plain(s):
    H, dk = s["v"].shape[1], s["q"].shape[-1]
    q, k = (x.float().repeat_interleave(H // x.shape[1], 1) for x in (s["q"], s["k"]))
    gamma = torch.exp(s["log_decay"].double()).float().view(1, H, 1, 1)
    s["s"].copy_(s["s"] * gamma + k[..., None] * s["v"].float()[:, :, None])
    y = (q[..., None] * s["s"]).sum(2) * dk ** -0.5
    return y.to(s["v"].dtype), s["s"]


def _act(name, u):
    """The activation and its derivative."""
    if name == "silu":
        g = 1.0 / (1.0 + torch.exp(-u))
        return u * g, g * (1.0 + u * (1.0 - g))
    if name == "gelu":
        p = 0.5 * (1.0 + torch.erf(u * (0.5 ** 0.5)))
        return u * p, p + u * torch.exp(-0.5 * u * u) * (0.5 / math.pi) ** 0.5
    if name == "relu":
        return u.clamp(min=0), (u > 0).to(u.dtype)
    return u, torch.ones_like(u)


def _norm_fwd_plain(s):
    B, L, C = s["x"].shape
    G = s["groups"]
    x = s["x"].float().view(B, L, G, C // G)
    mean = x.mean((1, 3), keepdim=True)
    d = x - mean
    rstd = torch.rsqrt((d * d).mean((1, 3), keepdim=True) + EPS)
    u = (d * rstd).view(B, L, C) * s["weight"] + s["bias"]
    y = _act(s["act"], u)[0] if s["gate"] is None else u * _act(s["act"], s["gate"].float())[0]
    return y.to(s["x"].dtype), mean.view(B, G), rstd.view(B, G)


def _norm_bwd_plain(s):
    B, L, C = s["x"].shape
    G, io = s["groups"], s["x"].dtype
    xh = (s["x"].float().view(B, L, G, C // G) - s["mean"].view(B, 1, G, 1)) * s["rstd"].view(B, 1, G, 1)
    xh, dy = xh.reshape(B, L, C), s["dy"].float()
    u = xh * s["weight"] + s["bias"]
    out = []
    if s["gate"] is None:
        du = dy * _act(s["act"], u)[1]
    else:
        a, da = _act(s["act"], s["gate"].float())
        du = dy * a
        out = [(dy * u * da).to(io)]
    dn = (du * s["weight"]).view(B, L, G, C // G)
    xg = xh.view(B, L, G, C // G)
    m1, m2 = dn.mean((1, 3), keepdim=True), (dn * xg).mean((1, 3), keepdim=True)
    dx = ((dn - m1 - xg * m2) * s["rstd"].view(B, 1, G, 1)).reshape(B, L, C)
    return [dx.to(io), (du * xh).sum((0, 1)), du.sum((0, 1))] + out


def run(state):
    s = state
    op = s["op"]
    if own:
        from state_space_lm_b200 import m3
        if op == "lin_fwd":
            return m3.linattn_chunked_fwd(s["q"], s["k"], s["v"], s["log_decay"], s0=s["s0"], lengths=s["lengths"])
        if op == "lin_step":
            return m3.linattn_step_decode(s["q"], s["k"], s["v"], s["log_decay"], s["s"]), s["s"]
        if op == "lin_bwd":
            g = m3.linattn_chunked_bwd(s["q"], s["k"], s["v"], s["log_decay"], s["dy"], s0=s["s0"], ds_final=s["ds"],
                                       lengths=s["lengths"])
            return g["dq"], g["dk"], g["dv"], g["ds0"]
        if op == "norm_fwd":
            return m3.group_norm_fwd(s["x"], s["groups"], s["weight"], s["bias"], gate=s["gate"], act=s["act"], eps=EPS)
        g = m3.group_norm_bwd(s["x"], s["dy"], s["mean"], s["rstd"], s["groups"], s["weight"], s["bias"],
                              gate=s["gate"], act=s["act"])
        return [g[k] for k in ("dx", "dweight", "dbias") + (() if s["gate"] is None else ("dgate",))]
    return {"lin_fwd": _fwd_plain, "lin_step": _step_plain, "lin_bwd": _bwd_plain, "norm_fwd": _norm_fwd_plain,
            "norm_bwd": _norm_bwd_plain}[op](s)


# ---- what a pass cannot do without -------------------------------------------------
def work(case):
    c, e = case, 2 if case["dtype"] == "bf16" else 4
    if c["op"].startswith("lin"):
        B, T, H, G, dk, dv = (c[k] for k in ("batch", "seqlen", "heads", "groups", "dk", "dv"))
        state, qk, vy = 4 * B * H * dk * dv, e * B * T * G * dk, e * B * T * H * dv
        mac = 2 * B * T * H * dk * dv                     # one product of a token with a state
        if c["op"] == "lin_step":
            return {"bytes": 2 * state + 2 * qk + 2 * vy + 4 * H, "flops": 2 * mac}
        if c["op"] == "lin_fwd":                          # the state's update and the answer
            return {"bytes": 2 * qk + 2 * vy + state * (2 if c["init"] else 1), "flops": 2 * mac}
        # two states (the forward's and the adjoint's) and three products with them
        return {"bytes": 4 * qk + 3 * vy + state * (3 if c["init"] else 1), "flops": 5 * mac}
    n = c["batch"] * c["seqlen"] * c["channels"]
    stats = 8 * c["batch"] * c["groups"] + 8 * c["channels"]
    if c["op"] == "norm_fwd":
        return {"bytes": n * e * (3 if c["gated"] else 2) + stats, "flops": 12 * n}
    return {"bytes": n * e * (5 if c["gated"] else 3) + 2 * stats, "flops": 24 * n}


# ---- the definition, in 64 bits ------------------------------------------------------
def _exact_lin(c, s):
    B, H, G, dk, dv = (c[k] for k in ("batch", "heads", "groups", "dk", "dv"))
    T = c["seqlen"]
    rep = H // G
    gamma = torch.exp(s["log_decay"].double()).view(1, H, 1, 1)
    scale = 1.0 / math.sqrt(dk)
    expand = lambda x: x.double().repeat_interleave(rep, -2)      # noqa: E731
    if c["op"] == "lin_step":
        S = s["s"].double() * gamma + torch.einsum("bhk,bhv->bhkv", expand(s["k"]), s["v"].double())
        return torch.einsum("bhk,bhkv->bhv", expand(s["q"]), S) * scale, S
    # time first, so that each token's slice is one block
    first = lambda x: x.transpose(0, 1).contiguous()              # noqa: E731
    q, k, v = first(expand(s["q"])), first(expand(s["k"])), first(s["v"].double())
    lens = torch.full((B,), T, device=q.device) if s["lengths"] is None else s["lengths"].long()
    on = (torch.arange(T, device=q.device)[:, None] < lens[None])
    q, k, v = (x * on[..., None, None] for x in (q, k, v))
    rate = torch.where(on[:, :, None], gamma.view(1, 1, H), 1.0)[..., None, None]
    S = torch.zeros(B, H, dk, dv, dtype=torch.float64, device=q.device) if s["s0"] is None else s["s0"].double()
    S = S.clone()
    if c["op"] == "lin_fwd":
        y = torch.empty_like(v)
        for t in range(T):
            S.mul_(rate[t]).addcmul_(k[t][..., None], v[t][:, :, None])
            y[t] = torch.matmul(q[t][:, :, None], S)[:, :, 0]
        return first(y) * scale, S
    dy = first(s["dy"].double()) * on[..., None, None]
    dq, dkk, dvv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    for t in range(T):
        S.mul_(rate[t]).addcmul_(k[t][..., None], v[t][:, :, None])
        dq[t] = torch.matmul(S, dy[t][..., None])[..., 0] * scale
    Z = torch.zeros_like(S) if s["ds"] is None else s["ds"].double().clone()
    for t in range(T - 1, -1, -1):
        Z.addcmul_(q[t][..., None], dy[t][:, :, None], value=scale)
        dkk[t] = torch.matmul(Z, v[t][..., None])[..., 0]
        dvv[t] = torch.matmul(k[t][:, :, None], Z)[:, :, 0]
        Z.mul_(rate[t])
    dq, dkk, dvv = (first(x * on[..., None, None]) for x in (dq, dkk, dvv))
    fold = lambda x: x.view(B, T, G, rep, dk).sum(3)              # noqa: E731
    return fold(dq), fold(dkk), dvv, Z


def _exact_norm(c, s):
    B, L, C, G = (c[k] for k in ("batch", "seqlen", "channels", "groups"))
    x = s["x"].double().requires_grad_()
    w, b = s["weight"].double().requires_grad_(), s["bias"].double().requires_grad_()
    z = None if s["gate"] is None else s["gate"].double().requires_grad_()
    act = {"silu": lambda u: u * torch.sigmoid(u), "relu": torch.relu, "none": lambda u: u,
           "gelu": lambda u: u * 0.5 * torch.erfc(-u / math.sqrt(2.0))}[c["act"]]
    xg = x.view(B, L, G, C // G)
    mean = xg.sum((1, 3)) / (L * (C // G))
    var = (xg - mean.view(B, 1, G, 1)).square().sum((1, 3)) / (L * (C // G))
    rstd = 1.0 / torch.sqrt(var + EPS)
    u = ((xg - mean.view(B, 1, G, 1)) * rstd.view(B, 1, G, 1)).reshape(B, L, C) * w + b
    y = act(u) if z is None else u * act(z)
    if c["op"] == "norm_fwd":
        return y.detach(), mean.detach(), rstd.detach()
    return list(torch.autograd.grad(y, [x, w, b] + ([] if z is None else [z]), s["dy"].double()))


def exact(case, seed):
    c = case
    if c["op"].startswith("lin") and c["batch"] * c["seqlen"] * c["heads"] * c["dk"] * c["dv"] > 3e10:
        return None          # the token loop would take too long
    s = prepare(c, seed)
    return _exact_lin(c, s) if c["op"].startswith("lin") else _exact_norm(c, s)
