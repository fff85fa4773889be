"""Plain 64-bit implementations of linear attention and group norm, and the
error bounds that the tests hold the kernels to.

Each bound is a sum of |products| times the roundings that a term meets: with
u the rounding of a type (half a step: 2^-24 for fp32, 2^-8 for bf16),
|fl(sum) - sum| <= (roundings of a term) u sum |terms|.  `mix64(..., absolute=
True)` gives that sum of |terms|.
"""
import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def heads(t, H):
    """(Bt,T,G,d) in 64 bits with one row per head: (Bt,H,T,d)."""
    t = t.double().transpose(1, 2)
    return t.repeat_interleave(H // t.shape[1], 1)


def powers(log_decay, n):
    """g_h^n, 0 where n < 0, 1 where n = 0 (a decay of zero too): (H, *n.shape)."""
    n = n.to(log_decay.device).double()
    lg = log_decay.double().view(-1, *([1] * n.dim()))
    p = torch.exp(torch.where(n > 0, lg * n.clamp(min=1), torch.zeros_like(lg * n)))
    return torch.where(n < 0, torch.zeros_like(p), p)


def live(lengths, B, T, dev):
    n = torch.full((B,), T, device=dev) if lengths is None else lengths.to(dev).long().clamp(0, T)
    return n, torch.arange(T, device=dev)[None] < n[:, None]


def forward64(q, k, v, ld, scale, s0=None, lengths=None, absolute=False):
    """y (Bt,T,H,dv), s_final: the sums over all pairs of tokens."""
    B, T, H, dv = v.shape
    n, on = live(lengths, B, T, v.device)
    q, k, v = (heads(t, H) for t in (q, k, v))
    # what stands behind the length is not read: garbage there must not matter
    q, k, v = (torch.where(on[:, None, :, None], t, torch.zeros_like(t)) for t in (q, k, v))
    s0 = None if s0 is None else s0.double()
    if absolute:
        q, k, v, s0 = (None if t is None else t.abs() for t in (q, k, v, s0))
    t = torch.arange(T, device=v.device)
    mask = powers(ld, t[:, None] - t[None]).unsqueeze(0)
    y = ((q @ k.transpose(-1, -2)) * mask) @ v
    left = powers(ld, n[:, None] - 1 - t[None]).transpose(0, 1)
    sf = (k * left[..., None]).transpose(-1, -2) @ v
    if s0 is not None:
        y = y + (q * powers(ld, t + 1).unsqueeze(0).unsqueeze(-1)) @ s0
        sf = sf + s0 * powers(ld, n).transpose(0, 1)[..., None, None]
    y = torch.where(on[:, None, :, None], y * scale, torch.zeros_like(y))
    return y.transpose(1, 2), sf


def backward64(q, k, v, ld, scale, dy, s0=None, ds=None, lengths=None, absolute=False):
    """dq, dk (Bt,T,G,dk), dv (Bt,T,H,dv), ds0."""
    B, T, H, dv = v.shape
    G, dkk = q.shape[2], q.shape[3]
    n, on = live(lengths, B, T, v.device)
    onb = on[:, None, :, None]
    q, k, v, dy = (torch.where(onb, x, torch.zeros_like(x)) for x in (heads(t, H) for t in (q, k, v, dy)))
    s0, ds = (None if t is None else t.double() for t in (s0, ds))
    if absolute:
        q, k, v, dy, s0, ds = (None if t is None else t.abs() for t in (q, k, v, dy, s0, ds))
    t = torch.arange(T, device=v.device)
    mask = powers(ld, t[:, None] - t[None]).unsqueeze(0)
    P = (q @ k.transpose(-1, -2)) * mask
    V = (dy @ v.transpose(-1, -2)) * mask
    dq, dk, dvv = scale * (V @ k), scale * (V.transpose(-1, -2) @ q), scale * (P.transpose(-1, -2) @ dy)
    grow = powers(ld, t + 1).unsqueeze(0).unsqueeze(-1)
    ds0 = scale * ((q * grow).transpose(-1, -2) @ dy)
    if s0 is not None:
        dq = dq + scale * grow * (dy @ s0.transpose(-1, -2))
    if ds is not None:
        left = powers(ld, n[:, None] - 1 - t[None]).transpose(0, 1)[..., None]
        dk = dk + left * (v @ ds.transpose(-1, -2))
        dvv = dvv + left * (k @ ds)
        ds0 = ds0 + ds * powers(ld, n).transpose(0, 1)[..., None, None]
    dq, dk, dvv = (torch.where(onb, x, torch.zeros_like(x)) for x in (dq, dk, dvv))
    dq, dk = (x.view(B, G, H // G, T, dkk).sum(2) for x in (dq, dk))
    return tuple(x.transpose(1, 2) for x in (dq, dk, dvv)) + (ds0,)


def mix_bound(ref, mass, io, T, da, tensor_cores, rep=1):
    """Bound of an answer's row (y, dq, dk, dv) of type io.  A term meets
    - in fp32: the dot product of its score (da) or with the state (da), the
      sum over a chunk (64 at most), the chunk chain (2 roundings a chunk, of
      16 tokens at least), its weights (8), the sum of shared heads (rep);
    - on the tensor cores one rounding of an operand to bf16 more (the score,
      or the state); q, k, v, dy enter exactly;
    and the result is rounded once to io."""
    u32 = (da + 64 + 2 * (T / 16 + 1) + 8 + rep) * U[torch.float32]
    return (u32 + (1.01 * U[torch.bfloat16] if tensor_cores else 0.0)) * mass + U[io] * ref.abs() * 1.01


def state_bound(ref, mass, T):
    """Bound of a final state or ds0, in fp32: the chunk's sum (64), the chain
    (3 roundings a chunk of 16 tokens at least) and the weights.  The tensor
    cores get the weighted rows in three bf16 pieces (exact to 2^-24 of the
    row) and so three times the terms."""
    return (3 * 64 + 3 * (T / 16 + 1) + 16) * U[torch.float32] * mass + U[torch.float32] * ref.abs()


def act64(name, u):
    if name == "silu":
        return u * torch.sigmoid(u)
    if name == "gelu":
        return 0.5 * u * torch.erfc(-u * 0.5 ** 0.5)
    if name == "relu":
        return torch.relu(u)
    return u


def norm64(x, groups, weight=None, bias=None, gate=None, act="none", eps=1e-5):
    """y, mean, rstd in 64 bits; differentiable."""
    B, C = x.shape[0], x.shape[-1]
    xg = x.double().reshape(B, -1, groups, C // groups)
    mean = xg.mean((1, 3))
    var = (xg - mean[:, None, :, None]).square().mean((1, 3))
    rstd = (var + eps) ** -0.5
    u = ((xg - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(x.shape)
    u = u if weight is None else u * weight.double()
    u = u if bias is None else u + bias.double()
    return (act64(act, u) if gate is None else u * act64(act, gate.double())), mean, rstd


def within(got, ref, bound, what=""):
    """|got - ref| <= bound everywhere, NaN and infinities only where ref has them."""
    g, r = got.double(), ref.double()
    bad = ~((g - r).abs() <= bound)
    bad &= ~((g == r) | (g.isnan() & r.isnan()))
    if bad.any():
        i = int(torch.argmax(torch.where(bad, (g - r).abs() / bound.clamp(min=1e-300), torch.zeros_like(g)).nan_to_num(
            nan=float("inf")).reshape(-1)))
        raise AssertionError("%s: %d of %d out of bounds, worst got %r ref %r bound %r at flat index %d" % (
            what, int(bad.sum()), bad.numel(), float(g.reshape(-1)[i]), float(r.reshape(-1)[i]),
            float(bound.expand_as(r).reshape(-1)[i]), i))
