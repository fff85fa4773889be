"""Group norm's formulas in 64 bits from given statistics, and error bounds of
each element from its own terms.

With u = 2^-24 (half a step of fp32), a sum of n terms that passes through r
roundings is off by r u sum |terms| at most.  R counts them for the longest way
through the kernels: values summed one after the other by a thread (32 in a
row of registers; a chunk's tokens over sequences; every 32nd channel of a wide
group), the lanes of a warp (5), the warps of a block, the phases of a vector, and
the chunks of a sequence, eight side by side.  `terms` are |values|, so a term that is left out, or a sum that is
zero, shows wherever it is larger than the roundings of what is there.
"""
import torch

from lin_reference import U

F32 = U[torch.float32]


def roundings(x, L, groups):
    B, C = x.shape[0], x.shape[-1]
    D = C // groups
    wide = 8 if x.dtype == torch.bfloat16 else 4
    vec = C // (wide if D % wide == 0 else 1)
    phases = max(1, 256 // vec)                             # threads that share a vector's tokens
    nch = max(1, min(296 // max(B, 1), -(-L // 4)))         # chunks of a sequence
    tokens = -(-(-(-L // nch)) // phases)                   # of a thread
    return 32 + 5 + 8 + phases + 2 * tokens + nch / 8 + D / 32 + 16


def act_parts(act, v):
    """act, act', in 64 bits."""
    if act == "silu":
        s = torch.sigmoid(v)
        return v * s, s * (1 + v * (1 - s))
    if act == "gelu":
        p = 0.5 * torch.erfc(-v * 0.5 ** 0.5)
        return v * p, p + v * torch.exp(-0.5 * v * v) * 0.3989422804014327
    if act == "relu":
        return torch.relu(v), (v > 0).double()
    return v, torch.ones_like(v)


def act_slack(io):
    """Error of act and act' as evaluated, relative to 1 + |v|: fp32 functions
    to 2 units in the last place and three operations; with 16-bit outputs the
    exponential and the reciprocal to 2^-22 each."""
    return 2.0 ** -20 if io == torch.bfloat16 else 16 * F32


def forward(x, groups, w, b, gate, act, eps=1e-5):
    """{y, mean, rstd: (value, bound)}."""
    io, C, B = x.dtype, x.shape[-1], x.shape[0]
    xg = x.double().reshape(B, -1, groups, C // groups)
    L = xg.shape[1]
    R = roundings(x, L, groups)
    over = lambda t: t[:, None, :, None]                   # noqa: E731
    mean = xg.mean((1, 3))
    d = xg - over(mean)
    var = d.square().mean((1, 3))
    rstd = (var + eps) ** -0.5
    far = d.abs().amax((1, 3))
    # one token: the values themselves are summed; more: differences from one of
    # them, which is added again by the thread, the phases' merge, the vectors'
    # merge and the chunks' merge: four roundings of the mean's own size
    e_mean = (R * F32 * xg.abs().mean((1, 3)) + F32 * mean.abs() if L == 1
              else R * F32 * (d.abs().mean((1, 3)) + far) + 4 * F32 * mean.abs())
    # squares of differences from the computed mean, or from a value, far^2 from it
    e_var = R * F32 * (var if L == 1 else 2 * (var + far ** 2)) + e_mean ** 2 + 2 * e_mean * F32 * far
    e_rstd = rstd * (0.5 * e_var / (var + eps) + 4 * F32)
    xh = d * over(rstd)
    e_xh = over(rstd * e_mean) + xh.abs() * (over(e_rstd / rstd) + 4 * F32)
    xh, e_xh = xh.reshape(x.shape), e_xh.reshape(x.shape)
    W, Bv = (1.0 if w is None else w.double()), (0.0 if b is None else b.double())
    u = xh * W + Bv
    e_u = e_xh * abs(W) + 3 * F32 * ((xh * W).abs() + abs(Bv))
    s = act_slack(io)
    if gate is None:
        f, _ = act_parts(act, u)
        e_y = 1.13 * e_u + s * (1 + u.abs()) * (act != "none") * (act != "relu")
        y = f
    else:
        f, _ = act_parts(act, gate.double())
        y = u * f
        e_f = s * (1 + gate.double().abs()) * (act not in ("none", "relu"))
        e_y = e_u * f.abs() + u.abs() * e_f + 2 * F32 * y.abs()
    return dict(y=(y, e_y + 1.01 * U[io] * y.abs()), mean=(mean, e_mean), rstd=(rstd, e_rstd))


def backward(x, dy, mean, rstd, groups, w, b, gate, act, leave_out=()):
    """{dx, dweight, dbias[, dgate]: (value, bound)} from the given statistics.
    leave_out names terms that the value then lacks: a planted mistake."""
    io, C, B = x.dtype, x.shape[-1], x.shape[0]
    D = C // groups
    xg = x.double().reshape(B, -1, groups, D)
    L = xg.shape[1]
    R = roundings(x, L, groups)
    over = lambda t: t.double()[:, None, :, None]          # noqa: E731
    group = lambda t: t.reshape(B, L, groups, D)           # noqa: E731
    xh = ((xg - over(mean)) * over(rstd)).reshape(x.shape)
    e_xh = 2.1 * F32 * xh.abs()
    W, Bv = (torch.ones(C, dtype=torch.float64, device=x.device) if w is None else w.double(),
             0.0 if b is None else b.double())
    u = xh * W + Bv
    e_u = e_xh * W.abs() + 2.1 * F32 * ((xh * W).abs() + abs(Bv))
    dyd, s, out = dy.double(), act_slack(io) * (act not in ("none", "relu")), {}
    if gate is None:
        _, df = act_parts(act, u)
        du = dyd * df
        # |act''| <= 0.8; the relu's derivative jumps, at 0 alone
        e_du = dyd.abs() * (0.8 * e_u * (act != "none") * (act != "relu") + s * (1 + u.abs())) + F32 * du.abs()
    else:
        z = gate.double()
        f, df = act_parts(act, z)
        du = dyd * f
        e_du = dyd.abs() * s * (1 + z.abs()) + 2 * F32 * du.abs()
        dg = dyd * u * df
        e_dg = dyd.abs() * (e_u * df.abs() + u.abs() * s * (1 + z.abs())) + 3 * F32 * dg.abs()
        out["dgate"] = (dg, e_dg + 1.01 * U[io] * dg.abs())
    dn = du * W
    e_dn = e_du * W.abs() + F32 * dn.abs()
    avg = lambda t: group(t).mean((1, 3), keepdim=True).expand(B, L, groups, D).reshape(x.shape)  # noqa: E731
    m1, m2 = avg(dn), avg(dn * xh)
    e_m1 = avg(e_dn) + R * F32 * avg(dn.abs())
    e_m2 = avg(e_dn * xh.abs() + dn.abs() * e_xh) + (R + 1) * F32 * avg((dn * xh).abs())
    r = over(rstd).expand(B, L, groups, D).reshape(x.shape)
    dx = r * (dn - (0 if "m1" in leave_out else m1) - (0 if "m2" in leave_out else xh * m2))
    e_dx = r * (e_dn + e_m1 + xh.abs() * e_m2 + e_xh * m2.abs() + 4 * F32 * (dn.abs() + m1.abs() + (xh * m2).abs()))
    out["dx"] = (dx, e_dx + 1.01 * U[io] * dx.abs())
    # sums over all rows: besides R, the rows of a slot one after the other (296
    # blocks of at least one row), or the sequences, eight side by side
    rows = x.numel() // C
    Rw = R + rows / 64 + B / 8 + 8
    total = lambda t: t.reshape(-1, C).sum(0)              # noqa: E731
    dw, db = total(du * xh), total(du)
    out["dweight"] = (torch.zeros_like(dw) if "dweight" in leave_out else dw,
                      total(e_du * xh.abs() + du.abs() * e_xh) + (Rw + 1) * F32 * total((du * xh).abs()) + F32 * dw.abs())
    out["dbias"] = (torch.zeros_like(db) if "dbias" in leave_out else db,
                    total(e_du) + Rw * F32 * total(du.abs()) + F32 * db.abs())
    return out
