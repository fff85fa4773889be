"""The bounds of norm_bounds on the CPU: arithmetic in 32 bits stays within
them, gradients agree with torch.autograd's in 64 bits, and a term that is
dropped or a sum that is zero does not pass."""
import pytest
import torch

import norm_bounds
from lin_reference import norm64, within

SHAPES = [((33, 64), 4), ((200, 128), 2), ((257, 1000), 8), ((3, 520), 1), ((2, 16384), 1), ((2, 5, 24), 3),
          ((3, 17, 64), 8), ((2, 100, 1024), 32), ((1, 1000, 70), 7), ((4, 33, 512), 1)]


def inputs(shape, groups, dtype, gated, act="silu", shift=0.25):
    """dy with a part along the norm's output and one along a constant, as a
    loss has: the two means that dx subtracts are then of its own size."""
    g = torch.Generator().manual_seed(sum(shape) + groups)
    n = lambda *s: torch.randn(*s, generator=g)            # noqa: E731
    C = shape[-1]
    x = (1.5 * n(*shape) + shift).to(dtype)
    gate = n(*shape).to(dtype) if gated else None
    dy = (n(*shape) + 0.7 + 0.4 * (x.float() - shift)).to(dtype)
    return x, dy, gate, 1 + 0.1 * n(C), 0.1 * n(C)


def plain32(x, dy, mean, rstd, groups, w, b, gate, act):
    """The same formulas in 32 bits, rounded once."""
    B, C = x.shape[0], x.shape[-1]
    shape = (B, -1, groups, C // groups)
    over = lambda t: t.float()[:, None, :, None]           # noqa: E731
    xh = ((x.float().view(shape) - over(mean)) * over(rstd))
    u = (xh.reshape(x.shape) * w + b)
    parts = lambda v: (p.float() for p in norm_bounds.act_parts(act, v.double()))  # noqa: E731
    out = {}
    if gate is None:
        du = dy.float() * tuple(parts(u))[1]
    else:
        f, df = parts(gate.float())
        du = dy.float() * f
        out["dgate"] = (dy.float() * u * df).to(x.dtype)
    dn = (du * w).view(shape)
    dx = (dn - dn.mean((1, 3), keepdim=True) - xh * (dn * xh).mean((1, 3), keepdim=True)) * over(rstd)
    out.update(dx=dx.reshape(x.shape).to(x.dtype), dweight=(du * xh.reshape(x.shape)).reshape(-1, C).sum(0),
               dbias=du.reshape(-1, C).sum(0))
    return out


def statistics(x, groups):
    _, mean, rstd = norm64(x, groups)
    return mean.float(), rstd.float()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("shape,groups", SHAPES, ids=lambda s: "x".join(map(str, s)) if isinstance(s, tuple) else str(s))
def test_the_bounds_take_32_bits_and_refuse_a_missing_term(shape, groups, gated, dtype):
    for act in ("none", "silu", "gelu"):
        for shift in (0.25, 4096.0) if dtype == torch.float32 else (0.25,):
            x, dy, gate, w, b = inputs(shape, groups, dtype, gated, act, shift)
            mean, rstd = statistics(x, groups)
            got = plain32(x, dy, mean, rstd, groups, w, b, gate, act)
            ref = norm_bounds.backward(x, dy, mean, rstd, groups, w, b, gate, act)
            for k in got:
                within(got[k], ref[k][0], ref[k][1], k)
            for term, name in (("m1", "dx"), ("m2", "dx"), ("dweight", "dweight"), ("dbias", "dbias")):
                broken = norm_bounds.backward(x, dy, mean, rstd, groups, w, b, gate, act, leave_out=(term,))[name][0]
                with pytest.raises(AssertionError):
                    within(broken.to(got[name].dtype), *ref[name], name)


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "relu"])
def test_the_formulas_are_the_gradients(act):
    for shape, groups, gated in (((7, 12), 3, True), ((2, 9, 8), 2, False), ((2, 9, 8), 2, True)):
        g = torch.Generator().manual_seed(3)
        n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)   # noqa: E731
        x, dy, w, b = n(*shape), n(*shape), n(shape[-1]), n(shape[-1])
        gate = n(*shape) if gated else None
        leaves = [t.requires_grad_() for t in (x, w, b)] + ([gate.requires_grad_()] if gated else [])
        y, mean, rstd = norm64(x, groups, w, b, gate, act)
        ref = torch.autograd.grad(y, leaves, dy)
        io = lambda t: t.detach()                          # noqa: E731
        norm_bounds.U[torch.float64] = 2.0 ** -53
        try:
            got = norm_bounds.backward(io(x), dy, io(mean), io(rstd), groups, io(w), io(b), None if gate is None else io(gate),
                                       act)
        finally:
            del norm_bounds.U[torch.float64]
        for k, r in zip(("dx", "dweight", "dbias", "dgate"), ref):
            assert torch.allclose(got[k][0], r, rtol=1e-11, atol=1e-12), k
