"""Differentiable Mamba-3 scan, linear attention and group norm for PyTorch:
each forward and its backward behind one torch.autograd.Function.

Argument marshalling only: the forward calls m3_siso_chunked_fwd or
m3_mimo_chunked_fwd, the backward calls m3_chunked_bwd (m3_linattn_* and
m3_group_norm_* for the other two), and every gradient comes from the CUDA
library (there is no other implementation behind these names).  The initial
states and the final states take part in autograd too, so a sequence can be
split into pieces whose states are chained.

A training step can be captured into a CUDA graph.  PyTorch ties a leaf's
gradient to the stream of the graph that used it first: drop every eager
graph of the same leaves (their losses) before the capture.
"""
import torch
from torch.autograd.function import once_differentiable

from . import m3

_SEQ = ("x", "dt", "A", "lam", "theta", "B", "C", "D")
_GRAD_OF = {"x": "dx", "dt": "ddt", "A": "dA", "lam": "dlam", "theta": "dtheta", "B": "dB", "C": "dC",
            "D": "dD", "W_x": "dW_x", "W_y": "dW_y", "h0": "dh0", "prevBx0": "dprevBx0", "angle0": "dangle0"}


class Mamba3Scan(torch.autograd.Function):
    """Inputs in the order of the C ABI; returns (y, h_final, prevBx_final,
    angle_final).  B, C with a rank axis (Bt,T,G,R,N) select the MIMO scan."""

    @staticmethod
    def forward(ctx, x, dt, A, lam, theta, B, C, D, W_x, W_y, h0, prevBx0, angle0, chunk):
        mimo = B.dim() == 5
        if not mimo and (W_x is not None or W_y is not None):
            raise ValueError("W_x, W_y need B and C with a rank axis (Bt,T,G,R,N)")
        if mimo:
            out = m3.mimo_chunked_fwd(x, dt, A, lam, theta, B, C, D, chunk, W_x=W_x, W_y=W_y, h0=h0,
                                      prevBx0=prevBx0, angle0=angle0)
        else:
            out = m3.siso_chunked_fwd(x, dt, A, lam, theta, B, C, D, chunk, h0=h0, prevBx0=prevBx0,
                                      angle0=angle0)
        ctx.save_for_backward(x, dt, A, lam, theta, B, C, D, W_x, W_y, h0, prevBx0, angle0)
        ctx.chunk = chunk
        ctx.mimo = mimo
        return out

    @staticmethod
    def backward(ctx, dy, dh, du, da):
        x, dt, A, lam, theta, B, C, D, W_x, W_y, h0, prevBx0, angle0 = ctx.saved_tensors
        inputs = dict(x=x, dt=dt, A=A, lam=lam, theta=theta, B=B, C=C, D=D, W_x=W_x, W_y=W_y, h0=h0,
                      prevBx0=prevBx0, angle0=angle0)
        names = ("x", "dt", "A", "lam", "theta", "B", "C", "D", "W_x", "W_y", "h0", "prevBx0", "angle0")
        want = tuple(_GRAD_OF[n] for n, need in zip(names, ctx.needs_input_grad[:13])
                     if need and (ctx.mimo or n not in ("W_x", "W_y")))
        if dy is None:
            dy = torch.zeros_like(x)
        cont = lambda t: None if t is None else t.contiguous()
        g = m3.chunked_bwd(x, dt, A, lam, theta, B, C, D, cont(dy.to(x.dtype)), ctx.chunk, W_x=W_x, W_y=W_y,
                           h0=h0, prevBx0=prevBx0, angle0=angle0, dh_final=cont(dh), dprevBx_final=cont(du),
                           dangle_final=cont(da), want=want)
        grads = []
        for n, need in zip(names, ctx.needs_input_grad[:13]):
            v = g.get(_GRAD_OF[n]) if need else None
            grads.append(None if v is None else v.to(inputs[n].dtype))
        return tuple(grads) + (None,)


def mamba3_scan(x, dt, A, lam, theta, B, C, D, chunk=64, W_x=None, W_y=None, h0=None, prevBx0=None,
                angle0=None):
    """Differentiable scan: returns y, h_final, prevBx_final, angle_final.
    Shapes and dtypes as in include/m3.h (x, B, C bf16 or fp32; the rest fp32)."""
    return Mamba3Scan.apply(x, dt, A, lam, theta, B, C, D, W_x, W_y, h0, prevBx0, angle0, chunk)


def _grad(t, dtype):
    """An incoming gradient as the library takes it: a view that autograd cut
    out of a larger one (by torch.cat, say) may start anywhere."""
    t = t.to(dtype).contiguous()
    return t.clone() if t.data_ptr() % 16 else t


def _shaped(g, t):
    """A gradient (or None) in its input's own shape: the library asks for
    element counts, so a gate may be (B, T, C) beside rows (B T, C)."""
    return None if g is None else g.view(t.shape)


class LinearAttention(torch.autograd.Function):
    """Returns (y, s_final); gradients of q, k, v and s0."""

    @staticmethod
    def forward(ctx, q, k, v, log_decay, scale, s0, lengths):
        if ctx.needs_input_grad[3]:
            raise ValueError("log_decay is a constant of linear_attention: it has no gradient (mamba3_scan with "
                             "lam = 1 and theta = 0 learns its decays)")
        y, sf = m3.linattn_chunked_fwd(q, k, v, log_decay, scale=scale, s0=s0, lengths=lengths)
        ctx.save_for_backward(q, k, v, log_decay, s0, lengths)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        return y, sf

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, ds):
        q, k, v, log_decay, s0, lengths = ctx.saved_tensors
        need = dict(zip(("dq", "dk", "dv"), ctx.needs_input_grad[:3]), ds0=ctx.needs_input_grad[5])
        want = tuple(n for n, on in need.items() if on)
        dy = torch.zeros_like(v, memory_format=torch.contiguous_format) if dy is None else _grad(dy, v.dtype)
        g = m3.linattn_chunked_bwd(q, k, v, log_decay, dy, scale=ctx.scale, s0=s0,
                                   ds_final=None if ds is None else _grad(ds, torch.float32), lengths=lengths, want=want)
        return g.get("dq"), g.get("dk"), g.get("dv"), None, None, _shaped(g.get("ds0"), s0), None


def linear_attention(q, k, v, log_decay, scale=None, s0=None, lengths=None):
    """Differentiable linear attention with a decay for each head: returns y
    and s_final (m3.linattn_chunked_fwd).  log_decay is a constant."""
    return LinearAttention.apply(q, k, v, log_decay, scale, s0, lengths)


class GroupNorm(torch.autograd.Function):
    """Returns y; gradients of x, weight, bias and gate."""

    @staticmethod
    def forward(ctx, x, groups, weight, bias, gate, act, eps):
        y, mean, rstd = m3.group_norm_fwd(x, groups, weight, bias, gate=gate, act=act, eps=eps)
        ctx.save_for_backward(x, weight, bias, gate, mean, rstd)
        ctx.groups, ctx.act = groups, act
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, bias, gate, mean, rstd = ctx.saved_tensors
        n = ctx.needs_input_grad
        want = tuple(k for k, on in (("dx", n[0]), ("dweight", n[2]), ("dbias", n[3]), ("dgate", n[4])) if on)
        g = m3.group_norm_bwd(x, _grad(dy, x.dtype), mean, rstd, ctx.groups, weight, bias, gate=gate, act=ctx.act,
                              want=want)
        return (g.get("dx"), None, _shaped(g.get("dweight"), weight), _shaped(g.get("dbias"), bias),
                _shaped(g.get("dgate"), gate), None, None)


def group_norm(x, groups, weight=None, bias=None, gate=None, act="none", eps=1e-5):
    """Differentiable group norm with an activation or a gate, channels last
    (m3.group_norm_fwd)."""
    return GroupNorm.apply(x, groups, weight, bias, gate, act, eps)
