"""The autograd wrappers with inputs whose element counts fit and whose shapes
differ from the library's: a gate (B, T, C) beside rows (B T, C), a state
(B, H, dk dv), a weight (1, C).  Their gradients have their own shapes."""
import torch

import lin_reference as ref
from state_space_lm_b200 import autograd as ag
from state_space_lm_b200 import m3


def gen(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, dtype=torch.float64).requires_grad_()   # noqa: E731


def test_group_norm(monkeypatch):
    def f(x, groups, weight=None, bias=None, gate=None, act="none", eps=1e-5, **kw):
        return tuple(t.detach() for t in ref.norm64(x, groups, weight.view(-1), bias.view(-1), gate.view(x.shape), act, eps))

    def g(x, dy, mean, rstd, groups, weight=None, bias=None, gate=None, act="none", want=None, **kw):
        with torch.enable_grad():
            ts = dict(dx=x, dweight=weight.view(-1), dbias=bias.view(-1), dgate=gate.view(x.shape))
            ts = {k: t.detach().requires_grad_() for k, t in ts.items()}
            y = ref.norm64(ts["dx"], groups, ts["dweight"], ts["dbias"], ts["dgate"], act)[0]
        return {k: t for k, t in zip(ts, torch.autograd.grad(y, list(ts.values()), dy)) if k in want}

    monkeypatch.setattr(m3, "group_norm_fwd", f)
    monkeypatch.setattr(m3, "group_norm_bwd", g)
    n = gen(1)
    x, w, b, z = n(6, 8), n(1, 8), n(2, 4), n(2, 3, 8)
    assert torch.autograd.gradcheck(lambda *a: ag.group_norm(a[0], 2, a[1], a[2], a[3], "silu"), (x, w, b, z))


def test_linear_attention(monkeypatch):
    def f(q, k, v, ld, scale=None, s0=None, lengths=None, **kw):
        y, s = ref.forward64(q, k, v, ld, scale, s0.view(2, 2, 3, 4), lengths)
        return y.contiguous(), s.reshape(s0.shape)

    def g(q, k, v, ld, dy, scale=None, s0=None, ds_final=None, lengths=None, want=None, **kw):
        out = ref.backward64(q, k, v, ld, scale, dy, s0.view(2, 2, 3, 4),
                             None if ds_final is None else ds_final.view(2, 2, 3, 4), lengths)
        return {k: t.contiguous() for k, t in zip(("dq", "dk", "dv", "ds0"), out) if k in want}

    monkeypatch.setattr(m3, "linattn_chunked_fwd", f)
    monkeypatch.setattr(m3, "linattn_chunked_bwd", g)
    n = gen(2)
    ld = torch.tensor([-0.3, -1.1], dtype=torch.float64)
    args = n(2, 5, 1, 3), n(2, 5, 1, 3), n(2, 5, 2, 4), n(2, 2, 12)
    assert torch.autograd.gradcheck(lambda *a: ag.linear_attention(a[0], a[1], a[2], ld, 0.7, a[3]), args)
