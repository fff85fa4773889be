"""Linear attention and group norm without a GPU: the binding's checks, the
library's own refusals (no call here passes validation, or it enqueues
nothing), and the autograd wrappers' plumbing with a 64-bit stand-in for the
library."""
import ctypes
import types

import pytest
import torch

import lin_reference as ref
from state_space_lm_b200 import autograd as ag
from state_space_lm_b200 import build as m3build
from state_space_lm_b200 import m3


@pytest.fixture(scope="module")
def L():
    m3build.build()
    return m3.lib()


FAKE, MIS, ODD = 0x10000, 0x10004, 0x10001      # never dereferenced: every call below is refused or empty


def ldims(**kw):
    b = dict(batch=2, seqlen=8, nheads=4, headdim=8, dstate=16, ngroups=2, ld_q=0, ld_k=0, ld_v=0)
    b.update(kw)
    return m3.LinattnDims(*[b[k] for k in ("batch", "seqlen", "nheads", "headdim", "dstate", "ngroups", "ld_q", "ld_k",
                                           "ld_v")])


def fwd(L, d, q=FAKE, k=FAKE, v=FAKE, dtype=m3.M3_BF16, ld=FAKE, scale=1.0, s0=None, lengths=None, y=FAKE, sf=None,
        ws=None, nbytes=0):
    return L.m3_linattn_chunked_fwd(q, k, v, dtype, ld, scale, s0, lengths, d, y, sf, ws, nbytes, None)


def bwd(L, d, q=FAKE, k=FAKE, v=FAKE, dtype=m3.M3_BF16, ld=FAKE, scale=1.0, dy=FAKE, g=None, ws=FAKE, nbytes=1 << 40):
    g = m3.LinattnGrads(FAKE, FAKE, FAKE, FAKE) if g is None else g
    return L.m3_linattn_chunked_bwd(q, k, v, dtype, ld, scale, None, None, d, dy, None, ctypes.byref(g) if g else None,
                                    ws, nbytes, None)


def step(L, d, q=FAKE, dtype=m3.M3_F32, ld=FAKE, scale=1.0, s=FAKE, y=FAKE):
    return L.m3_linattn_step_decode(q, FAKE, FAKE, dtype, ld, scale, d, s, y, None)


def test_linattn_refusals(L):
    INV, UNS = m3.M3_ERR_INVALID_ARG, m3.M3_ERR_UNSUPPORTED
    n0 = m3.launch_count()
    for call in (lambda **kw: fwd(L, ldims(**kw)), lambda **kw: bwd(L, ldims(**kw)), lambda **kw: step(L, ldims(**kw))):
        assert call(batch=-1) == INV and call(nheads=0) == INV and call(headdim=0) == INV and call(dstate=0) == INV
        assert call(ngroups=3) == INV and call(ngroups=-1) == INV
        assert call(ld_q=31) == INV and call(ld_k=-8) == INV and call(ld_v=31) == INV     # rows would overlap
        assert call(dstate=257) == UNS and call(headdim=257) == UNS and call(dstate=256, headdim=128) == UNS
        assert call(nheads=4098, ngroups=1) == UNS and call(batch=(1 << 24) + 1) == UNS
        assert call(batch=1 << 20, ld_q=1 << 40) == UNS
    for call in (lambda **kw: fwd(L, ldims(), **kw), lambda **kw: bwd(L, ldims(), **kw), lambda **kw: step(L, ldims(), **kw)):
        assert call(q=None) == INV and call(q=ODD) == INV and call(ld=None) == INV and call(ld=MIS) == INV
        assert call(dtype=5) == INV and call(scale=float("nan")) == INV and call(scale=float("inf")) == INV
    assert fwd(L, ldims(seqlen=-1)) == INV and fwd(L, ldims(seqlen=(1 << 30) + 1, batch=1)) == UNS
    assert fwd(L, ldims(), y=None) == INV and fwd(L, ldims(), y=MIS) == INV and fwd(L, ldims(), s0=MIS) == INV
    assert fwd(L, ldims(), lengths=MIS) == INV and fwd(L, ldims(), sf=MIS) == INV
    assert step(L, ldims(), s=None) == INV and step(L, ldims(), y=MIS) == INV and step(L, ldims(), q=0x10002) == INV
    assert bwd(L, ldims(), dy=None) == INV and bwd(L, ldims(), dy=MIS) == INV and bwd(L, ldims(), g=0) == INV
    assert bwd(L, ldims(), g=m3.LinattnGrads(MIS, None, None, None)) == INV
    # shared heads need a workspace; a long sequence over few lanes too
    assert bwd(L, ldims(), ws=None, nbytes=0) == m3.M3_ERR_WORKSPACE
    d = ldims(batch=1, nheads=1, ngroups=1, seqlen=32768, dstate=128, headdim=64)
    need = L.m3_linattn_workspace_bytes(m3.M3_WS_LINATTN_FWD, d, m3.M3_BF16)
    assert need > 0
    assert fwd(L, d) == m3.M3_ERR_WORKSPACE and fwd(L, d, ws=FAKE, nbytes=need - 1) == m3.M3_ERR_WORKSPACE
    # queries of what the calls refuse
    assert L.m3_linattn_workspace_bytes(7, d, m3.M3_BF16) == 0
    assert L.m3_linattn_workspace_bytes(0, ldims(dstate=0), m3.M3_BF16) == 0
    # an empty batch is valid and enqueues nothing
    assert fwd(L, ldims(batch=0), q=None, k=None, v=None, y=None) == m3.M3_OK
    assert bwd(L, ldims(batch=0), q=None, k=None, v=None, dy=None) == m3.M3_OK
    assert step(L, ldims(batch=0), q=None, s=None, y=None) == m3.M3_OK
    assert m3.launch_count() == n0


def test_group_norm_refusals(L):
    INV, UNS = m3.M3_ERR_INVALID_ARG, m3.M3_ERR_UNSUPPORTED
    nd = lambda **kw: m3.NormDims(*[{**dict(batch=2, seqlen=8, channels=12, ngroups=3), **kw}[k]  # noqa: E731
                                    for k in ("batch", "seqlen", "channels", "ngroups")])
    f = lambda d=None, x=FAKE, dt=0, w=None, gate=None, act=1, eps=1e-5, y=FAKE, mean=FAKE, ws=FAKE, nb=1 << 40: (  # noqa: E731
        L.m3_group_norm_fwd(x, dt, w, None, gate, act, eps, d or nd(), y, mean, None, ws, nb, None))
    b = lambda d=None, x=FAKE, dt=0, gate=None, act=1, mean=FAKE, dx=FAKE, dg=None, ws=FAKE, nb=1 << 40: (  # noqa: E731
        L.m3_group_norm_bwd(x, FAKE, dt, None, None, gate, act, mean, FAKE, d or nd(), dx, None, None, dg, ws, nb, None))
    n0 = m3.launch_count()
    for c in (f, b):
        assert c(nd(ngroups=5)) == INV and c(nd(ngroups=0)) == INV and c(nd(channels=0)) == INV
        assert c(nd(batch=-1)) == INV and c(nd(seqlen=-1)) == INV and c(dt=3) == INV
        assert c(act=4) == INV and c(act=-1) == INV and c(x=None) == INV and c(x=MIS) == INV and c(gate=MIS) == INV
        assert c(nd(channels=16386)) == UNS and c(nd(seqlen=(1 << 30) + 1)) == UNS and c(nd(batch=(1 << 24) + 1)) == UNS
        assert c(ws=None, nb=0) == m3.M3_ERR_WORKSPACE and c(ws=FAKE, nb=3) == m3.M3_ERR_WORKSPACE
    assert f(eps=-1.0) == INV and f(eps=float("nan")) == INV and f(y=None) == INV and f(mean=MIS) == INV and f(w=MIS) == INV
    assert b(mean=None) == INV and b(dg=FAKE) == INV and b(dx=MIS) == INV          # dgate without a gate
    assert f(nd(batch=0), x=None, y=None) == m3.M3_OK and f(nd(seqlen=0), x=None, y=None) == m3.M3_OK
    assert m3.launch_count() == n0


def _stops_at_the_pointers(fn):
    with pytest.raises(ValueError, match="expected a CUDA tensor"):
        fn()


def test_binding_checks_linattn():
    m3build.build()
    z = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t)  # noqa: E731
    q, v, ld = z(2, 6, 2, 8), z(2, 6, 4, 16), z(4)
    dy, S = z(2, 6, 4, 16), z(2, 4, 8, 16)
    _stops_at_the_pointers(lambda: m3.linattn_chunked_fwd(q, q, v, ld))
    _stops_at_the_pointers(lambda: m3.linattn_chunked_bwd(q, q, v, ld, dy))
    _stops_at_the_pointers(lambda: m3.linattn_step_decode(q[:, 0], q[:, 0], v[:, 0], ld, S))
    for call in (lambda a, b, c, l: m3.linattn_chunked_fwd(a, b, c, l), lambda a, b, c, l: m3.linattn_chunked_bwd(a, b, c, l, dy)):
        for args, word in (((q, z(2, 6, 2, 7), v, ld), "k has"), ((z(2, 5, 2, 8), q, v, ld), "q has"),
                           ((q, q, v, z(3)), "log_decay"), ((q, q.bfloat16(), v, ld), "k is torch.bfloat16"),
                           ((q, q, v, ld.double()), "log_decay is"), ((q[:, 0], q, v, ld), "are"),
                           ((z(2, 6, 3, 8), z(2, 6, 3, 8), v, ld), "3 groups"), ((q.half(), q.half(), v.half(), ld), "bfloat16"),
                           ((z(2, 6, 8, 2), q, v, ld), "q is|k is"),
                           ((q.transpose(2, 3).contiguous().transpose(2, 3), q, v, ld), "strides"),
                           ((z(1, 1, 2, 8).expand(2, 6, 2, 8), q, v, ld), "strides"),
                           ((z(2, 9, 2, 8)[:, :6], q, v, ld), "strides")):
            with pytest.raises(ValueError, match=word):
                call(*args)
    with pytest.raises(ValueError, match="s0"):
        m3.linattn_chunked_fwd(q, q, v, ld, s0=z(2, 4, 8, 15))
    with pytest.raises(ValueError, match="lengths is torch.int64"):
        m3.linattn_chunked_fwd(q, q, v, ld, lengths=z(2, t=torch.int64))
    with pytest.raises(ValueError, match="y has"):
        m3.linattn_chunked_fwd(q, q, v, ld, out=(z(2, 6, 4, 15), None))
    with pytest.raises(ValueError, match="dy has"):
        m3.linattn_chunked_bwd(q, q, v, ld, z(2, 6, 4, 15))
    with pytest.raises(ValueError, match="no gradient 'dld'"):
        m3.linattn_chunked_bwd(q, q, v, ld, dy, want=("dld",))
    with pytest.raises(ValueError, match="ds0 is"):
        m3.linattn_chunked_bwd(q, q, v, ld, dy, out={"ds0": S.bfloat16()})
    with pytest.raises(ValueError, match=": s has"):
        m3.linattn_step_decode(q[:, 0], q[:, 0], v[:, 0], ld, S[:1])
    other = types.SimpleNamespace(device=torch.device("cuda", 1))
    for call in (lambda: m3.linattn_chunked_fwd(q, q, v, ld, stream=other),
                 lambda: m3.linattn_chunked_bwd(q, q, v, ld, dy, stream=other),
                 lambda: m3.linattn_step_decode(q[:, 0], q[:, 0], v[:, 0], ld, S, stream=other),
                 lambda: m3.group_norm_fwd(dy, 4, stream=other),
                 lambda: m3.group_norm_bwd(dy, dy, z(2, 4), z(2, 4), 4, stream=other)):
        with pytest.raises(ValueError, match="stream is on cuda:1"):
            call()
    with pytest.raises(ValueError, match="0 wide"):
        m3.linattn_chunked_fwd(z(2, 6, 2, 0), z(2, 6, 2, 0), v, ld)
    # what the binding takes as it is: slices of a fused projection, one token of a longer tensor
    flat = z(2, 6, 100)
    a, b, c = flat[..., :16].unflatten(-1, (2, 8)), flat[..., 16:32].unflatten(-1, (2, 8)), flat[..., 36:100].unflatten(-1, (4, 16))
    d = m3._linattn_dims("w", a, b, c, True)[0]
    assert (d.ld_q, d.ld_k, d.ld_v) == (100, 100, 100)
    d = m3._linattn_dims("w", q[:, 3], q[:, 3], v[:, 3], False)[0]
    assert (d.ld_q, d.ld_v, d.batch, d.ngroups) == (6 * 16, 6 * 64, 2, 2)
    d = m3._linattn_dims("w", q[:1, :1], q[:1, :1], v[:1, :1], True)[0]
    assert (d.ld_q, d.ld_v) == (16, 64)


def test_binding_checks_group_norm():
    m3build.build()
    z = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t)  # noqa: E731
    x, st = z(3, 5, 12), z(3, 4)
    _stops_at_the_pointers(lambda: m3.group_norm_fwd(x, 4, z(12), z(12), gate=x, act="silu"))
    _stops_at_the_pointers(lambda: m3.group_norm_bwd(x, x, st, st, 4))
    for kw, word in ((dict(weight=z(11)), "weight"), (dict(bias=z(12, t=torch.bfloat16)), "bias is"),
                     (dict(gate=z(3, 5, 11)), "gate has"), (dict(act="tanh"), "act is one of")):
        with pytest.raises(ValueError, match=word):
            m3.group_norm_fwd(x, 4, **kw)
        with pytest.raises(ValueError, match=word):
            m3.group_norm_bwd(x, x, st, st, 4, **kw)
    with pytest.raises(ValueError, match="bfloat16"):
        m3.group_norm_fwd(x.half(), 4)
    with pytest.raises(ValueError, match="dy has"):
        m3.group_norm_bwd(x, z(3, 5, 11), st, st, 4)
    with pytest.raises(ValueError, match="rstd has"):
        m3.group_norm_bwd(x, x, st, z(3, 3), 4)
    with pytest.raises(ValueError, match="no gradient 'dgate'"):
        m3.group_norm_bwd(x, x, st, st, 4, want=("dgate",))
    with pytest.raises(ValueError, match="mean has"):
        m3.group_norm_fwd(x, 4, out=(x, z(3, 5), None))


# ---- autograd plumbing --------------------------------------------------------
def test_linear_attention_gradients_route_to_their_inputs(monkeypatch):
    def f(q, k, v, ld, scale=None, s0=None, lengths=None, **kw):
        return tuple(t.contiguous() for t in ref.forward64(q, k, v, ld, q.shape[-1] ** -0.5 if scale is None else scale, s0, lengths))

    def g(q, k, v, ld, dy, scale=None, s0=None, ds_final=None, lengths=None, want=None, **kw):
        out = ref.backward64(q, k, v, ld, q.shape[-1] ** -0.5 if scale is None else scale, dy, s0, ds_final, lengths)
        return {n: t.contiguous() for n, t in zip(("dq", "dk", "dv", "ds0"), out) if n in want}

    monkeypatch.setattr(m3, "linattn_chunked_fwd", f)
    monkeypatch.setattr(m3, "linattn_chunked_bwd", g)
    gen = torch.Generator().manual_seed(2)
    n = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64).requires_grad_()  # noqa: E731
    q, k, v, s0 = n(2, 5, 1, 3), n(2, 5, 1, 3), n(2, 5, 2, 4), n(2, 2, 3, 4)
    ld, lens = torch.tensor([-0.3, -1.1], dtype=torch.float64), torch.tensor([5, 3], dtype=torch.int32)
    assert torch.autograd.gradcheck(lambda *a: ag.linear_attention(a[0], a[1], a[2], ld, 0.7, a[3], lens), (q, k, v, s0))
    assert torch.autograd.gradcheck(lambda *a: ag.linear_attention(*a, ld), (q, k, v))
    # a part of the inputs only
    y, _ = ag.linear_attention(q, k.detach(), v, ld)
    y.sum().backward()
    assert q.grad is not None and v.grad is not None and k.grad is None
    with pytest.raises(ValueError, match="constant"):
        ag.linear_attention(q, k, v, ld.clone().requires_grad_())


def test_group_norm_gradients_route_to_their_inputs(monkeypatch):
    def f(x, groups, weight=None, bias=None, gate=None, act="none", eps=1e-5, **kw):
        return tuple(t.detach() for t in ref.norm64(x, groups, weight, bias, gate, act, eps))

    def g(x, dy, mean, rstd, groups, weight=None, bias=None, gate=None, act="none", want=None, **kw):
        leaves = {"dx": x, "dweight": weight, "dbias": bias, "dgate": gate}
        with torch.enable_grad():
            ts = {n: t.detach().requires_grad_() for n, t in leaves.items() if t is not None}
            y = ref.norm64(ts["dx"], groups, ts.get("dweight"), ts.get("dbias"), ts.get("dgate"), act)[0]
        return {n: t for n, t in zip(ts, torch.autograd.grad(y, list(ts.values()), dy)) if n in want}

    monkeypatch.setattr(m3, "group_norm_fwd", f)
    monkeypatch.setattr(m3, "group_norm_bwd", g)
    gen = torch.Generator().manual_seed(4)
    n = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64).requires_grad_()  # noqa: E731
    x, w, b, z = n(2, 3, 8), n(8), n(8), n(2, 3, 8)
    assert torch.autograd.gradcheck(lambda *a: ag.group_norm(a[0], 2, a[1], a[2], a[3], "silu"), (x, w, b, z))
    assert torch.autograd.gradcheck(lambda *a: ag.group_norm(a[0], 4, act="gelu"), (x,))
    y = ag.group_norm(x, 2, w.detach(), b, act="silu")
    y.sum().backward()
    assert x.grad is not None and b.grad is not None and w.grad is None
