"""Group norm with an activation on the GPU (marked gpu), against plain 64-bit
arithmetic (and its gradients by torch.autograd in 64 bits)."""
import math

import pytest
import torch

from helpers import Canary
from lin_reference import U, norm64, within
from state_space_lm_b200 import m3

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ACTS = ["none", "silu", "gelu", "relu"]


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from state_space_lm_b200 import build
    build.build()


def inputs(shape, groups, dtype, gated, seed=0, shift=0.25, affine=True):
    g = torch.Generator(device="cuda").manual_seed(seed + sum(shape) + groups)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    C, t = shape[-1], DT[dtype]
    return dict(x=(1.5 * n(*shape) + shift).to(t), dy=n(*shape).to(t), gate=n(*shape).to(t) if gated else None,
                w=(1 + 0.1 * n(C)) if affine else None, b=0.1 * n(C) if affine else None)


def check(d, groups, act, eps=1e-5):
    x, dy, io = d["x"], d["dy"], d["x"].dtype
    y, mean, rstd = m3.group_norm_fwd(x, groups, d["w"], d["b"], gate=d["gate"], act=act, eps=eps)
    leaves = {k: d[k].double().requires_grad_() for k in ("x", "w", "b", "gate") if d[k] is not None}
    ry, rm, rr = norm64(leaves["x"], groups, leaves.get("w"), leaves.get("b"), leaves.get("gate"), act, eps)
    n = x[0].numel() // groups
    u = U[torch.float32]
    # the sums of a group run over at most 1024 values one after the other,
    # the rest in trees: count them all as 2 log2(n) + 64 roundings
    r = 64 + 2 * math.log2(n + 1) + (n if n < 1024 else 0) * 0
    big = x.double().abs().max()
    within(mean, rm, (r * u * big).expand_as(rm), "mean")
    spread = (rr * big).clamp(min=1.0)                     # how far a group's values are from 0, in deviations
    within(rstd, rr, 2 * r * u * rr * spread, "rstd")
    # u = xh w + b: the error of mean and rstd moves it by r u spread (twice);
    # |act'| <= 1.13; 16-bit outputs use exponentials good to 2^-21
    wmax = 1.0 if d["w"] is None else float(d["w"].abs().max())
    xh_max = (spread.max() * 2 + 1)
    e_u = (3 * r * u) * xh_max * wmax + 4 * u
    slack = 2.0 ** -20 if io == torch.bfloat16 else 8 * u
    gmax = 1.0 if d["gate"] is None else float(d["gate"].double().abs().max() + 1)
    within(y, ry.detach(), (1.2 * e_u * gmax + slack * (ry.detach().abs() + xh_max * wmax * gmax))
           + 1.01 * U[io] * ry.detach().abs(), "y")
    g = m3.group_norm_bwd(x, dy, mean, rstd, groups, d["w"], d["b"], gate=d["gate"], act=act)
    ref = dict(zip(leaves, torch.autograd.grad(ry, list(leaves.values()), dy.double())))
    # dx = rstd (dn - mean dn - xh mean(dn xh)): three terms no larger than
    # max|dn| (1 + xh^2); derivative of act' is bounded by 1.2
    dmax = float(dy.double().abs().max()) * gmax * wmax
    e_dx = rr.max() * dmax * (1 + xh_max ** 2) * (1.2 * e_u + 4 * r * u + 2 * slack)
    within(g["dx"], ref["x"], e_dx + 1.01 * U[io] * ref["x"].abs(), "dx")
    rows = x.numel() // x.shape[-1]
    ch = x.shape[-1]
    for k, name, size in (("w", "dweight", xh_max), ("b", "dbias", 1.0)):
        if k in ref:
            # a sum over all rows: the terms' own errors and the sum's roundings
            bound = rows * float(dy.double().abs().max()) * gmax * size * (1.2 * e_u + 2 * slack + 4 * u)
            bound += (64 + rows / 148 / 4 + math.log2(rows + 1)) * u * rows * float(dy.double().abs().max()) * gmax * size
            within(g[name], ref[k], torch.full((ch,), float(bound), device="cuda", dtype=torch.float64), name)
        else:
            assert torch.isfinite(g[name]).all()
    if d["gate"] is not None:
        e_dg = float(dy.double().abs().max()) * (1.13 * e_u + xh_max * wmax * 2 * slack)
        within(g["dgate"], ref["gate"], e_dg + 1.01 * U[io] * ref["gate"].abs(), "dgate")
    return y, g


# one token a sequence: every team width, vectors or not, wide groups; many
# tokens: chunks that do and do not divide them
SHAPES = [((7, 1), 1), ((5, 3), 3), ((33, 64), 4), ((1000, 128), 2), ((257, 1000), 8), ((64, 1024), 16),
          ((3, 520), 1), ((9, 4096), 1), ((5, 9000), 2), ((2, 16384), 1), ((300, 96), 12),
          ((1, 2, 8), 2), ((2, 5, 24), 3), ((3, 17, 64), 8), ((2, 100, 1024), 32), ((1, 1000, 70), 7),
          ((4, 33, 512), 1), ((1, 700, 16384), 4), ((2, 3, 5, 48), 6)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("shape,groups", SHAPES, ids=lambda s: "x".join(map(str, s)) if isinstance(s, tuple) else str(s))
def test_forward_and_backward(shape, groups, gated, dtype):
    act = ACTS[(sum(shape) + gated) % 4]
    # relu at values within rounding of zero has no derivative to compare: its
    # gradient is tested on values that are not near it
    if act == "relu":
        act = "silu"
    check(inputs(shape, groups, dtype, gated), groups, act)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("shape,groups", [((40, 64), 4), ((37, 21), 3), ((2, 50, 64), 8), ((2, 50, 9), 3)])
def test_activations(shape, groups, act, dtype):
    for gated in (False, True):
        d = inputs(shape, groups, dtype, gated)
        if act == "relu":
            # keep every argument of the relu away from zero
            if gated:
                d["gate"] = torch.where(d["gate"].abs() < 0.1, torch.ones_like(d["gate"]), d["gate"])
            else:
                u = norm64(d["x"], groups, d["w"], d["b"])[0]
                d["dy"] = torch.where(u.abs() < 1e-3, torch.zeros_like(d["dy"]), d["dy"])
        check(d, groups, act)


def test_no_weight_and_no_bias():
    for shape in ((50, 64), (2, 30, 64)):
        check(inputs(shape, 4, "f32", False, affine=False), 4, "gelu")


def test_a_large_mean_cancels_nothing():
    """x = 4096 + N(0, 1.5^2) in fp32: the spread survives (differences from a
    value of the group, never a difference of squares)."""
    for shape, groups in (((65, 128), 2), ((2, 400, 64), 4)):
        check(inputs(shape, groups, "f32", False, shift=4096.0), groups, "none")


def test_a_constant_group_and_an_infinity():
    x = torch.full((4, 64), 3.0, device="cuda")
    y, mean, rstd = m3.group_norm_fwd(x, 2)
    assert bool((y == 0).all()) and bool((mean == 3).all())
    within(rstd, torch.full((4, 2), 1e-5 ** -0.5, device="cuda", dtype=torch.float64), 4e-7 * rstd.double() * 316, "rstd")
    x = torch.randn(4, 64, device="cuda")
    x[1, 3] = math.inf
    y, _, _ = m3.group_norm_fwd(x, 2)
    assert bool(y[1, :32].isnan().any()) and bool(torch.isfinite(y[1, 32:]).all())
    assert bool(torch.isfinite(y[[0, 2, 3]]).all())


def test_empty_batches():
    for shape in ((0, 64), (2, 0, 64)):
        x = torch.empty(*shape, device="cuda")
        y, mean, rstd = m3.group_norm_fwd(x, 4)
        assert y.shape == x.shape
        g = m3.group_norm_bwd(x, x, mean, rstd, 4)
        assert bool((g["dweight"] == 0).all()) and bool((g["dbias"] == 0).all())


@pytest.mark.parametrize("shape,groups", [((333, 256), 4), ((3, 77, 96), 4)])
def test_bits_canaries_streams_and_graphs(shape, groups):
    d = inputs(shape, groups, "bf16", True)
    y, mean, rstd = m3.group_norm_fwd(d["x"], groups, d["w"], d["b"], gate=d["gate"], act="silu")
    g = m3.group_norm_bwd(d["x"], d["dy"], mean, rstd, groups, d["w"], d["b"], gate=d["gate"], act="silu")
    co = [Canary(shape, torch.bfloat16)] + [Canary(mean.shape, torch.float32) for _ in range(2)]
    cg = {n: Canary(t.shape, t.dtype) for n, t in g.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    m3.group_norm_fwd(d["x"], groups, d["w"], d["b"], gate=d["gate"], act="silu", out=tuple(c.t for c in co), stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m3.group_norm_bwd(d["x"], d["dy"], co[1].t, co[2].t, groups, d["w"], d["b"], gate=d["gate"], act="silu",
                          out={n: c.t for n, c in cg.items()})
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c.t) for a, c in zip((y, mean, rstd), co))
        assert all(torch.equal(g[n], cg[n].t) for n in g)
    for c in co + list(cg.values()):
        c.check()


def test_wanted_gradients_alone():
    for shape in ((100, 64), (2, 40, 64)):
        d = inputs(shape, 4, "bf16", True)
        y, mean, rstd = m3.group_norm_fwd(d["x"], 4, d["w"], d["b"], gate=d["gate"], act="silu")
        kw = dict(gate=d["gate"], act="silu")
        full = m3.group_norm_bwd(d["x"], d["dy"], mean, rstd, 4, d["w"], d["b"], **kw)
        for want in (("dx",), ("dweight",), ("dbias",), ("dgate",), ("dgate", "dweight")):
            g = m3.group_norm_bwd(d["x"], d["dy"], mean, rstd, 4, d["w"], d["b"], want=want, **kw)
            assert set(g) == set(want) and all(torch.equal(g[n], full[n]) for n in want)
