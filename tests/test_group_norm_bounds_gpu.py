"""Group norm on the GPU (marked gpu), each element of its outputs and gradients
against 64-bit formulas within a bound from that element's own terms."""
import pytest
import torch

import norm_bounds
from lin_reference import norm64, within
from state_space_lm_b200 import m3

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from state_space_lm_b200 import build
    build.build()


def check(shape, groups, dtype, gated, act, shift=0.25, affine=True):
    g = torch.Generator(device="cuda").manual_seed(sum(shape) + groups)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
    C, t = shape[-1], DT[dtype]
    x = (1.5 * n(*shape) + shift).to(t)
    gate = n(*shape).to(t) if gated else None
    # parts along a constant and along the output, as a loss has: the means that
    # dx subtracts are of its own size
    dy = (n(*shape) + 0.7 + 0.4 * (x.float() - shift)).to(t)
    w, b = (1 + 0.1 * n(C), 0.1 * n(C)) if affine else (None, None)
    if act == "relu":                                      # keep its argument off the jump of the derivative
        if gated:
            gate = torch.where(gate.abs() < 0.1, torch.ones_like(gate), gate)
        else:
            dy = torch.where(norm64(x, groups, w, b)[0].abs() < 1e-2, torch.zeros_like(dy), dy)
    kw = dict(gate=gate, act=act)
    y, mean, rstd = m3.group_norm_fwd(x, groups, w, b, **kw)
    ref = norm_bounds.forward(x, groups, w, b, gate, act)
    for k, got in (("mean", mean), ("rstd", rstd), ("y", y)):
        within(got, *ref[k], k)
    g = m3.group_norm_bwd(x, dy, mean, rstd, groups, w, b, **kw)
    ref = norm_bounds.backward(x, dy, mean, rstd, groups, w, b, gate, act)
    assert set(g) == set(ref)
    for k in ref:
        within(g[k], *ref[k], k)


# one token a sequence: every team width, with and without vectors, groups past
# the registers; many tokens: one vector a thread and several, phases, chunks
# that do and do not divide, more sequences than CTAs fit
SHAPES = [((33, 64), 4), ((1000, 128), 2), ((257, 1000), 8), ((64, 1024), 16), ((3, 520), 1), ((9, 4096), 1),
          ((5, 9000), 2), ((2, 16384), 1), ((300, 96), 12), ((2, 5, 24), 3), ((3, 17, 64), 8), ((2, 100, 1024), 32),
          ((1, 1000, 70), 7), ((4, 33, 512), 1), ((1, 700, 16384), 4), ((8, 300, 1024), 32), ((1, 5000, 264), 3),
          ((400, 30, 40), 5), ((2, 3, 5, 48), 6)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("shape,groups", SHAPES, ids=lambda s: "x".join(map(str, s)) if isinstance(s, tuple) else str(s))
def test_every_element(shape, groups, gated, dtype):
    for act in ("silu", "gelu") if gated else ("none", "silu", "relu"):
        check(shape, groups, dtype, gated, act)


def test_a_large_mean():
    for shape, groups in (((65, 128), 2), ((300, 70), 2), ((2, 400, 64), 4), ((1, 900, 18), 2)):
        for act in ("none", "silu"):
            check(shape, groups, "f32", False, act, shift=4096.0)


# phases of a vector that share its tokens: 256, 85 and 64 of them; hundreds of
# sequences, one chunk each
@pytest.mark.parametrize("shape,groups", [((300, 1000, 4), 1), ((2, 3000, 4), 1), ((3, 3000, 8), 2), ((1, 3000, 3), 3), ((308, 6, 3), 3),
                                          ((928, 3, 3), 3), ((310, 3, 8), 8), ((40, 900, 16), 1)],
                         ids=lambda s: "x".join(map(str, s)) if isinstance(s, tuple) else str(s))
def test_the_mean_of_means(shape, groups):
    for shift in (100.0, 4096.0, -4096.0):
        check(shape, groups, "f32", False, "none", shift=shift)


def test_no_weight_and_no_bias():
    for shape in ((50, 64), (2, 30, 64)):
        check(shape, 4, "f32", False, "gelu", affine=False)
