"""Infinities and NaN in group norm on the GPU (marked gpu): they reach what
the definition says and nothing else, in both plans (one token a sequence,
statistics over many tokens), forwards and backwards."""
import math

import pytest
import torch

from lin_reference import norm64
from state_space_lm_b200 import m3

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
# a row of registers with and without vectors; chunks of tokens with and
# without vectors, one vector a thread and several, one token of wide groups
SHAPES = [((6, 64), 2), ((6, 70), 2), ((2, 100, 64), 4), ((2, 100, 18), 2), ((1, 1000, 512), 4), ((2, 9, 4096), 2),
          ((3, 16384), 2)]
BAD = {"inf": (math.inf,), "-inf": (-math.inf,), "nan": (math.nan,), "both": (math.inf, -math.inf)}


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from state_space_lm_b200 import build
    build.build()


def inputs(shape, dtype):
    g = torch.Generator(device="cuda").manual_seed(sum(shape))
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    t, C = DT[dtype], shape[-1]
    return n(*shape).to(t), n(*shape).to(t), n(*shape).to(t), 1 + 0.1 * n(C), 0.1 * n(C)


def same_kind(got, ref):
    """NaN where ref is NaN, the same infinities, finite elsewhere."""
    return bool(((got.isnan() == ref.isnan()) & (got.isposinf() == ref.isposinf()) &
                 (got.isneginf() == ref.isneginf())).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", list(BAD))
@pytest.mark.parametrize("shape,groups", SHAPES, ids=lambda s: "x".join(map(str, s)) if isinstance(s, tuple) else str(s))
def test_what_an_infinity_or_a_nan_reaches(shape, groups, bad, dtype):
    x0, dy, gate, w, b = inputs(shape, dtype)
    B, C = shape[0], shape[-1]
    L = x0[0].numel() // C
    D = C // groups
    last = groups - 1
    for act, z in (("none", None), ("silu", None), ("relu", None), ("silu", gate)):
        y0, mean0, rstd0 = m3.group_norm_fwd(x0, groups, w, b, gate=z, act=act)
        g0 = m3.group_norm_bwd(x0, dy, mean0, rstd0, groups, w, b, gate=z, act=act)
        for t in sorted({0, L // 2, L - 1}):               # the first chunk, one between, the last
            x = x0.clone()
            for i, v in enumerate(BAD[bad]):
                x.view(B, L, groups, D)[0, (t + i) % L, last, (D // 3 + 2 * i) % D] = v
            y, mean, rstd = m3.group_norm_fwd(x, groups, w, b, gate=z, act=act)
            ry, rm, rr = norm64(x, groups, w, b, z, act)
            assert same_kind(mean, rm), (act, t)
            assert same_kind(rstd, rr) and bool(rstd[0, last].isnan()), (act, t)
            assert same_kind(y, ry) and bool(y.view(B, L, groups, D)[0, :, last].isnan().all()), (act, t)
            g = m3.group_norm_bwd(x, dy, mean, rstd, groups, w, b, gate=z, act=act)
            hit = torch.zeros(B, L, groups, D, dtype=torch.bool, device="cuda")
            hit[0, :, last] = True
            hit = hit.view(shape)
            cols = torch.arange(C, device="cuda") >= C - D
            # every element of the group moves its statistics, and none elsewhere does
            assert torch.equal(g["dx"].isnan(), hit), (act, t)
            assert torch.equal(y[~hit], y0[~hit]) and torch.equal(g["dx"][~hit], g0["dx"][~hit])
            assert torch.equal(g["dweight"].isnan(), cols), (act, t)
            assert torch.equal(g["dweight"][~cols], g0["dweight"][~cols])
            assert torch.equal(g["dbias"][~cols], g0["dbias"][~cols])
            if z is not None:
                assert torch.equal(g["dgate"].isnan(), hit) and torch.equal(g["dgate"][~hit], g0["dgate"][~hit])


def test_statistics_of_no_positions():
    """The mean of nothing is NaN, not what the memory held."""
    held = torch.ones(2, 2, 4, device="cuda")
    del held
    x = torch.empty(2, 0, 64, device="cuda")
    y, mean, rstd = m3.group_norm_fwd(x, 4)
    assert y.shape == x.shape and bool(mean.isnan().all()) and bool(rstd.isnan().all())
    out = [torch.empty_like(x), torch.ones(2, 4, device="cuda"), None]
    m3.group_norm_fwd(x, 4, out=out)
    assert bool(out[1].isnan().all())
