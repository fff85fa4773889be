"""Group norm over sequences with thousands of groups on the GPU (marked gpu):
the statistics of all groups stand in shared memory, around and above what a
launch gets without asking for more, in any order of the calls."""
import threading

import pytest
import torch

from lin_reference import U, norm64, within
from state_space_lm_b200 import m3

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from state_space_lm_b200 import build
    build.build()


def inputs(L, C, dtype, gated=False):
    g = torch.Generator(device="cuda").manual_seed(C)
    n = lambda: torch.randn(2, L, C, generator=g, device="cuda").to(DT[dtype])  # noqa: E731
    return n(), n() if gated else None


def check(L, C, groups, dtype, gated):
    x, gate = inputs(L, C, dtype, gated)
    y, mean, rstd = m3.group_norm_fwd(x, groups, gate=gate, act="relu" if gated else "none")
    ry, rm, rr = norm64(x, groups, None, None, gate, "relu" if gated else "none")
    # at most 100 values of a group are summed, from differences of one of them
    # (6 deviations at the most): 140 roundings, of the spread or its square
    xh = ((x.double().view(2, L, groups, -1) - rm[:, None, :, None]) * rr[:, None, :, None]).abs().amax((1, 3))
    u = U[torch.float32]
    within(mean, rm, 140 * u * (rm.abs() + xh / rr), "mean")
    within(rstd, rr, 140 * u * rr * (1 + xh ** 2), "rstd")
    z = 1.0 if gate is None else gate.double().abs()
    e = (3 * 140 * u * (1 + xh) * (1 + xh ** 2))[:, None, :, None].expand(2, L, groups, C // groups).reshape(x.shape)
    within(y, ry, e * z + 1.01 * U[x.dtype] * ry.abs(), "y")


# 8 bytes a group beside 2 KB: 5888 groups are 48 KB together, 6144 alone;
# ascending, so that no larger call has gone before (vectors and single elements)
@pytest.mark.parametrize("groups", [5119, 5121, 5888, 5889, 6000, 6144, 6145, 16384])
def test_forward_and_backward(groups):
    for dtype, gated in (("f32", False), ("bf16", True)):
        check(40, groups, groups, dtype, gated)
    x, _ = inputs(40, groups, "f32")
    y, mean, rstd = m3.group_norm_fwd(x, groups, act="silu")
    g = m3.group_norm_bwd(x, x, mean, rstd, groups, act="silu")
    leaf = x.double().requires_grad_()
    ref, = torch.autograd.grad(norm64(leaf, groups, act="silu")[0], leaf, x.double())
    # terms of dx are below rstd max|dn| (1 + xh^2), with |xh| < 6 and as many roundings
    big = float(rstd.max() * x.abs().max()) * 1.2 * 37
    within(g["dx"], ref, torch.full_like(ref, 3 * 140 * U[torch.float32] * big * 37), "dx")


def test_two_sizes_from_two_threads():
    """Each thread's calls need another amount of shared memory of one kernel."""
    a, b = inputs(8, 16384, "f32")[0], inputs(8, 6000, "f32")[0]
    want = [m3.group_norm_fwd(a, 16384)[0], m3.group_norm_fwd(b, 6000)[0]]
    torch.cuda.synchronize()
    errors = []

    def calls(x, groups, ref):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(200):
                    y = m3.group_norm_fwd(x, groups)[0]
                torch.cuda.current_stream().synchronize()
                assert torch.equal(y, ref)
        except Exception as e:                             # a thread's exception would be lost
            errors.append(e)

    ts = [threading.Thread(target=calls, args=(x, x.shape[-1], r)) for x, r in zip((a, b), want)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not errors, errors
