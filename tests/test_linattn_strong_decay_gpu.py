"""Linear attention with strong decays on the GPU (marked gpu): what is left of
an old state is a small multiple of it, and the new tokens and that multiple
keep their own digits however large the old state was."""
import math

import pytest
import torch

from lin_reference import U, forward64, within
from state_space_lm_b200 import m3

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
F32 = U[torch.float32]
# no memory, g = 1e-13, 7e-3, around 1/2 on both sides, weak, none
DECAYS = [-math.inf, -30.0, -5.0, -0.7, -0.69, -1e-3, 0.0]


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from state_space_lm_b200 import build
    build.build()


def inputs(B, T, H, dk, dv, dtype, state):
    g = torch.Generator(device="cuda").manual_seed(B + T + dk)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    t = DT[dtype]
    return (n(B, T, H, dk).to(t), n(B, T, H, dk).to(t), n(B, T, H, dv).to(t), torch.tensor(DECAYS[:H], device="cuda"),
            state * n(B, H, dk, dv))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(128, 64), (37, 29), (256, 64)])
@pytest.mark.parametrize("state", [1.0, 1e3, 1e8])
def test_step(state, dk, dv, dtype):
    q, k, v, ld, s0 = inputs(3, 1, len(DECAYS), dk, dv, dtype, state)
    S = s0.clone()
    y = m3.linattn_step_decode(q[:, 0], k[:, 0], v[:, 0], ld, S)
    ry, rs = forward64(q, k, v, ld, dk ** -0.5, s0)
    ay, as_ = forward64(q, k, v, ld, dk ** -0.5, s0, absolute=True)
    # as_ = g |S| + |k v|.  g or g - 1 to 2 units in the last place (4 half
    # steps; of g - 1 that is no more than 4 of g where g >= 1/2), the product
    # k v, the sum with the product, the sum with the state
    within(S, rs, 8 * F32 * as_, "s")
    within(y[:, None], ry, (dk + 12) * F32 * ay + 1.01 * U[y.dtype] * ry.abs(), "y_t")
    assert bool(torch.isfinite(S).all())


def test_no_memory_is_none():
    """log_decay = -inf: the new state is k v, whatever the old one was."""
    q, k, v, ld, s0 = inputs(2, 1, 1, 64, 32, "f32", 1e30)
    S = s0.clone()
    m3.linattn_step_decode(q[:, 0], k[:, 0], v[:, 0], ld, S)
    assert torch.equal(S, k[:, 0, :, :, None] * v[:, 0, :, None, :])
