"""Linear attention with strong decays on the GPU (marked gpu): what is left of
an old state is a small multiple of it, and the new tokens and that multiple
keep their own digits however large the old state was."""
import math

import pytest
import torch

from lin_reference import U, backward64, forward64, mix_bound, within
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


# What 32 bits hold of a vanishing state: below this nothing is asked (the
# smallest normal number, times 2^16 for the bf16 pieces of weighted rows)
FLOOR = 2.0 ** -110


def on_tensor_cores(q, v):
    return q.dtype == torch.bfloat16 and q.shape[-1] <= 128 and v.shape[-1] <= 128


def chain_bound(ref, mass, T):
    """A state in fp32: a chunk's own sum (3 x 64, as in state_bound), and for
    each chunk of 16 tokens at least: its power (expf to 2 units in the last
    place, two more roundings; or expm1f and one), the product and the sum."""
    return (3 * 64 + 16 + 8 * (T / 16 + 1)) * F32 * mass + F32 * ref.abs() + FLOOR


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [16, 64, 65, 200, 1100])
@pytest.mark.parametrize("dk,dv", [(128, 64), (64, 96), (37, 29)])
@pytest.mark.parametrize("first", [0, 10])
def test_a_state_decays_through_tokens_that_add_nothing(first, dk, dv, T, dtype):
    """Keys and queries (the adjoint's keys) are zero behind the first 10 tokens
    or from the start: s_final = g^T s0 + ..., ds0 = g^T ds + ... to their own
    digits, and so are the answers and gradients that read them."""
    q, k, v, _, s0 = inputs(2, T, 7, dk, dv, dtype, 1.0)
    ld = torch.tensor([-math.inf, -5.0, -0.3, -0.25, -0.05, -1e-3, 0.0], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(T)
    dy = torch.randn(v.shape, generator=g, device="cuda").to(v.dtype)
    ds = torch.randn(s0.shape, generator=g, device="cuda")
    k[:, first:] = 0
    sc, tc = dk ** -0.5, on_tensor_cores(q, v)
    y, sf = m3.linattn_chunked_fwd(q, k, v, ld, s0=s0)
    ry, rs = forward64(q, k, v, ld, sc, s0)
    ay, as_ = forward64(q, k, v, ld, sc, s0, absolute=True)
    within(sf, rs, chain_bound(rs, as_, T), "s_final")
    within(y, ry, mix_bound(ry, ay, v.dtype, 4 * T, dk, tc) + FLOOR, "y")
    q2 = q.clone()
    q2[:, :T - first] = 0
    got = m3.linattn_chunked_bwd(q2, k, v, ld, dy, s0=s0, ds_final=ds)
    ref = backward64(q2, k, v, ld, sc, dy, s0, ds)
    mass = backward64(q2, k, v, ld, sc, dy, s0, ds, absolute=True)
    within(got["ds0"], ref[3], chain_bound(ref[3], mass[3], T), "ds0")
    for name, r, a, da in zip(("dq", "dk", "dv"), ref, mass, (dv, dv, dk)):
        within(got[name], r, mix_bound(r, a, v.dtype, 4 * T, da, tc) + FLOOR, name)
    assert m3.device_error() == m3.M3_OK


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_large_old_state_behind_a_strong_decay(dtype):
    """The new tokens keep their digits beside what 100 tokens leave of 1e8."""
    q, k, v, ld, s0 = inputs(2, 100, len(DECAYS), 64, 64, dtype, 1e8)
    _, sf = m3.linattn_chunked_fwd(q, k, v, ld, s0=s0)
    rs = forward64(q, k, v, ld, 0.125, s0)[1]
    within(sf, rs, chain_bound(rs, forward64(q, k, v, ld, 0.125, s0, absolute=True)[1], 100), "s_final")
