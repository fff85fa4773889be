"""Gradients in their inputs' own shapes through the library (marked gpu)."""
import pytest
import torch

from state_space_lm_b200 import group_norm, linear_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from state_space_lm_b200 import build
    build.build()


def test_a_gate_of_three_axes_and_a_flat_state():
    g = torch.Generator(device="cuda").manual_seed(5)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
    B, T, H, dk, dv = 2, 40, 4, 16, 8
    ld = torch.full((H,), -0.1, device="cuda")
    base = dict(q=n(B, T, H, dk), k=n(B, T, H, dk), v=n(B, T, H, dv), s0=n(B, H, dk, dv), z=n(B * T, H * dv),
                w=1 + 0.1 * n(H * dv), b=n(H * dv))
    dy, ds = n(B * T, H * dv), n(B, H, dk, dv)

    def grads(shapes):
        x = {k: t.detach().view(shapes.get(k, t.shape)).requires_grad_() for k, t in base.items()}
        y, s = linear_attention(x["q"], x["k"], x["v"], ld, s0=x["s0"])
        o = group_norm(y.reshape(B * T, -1), H, x["w"], x["b"], x["z"], "silu")
        ((o * dy).sum() + (s * ds.view(s.shape)).sum()).backward()
        return {k: t.grad for k, t in x.items()}

    want = grads({})
    shapes = dict(z=(B, T, H * dv), s0=(B, H, dk * dv), w=(1, H * dv), b=(H, dv))
    got = grads(shapes)
    for k, t in want.items():
        assert got[k].shape == shapes.get(k, t.shape) and torch.equal(got[k].view(t.shape), t), k
