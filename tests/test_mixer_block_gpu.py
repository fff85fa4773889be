"""Linear attention and the gated group norm together, as a layer uses them
(marked gpu): training through torch.autograd, a prompt followed by single
tokens, calls that overlap on two streams, a captured layer, offsets past 32
bits, and the host-side failure hook."""
import math

import pytest
import torch

from lin_reference import U, act64, forward64, live, norm64, powers, heads, within
from state_space_lm_b200 import group_norm, linear_attention, m3

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from state_space_lm_b200 import build
    build.build()


def layer_inputs(B, T, H, G, dk, dv, dtype, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    ld = torch.log1p(-torch.exp2(-torch.linspace(2.0, 8.0, H, device="cuda")))
    w, b = 1 + 0.1 * n(H * dv).float(), 0.1 * n(H * dv).float()
    return dict(flat=n(B, T, 2 * G * dk + H * dv), z=n(B, T, H * dv), w=w, b=b, ld=ld, H=H, G=G, dk=dk, dv=dv)


def split(flat, G, dk, H, dv):
    q = flat[..., :G * dk].unflatten(-1, (G, dk))
    k = flat[..., G * dk:2 * G * dk].unflatten(-1, (G, dk))
    return q, k, flat[..., 2 * G * dk:].unflatten(-1, (H, dv))


def layer(x, flat, z, w, b, lengths=None, s0=None):
    """One layer: attention over slices of a projection, the norm of each head
    of each token, the gate."""
    B, T = flat.shape[:2]
    y, s = linear_attention(*split(flat, x["G"], x["dk"], x["H"], x["dv"]), x["ld"], s0=s0, lengths=lengths)
    return group_norm(y.reshape(B * T, -1), x["H"], w, b, z.reshape(B * T, -1), "silu").view(B, T, -1), s


def layer64(x, flat, z, w, b, lengths=None):
    """The same in 64 bits, with torch.autograd behind it."""
    B, T = flat.shape[:2]
    q, k, v = (heads(t, x["H"]) for t in split(flat, x["G"], x["dk"], x["H"], x["dv"]))
    n, on = live(lengths, B, T, flat.device)
    on = on[:, None, :, None]
    t = torch.arange(T, device=flat.device)
    k, v = k * on, v * on
    mask = powers(x["ld"], t[:, None] - t[None]).unsqueeze(0)
    y = (((q @ k.transpose(-1, -2)) * mask) @ v) * x["dk"] ** -0.5 * on
    y = y.transpose(1, 2).reshape(B * T, -1)
    return norm64(y, x["H"], w, b, z.reshape(B * T, -1), "silu")[0].view(B, T, -1)


@pytest.mark.parametrize("lens", [None, (130, 77, 0)])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_training_through_a_layer(dtype, lens):
    """Gradients of the projection, the gate and the norm's parameters, q and k
    shared by two heads each.  fp32: within 2-norm 5e-5 of the 64-bit layer's
    (a few hundred roundings of 2^-24 in each of the three stages).  bf16: the
    attention's outputs and gradients are rounded to 2^-8 twice on the way
    (y, and dy of the norm), and the norm of a head of a nearly empty row
    amplifies y's rounding by rstd: 5e-2."""
    x = layer_inputs(3, 130, 4, 2, 64, 32, dtype)
    lengths = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    names = ("flat", "z", "w", "b")
    a = [x[n].clone().requires_grad_() for n in names]
    r = [x[n].double().requires_grad_() for n in names]
    o, _ = layer(x, *a, lengths=lengths)
    ref = layer64(x, *r, lengths=lengths)
    dy = torch.randn(o.shape, generator=torch.Generator(device="cuda").manual_seed(9), device="cuda").to(dtype)
    o.backward(dy)
    ref.backward(dy.double())
    tol = 5e-5 if dtype == torch.float32 else 5e-2
    assert float((o.double() - ref).norm() / ref.norm()) <= tol
    for n, p, t in zip(names, a, r):
        err = float((p.grad.double() - t.grad).norm() / t.grad.norm())
        assert err <= tol, (n, err)
        assert torch.isfinite(p.grad).all(), n


def test_second_derivatives_are_refused():
    x = layer_inputs(1, 20, 2, 2, 16, 16, torch.float32)
    flat = x["flat"].requires_grad_()
    o, _ = layer(x, flat, x["z"], x["w"], x["b"])
    g, = torch.autograd.grad(o.square().sum(), flat, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiate twice|once_differentiable"):
        g.sum().backward()


def test_a_prompt_then_single_tokens_with_the_norm_behind():
    """Prefill of a ragged batch, then 6 tokens one by one, each followed by
    the gated norm, against the 64-bit layer over the whole sequences."""
    B, T, H, G, dk, dv = 3, 96, 4, 4, 128, 64
    x = layer_inputs(B, T + 6, H, G, dk, dv, BF)
    lens = [96, 41, 1]
    # each sequence's tokens: a prompt of lens[b], then six more
    own = torch.stack([x["flat"][b, :T + 6] for b in range(B)])
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q, k, v = split(own[:, :T].contiguous(), G, dk, H, dv)
    y, S = m3.linattn_chunked_fwd(q, k, v, x["ld"], lengths=lengths)
    steps = []
    for i in range(6):
        tok = torch.stack([own[b, lens[b] + i] for b in range(B)])
        qt, kt, vt = split(tok, G, dk, H, dv)
        steps.append(m3.linattn_step_decode(qt, kt, vt, x["ld"], S))
    for b in range(B):
        n = lens[b] + 6
        seq = own[b:b + 1, :n].contiguous()
        ry, rs = forward64(*split(seq, G, dk, H, dv), x["ld"], dk ** -0.5)
        ay, as_ = forward64(*split(seq, G, dk, H, dv), x["ld"], dk ** -0.5, absolute=True)
        got = torch.cat([y[b, :lens[b]], torch.stack([s[b] for s in steps])])
        u32 = (dk + 64 + 2 * (n / 16 + 1) + 60) * U[torch.float32]
        within(got[None], ry, (u32 + 1.01 * U[BF]) * ay + 1.01 * U[BF] * ry.abs(), "y of sequence %d" % b)
        within(S[b:b + 1], rs, (3 * 64 + 3 * (n / 16 + 1) + 60) * U[torch.float32] * as_, "state")
        z = x["z"][b, :n]
        o, mean, rstd = m3.group_norm_fwd(got.reshape(n, H * dv), H, x["w"], x["b"], gate=z, act="silu")
        # the norm against 64 bits of what it was given: its own roundings only
        ro, _, rr = norm64(got.reshape(n, H * dv), H, x["w"], x["b"], z, "silu")
        size = (9.0 * float(x["w"].abs().max()) + 1) * act64("silu", z.double()).abs()
        within(o, ro, 200 * U[torch.float32] * size * 9 + 2.0 ** -19 * size + 1.01 * U[BF] * ro.abs(), "norm")


def test_two_streams_at_once_and_a_captured_layer():
    """Two layers that overlap on two streams, each with its own workspace, and
    one captured layer replayed on new inputs: the bits of calls one by one."""
    xs = [layer_inputs(1, 1100, 2, 2, 128, 64, BF, seed=s) for s in (3, 4)]

    def fwd(x, stream=None):
        y, s = m3.linattn_chunked_fwd(*split(x["flat"], 2, 128, 2, 64), x["ld"], stream=stream)
        o, _, _ = m3.group_norm_fwd(y.view(1100, 128), 2, x["w"], x["b"], gate=x["z"].view(1100, 128), act="silu",
                                    stream=stream)
        return o, s

    alone = [fwd(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        out = [fwd(x, st) for x, st in zip(xs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(alone, out):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    x = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in xs[0].items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = fwd(x)
    for i in (1, 0, 1):
        for k, v in xs[i].items():
            if isinstance(v, torch.Tensor):
                x[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(cap[0], alone[i][0]) and torch.equal(cap[1], alone[i][1])


def test_offsets_past_32_bits():
    """q and k of 2.2e9 elements each: the last tokens of the long sequence
    equal those of a short one that continues from the state before them, and a
    norm over 2.2e9 elements equals the norm of its last rows alone."""
    H, dk, dv, T, tail = 16, 128, 16, 1_075_000, 200
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    g = torch.Generator(device="cuda").manual_seed(6)
    q = torch.randn(1, T, H, dk, generator=g, device="cuda", dtype=BF)
    k = torch.randn(1, T, H, dk, generator=g, device="cuda", dtype=BF)
    v = torch.randn(1, T, H, dv, generator=g, device="cuda", dtype=BF)
    assert q.numel() > 1 << 31
    ld = torch.full((H,), -0.05, device="cuda")
    y, S = m3.linattn_chunked_fwd(q, k, v, ld)
    cut = T - tail
    warm = 2000                                             # e^(-0.05 * 2000) = 4e-44: nothing is left of what came before
    a = slice(cut - warm, cut)
    _, s0 = m3.linattn_chunked_fwd(q[:, a].contiguous(), k[:, a].contiguous(), v[:, a].contiguous(), ld)
    ry, rs = forward64(q[:, cut:], k[:, cut:], v[:, cut:], ld, dk ** -0.5, s0)
    ay, as_ = forward64(q[:, cut:], k[:, cut:], v[:, cut:], ld, dk ** -0.5, s0, absolute=True)
    within(y[:, cut:], ry, 1.05 * U[BF] * (ay + ry.abs()), "y")
    within(S, rs, 1e-4 * as_, "s_final")
    assert m3.device_error() == m3.M3_OK
    del k, v, y
    x = q.view(-1, 1024)
    o, mean, rstd = m3.group_norm_fwd(x, 16, act="none")
    last = x[-50:].clone()
    ol, ml, rl = m3.group_norm_fwd(last, 16, act="none")
    assert torch.equal(o[-50:], ol) and torch.equal(mean[-50:], ml) and torch.equal(rstd[-50:], rl)


def test_injected_launch_failures_raise_and_enqueue_nothing():
    x = layer_inputs(1, 30, 2, 2, 64, 64, BF)
    q, k, v = split(x["flat"], 2, 64, 2, 64)
    y, s = torch.full((1, 30, 2, 64), -7.0, device="cuda", dtype=BF), torch.full((1, 2, 64, 64), -7.0, device="cuda")
    calls = [lambda: m3.linattn_chunked_fwd(q, k, v, x["ld"], out=(y, s)),
             lambda: m3.linattn_step_decode(q[:, 0], k[:, 0], v[:, 0], x["ld"], s, y_out=y[:, 0].contiguous()),
             lambda: m3.linattn_chunked_bwd(q, k, v, x["ld"], y.clone(), out={"dv": y}, want=("dv",)),
             lambda: m3.group_norm_fwd(y.view(30, 128), 2, out=(y.clone().view(30, 128), None, None)),
             lambda: m3.group_norm_bwd(y.view(30, 128), y.view(30, 128), s[0, 0, 0:30, 0:2].contiguous(),
                                       s[0, 0, 0:30, 0:2].contiguous(), 2)]
    for call in calls:
        n0 = m3.launch_count()
        m3.debug_fail_next_launches(1)
        with pytest.raises(m3.M3Error) as e:
            call()
        assert e.value.status == m3.M3_ERR_CUDA and m3.launch_count() == n0
    torch.cuda.synchronize()
    assert bool((y == -7).all()) and bool((s == -7).all())
    m3.linattn_chunked_fwd(q, k, v, x["ld"], out=(y, s))
    assert not bool((y == -7).all())


def test_results_on_another_stream_take_no_memory_with_work_pending():
    """A block of memory that the current stream has freed but is still to
    write goes to nobody on another stream."""
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k, v = (torch.randn(2, 4096, 4, 64, generator=g, device="cuda").bfloat16() for _ in range(3))
    ld = torch.full((4,), -0.05, device="cuda")
    x = torch.randn(2, 4096, 256, generator=g, device="cuda").bfloat16()
    w = torch.randn(256, generator=g, device="cuda")
    ref, _ = m3.linattn_chunked_fwd(q, k, v, ld)
    gref = m3.linattn_chunked_bwd(q, k, v, ld, v)
    nref, mean, rstd = m3.group_norm_fwd(x, 4, w)
    bref = m3.group_norm_bwd(x, x, mean, rstd, 4, w)
    state = torch.zeros(2, 4, 64, 64, device="cuda")
    sref = m3.linattn_step_decode(q[:, 0], k[:, 0], v[:, 0], ld, state.clone())
    side = torch.cuda.Stream()
    calls = [
        lambda: (m3.linattn_chunked_fwd(q, k, v, ld, stream=side)[0], ref),
        lambda: (m3.linattn_chunked_bwd(q, k, v, ld, v, stream=side)["dk"], gref["dk"]),
        lambda: (m3.group_norm_fwd(x, 4, w, stream=side)[0], nref),
        lambda: (m3.group_norm_bwd(x, x, mean, rstd, 4, w, stream=side)["dx"], bref["dx"]),
        lambda: (m3.linattn_step_decode(q[:, 0], k[:, 0], v[:, 0], ld, state, stream=side), sref),
    ]
    for call in calls:
        side.wait_stream(torch.cuda.current_stream())
        torch.cuda._sleep(20_000_000)                        # ~10 ms of the current stream
        for _ in range(8):
            late = [torch.empty_like(t).fill_(7) for t in (ref, sref, gref["dk"], nref)]
            del late
        got, want = call()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_incoming_gradients_that_start_anywhere():
    """torch.cat hands back slices of one gradient: contiguous, but not on 16
    bytes."""
    for dtype in (torch.float32, torch.bfloat16):
        g = torch.Generator(device="cuda").manual_seed(6)
        q, k, v = (torch.randn(1, 33, 2, 24, generator=g, device="cuda").to(dtype).requires_grad_() for _ in range(3))
        ld = torch.full((2,), -0.1, device="cuda")
        w = torch.randn(48, generator=g, device="cuda").requires_grad_()
        first = torch.zeros(3, device="cuda", dtype=dtype, requires_grad=True)
        up = torch.randn(3 + 33 * 48, generator=g, device="cuda").to(dtype)

        def grads(cat):
            y, s = linear_attention(q, k, v, ld)
            z = group_norm(y.reshape(33, 48), 2, w)
            for out in (y, z):
                flat = out.reshape(-1)
                loss = (torch.cat([first, flat]) * up).sum() if cat else (flat * up[3:].clone()).sum()
                up_s = torch.ones(s.numel() + 1, device="cuda")
                loss = loss.float() + ((torch.cat([first[:1].float(), s.reshape(-1)]) * up_s).sum() if cat else s.sum())
                yield torch.autograd.grad(loss, (q, k, v) if out is y else (q, k, v, w), retain_graph=True)

        for a, b in zip(grads(True), grads(False)):
            assert all(torch.equal(x, z) for x, z in zip(a, b))
