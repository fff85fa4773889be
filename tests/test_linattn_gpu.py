"""Linear attention with a decay for each head on the GPU (marked gpu): the
chunked forward, the step and the backward against plain 64-bit sums over all
pairs of tokens, within bounds counted from the roundings (lin_reference)."""
import math

import pytest
import torch

from helpers import Canary
from lin_reference import U, backward64, forward64, mix_bound, state_bound, within
from state_space_lm_b200 import m3

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from state_space_lm_b200 import build
    build.build()


def decays(H, kind="spread"):
    if kind == "none":
        return torch.zeros(H, device="cuda")
    if kind == "edges":      # no memory, strong, weak, none
        return torch.tensor(([-math.inf, -30.0, -0.7, -1e-6, 0.0] * H)[:H], device="cuda")
    return torch.log1p(-torch.exp2(-torch.linspace(1.0, 12.0, H, dtype=torch.float64))).float().cuda()


def inputs(B, T, H, G, dk, dv, dtype, seed=0, fused=False, init=True, kind="spread", ragged=False):
    g = torch.Generator(device="cuda").manual_seed(seed + 1000 * B + T)
    n = lambda *s, t=DT[dtype]: torch.randn(*s, generator=g, device="cuda").to(t)  # noqa: E731
    if fused:
        # slices of one projection, the first 8 columns someone else's
        flat = n(B, T, 8 + 2 * G * dk + H * dv)
        q = flat[..., 8:8 + G * dk].unflatten(-1, (G, dk))
        k = flat[..., 8 + G * dk:8 + 2 * G * dk].unflatten(-1, (G, dk))
        v = flat[..., 8 + 2 * G * dk:].unflatten(-1, (H, dv))
    else:
        q, k, v = n(B, T, G, dk), n(B, T, G, dk), n(B, T, H, dv)
    f = torch.float32
    d = dict(q=q, k=k, v=v, ld=decays(H, kind), s0=n(B, H, dk, dv, t=f) if init else None,
             dy=n(B, T, H, dv), ds=n(B, H, dk, dv, t=f) if init else None, lengths=None)
    if ragged:
        ln = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        ln[0] = T
        if B > 1:
            ln[1] = 0
        d["lengths"] = ln
    return d


def on_tensor_cores(q, v):
    return q.dtype == torch.bfloat16 and all(e <= 128 for e in (q.shape[-1], v.shape[-1]))


def check_forward(d, scale=None, **kw):
    q, k, v = d["q"], d["k"], d["v"]
    sc = q.shape[-1] ** -0.5 if scale is None else scale
    y, sf = m3.linattn_chunked_fwd(q, k, v, d["ld"], scale=scale, s0=d["s0"], lengths=d["lengths"], **kw)
    ry, rs = forward64(q, k, v, d["ld"], sc, d["s0"], d["lengths"])
    ay, as_ = forward64(q, k, v, d["ld"], abs(sc), d["s0"], d["lengths"], absolute=True)
    T = v.shape[1]
    within(y, ry, mix_bound(ry, ay, v.dtype, T, q.shape[-1], on_tensor_cores(q, v)), "y")
    within(sf, rs, state_bound(rs, as_, T), "s_final")
    assert m3.device_error() == m3.M3_OK
    return y, sf


def check_backward(d, scale=None):
    q, k, v = d["q"], d["k"], d["v"]
    sc = q.shape[-1] ** -0.5 if scale is None else scale
    g = m3.linattn_chunked_bwd(q, k, v, d["ld"], d["dy"], scale=scale, s0=d["s0"], ds_final=d["ds"],
                               lengths=d["lengths"])
    ref = backward64(q, k, v, d["ld"], sc, d["dy"], d["s0"], d["ds"], d["lengths"])
    mass = backward64(q, k, v, d["ld"], abs(sc), d["dy"], d["s0"], d["ds"], d["lengths"], absolute=True)
    T, rep, tc = v.shape[1], v.shape[2] // q.shape[2], on_tensor_cores(q, v)
    for name, r, a, da in zip(("dq", "dk", "dv"), ref, mass, (v.shape[-1], v.shape[-1], q.shape[-1])):
        within(g[name], r, mix_bound(r, a, v.dtype, T, da, tc, rep), name)
    within(g["ds0"], ref[3], state_bound(ref[3], mass[3], T), "ds0")
    assert m3.device_error() == m3.M3_OK
    return g


# sizes around every edge: one token, the blocks of 16 and 64, several
# segments; widths with and without vectors, past a column tile, the largest
SHAPES = [
    (1, 1, 1, 1, 1, 1), (2, 1, 3, 3, 64, 64), (1, 15, 2, 1, 7, 5), (2, 16, 2, 2, 16, 32), (1, 17, 2, 2, 33, 33),
    (2, 63, 4, 2, 64, 64), (1, 64, 2, 2, 128, 64), (3, 65, 2, 1, 128, 128), (1, 127, 5, 5, 8, 8), (2, 128, 4, 4, 128, 64),
    (1, 129, 6, 2, 64, 128), (2, 200, 3, 3, 120, 72), (1, 300, 2, 2, 40, 24), (1, 100, 1, 1, 256, 64),
    (1, 100, 2, 1, 64, 256), (1, 1100, 2, 2, 128, 64), (1, 777, 8, 2, 64, 64), (1, 1024, 1, 1, 37, 29),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward(shape, dtype):
    check_forward(inputs(*shape, dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_backward(shape, dtype):
    check_backward(inputs(*shape, dtype))


@pytest.mark.parametrize("kind", ["none", "edges"])
@pytest.mark.parametrize("shape", [(1, 150, 5, 5, 128, 64), (2, 90, 5, 1, 21, 10), (1, 700, 5, 5, 64, 64)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decays_from_none_to_no_memory(shape, dtype, kind):
    d = inputs(*shape, dtype, kind=kind)
    check_forward(d)
    check_backward(d)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(5, 130, 4, 2, 64, 64), (4, 64, 2, 2, 128, 64), (3, 1000, 2, 1, 128, 128),
                                   (6, 70, 2, 2, 12, 20)], ids=lambda s: "x".join(map(str, s)))
def test_ragged_batches_with_garbage_behind_the_lengths(shape, dtype):
    """Lengths 0, T and between; what stands behind them is NaN and infinity
    and reaches nothing; rows of y and of the gradients there are zeros."""
    d = inputs(*shape, dtype, ragged=True)
    T = shape[1]
    behind = torch.arange(T, device="cuda")[None] >= d["lengths"].long()[:, None]
    clean = {k: d[k].clone() for k in ("q", "k", "v", "dy")}
    for i, k in enumerate(("q", "k", "v", "dy")):
        d[k][behind] = math.inf if i % 2 else math.nan
    y, sf = check_forward(d)
    assert bool((y[behind] == 0).all())
    assert torch.equal(sf[1], d["s0"][1])                       # no token: the state as it was
    g = check_backward(d)
    for k in ("dq", "dk", "dv"):
        assert bool((g[k][behind] == 0).all())
    assert torch.equal(g["ds0"][1], d["ds"][1])
    y2, sf2 = m3.linattn_chunked_fwd(clean["q"], clean["k"], clean["v"], d["ld"], s0=d["s0"], lengths=d["lengths"])
    assert torch.equal(y, y2) and torch.equal(sf, sf2)


@pytest.mark.parametrize("shape", [(129, 1, 2, 2, 64, 64), (20, 16, 16, 4, 128, 64), (65, 7, 4, 1, 36, 20),
                                   (128, 16, 2, 2, 64, 64), (300, 3, 1, 1, 8, 72)],
                         ids=lambda s: "x".join(map(str, s)))
def test_many_short_sequences(shape):
    """Both sides of the rule that gives up to 256 lanes of up to 16 tokens to
    the fp32 kernel and more of them to the tensor cores."""
    d = inputs(*shape, "bf16", ragged=True)
    check_forward(d)
    check_backward(d)


def test_a_nan_stays_out_of_the_chunks_before_it():
    for dtype, block in (("f32", 1), ("bf16", 64)):
        d = inputs(1, 300, 2, 2, 64, 64, dtype)
        y, _ = m3.linattn_chunked_fwd(d["q"], d["k"], d["v"], d["ld"], s0=d["s0"])
        for name in "qkv":
            bad = dict(d)
            bad[name] = d[name].clone()
            bad[name][:, 200] = math.nan
            y2, _ = m3.linattn_chunked_fwd(bad["q"], bad["k"], bad["v"], d["ld"], s0=d["s0"])
            first = 200 - 200 % block
            assert torch.equal(y2[:, :first], y[:, :first]), name
            assert bool(torch.isnan(y2[:, 200]).all()), name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_growing_decays(dtype):
    d = inputs(2, 200, 3, 3, 64, 48, dtype)
    d["ld"] = torch.tensor([0.02, 0.001, 0.1], device="cuda")    # up to e^20 over the sequence
    check_forward(d)
    check_backward(d)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_tensor_as_q_k_v_and_dy(dtype):
    d = inputs(2, 150, 3, 3, 64, 64, dtype)
    d["q"] = d["k"] = d["dy"] = d["v"]
    check_forward(d)
    check_backward(d)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_most_heads(dtype):
    d = inputs(1, 20, 4096, 64, 8, 8, dtype)
    check_forward(d)
    check_backward(d)
    m3.linattn_step_decode(d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["ld"], d["s0"])


def test_lengths_outside_the_range_are_taken_into_it():
    d = inputs(3, 40, 2, 2, 64, 64, "bf16")
    d["lengths"] = torch.tensor([-5, 999, 40], dtype=torch.int32, device="cuda")
    check_forward(d)
    check_backward(d)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_slices_of_a_fused_projection(dtype):
    d = inputs(2, 97, 4, 2, 64, 32, dtype, fused=True)
    y, sf = check_forward(d)
    g = check_backward(d)
    c = {k: d[k].contiguous() for k in ("q", "k", "v")}
    y2, sf2 = m3.linattn_chunked_fwd(c["q"], c["k"], c["v"], d["ld"], s0=d["s0"])
    g2 = m3.linattn_chunked_bwd(c["q"], c["k"], c["v"], d["ld"], d["dy"], s0=d["s0"], ds_final=d["ds"])
    assert torch.equal(y, y2) and torch.equal(sf, sf2)
    assert all(torch.equal(g[k], g2[k]) for k in g)


def test_strides_and_bases_that_tma_cannot_address():
    """Row strides that are no multiple of 8 (padded copies on the way), and
    bases on two bytes (fp32 arithmetic, within the same bounds)."""
    g = torch.Generator(device="cuda").manual_seed(3)
    B, T, H, dk, dv = 2, 70, 2, 64, 64
    big = torch.randn(B, T, 3 * H * 64 + 3, generator=g, device="cuda").bfloat16()
    q, k, v = (big[..., i * 128:(i + 1) * 128].unflatten(-1, (H, 64)) for i in range(3))
    d = dict(q=q, k=k, v=v, ld=decays(H), s0=None, ds=None, lengths=None,
             dy=torch.randn(B, T, H, dv, generator=g, device="cuda").bfloat16())
    check_forward(d)
    check_backward(d)
    flat = torch.randn(B, T, 1 + 3 * H * 64 + 7, generator=g, device="cuda").bfloat16()
    q, k, v = (flat[..., 1 + i * 128:1 + (i + 1) * 128].unflatten(-1, (H, 64)) for i in range(3))
    assert q.data_ptr() % 4 == 2 and q.stride(1) % 8 == 0
    d.update(q=q, k=k, v=v)
    check_forward(d)
    check_backward(d)


def test_no_initial_state_zero_scale_and_negative_scale():
    for scale in (0.0, -0.3):
        d = inputs(2, 80, 2, 2, 64, 64, "bf16", init=False)
        y, _ = check_forward(d, scale=scale)
        if scale == 0.0:
            assert bool((y == 0).all())
        check_backward(d, scale=scale)


def test_empty_sequences_pass_the_state_through():
    for dtype in ("f32", "bf16"):
        q = torch.empty(2, 0, 1, 64, device="cuda", dtype=DT[dtype])
        v = torch.empty(2, 0, 2, 64, device="cuda", dtype=DT[dtype])
        s0 = torch.randn(2, 2, 64, 64, device="cuda")
        y, sf = m3.linattn_chunked_fwd(q, q, v, decays(2), s0=s0)
        assert y.shape == v.shape and torch.equal(sf, s0)
        g = m3.linattn_chunked_bwd(q, q, v, decays(2), v, s0=s0, ds_final=s0)
        assert torch.equal(g["ds0"], s0)
    e = torch.empty(0, 5, 2, 8, device="cuda")
    y, sf = m3.linattn_chunked_fwd(e, e, e, decays(2))
    assert y.numel() == 0 and sf.numel() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 1), (3, 4, 2, 64, 64), (2, 2, 2, 128, 64), (5, 3, 1, 37, 29),
                                   (2, 2, 1, 256, 64), (1, 2, 2, 64, 256), (4, 2, 2, 100, 130)],
                         ids=lambda s: "x".join(map(str, s)))
def test_step(shape, dtype):
    B, H, G, dk, dv = shape
    d = inputs(B, 1, H, G, dk, dv, dtype)
    S = d["s0"].clone()
    y = m3.linattn_step_decode(d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["ld"], S)
    sc = dk ** -0.5
    ry, rs = forward64(d["q"], d["k"], d["v"], d["ld"], sc, d["s0"])
    ay, as_ = forward64(d["q"], d["k"], d["v"], d["ld"], sc, d["s0"], absolute=True)
    # the state: decay, product and two sums; y: those, and a sum over dk rows
    within(S, rs, 4 * U[torch.float32] * as_, "s")
    within(y[:, None], ry, (dk + 8) * U[torch.float32] * ay + 1.01 * U[y.dtype] * ry.abs(), "y_t")


@pytest.mark.parametrize("dtype,dk,dv", [("bf16", 128, 64), ("f32", 21, 12)])
def test_prefill_then_steps_equal_one_prompt(dtype, dk, dv):
    """A prompt of 90 tokens, then 10 single steps, against 100 at once, in 64 bits."""
    d = inputs(2, 100, 4, 2, dk, dv, dtype)
    q, k, v = d["q"], d["k"], d["v"]
    y, S = m3.linattn_chunked_fwd(q[:, :90].contiguous(), k[:, :90].contiguous(), v[:, :90].contiguous(), d["ld"],
                                  s0=d["s0"])
    ys = [y] + [m3.linattn_step_decode(q[:, t], k[:, t], v[:, t], d["ld"], S)[:, None] for t in range(90, 100)]
    ry, rs = forward64(q, k, v, d["ld"], dk ** -0.5, d["s0"])
    ay, as_ = forward64(q, k, v, d["ld"], dk ** -0.5, d["s0"], absolute=True)
    within(torch.cat(ys, 1), ry, mix_bound(ry, ay, v.dtype, 200, dk, on_tensor_cores(q, v)), "y")
    within(S, rs, state_bound(rs, as_, 260), "s")


def test_a_sequence_cut_in_two_chains_its_states():
    d = inputs(1, 500, 2, 2, 128, 64, "bf16")
    cut = lambda a, b: [d[x][:, a:b].contiguous() for x in ("q", "k", "v")]  # noqa: E731
    y1, s1 = m3.linattn_chunked_fwd(*cut(0, 213), d["ld"], s0=d["s0"])
    y2, s2 = m3.linattn_chunked_fwd(*cut(213, 500), d["ld"], s0=s1)
    ry, rs = forward64(d["q"], d["k"], d["v"], d["ld"], 128 ** -0.5, d["s0"])
    ay, as_ = forward64(d["q"], d["k"], d["v"], d["ld"], 128 ** -0.5, d["s0"], absolute=True)
    within(torch.cat([y1, y2], 1), ry, mix_bound(ry, ay, torch.bfloat16, 600, 128, True), "y")
    within(s2, rs, state_bound(rs, as_, 600), "s")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_repeated_calls_give_identical_bits_and_stay_inside_their_outputs(dtype):
    d = inputs(3, 210, 4, 2, 64, 96, dtype, ragged=True)
    first = None
    for _ in range(3):
        y, s = Canary(d["v"].shape, d["v"].dtype), Canary((3, 4, 64, 96), torch.float32)
        m3.linattn_chunked_fwd(d["q"], d["k"], d["v"], d["ld"], s0=d["s0"], lengths=d["lengths"], out=(y.t, s.t))
        out = {n: Canary(t.shape, t.dtype) for n, t in (("dq", d["q"]), ("dk", d["k"]), ("dv", d["v"]), ("ds0", s.t))}
        m3.linattn_chunked_bwd(d["q"], d["k"], d["v"], d["ld"], d["dy"], s0=d["s0"], ds_final=d["ds"],
                               lengths=d["lengths"], out={n: c.t for n, c in out.items()})
        for c in (y, s, *out.values()):
            c.check()
        now = [y.t, s.t] + [c.t for c in out.values()]
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, now))
        first = first or [t.clone() for t in now]


def test_wanted_gradients_alone():
    d = inputs(2, 100, 4, 2, 64, 64, "bf16")
    full = m3.linattn_chunked_bwd(d["q"], d["k"], d["v"], d["ld"], d["dy"], s0=d["s0"], ds_final=d["ds"])
    for want in (("dq",), ("dk",), ("dv",), ("ds0",), ("dk", "ds0"), ()):
        g = m3.linattn_chunked_bwd(d["q"], d["k"], d["v"], d["ld"], d["dy"], s0=d["s0"], ds_final=d["ds"], want=want)
        assert set(g) == set(want) and all(torch.equal(g[n], full[n]) for n in want)


def test_gradients_against_differences():
    """Central differences of <dy, y> + <ds, s_final> in fp32 along random
    directions: the loss is linear in each of q, k, v, s0, so the difference
    quotient has no truncation error, only the roundings of the two losses."""
    d = inputs(1, 70, 4, 2, 24, 20, "f32")
    dirs = {n: torch.randn_like(d[n]) for n in ("q", "k", "v", "s0")}
    g = m3.linattn_chunked_bwd(d["q"], d["k"], d["v"], d["ld"], d["dy"], s0=d["s0"], ds_final=d["ds"])

    def loss(x):
        y, s = m3.linattn_chunked_fwd(x["q"], x["k"], x["v"], d["ld"], s0=x["s0"])
        return float((y.double() * d["dy"].double()).sum() + (s.double() * d["ds"].double()).sum())

    for n, name in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("s0", "ds0")):
        up, dn = dict(d), dict(d)
        up[n], dn[n] = d[n] + dirs[n], d[n] - dirs[n]
        fd = (loss(up) - loss(dn)) / 2
        an = float((g[name].double() * dirs[n].double()).sum())
        ay, as_ = forward64(up["q"].abs() + dn["q"].abs(), up["k"].abs() + dn["k"].abs(), up["v"].abs() + dn["v"].abs(),
                            d["ld"], 24 ** -0.5, up["s0"].abs() + dn["s0"].abs(), absolute=True)
        mass = float((ay * d["dy"].double().abs()).sum() + (as_ * d["ds"].double().abs()).sum())
        assert abs(fd - an) <= 400 * U[torch.float32] * mass, (n, fd, an, mass)


def test_streams_graphs_and_workspaces():
    """Another stream than the current one, a captured and replayed call, and a
    caller's workspace that the calls share."""
    d = inputs(1, 1500, 2, 2, 128, 64, "bf16")
    ref, sref = m3.linattn_chunked_fwd(d["q"], d["k"], d["v"], d["ld"], s0=d["s0"])
    gref = m3.linattn_chunked_bwd(d["q"], d["k"], d["v"], d["ld"], d["dy"], s0=d["s0"], ds_final=d["ds"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, s = torch.empty_like(ref), torch.empty_like(sref)
    m3.linattn_chunked_fwd(d["q"], d["k"], d["v"], d["ld"], s0=d["s0"], out=(y, s), stream=side)
    side.synchronize()
    assert torch.equal(y, ref) and torch.equal(s, sref)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    out = {n: torch.empty_like(t) for n, t in gref.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m3.linattn_chunked_fwd(d["q"], d["k"], d["v"], d["ld"], s0=d["s0"], out=(y, s), workspace=ws)
        m3.linattn_chunked_bwd(d["q"], d["k"], d["v"], d["ld"], d["dy"], s0=d["s0"], ds_final=d["ds"], out=out,
                               workspace=ws)
    for _ in range(2):
        for t in (y, s, *out.values()):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref) and torch.equal(s, sref)
        assert all(torch.equal(out[n], gref[n]) for n in out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_sequences_over_few_lanes(dtype):
    """The split time axis (T = 5000 over two lanes), against the 64-bit
    recurrence chunk by chunk; odd lengths cut a segment short."""
    B, T, H, dk, dv = 2, 5000, 1, 128, 64
    d = inputs(B, T, H, 1, dk, dv, dtype)
    d["lengths"] = torch.tensor([T, 3333], dtype=torch.int32, device="cuda")
    check_forward(d)
    check_backward(d)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_step_of_the_most_heads(dtype):
    d = inputs(2, 1, 4096, 64, 8, 8, dtype)
    S = d["s0"].clone()
    y = m3.linattn_step_decode(d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["ld"], S)
    ry, rs = forward64(d["q"], d["k"], d["v"], d["ld"], 8 ** -0.5, d["s0"])
    ay, as_ = forward64(d["q"], d["k"], d["v"], d["ld"], 8 ** -0.5, d["s0"], absolute=True)
    # g or g - 1 (4 half steps), a product and two sums; y: those, and a sum over 8 rows
    within(S, rs, 8 * U[torch.float32] * as_, "s")
    within(y[:, None], ry, (8 + 12) * U[torch.float32] * ay + 1.01 * U[y.dtype] * ry.abs(), "y_t")
