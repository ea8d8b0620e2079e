"""The gated feed-forward block and its backward pass on the GPU against their formulas in 64 bits.

Tolerances count roundings.  u = 2^-24 is half a step of fp32.  A sum of `depth` products on the matrix
cores adds them in an order of its own: at most depth / 16 additions to the running sum and 16 inside an
instruction for the 16-bit types, whose products are exact, and `depth` fused ones for fp32; each is
taken to be off by a whole step (2 u) of at most the sum of the magnitudes.  The activations are off by
a few u, and where their argument is rounded (by v: |v| u) by what their slope makes of it.  The result
is rounded once, by at most half a step of its type.  Integers, whose sums are exact, come out equal.
"""
import math

import pytest
import torch

import gradient_compression_amd as gca
from tests.gpu_helpers import log

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = 2.0 ** -24
SMALLEST = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}     # half a step, relative
ACTS = ("silu", "gelu", "gelu_tanh")


def act64(name, g):
    """act(g), act'(g) in 64 bits, and bounds on what fp32 makes of them, in u."""
    if name == "gelu":
        p = 0.5 * torch.special.erfc(g / -math.sqrt(2.0))
        d = g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
        return g * p, p + d, 16 * ((g * p).abs() + (g * d).abs()), 16 * (
            p + d.abs() * (2 + g * g))
    if name == "silu":
        v, dv = g, torch.ones_like(g)
    else:
        k = 2.0 * math.sqrt(2.0 / math.pi)
        v, dv = k * (g + 0.044715 * g ** 3), k * (1.0 + 3 * 0.044715 * g * g)
    p, q = torch.sigmoid(v), torch.sigmoid(-v)
    t = g * p * q
    around = 1 + (v.abs() if name == "gelu_tanh" else 0)
    return g * p, p + t * dv, 16 * ((g * p).abs() + t.abs() * around), 16 * (
        p + (t * dv).abs() * around)


def sums64(x, w, dtype):
    """x w^T in 64 bits and the bound on what fp32 sums make of it."""
    depth = x.shape[-1]
    steps = depth + 4 if dtype == "f32" else depth / 16 + 17
    return x @ w.t().contiguous(), 2 * U * steps * (x.abs() @ w.abs().t().contiguous())


def close(got, want, bound, dtype, what):
    got = got.double()
    err = (got - want).abs()
    tol = bound + HALF[dtype] * (want.abs() + bound) + SMALLEST[dtype] / 2 + 2.0 ** -126
    worst = (err / tol).max().item() if err.numel() else 0.0
    log(f"[gated] {what}: worst {worst:.3f} of the bound")
    assert not torch.isnan(got).any(), f"{what}: NaN"
    assert worst <= 1.0, f"{what}: {worst} of the bound"


def randn(gen, *shape, scale=1.0, dtype="f32"):
    return (scale * torch.randn(*shape, generator=gen, device="cuda")).to(TYPES[dtype])


def strided(t, pad, shift=0, fill=float("nan")):
    """The matrix in a wider buffer of `fill` (rows `pad` elements apart, `shift` off its start)."""
    rows, cols = t.shape
    buf = torch.full((rows * (cols + pad) + shift + 8,), fill, dtype=t.dtype, device=t.device)
    view = buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(t)
    return view, buf


def untouched(buf, view, fill):
    mask = torch.ones_like(buf, dtype=torch.bool)
    torch.as_strided(mask, view.shape, view.stride(), view.storage_offset()).fill_(False)
    return bool((buf[mask] == fill).all())


def check_forward(rows, n, cols, dtype, act, pad=0, shift=0, keep=True, seed=0):
    what = f"{dtype} {act} {rows} x {cols} -> {n}, pad {pad} shift {shift}"
    log(f"[gated] forward {what}")
    gen = torch.Generator("cuda").manual_seed(seed * 1000003 + rows * 7919 + n * 31 + cols)
    x0 = randn(gen, rows, cols, dtype=dtype)
    w0 = [randn(gen, n, cols, scale=1.5 / math.sqrt(cols), dtype=dtype) for _ in range(2)]
    x, _ = strided(x0, pad, shift)
    wg, _ = strided(w0[0], pad, shift)
    wu, _ = strided(w0[1], 2 * pad, 0)
    zeros = torch.zeros(rows, n, dtype=TYPES[dtype], device="cuda")
    outs = [strided(zeros, pad, shift, 7.0) for _ in range(3 if keep else 1)]
    views = [v for v, _ in outs] + [None] * (0 if keep else 2)
    gca.gated_linear(x, wg, wu, views[0], gate=views[1], up=views[2], activation=act)
    torch.cuda.synchronize()
    gate, eg = sums64(x0.double(), w0[0].double(), dtype)
    up, eu = sums64(x0.double(), w0[1].double(), dtype)
    a, _, ea, _ = act64(act, gate)
    ea = U * ea + 1.13 * eg      # no activation's slope is above 1.13
    eh = ea * up.abs() + eu * a.abs() + ea * eu + 2 * U * (a * up).abs()
    close(views[0], a * up, eh, dtype, f"h of {what}")
    if keep:
        close(views[1], gate, eg, dtype, f"gate of {what}")
        close(views[2], up, eu, dtype, f"up of {what}")
    for v, buf in outs:
        assert untouched(buf, v, 7.0), what


def check_backward(rows, n, cols, dtype, act, pad=0, shift=0, in_place=False, seed=0):
    what = f"{dtype} {act} {rows} x {n} -> {cols}, pad {pad} shift {shift}"
    log(f"[gated] backward {what}")
    gen = torch.Generator("cuda").manual_seed(seed * 1000003 + rows * 7919 + n * 31 + cols)
    src = [randn(gen, rows, n, scale=s, dtype=dtype) for s in (0.05, 1.5, 1.0)]
    w0 = [randn(gen, n, cols, scale=1.0 / math.sqrt(cols), dtype=dtype) for _ in range(2)]
    dh, gate, up = (strided(t, pad, shift, 7.0) for t in src)
    wg, _ = strided(w0[0], pad, shift)
    wu, _ = strided(w0[1], 2 * pad, 0)
    zeros = torch.zeros(rows, n, dtype=TYPES[dtype], device="cuda")
    dgate, dup = (gate, dh) if in_place else (strided(zeros, pad, shift, 7.0) for _ in range(2))
    dx, xbuf = strided(torch.zeros(rows, cols, dtype=TYPES[dtype], device="cuda"), pad, shift, 7.0)
    gca.gated_linear_backward(dh[0], gate[0], up[0], dgate[0], dup[0], w_gate=wg, w_up=wu, dx=dx,
                              activation=act)
    torch.cuda.synchronize()
    d, g, u = (t.double() for t in src)
    a, s, ea, es = act64(act, g)
    close(dgate[0], d * u * s, U * (es + 4 * s.abs()) * (d * u).abs(), dtype, f"dgate of {what}")
    close(dup[0], d * a, U * (ea + 4 * a.abs()) * d.abs(), dtype, f"dup of {what}")
    stored = torch.cat((dgate[0], dup[0]), 1).double()
    want, bound = sums64(stored, torch.cat((w0[0], w0[1]), 0).double().t(), dtype)
    close(dx, want, bound, dtype, f"dx of {what}")
    assert untouched(xbuf, dx, 7.0) and untouched(up[1], up[0], 7.0)
    for v, buf in (dgate, dup):
        assert untouched(buf, v, 7.0), what
    assert torch.equal(up[0], src[2])


# one to long, across the tiles' sizes, odd and even
SHAPES = [(1, 1, 1), (1, 33, 64), (2, 7, 129), (3, 64, 8), (16, 16, 32), (17, 40, 200), (31, 65, 63),
          (64, 128, 64), (65, 63, 1000), (100, 200, 40), (128, 64, 128), (129, 129, 129),
          (200, 1000, 72), (257, 300, 520), (300, 77, 4100), (640, 512, 256), (1030, 520, 264)]


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_forward_matches_the_formula(dtype):
    for i, (rows, n, cols) in enumerate(SHAPES):
        check_forward(rows, n, cols, dtype, ACTS[i % 3], keep=i % 4 != 3)


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_backward_matches_the_formula(dtype):
    for i, (rows, n, cols) in enumerate(SHAPES):
        check_backward(rows, n, cols, dtype, ACTS[i % 3])


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_strided_unaligned_and_in_place(dtype, act):
    """Rows at any pitch and place, NaN between the inputs' rows and sevens between the outputs'."""
    for pad, shift in ((8, 0), (8, 8), (3, 0), (5, 1), (16, 3)):
        for rows, n, cols in ((5, 40, 72), (70, 137, 203), (150, 256, 192)):
            check_forward(rows, n, cols, dtype, act, pad, shift)
            check_backward(rows, n, cols, dtype, act, pad, shift, in_place=True)


def integers(gen, *shape, most=3):
    return torch.randint(-most, most + 1, shape, generator=gen, device="cuda")


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_integers_are_exact(dtype):
    """Sums of integers within each type's whole numbers come out equal, in every place of every
    tile: gate and up of the forward pass, and dx where the activation's slope is 1 (silu at 64)."""
    gen = torch.Generator("cuda").manual_seed(11)
    t = TYPES[dtype]
    for rows, n, cols in SHAPES + [(19, 2000, 48), (1500, 24, 80), (33, 300, 2064)]:
        log(f"[gated] integers {dtype} {rows} {n} {cols}")
        # few products other than 0, so that bf16's 8 bits hold the sums (the bound is checked)
        few = min(1.0, 24 / cols)
        x = integers(gen, rows, cols) * (torch.rand(rows, cols, generator=gen, device="cuda") < few)
        wg, wu = integers(gen, n, cols, most=1), integers(gen, n, cols, most=2)
        h, gate, up = (torch.empty(rows, n, dtype=t, device="cuda") for _ in range(3))
        gca.gated_linear(x.to(t), wg.to(t), wu.to(t), h, gate=gate, up=up)
        for got, w in ((gate, wg), (up, wu)):
            want = x.double() @ w.double().t().contiguous()
            assert want.abs().max() <= 256
            assert torch.equal(got.double(), want), f"{dtype} {rows} {n} {cols}"
        few = min(1.0, 24 / n)
        dh = integers(gen, rows, n, most=1) * (torch.rand(rows, n, generator=gen, device="cuda") < few)
        big = torch.full((rows, n), 64.0, dtype=t, device="cuda")
        wg, wu = integers(gen, n, cols, most=2), integers(gen, n, cols, most=1)
        dx = torch.empty(rows, cols, dtype=t, device="cuda")
        up = integers(gen, rows, n, most=2)
        gca.gated_linear_backward(dh.to(t), big, up.to(t), gate, h, w_gate=wg.to(t),
                                  w_up=(wu / 64).to(t), dx=dx)
        assert torch.equal(gate.double(), (dh * up).double())
        assert torch.equal(h.double(), 64 * dh.double())
        want = (dh * up).double() @ wg.double() + dh.double() @ wu.double()
        assert want.abs().max() <= 256
        assert torch.equal(dx.double(), want), f"{dtype} {rows} {n} {cols}"


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_activations_over_their_range(dtype, act):
    """act and its slope from the smallest to the largest arguments, through the backward pass
    (dgate = slope where dh = up = 1, dup = act)."""
    g = torch.cat([torch.linspace(-30, 30, 4001), torch.logspace(-30, 4, 400),
                   -torch.logspace(-30, 4, 400), torch.tensor([0.0, -0.0, 88.0, -88.0, -104.0, 6e4])])
    g = g.view(1, -1).to(TYPES[dtype]).cuda()
    one, dg, du = torch.ones_like(g), torch.empty_like(g), torch.empty_like(g)
    gca.gated_linear_backward(one, g, one, dg, du, activation=act)
    a, s, ea, es = act64(act, g.double())
    close(du, a, U * (ea + 4 * a.abs()), dtype, f"{act} {dtype}")
    close(dg, s, U * (es + 4 * s.abs()), dtype, f"{act} slope {dtype}")


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_inf_and_nan_stay_in_their_rows_and_columns(dtype):
    gen = torch.Generator("cuda").manual_seed(2)
    rows, n, cols = 150, 140, 100
    x, wg, wu = randn(gen, rows, cols, dtype=dtype), randn(gen, n, cols, dtype=dtype), randn(
        gen, n, cols, dtype=dtype)
    h, gate, up = (torch.empty(rows, n, dtype=TYPES[dtype], device="cuda") for _ in range(3))
    gca.gated_linear(x, wg, wu, h, gate=gate, up=up)
    clean = [t.clone() for t in (h, gate, up)]
    x[3, 99], x[140, 0], wg[5, 50], wu[139, 99] = (float("nan"), float("inf"), float("nan"),
                                                  float("nan"))
    gca.gated_linear(x, wg, wu, h, gate=gate, up=up)
    bad_rows = torch.zeros(rows, 1, dtype=torch.bool, device="cuda")
    bad_rows[3], bad_rows[140] = True, True
    for got, want, columns in ((h, clean[0], (5, 139)), (gate, clean[1], (5,)),
                               (up, clean[2], (139,))):
        bad = bad_rows.expand(rows, n).clone()
        bad[:, list(columns)] = True
        assert torch.equal(got[~bad], want[~bad])
        assert torch.isnan(got[3]).all() and torch.isnan(got[:, list(columns)]).all()
        assert not torch.isfinite(got[140]).any()
    gate, up, dh = clean[1], clean[2], randn(gen, rows, n, dtype=dtype)
    wg, wu = randn(gen, n, cols, dtype=dtype), randn(gen, n, cols, dtype=dtype)
    dg, du, dx = torch.empty_like(dh), torch.empty_like(dh), torch.empty_like(x)
    gca.gated_linear_backward(dh, gate, up, dg, du, w_gate=wg, w_up=wu, dx=dx)
    clean = dx.clone()
    dh[7, 139], wu[0, 64] = float("nan"), float("inf")
    gca.gated_linear_backward(dh, gate, up, dg, du, w_gate=wg, w_up=wu, dx=dx)
    bad = torch.zeros_like(dx, dtype=torch.bool)
    bad[7], bad[:, 64] = True, True
    assert torch.equal(dx[~bad], clean[~bad])
    assert torch.isnan(dx[7]).all() and not torch.isfinite(dx[:, 64]).any()
    # a gate without bounds: its limits, or NaN where the formula has Inf * 0
    g = torch.tensor([[float("inf"), float("nan")]], dtype=TYPES[dtype], device="cuda")
    one, dg, du = torch.ones_like(g), torch.empty_like(g), torch.empty_like(g)
    gca.gated_linear_backward(one, g, one, dg, du)
    assert du[0, 0] == float("inf") and torch.isnan(du[0, 1]) and torch.isnan(dg[0, 1])


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_empty_dimensions(dtype):
    empty = lambda *s: torch.empty(*s, dtype=TYPES[dtype], device="cuda")  # noqa: E731
    h = torch.full((3, 5), 7.0, dtype=TYPES[dtype], device="cuda")
    gate, up = h.clone(), h.clone()
    gca.gated_linear(empty(3, 0), empty(5, 0), empty(5, 0), h, gate=gate, up=up)
    assert not h.any() and not gate.any() and not up.any()
    gca.gated_linear(empty(0, 4), empty(5, 4), empty(5, 4), empty(0, 5))
    gca.gated_linear(empty(3, 4), empty(0, 4), empty(0, 4), empty(3, 0))
    dx = torch.full((3, 4), 7.0, dtype=TYPES[dtype], device="cuda")
    gca.gated_linear_backward(empty(3, 0), empty(3, 0), empty(3, 0), empty(3, 0), empty(3, 0),
                              w_gate=empty(0, 4), w_up=empty(0, 4), dx=dx)
    assert not dx.any()
    gca.gated_linear_backward(empty(0, 2), empty(0, 2), empty(0, 2), empty(0, 2), empty(0, 2),
                              w_gate=empty(2, 4), w_up=empty(2, 4), dx=empty(0, 4))
    gca.gated_linear_backward(empty(2, 3).zero_(), empty(2, 3).zero_(), empty(2, 3).zero_(),
                              empty(2, 3), empty(2, 3), w_gate=empty(3, 0), w_up=empty(3, 0),
                              dx=empty(2, 0))


def test_leading_dimensions_and_halves_of_one_weight():
    gen = torch.Generator("cuda").manual_seed(5)
    x = randn(gen, 2, 3, 7, 64, dtype="bf16")
    w = randn(gen, 2 * 96, 64, scale=0.2, dtype="bf16")
    both = torch.empty(42, 192, dtype=torch.bfloat16, device="cuda")
    h, h2 = (torch.empty(2, 3, 7, 96, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gate, up = both.view(2, 3, 7, 192)[..., :96], both.view(2, 3, 7, 192)[..., 96:]
    gca.gated_linear(x, w[:96], w[96:], h, gate=gate, up=up)
    flat = [torch.empty(42, 96, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    gca.gated_linear(x.view(42, 64), w[:96].clone(), w[96:].clone(), h2.view(42, 96), gate=flat[0],
                     up=flat[1])
    assert torch.equal(h, h2) and torch.equal(both, torch.cat(flat, 1))
    # the gradients of both side by side, as one weight gradient takes them, over their inputs
    dx, dx2 = torch.empty_like(x), torch.empty_like(x)
    gca.gated_linear_backward(h, gate, up, gate, up, w_gate=w[:96], w_up=w[96:], dx=dx)
    gca.gated_linear_backward(h.view(42, 96), flat[0], flat[1], flat[0], flat[1], w_gate=w[:96],
                              w_up=w[96:], dx=dx2.view(42, 64))
    assert torch.equal(dx, dx2) and torch.equal(both, torch.cat(flat, 1))


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_two_streams_repeats_and_the_callers_workspace(dtype):
    """Calls at once on two streams, each with a workspace of its own, give the bits of calls one after
    the other."""
    gen = torch.Generator("cuda").manual_seed(9)
    shapes = [(3, 500, 700), (130, 384, 512), (300, 1000, 130), (64, 264, 2000)]
    data, want = [], []
    for rows, n, cols in shapes:
        x, dh = randn(gen, rows, cols, dtype=dtype), randn(gen, rows, n, dtype=dtype)
        wg, wu = (randn(gen, n, cols, scale=0.05, dtype=dtype) for _ in range(2))
        data.append((x, wg, wu, dh))

    def outputs():
        return [[torch.full((r, c), 7.0, dtype=TYPES[dtype], device="cuda")
                 for c in (n, n, n, n, n, cols)] for r, n, cols in shapes]

    def work(i, o, stream=None):
        x, wg, wu, dh = data[i]
        rows, n, cols = shapes[i]
        sizes = [f(rows, n, cols, TYPES[dtype]) for f in (gca.gated_linear_workspace,
                                                          gca.gated_linear_backward_workspace)]
        ws = [torch.empty(max(s, 16), dtype=torch.uint8, device="cuda") for s in sizes]
        torch.cuda.current_stream().synchronize()
        gca.gated_linear(x, wg, wu, o[0], gate=o[1], up=o[2], workspace=ws[0], stream=stream)
        gca.gated_linear_backward(dh, o[1], o[2], o[3], o[4], w_gate=wg, w_up=wu, dx=o[5],
                                  workspace=ws[1], stream=stream)
        return ws

    want = outputs()
    for i in range(len(shapes)):
        work(i, want[i])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = outputs()
        torch.cuda.synchronize()
        keep = [work(i, got[i], streams[i % 2]) for i in range(len(shapes))]
        torch.cuda.synchronize()
        del keep
        for w, g in zip(want, got):
            for a, b in zip(w, g):
                assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_graph_replays_match_eager_calls(dtype):
    """A captured block (forward, backward) replayed on new inputs, with eager calls between the
    replays, gives what eager calls give."""
    gen = torch.Generator("cuda").manual_seed(4)
    for rows, n, cols in ((2, 300, 260), (140, 264, 1030), (65, 100, 72)):
        t = TYPES[dtype]
        x, dh = randn(gen, rows, cols, dtype=dtype), randn(gen, rows, n, dtype=dtype)
        wg, wu = (randn(gen, n, cols, scale=0.1, dtype=dtype) for _ in range(2))
        out = [torch.empty(rows, n, dtype=t, device="cuda") for _ in range(5)]
        out.append(torch.empty(rows, cols, dtype=t, device="cuda"))

        def step(o):
            gca.gated_linear(x, wg, wu, o[0], gate=o[1], up=o[2], activation="gelu")
            gca.gated_linear_backward(dh, o[1], o[2], o[3], o[4], w_gate=wg, w_up=wu, dx=o[5],
                                      activation="gelu")

        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            step(out)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(out)
        for _ in range(4):
            x.copy_(randn(gen, rows, cols, dtype=dtype))
            dh.copy_(randn(gen, rows, n, dtype=dtype))
            eager = [torch.empty_like(o) for o in out]
            step(eager)
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(out, eager):
                assert torch.equal(a, b)


def test_versions_are_raised_and_outputs_are_constants():
    gen = torch.Generator("cuda").manual_seed(6)
    x = randn(gen, 4, 32).requires_grad_()
    w = randn(gen, 8, 32)
    h, gate, up, other = (torch.empty(4, 8, device="cuda") for _ in range(4))
    before = [t._version for t in (h, gate, up, other, w)]
    gca.gated_linear(x, w, w, h, gate=gate, up=up)
    assert [t._version > b for t, b in zip((h, gate, up, other, w), before)] == [
        True, True, True, False, False]
    assert not h.requires_grad
    dx = torch.empty(4, 32, device="cuda")
    before = [t._version for t in (h, gate, up, dx, w)]
    gca.gated_linear_backward(h, gate, up, gate, up, w_gate=w, w_up=w, dx=dx)
    assert [t._version > b for t, b in zip((h, gate, up, dx, w), before)] == [
        False, True, True, True, False]
