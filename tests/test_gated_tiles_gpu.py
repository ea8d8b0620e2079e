"""The gated block at sizes that take every tile, whole sums and sums in parts, and at random ones, against
the formulas in 64 bits; far apart rows, more than 2^31 elements, and ends of the number range.

Tolerances as derived beside the checks that these tests call."""
import math
import random

import pytest
import torch

import gradient_compression_amd as gca
from tests.gpu_helpers import log
from tests.test_gated_gpu import (ACTS, HALF, TYPES, U, act64, check_backward, check_forward, close,
                                  randn, sums64)

pytestmark = pytest.mark.gpu

# large and small tiles with whole sums and sums in parts, last tiles of one row or column
SHAPES = [(2000, 3000, 1000), (1300, 2100, 800), (3000, 4100, 700), (700, 1500, 2000),
          (2500, 1100, 3000), (1000, 4000, 520), (4100, 2100, 1030), (513, 2049, 1025), (32, 3000, 2050),
          (33, 3000, 2050), (128, 1000, 4096), (129, 1000, 4096), (7, 129, 9000)]


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_every_tile(shape, dtype):
    rows, n, cols = shape
    check_forward(rows, n, cols, dtype, ACTS[(rows + n) % 3])
    check_backward(rows, n, cols, dtype, ACTS[(rows + cols) % 3])


@pytest.mark.parametrize("seed", range(6))
def test_random_configurations(seed):
    rng = random.Random(seed)
    size = lambda most: int(round(most ** rng.random()))  # noqa: E731
    for i in range(12):
        rows, n, cols = size(3000), size(3000), size(3000)
        if rng.random() < 0.3:
            rows, n, cols = (max(8, v // 8 * 8) for v in (rows, n, cols))
        dtype, act = rng.choice(sorted(TYPES)), rng.choice(ACTS)
        pad, shift = rng.choice([(0, 0), (0, 0), (8, 0), (1, 0), (5, 3), (24, 16)])
        check_forward(rows, n, cols, dtype, act, pad, shift, keep=rng.random() < 0.7, seed=seed + i)
        check_backward(rows, n, cols, dtype, act, pad, shift, in_place=rng.random() < 0.5,
                       seed=seed + i)


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_far_apart_rows(dtype):
    """Rows 2^21 and more elements apart, whose offsets in a tile pass 32 bits."""
    gen = torch.Generator("cuda").manual_seed(1)
    rows, n, cols = 300, 140, 200
    far = {"f32": (1 << 22) + 3, "bf16": (1 << 23) + 8, "f16": (1 << 22) + 1}[dtype]
    big = torch.empty(rows * far + cols, dtype=TYPES[dtype], device="cuda")
    x = big[:rows * far].view(rows, far)[:, :cols]
    x0 = randn(gen, rows, cols, dtype=dtype)
    x.copy_(x0)
    wg, wu = (randn(gen, n, cols, scale=0.1, dtype=dtype) for _ in range(2))
    h, gate, up = (torch.empty(rows, n, dtype=TYPES[dtype], device="cuda") for _ in range(3))
    near = [torch.empty_like(t) for t in (h, gate, up)]
    gca.gated_linear(x, wg, wu, h, gate=gate, up=up)
    gca.gated_linear(x0, wg, wu, near[0], gate=near[1], up=near[2])
    assert all(torch.equal(a, b) for a, b in zip((h, gate, up), near))
    gca.gated_linear(x[:20], wg, wu, h[:20])
    gca.gated_linear(x0[:20], wg, wu, near[0][:20])
    assert torch.equal(h[:20], near[0][:20])
    # weights, gradients and results far apart
    w = big[:n * far].view(n, far)[:, :cols]
    w.copy_(wg)
    dx, dx_near = (torch.empty(rows, cols, dtype=TYPES[dtype], device="cuda") for _ in range(2))
    gca.gated_linear_backward(h, gate, up, gate, up, w_gate=w, w_up=wu, dx=dx)
    gca.gated_linear_backward(near[0], near[1], near[2], near[1], near[2], w_gate=wg, w_up=wu,
                              dx=dx_near)
    assert torch.equal(dx, dx_near) and torch.equal(gate, near[1])
    out = big[:rows * far].view(rows, far)[:, 7:7 + cols]
    gca.gated_linear_backward(near[0], near[1], near[2], gate, up, w_gate=wg, w_up=wu, dx=out)
    gca.gated_linear_backward(near[0], near[1], near[2], gate, up, w_gate=wg, w_up=wu, dx=dx)
    assert torch.equal(out, dx)


def test_more_than_2_to_31_elements():
    """Weights, rows and results of more than 2^31 elements: integers, compared where they are wanted."""
    t = torch.bfloat16
    log("[gated] long weights")
    n, cols, rows = 33000, 66000, 5
    wg = torch.zeros(n, cols, dtype=t, device="cuda")
    wu = torch.zeros(n, cols, dtype=t, device="cuda")
    x = torch.zeros(rows, cols, dtype=t, device="cuda")
    picks = [(0, 0), (n - 1, cols - 1), (n - 1, 0), (n // 2, cols - 7), (32768, 65535)]
    for i, (r, c) in enumerate(picks):
        wg[r, c], wu[r, c], x[i % rows, c] = 64.0, 3.0 + i, 1.0
    h, gate, up = (torch.empty(rows, n, dtype=t, device="cuda") for _ in range(3))
    gca.gated_linear(x, wg, wu, h, gate=gate, up=up)
    want_g, want_u = torch.zeros(rows, n), torch.zeros(rows, n)
    for m in range(rows):
        for i, (r, c) in enumerate(picks):
            if x[m, c] == 1.0:
                want_g[m, r] += 64.0
                want_u[m, r] += 3.0 + i
    assert torch.equal(gate.float().cpu(), want_g) and torch.equal(up.float().cpu(), want_u)
    dh = torch.zeros(rows, n, dtype=t, device="cuda")
    dh[0, n - 1], dh[4, 0] = 1.0, 2.0
    dx = torch.empty(rows, cols, dtype=t, device="cuda")
    gate.fill_(64.0)
    up.fill_(1.0)
    gca.gated_linear_backward(dh, gate, up, gate, up, w_gate=wg, w_up=wu, dx=dx)
    want = torch.zeros(rows, cols)
    want[0] = (wg[n - 1].float() + 64.0 * wu[n - 1].float()).cpu()
    want[4] = (2.0 * wg[0].float() + 128.0 * wu[0].float()).cpu()
    assert torch.equal(dx.float().cpu(), want)
    del wg, wu, x, h, gate, up, dh, dx
    torch.cuda.empty_cache()
    log("[gated] many rows")
    rows, n, cols = (1 << 23) + 77, 264, 16
    gen = torch.Generator("cuda").manual_seed(0)
    x = torch.randint(-2, 3, (rows, cols), generator=gen, device="cuda").to(t)
    wg, wu = (torch.randint(-2, 3, (n, cols), generator=gen, device="cuda").to(t) for _ in range(2))
    h, up = torch.empty(rows, n, dtype=t, device="cuda"), torch.empty(rows, n, dtype=t, device="cuda")
    gca.gated_linear(x, wg, wu, h, up=up)
    for at in (slice(0, 300), slice(rows // 2, rows // 2 + 300), slice(rows - 300, rows)):
        want = x[at].float() @ wu.float().t().contiguous()
        assert torch.equal(up[at].float(), want)
        a = act64("silu", (x[at].double() @ wg.double().t().contiguous()))[0] * want.double()
        assert bool(((h[at].double() - a).abs() <= (HALF["bf16"] + 40 * U) * a.abs()).all())
    dgate = torch.empty_like(h)
    dx = torch.empty(rows, cols, dtype=t, device="cuda")
    h.fill_(64.0)                       # a gate at which silu is 64 and its slope 1
    one = torch.ones(1, 1, dtype=t, device="cuda").expand(rows, n).contiguous()
    gca.gated_linear_backward(one, h, up, dgate, h, w_gate=wg, w_up=wu / 64, dx=dx)
    for at in (slice(0, 300), slice(rows - 300, rows)):
        want = up[at].float() @ wg.float() + wu.float().sum(0)
        assert torch.equal(dx[at].float(), want.to(t).float())


def test_fp32_from_the_smallest_to_the_largest_numbers():
    """fp32 products over its whole range, each row and column of a magnitude of its own: the bf16 parts of a
    value hold it, what is below 2^-126 may count as 0, and what passes the range is Inf as in one sum."""
    gen = torch.Generator("cuda").manual_seed(3)
    rows, n, cols = 96, 160, 72
    x, wg, wu = randn(gen, rows, cols), randn(gen, n, cols), randn(gen, n, cols)
    sx = 2.0 ** torch.arange(-60, 36, device="cuda").float()
    sw = 2.0 ** torch.linspace(-40, 60, n, device="cuda").round()
    x, wg, wu = x * sx[:, None], wg * sw[:, None], wu * sw[:, None]
    h, gate, up = (torch.empty(rows, n, device="cuda") for _ in range(3))
    gca.gated_linear(x, wg, wu, h, gate=gate, up=up)
    for got, w in ((gate, wg), (up, wu)):
        want, bound = sums64(x.double(), w.double(), "f32")
        # 6 products of parts a value, each part's low bits below 2^-126 dropped
        low = 6 * 2.0 ** -126 * (x.abs().sum(1, keepdim=True) + w.abs().sum(1)).double()
        close(got, want, bound + low, "f32", "range")
    # the largest: hi rounds to Inf, and the whole element says what it is
    top = torch.finfo(torch.float32).max
    x = torch.zeros(40, 64, device="cuda")
    x[0, 0], x[1, 1], x[2, 2], x[3, 3] = top, float("inf"), -float("inf"), 3.39e38
    w = torch.zeros(64, 64, device="cuda")
    w[:, 0], w[:, 1], w[:, 2], w[:, 3] = 0.5, 1.0, 2.0, 1.0
    w[5, 1] = 0.0
    gate, up, h = (torch.empty(40, 64, device="cuda") for _ in range(3))
    gca.gated_linear(x, w, w, h, gate=gate, up=up)
    assert torch.equal(gate[0], torch.full((64,), top / 2, device="cuda"))
    assert bool((gate[1][torch.arange(64) != 5] == float("inf")).all()) and torch.isnan(gate[1, 5])
    assert bool((gate[2] == -float("inf")).all())
    assert bool((gate[3] == torch.tensor(3.39e38, device="cuda")).all())
    assert not gate[4:].any()
    # the same through the backward pass's product
    dh = torch.zeros(40, 64, device="cuda")
    dh[1, 3] = float("inf")
    one = torch.ones_like(dh)
    dx, dg, du = torch.empty(40, 64, device="cuda"), torch.empty_like(dh), torch.empty_like(dh)
    gca.gated_linear_backward(dh, 64 * one, one, dg, du, w_gate=torch.ones(64, 64, device="cuda"),
                              w_up=torch.zeros(64, 64, device="cuda") + 0.5, dx=dx)
    assert bool((dx[1] == float("inf")).all()) and not dx[0].any() and not dx[2:].any()


def test_what_lies_behind_the_last_row_stays():
    """Rows behind the last sequence's, in every path: left as they were."""
    gen = torch.Generator("cuda").manual_seed(8)
    for dtype in sorted(TYPES):
        for rows, n, cols in ((5, 100, 300), (70, 130, 520), (700, 1500, 2000), (300, 77, 4100)):
            x, dh = randn(gen, rows, cols, dtype=dtype), randn(gen, rows, n, dtype=dtype)
            wg, wu = (randn(gen, n, cols, scale=0.1, dtype=dtype) for _ in range(2))
            outs = [torch.full((rows + 40, c), 7.0, dtype=TYPES[dtype], device="cuda")
                    for c in (n, n, n, n, n, cols)]
            v = [o[20:20 + rows] for o in outs]
            gca.gated_linear(x, wg, wu, v[0], gate=v[1], up=v[2])
            gca.gated_linear_backward(dh, v[1], v[2], v[3], v[4], w_gate=wg, w_up=wu, dx=v[5])
            for o in outs:
                assert bool((o[:20] == 7.0).all()) and bool((o[20 + rows:] == 7.0).all())


def test_fp32_products_just_below_the_largest_number():
    """A value whose first bf16 part is a power of two above it: that part's product passes fp32's range where the
    value's own, exact here, does not."""
    rows, n, cols = 70, 100, 520
    near = 2.0 ** 65 - 2.0 ** 55
    x = torch.zeros(rows, cols, device="cuda")
    wg, wu = torch.zeros(n, cols, device="cuda"), torch.zeros(n, cols, device="cuda")
    x[3, 5], wg[:, 5], wu[:, 5] = near, 2.0 ** 63, 2.0 ** -100
    h, gate, up = (torch.empty(rows, n, device="cuda") for _ in range(3))
    gca.gated_linear(x, wg, wu, h, gate=gate, up=up)
    want = torch.zeros(rows, n, dtype=torch.float64, device="cuda")
    want[3] = near * 2.0 ** 63
    assert torch.equal(gate.double(), want)
    want[3] *= near * 2.0 ** -100      # silu is the identity there, to 16 * 2^-24 of it as everywhere
    assert bool(((h.double() - want).abs() <= 17 * 2.0 ** -24 * want).all())
    # dgate = 2^65 - 2^55 to a few units, as silu's slope at 100 is 1 to 16 * 2^-24; dup's weights are 0
    dh = torch.zeros(rows, n, device="cuda")
    dh[2, 4] = near
    wg, wu = torch.zeros(n, cols, device="cuda"), torch.zeros(n, cols, device="cuda")
    wg[4] = 2.0 ** 63
    dx, dg, du = torch.empty(rows, cols, device="cuda"), torch.empty_like(dh), torch.empty_like(dh)
    gca.gated_linear_backward(dh, torch.full_like(dh, 100.0), torch.ones_like(dh), dg, du, w_gate=wg,
                              w_up=wu, dx=dx)
    want = torch.zeros(rows, cols, dtype=torch.float64, device="cuda")
    want[2] = near * 2.0 ** 63
    assert bool(((dx.double() - want).abs() <= 20 * 2.0 ** -24 * want).all())
