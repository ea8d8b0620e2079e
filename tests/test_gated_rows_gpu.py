"""What stands in one row of the gated block reaches no other row, and the forward pass's activation is a
function of the gate alone, right over its range.

Gates stay below 8 where nothing was planted (unit rows through weights of 1.2 / sqrt(columns)), so that a
planted one is the only large one in its kernel's wave."""
import math

import pytest
import torch

import gradient_compression_amd as gca
from tests.gpu_helpers import log
from tests.test_gated_gpu import ACTS, TYPES, U, act64, close, randn

pytestmark = pytest.mark.gpu

# (rows, n, cols): up to 32 rows, and tiles of each size with whole sums and sums in parts
SHAPES = [(4, 100, 72), (20, 264, 200), (40, 264, 200), (64, 264, 2000), (130, 384, 512), (300, 77, 4100),
          (700, 1500, 2000), (1030, 2100, 264), (2000, 3000, 200)]


def inputs(shape, dtype, seed):
    rows, n, cols = shape
    gen = torch.Generator("cuda").manual_seed(seed)
    x = randn(gen, rows, cols, dtype=dtype)
    wg, wu = (randn(gen, n, cols, scale=1.2 / math.sqrt(cols), dtype=dtype) for _ in range(2))
    return gen, x, wg, wu


def forward(x, wg, wu, act):
    outs = [torch.empty(x.shape[0], wg.shape[0], dtype=x.dtype, device="cuda") for _ in range(3)]
    gca.gated_linear(x, wg, wu, outs[0], gate=outs[1], up=outs[2], activation=act)
    return outs


def plant(t, kind):
    """Spoils two rows (one where there are few) and says which."""
    rows = sorted({t.shape[0] // 3, t.shape[0] - 1} if t.shape[0] > 4 else {1})
    for i, r in enumerate(rows):
        if kind == "large":
            t[r] *= 300.0
        else:
            t[r, (7 * i) % t.shape[1]] = float(kind)
    clean = torch.ones(t.shape[0], dtype=torch.bool, device="cuda")
    clean[rows] = False
    return clean


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_other_rows_keep_their_bits(dtype, act):
    for i, shape in enumerate(SHAPES):
        gen, x, wg, wu = inputs(shape, dtype, i)
        want = forward(x, wg, wu, act)
        assert want[1].abs().max() < 16
        rows, n, cols = shape
        dh = randn(gen, rows, n, dtype=dtype)
        grads = lambda d, g, u: [torch.empty_like(g), torch.empty_like(u),  # noqa: E731
                                 torch.empty(rows, cols, dtype=TYPES[dtype], device="cuda")]
        back = grads(dh, *want[1:])
        gca.gated_linear_backward(dh, want[1], want[2], back[0], back[1], w_gate=wg, w_up=wu, dx=back[2],
                                  activation=act)
        for kind in ("large", "inf", "-inf", "nan"):
            log(f"[gated] rows {dtype} {act} {shape} {kind}")
            bad = x.clone()
            clean = plant(bad, kind)
            got = forward(bad, wg, wu, act)
            for name, a, b in zip(("h", "gate", "up"), got, want):
                assert torch.equal(a[clean], b[clean]), f"{name} of {shape}, {kind}"
            gate = want[1].clone()
            clean = plant(gate, kind)
            got = grads(dh, gate, want[2])
            gca.gated_linear_backward(dh, gate, want[2], got[0], got[1], w_gate=wg, w_up=wu, dx=got[2],
                                      activation=act)
            for name, a, b in zip(("dgate", "dup", "dx"), got, back):
                assert torch.equal(a[clean], b[clean]), f"{name} of {shape}, {kind}"


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_other_columns_keep_their_bits(dtype, act):
    """A large or infinite gate in one column of h, from its weight alone."""
    for i, shape in enumerate(SHAPES):
        _, x, wg, wu = inputs(shape, dtype, 100 + i)
        want = forward(x, wg, wu, act)
        for kind in ("large", "inf", "nan"):
            log(f"[gated] columns {dtype} {act} {shape} {kind}")
            bad = wg.clone()
            clean = plant(bad, kind)
            got = forward(x, bad, wu, act)
            for a, b in zip(got, want):
                assert torch.equal(a[:, clean], b[:, clean]), f"{shape}, {kind}"


def around(dtype):
    """Gates over the activations' range, each type's numbers around 16 among them."""
    t = TYPES[dtype]
    top = 6e4 if dtype == "f16" else 1e9
    g = torch.cat([torch.linspace(-30, 30, 4001), torch.linspace(-110, 110, 1001),
                   torch.logspace(-12, math.log10(top), 400), -torch.logspace(-12, math.log10(top), 400),
                   torch.tensor([0.0, -0.0, 88.0, -88.0, -104.0])])
    at = torch.tensor([16.0, -16.0]).to(t)
    edge = torch.cat([at.float() * (1 + k * torch.finfo(t).eps) for k in range(-3, 4)])
    return torch.cat([g, edge]).to(t)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_the_activation_over_its_range(dtype, act):
    """x = (gates, 1), w_gate = (identity, 0), w_up = (0, 1): h is act of the gates.  The tolerance: as in
    the tests of the block's sums, without the sums, whose one product and zeros are exact."""
    g = around(dtype)
    n = 64
    g = torch.cat([g, g[:-g.numel() % n]]) if g.numel() % n else g
    g = g.cuda()
    wg, wu = (torch.zeros(n, n + 8, dtype=TYPES[dtype], device="cuda") for _ in range(2))
    wg[:, :n], wu[:, n] = torch.eye(n), 1.0

    def h_of(gates):
        x = torch.zeros(gates.shape[0], n + 8, dtype=TYPES[dtype], device="cuda")
        x[:, :n], x[:, n] = gates, 1.0
        h, gate, up = forward(x, wg, wu, act)
        assert torch.equal(gate, gates) and bool((up == 1.0).all())
        return h

    gates = g.view(-1, n)
    a, _, ea, _ = act64(act, gates.double())
    ordered = h_of(gates)
    close(ordered, a, U * (ea + 4 * a.abs()), dtype, f"forward {act} {dtype}")
    # the same gates beside other ones, in other rows and columns, and by the kernel of few rows
    mixed = torch.randperm(g.numel(), generator=torch.Generator().manual_seed(3)).cuda()
    assert torch.equal(h_of(g[mixed].view(-1, n)).view(-1), ordered.view(-1)[mixed])
    few = torch.cat([h_of(part) for part in g[mixed].view(-1, n).split(16)])
    assert torch.equal(few.view(-1), ordered.view(-1)[mixed])
    # and among small ones only
    order = g.float().abs().argsort()
    assert torch.equal(h_of(g[order].view(-1, n)).view(-1), ordered.view(-1)[order])
