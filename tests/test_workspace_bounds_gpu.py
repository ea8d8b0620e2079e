"""Workspaces of exactly the stated size: nothing is written around them, and what they hold before a call
does not matter."""
import pytest
import torch

import gradient_compression_amd as gca
from tests.test_gated_gpu import TYPES, randn

pytestmark = pytest.mark.gpu


def around(size):
    """A workspace of `size` bytes, 16-byte aligned, in a buffer of sevens."""
    buf = torch.full((size + 512,), 7, dtype=torch.uint8, device="cuda")
    return buf, buf[256:256 + size]


def untouched(buf):
    return bool((buf[:256] == 7).all()) and bool((buf[-256:] == 7).all())


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("shape", [(64, 264, 2000), (300, 77, 4100), (512, 1024, 4096), (130, 384, 512),
                                   (129, 1000, 4096), (1537, 1001, 2731)], ids=str)
def test_the_block_s_parts_stay_inside(shape, dtype):
    """Forward and backward, from a workspace of sevens and from one of NaN: the same bits."""
    rows, n, cols = shape
    gen = torch.Generator("cuda").manual_seed(rows)
    t = TYPES[dtype]
    x, dh = randn(gen, rows, cols, dtype=dtype), randn(gen, rows, n, dtype=dtype)
    wg, wu = (randn(gen, n, cols, scale=0.03, dtype=dtype) for _ in range(2))
    results = []
    for fill in (7, 255):
        out = [torch.empty(rows, n, dtype=t, device="cuda") for _ in range(5)]
        dx = torch.empty(rows, cols, dtype=t, device="cuda")
        bufs = [around(f(rows, n, cols, t)) for f in (gca.gated_linear_workspace,
                                                      gca.gated_linear_backward_workspace)]
        for _, ws in bufs:
            ws.fill_(fill)
        gca.gated_linear(x, wg, wu, out[0], gate=out[1], up=out[2],
                         workspace=bufs[0][1] if bufs[0][1].numel() else None)
        gca.gated_linear_backward(dh, out[1], out[2], out[3], out[4], w_gate=wg, w_up=wu, dx=dx,
                                  workspace=bufs[1][1] if bufs[1][1].numel() else None)
        assert all(untouched(b) for b, _ in bufs)
        results.append([*out, dx])
    assert all(torch.equal(a, b) for a, b in zip(*results))
    assert all(bool(torch.isfinite(a).all()) for a in results[0])


@pytest.mark.parametrize("sizes", [[1], [0, 5], [300000] * 3, [16384, 0, 16385] * 200, [1 << 24]], ids=len)
def test_the_norm_s_sums_stay_inside(sizes):
    ts = [torch.full((n,), 0.5, device="cuda") for n in sizes]
    want = 0.5 * sum(sizes) ** 0.5
    for fill in (7, 255):
        buf, ws = around(gca.grad_norm_workspace(sizes))
        ws.fill_(fill)
        norm, norms = torch.empty(1, device="cuda"), torch.empty(len(sizes), device="cuda")
        gca.grad_norm(ts, norm, norms=norms, workspace=ws)
        assert untouched(buf)
        assert abs(norm.item() - want) <= 2.0 ** -23 * want
        each = 0.5 * torch.tensor(sizes, dtype=torch.float64, device="cuda").sqrt()
        assert bool(((norms.double() - each).abs() <= 2.0 ** -23 * each).all())


@pytest.mark.parametrize("n", [1, 1000, 16385, 300001, 4000003])
def test_one_tensor_is_clipped_as_by_the_plan(n):
    """Whether or not the two norms are equal: each is within a step (2^-23) of the other's, so that the
    factors, rounded once each, are within two, and the products within three steps of each other."""
    gen = torch.Generator("cuda").manual_seed(n)
    g = torch.randn(n, generator=gen, device="cuda")
    limit = 0.3 * g.double().norm().item()
    plan = gca.Plan([0, n], k=[0])
    clipped, theirs = g.clone(), torch.empty(1, device="cuda")
    plan.clip_by_norm(clipped, torch.tensor([limit], device="cuda"), norms_out=theirs)
    norm, mine, flat = torch.empty(1, device="cuda"), g.clone(), torch.empty(n, device="cuda")
    gca.clip_grad_norm([mine], limit, norm, out=flat)
    gca.grad_clip([mine], limit, norm)
    assert torch.equal(mine, flat)
    assert abs(norm.item() - theirs.item()) <= 2.0 ** -23 * theirs.item()
    assert bool(((mine.double() - clipped.double()).abs() <= 3 * 2.0 ** -23 * clipped.double().abs()).all())
    want = g.double() * (limit / g.double().norm())
    assert bool(((mine.double() - want).abs() <= 3 * 2.0 ** -23 * want.abs()).all())
    plan.close()
