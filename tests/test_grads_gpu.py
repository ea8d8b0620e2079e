"""The norm over many tensors and their clipping on the GPU.

The norm is a sum in double, rounded once: within a step of fp32 (2^-23) of the one in 64 bits.  What is
scaled is compared bit for bit with its definition, from the GPU's own norm."""
import numpy as np
import pytest
import torch

import gradient_compression_amd as gca
from tests.gpu_helpers import log

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
STEP = 2.0 ** -23


def gradients(sizes, seed, types=(F32, BF16, F16), scale=1e-3):
    gen = torch.Generator("cuda").manual_seed(seed)
    return [(scale * torch.randn(n, generator=gen, device="cuda")).to(types[i % len(types)])
            for i, n in enumerate(sizes)]


def norms64(ts):
    s = torch.stack([t.double().square().sum() for t in ts]) if ts else torch.zeros(0).cuda().double()
    return s.sum().sqrt(), s.sqrt()


def near(got, want):
    assert bool(((got.double() - want).abs() <= STEP * want.abs()).all()), (got, want)


def factor(norm, max_norm):
    n, m = np.float32(norm.item()), np.float32(max_norm)
    return m / n if n > m and np.isfinite(n) else np.float32(1.0)


def check(sizes, seed=0, types=(F32, BF16, F16), clip=0.5):
    log(f"[grads] {len(sizes)} tensors, {sum(sizes)} elements")
    ts = gradients(sizes, seed, types)
    before = [t.clone() for t in ts]
    want, wants = norms64(ts)
    max_norm = clip * want.item()
    norm = torch.full((3,), 7.0, device="cuda")
    norms = torch.full((len(ts) + 1,), 7.0, device="cuda")
    gca.grad_norm(ts, norm[1:2], norms=norms[:len(ts)])
    near(norm[1], want)
    near(norms[:len(ts)], wants)
    assert norm[0] == 7.0 and norm[2] == 7.0 and norms[-1] == 7.0
    only = torch.zeros(1, device="cuda")
    gca.grad_norm(ts, only)
    assert torch.equal(only, norm[1:2])
    f = torch.tensor(factor(norm[1], max_norm), device="cuda")
    # into a flat fp32 gradient, between sevens
    total = sum(sizes)
    flat = torch.full((total + 2,), 7.0, device="cuda")
    got = torch.empty(1, device="cuda")
    factors = torch.full((5,), 7.0, device="cuda")
    gca.clip_grad_norm(ts, max_norm, got, out=flat[1:-1], factors=factors[1:4])
    assert torch.equal(got, only) and flat[0] == 7.0 and flat[-1] == 7.0
    assert bool((factors[1:4] == f).all()) and factors[0] == 7.0 and factors[4] == 7.0
    scaled = [t.float() * f for t in before]
    assert torch.equal(flat[1:-1], torch.cat(scaled) if scaled else flat[1:-1])
    assert all(torch.equal(a, b) for a, b in zip(ts, before))
    # into tensors of other types
    for shift in (1, 2):
        other = [torch.empty(n, dtype=types[(i + shift) % len(types)], device="cuda")
                 for i, n in enumerate(sizes)]
        gca.grad_clip(ts, max_norm, norm[1:2], out=other)
        assert all(torch.equal(o, s.to(o.dtype)) for o, s in zip(other, scaled))
    # in place
    gca.clip_grad_norm(ts, max_norm, got, norms=norms[:len(ts)])
    assert all(torch.equal(t, s.to(t.dtype)) for t, s in zip(ts, scaled))


SIZES = [[1], [0], [], [7], [0, 0, 3, 0], [8, 9, 15, 16, 17], [16383, 16384, 16385],
         [100, 0, 50000, 1, 0, 0, 32768, 2049, 0], [1 << 20, 3, (1 << 20) + 1], [40 << 20, 5, 77777]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}_{sum(s)}")
def test_norm_and_clip(sizes):
    check(sizes)


@pytest.mark.parametrize("count", [159, 160, 161, 239, 240, 241, 479, 481, 1000])
def test_as_many_tensors_as_launches_hold(count):
    rng = np.random.default_rng(count)
    sizes = [int(n) for n in rng.integers(0, 40000, count)]
    sizes[::7] = [0] * len(sizes[::7])
    if count == 481:
        sizes[:240] = [0] * 240       # a launch without elements
    check(sizes, seed=count)


def test_small_norms_change_nothing():
    ts = gradients([1000, 70000, 3], 1)
    ts[0][5], ts[1][7] = -0.0, 1e-30
    before = [t.clone() for t in ts]
    version = [t._version for t in ts]
    norm, factors = torch.empty(1, device="cuda"), torch.empty(4, device="cuda")
    gca.clip_grad_norm(ts, 1e9, norm, factors=factors)
    assert all(torch.equal(t.view(torch.uint8), b.view(torch.uint8)) for t, b in zip(ts, before))
    assert bool((factors == 1.0).all())
    assert all(t._version > v for t, v in zip(ts, version))
    # at the limit itself nothing is scaled
    gca.clip_grad_norm(ts, norm.item(), norm, factors=factors)
    assert bool((factors == 1.0).all())


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_inf_and_nan_are_told_and_left(dtype):
    for bad in (float("inf"), -float("inf"), float("nan")):
        ts = gradients([1000, 40000, 9], 2, (dtype,))
        ts[1][39999] = bad
        before = [t.clone() for t in ts]
        norm, norms, factors = (torch.empty(n, device="cuda") for n in (1, 3, 2))
        gca.clip_grad_norm(ts, 0.25, norm, norms=norms, factors=factors)
        for n in (norm[0], norms[1]):
            assert torch.isnan(n) if bad != bad else n == float("inf")
        assert torch.isfinite(norms[0]) and torch.isfinite(norms[2])
        assert bool((factors == 1.0).all())
        assert all(torch.equal(t.view(torch.uint8), b.view(torch.uint8)) for t, b in zip(ts, before))


def test_range_of_the_squares():
    """Elements whose squares fp32 has not: the norm is right up to fp32's range, Inf above it."""
    for v in (1e30, 1e-30, 1e-42):
        ts = [torch.full((1000,), v, device="cuda"), torch.full((44,), -v, device="cuda")]
        want, _ = norms64(ts)
        norm = torch.empty(1, device="cuda")
        gca.clip_grad_norm(ts, 0.0, norm)
        # 1e-42 is a denormal: half a step of those
        assert abs(norm.item() - want.item()) <= max(STEP * want.item(), 2.0 ** -150)
        assert all(not t.any() for t in ts)
    ts = [torch.full((100,), 3e38, device="cuda")]
    norm = torch.empty(1, device="cuda")
    gca.clip_grad_norm(ts, 1.0, norm)
    assert norm.item() == float("inf") and bool((ts[0] == ts[0][0]).all()) and ts[0][0] > 2e38


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_tensors_at_any_element(dtype):
    """Tensors back to back in one bucket, and into places of a flat gradient, at every offset."""
    gen = torch.Generator("cuda").manual_seed(3)
    sizes = [1, 2, 3, 5, 8, 13, 21, 4099, 8191, 16383, 20001, 2, 65539]
    bucket = torch.randn(sum(sizes) + 2, generator=gen, device="cuda").to(dtype)
    first = bucket.clone()
    views = list(bucket[1:-1].split(sizes))
    want, _ = norms64(views)
    norm, flat = torch.empty(1, device="cuda"), torch.full((sum(sizes) + 8,), 7.0, device="cuda")
    gca.clip_grad_norm(views, 0.1 * want.item(), norm, out=flat[3:-5])
    near(norm[0], want)
    f = torch.tensor(factor(norm[0], 0.1 * want.item()), device="cuda")
    assert torch.equal(flat[3:-5], first[1:-1].float() * f)
    assert bool((flat[:3] == 7.0).all()) and bool((flat[-5:] == 7.0).all())
    gca.grad_clip(views, 0.1 * want.item(), norm)
    assert torch.equal(bucket[1:-1], (first[1:-1].float() * f).to(dtype))
    assert bucket[0] == first[0] and bucket[-1] == first[-1]


def test_a_long_tensor():
    """More than 2^31 elements in one tensor and 2^32 in all."""
    ts = [torch.empty((1 << 31) + 12345, dtype=BF16, device="cuda"),
          torch.empty((1 << 31) + 5, dtype=F16, device="cuda")]
    for i, t in enumerate(ts):
        t.fill_(0.5)
        t[-1] = 3.0 + i
    n0, n1 = (t.numel() for t in ts)
    want = (0.25 * (n0 + n1 - 2) + 9 + 16) ** 0.5
    norm, norms = torch.empty(1, device="cuda"), torch.empty(2, device="cuda")
    gca.clip_grad_norm(ts, want / 2, norm, norms=norms)
    assert abs(norm.item() - want) <= STEP * want
    for i, (t, n) in enumerate(zip(ts, (n0, n1))):
        one = (0.25 * (n - 1) + (3.0 + i) ** 2) ** 0.5
        assert abs(norms[i].item() - one) <= STEP * one
        f = factor(norm[0], want / 2)
        low = torch.tensor(0.5 * f).to(t.dtype).item()
        assert t[-1].item() == torch.tensor(np.float32(3.0 + i) * f).to(t.dtype).item()
        assert bool((t[:-1] == low).all())


def test_two_streams_repeats_and_the_callers_workspace():
    sizes = [300000, 5, 0, 70001, 16384, 9] * 20
    sets = [gradients(sizes, s) for s in range(3)]
    ws = [torch.empty(gca.grad_norm_workspace(sizes), dtype=torch.uint8, device="cuda")
          for _ in sets]
    norms = [torch.empty(1, device="cuda") for _ in sets]
    flats = [torch.empty(sum(sizes), device="cuda") for _ in sets]
    for i, ts in enumerate(sets):
        gca.clip_grad_norm(ts, 0.3, norms[i], out=flats[i], workspace=ws[i])
    torch.cuda.synchronize()
    want = [(n.clone(), f.clone()) for n, f in zip(norms, flats)]
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        for f in flats:
            f.fill_(7.0)
        torch.cuda.synchronize()
        for i, ts in enumerate(sets):
            gca.clip_grad_norm(ts, 0.3, norms[i], out=flats[i], workspace=ws[i], stream=streams[i])
        torch.cuda.synchronize()
        for (n, f), n2, f2 in zip(want, norms, flats):
            assert torch.equal(n, n2) and torch.equal(f, f2)


def test_graph_replays_match_eager_calls():
    sizes = [40000, 3, 0, 100001] * 70        # two launches of each kernel
    ts = gradients(sizes, 8)
    norm, norms = torch.empty(1, device="cuda"), torch.empty(len(sizes), device="cuda")
    flat = torch.empty(sum(sizes), device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        gca.clip_grad_norm(ts, 0.5, norm, out=flat, norms=norms)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gca.clip_grad_norm(ts, 0.5, norm, out=flat, norms=norms)
    for i in range(4):
        for t, new in zip(ts, gradients(sizes, 100 + i, scale=(1e-3, 1e-5, 1e-2, 1e-4)[i])):
            t.copy_(new)
        eager = [torch.empty_like(t) for t in (norm, norms, flat)]
        gca.clip_grad_norm(ts, 0.5, eager[0], out=eager[2], norms=eager[1])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((norm, norms, flat), eager):
            assert torch.equal(a, b)


def test_one_tensor_agrees_with_the_plan_s_clipping():
    """A gradient of one segment: the global norm is the segment's."""
    n = 300001
    g = torch.randn(n, device="cuda")
    plan = gca.Plan([0, n], k=[0])
    limit, theirs = torch.tensor([20.0], device="cuda"), torch.empty(1, device="cuda")
    clipped = g.clone()
    plan.clip_by_norm(clipped, limit, norms_out=theirs)
    norm = torch.empty(1, device="cuda")
    mine = g.clone()
    gca.clip_grad_norm([mine], 20.0, norm)
    near(norm[0], theirs[0].double())
    if torch.equal(norm, theirs):
        assert torch.equal(mine, clipped)
    plan.close()


def test_factors_go_into_the_compressors():
    """The global factor through Plan.set_gradient_scale gives what compressing the clipped gradient
    gives."""
    sizes = [5000, 33, 70000, 20001]
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int64)
    n = int(off[-1])
    parts = gradients(sizes, 12)
    plan = gca.Plan(off, ratio=0.01)
    norm, factors = torch.empty(1, device="cuda"), torch.empty(len(sizes), device="cuda")
    results = []
    for folded in (False, True):
        flat = torch.empty(n, device="cuda")
        e = torch.zeros(n, device="cuda")
        vals = torch.empty(plan.total_k, device="cuda")
        idx = torch.empty(plan.total_k, dtype=torch.int32, device="cuda")
        if folded:
            gca.grad_norm(parts, norm)
            gca.grad_clip(parts, float("inf"), norm, out=flat)        # as they are
            gca.grad_clip([], 0.05, norm, factors=factors)
            plan.set_gradient_scale(factors)
        else:
            gca.clip_grad_norm(parts, 0.05, norm, out=flat)
        plan.compress(flat, e, vals, idx)
        torch.cuda.synchronize()
        results.append((vals, idx, e))
    plan.set_gradient_scale(None)
    assert norm.item() > 0.05
    for a, b in zip(*results):
        assert torch.equal(a, b)
    plan.close()
