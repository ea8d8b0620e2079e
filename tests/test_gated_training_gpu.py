"""The operators together, as a training step has them: the norm that keeps its row in 8 bits, the gated
block, the layer behind it, their backward passes and weight gradients, and all gradients clipped by their
global norm into the flat gradient that the compressor takes.  The gradients are compared with autograd's
in 64 bits, and those with differences."""
import numpy as np
import pytest
import torch

import gradient_compression_amd as gca

pytestmark = pytest.mark.gpu

ROWS, COLS, N = 96, 160, 224


class Block:
    """norm -> gated -> down, with its weights; `n` as one name for each of its tensors."""

    def __init__(self, dtype, seed):
        gen = torch.Generator("cuda").manual_seed(seed)
        r = lambda *s, k=1.0: (k * torch.randn(*s, generator=gen, device="cuda")).to(dtype)  # noqa: E731
        self.x, self.dout = r(ROWS, COLS), r(ROWS, COLS, k=0.1)
        self.w = (1.0 + 0.1 * torch.randn(COLS, generator=gen, device="cuda")).to(dtype)
        self.wg, self.wu = r(N, COLS, k=1.3 * COLS ** -0.5), r(N, COLS, k=COLS ** -0.5)
        self.wd = r(COLS, N, k=N ** -0.5)

    def weights(self):
        return [self.w, self.wg, self.wu, self.wd]

    def step(self, act):
        """dx and the gradients of the four weights, through the library."""
        t = self.x.dtype
        empty = lambda *s, d=t: torch.empty(*s, dtype=d, device="cuda")  # noqa: E731

        def kept(cols):
            pitch, groups = gca.act_layout(cols)
            return empty(ROWS, pitch, d=torch.int8), empty(ROWS, groups, d=torch.uint8)

        codes, exps = kept(COLS)
        rstd, y = empty(ROWS, d=torch.float32), empty(ROWS, COLS)
        gca.rmsnorm(self.x, weight=self.w, eps=1e-5, y=y, rstd=rstd, codes=codes, exps=exps)
        h, both = empty(ROWS, N), empty(ROWS, 2 * N)
        gate, up = both[:, :N], both[:, N:]
        gca.gated_linear(y, self.wg, self.wu, h, gate=gate, up=up, activation=act)
        hcodes, hexps = kept(N)
        gca.act_quant(h, hcodes, hexps)
        # backward
        grads = [empty(COLS, d=torch.float32), empty(2 * N, COLS, d=torch.float32),
                 empty(COLS, N, d=torch.float32)]
        gca.act_weight_grad(self.dout, hcodes, hexps, grads[2])
        dh = (self.dout.float() @ self.wd.float()).to(t)
        dy = empty(ROWS, COLS)
        gca.gated_linear_backward(dh, gate, up, gate, up, w_gate=self.wg, w_up=self.wu, dx=dy,
                                  activation=act)
        gca.act_weight_grad(both, codes, exps, grads[1], col_scale=self.w)   # both weights at once
        dx = empty(ROWS, COLS)
        gca.rmsnorm_backward(dy, codes, exps, rstd, dx, weight=self.w, dweight=grads[0])
        return h, dx, [grads[0], grads[1][:N], grads[1][N:], grads[2]]

    def plain(self, act, x, w, wg, wu, wd):
        y = x * (x.square().mean(1, keepdim=True) + 1e-5).rsqrt() * w
        g = y @ wg.t()
        a = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
             "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[act](g)
        return (a * (y @ wu.t())) @ wd.t()

    def autograd(self, act):
        """The same in 64 bits on the CPU, and its loss as a function of the leaves."""
        leaves = [t.detach().double().cpu().requires_grad_() for t in (self.x, *self.weights())]
        dout = self.dout.double().cpu()
        loss = lambda *v: (self.plain(act, *v) * dout).sum()  # noqa: E731
        return torch.autograd.grad(loss(*leaves), leaves), loss, [v.detach() for v in leaves]


def off(got, want):
    return ((got.double().cpu() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("act", sorted(gca.ACTIVATIONS))
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_gradients_against_autograd_and_differences(dtype, act):
    b = Block(dtype, 3)
    _, dx, grads = b.step(act)
    want, loss, leaves = b.autograd(act)
    # A code is off by at most half a unit 2^e, evenly: 2^e / sqrt(12) in the root mean square, and 2^e < A /
    # 63 with A the group's largest, which is at most sqrt(32) times the group's root mean square: 0.289 * 5.66
    # / 63 = 0.026 of it.  Gradients are linear in the kept rows (the norm's quadratic): that share, twice.
    # The other intermediates are off by half a step of the type; a gradient passes at most 8 of them.
    bound = 2 * 0.026 + 8 * torch.finfo(dtype).eps / 2
    for got, w in zip([dx, *grads], want):
        assert off(got, w) <= bound
    # and the 64-bit gradients against differences along random directions
    gen = torch.Generator().manual_seed(0)
    for i, (leaf, w) in enumerate(zip(leaves, want)):
        d = torch.randn(leaf.shape, generator=gen, dtype=torch.float64)
        step = 1e-5
        up, down = ([v + s * step * d if j == i else v for j, v in enumerate(leaves)] for s in (1, -1))
        slope = ((loss(*up) - loss(*down)) / (2 * step)).item()
        assert abs(slope - (w * d).sum().item()) <= 1e-6 * (w.norm() * d.norm()).item()


def test_clipped_gradients_go_through_the_compressor():
    """The gradients of two blocks, clipped by their global norm into the flat gradient, compress to what the
    flat gradient clipped by hand compresses to."""
    parts = []
    for seed in (1, 2):
        parts += Block(torch.bfloat16, seed).step("silu")[2]
    sizes = [p.numel() for p in parts]
    off_ = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int64)
    total = int(off_[-1])
    tensors = [p.contiguous().to(torch.bfloat16 if i % 2 else torch.float32)
               for i, p in enumerate(parts)]
    norm64 = torch.cat([t.double().flatten() for t in tensors]).norm()
    max_norm = 0.3 * norm64.item()
    norm, flat = torch.empty(1, device="cuda"), torch.empty(total, device="cuda")
    gca.clip_grad_norm(tensors, max_norm, norm, out=flat)
    assert abs(norm.double() - norm64) <= 2.0 ** -23 * norm64
    f = torch.tensor(np.float32(max_norm) / np.float32(norm.item()), device="cuda")
    by_hand = torch.cat([t.float().flatten() for t in tensors]) * f
    assert torch.equal(flat, by_hand)
    plan = gca.Plan(off_, ratio=0.01)
    results = []
    for g in (flat, by_hand):
        e = torch.zeros(total, device="cuda")
        vals = torch.empty(plan.total_k, device="cuda")
        idx = torch.empty(plan.total_k, dtype=torch.int32, device="cuda")
        plan.compress(g, e, vals, idx)
        results.append((vals, idx, e))
    torch.cuda.synchronize()
    for a, c in zip(*results):
        assert torch.equal(a, c)
    plan.close()


def test_a_captured_step_replays():
    """The whole step captured into a graph, replayed on new inputs with eager steps in between."""
    b = Block(torch.bfloat16, 5)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b.step("silu")
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, dx, grads = b.step("silu")
        norm, flat = torch.empty(1, device="cuda"), torch.empty(sum(g.numel() for g in grads),
                                                               device="cuda")
        gca.clip_grad_norm([g.view(-1) for g in grads], 0.01, norm, out=flat)
    for seed in range(6, 9):
        new = Block(torch.bfloat16, seed)
        for name in ("x", "dout", "w", "wg", "wu", "wd"):
            getattr(b, name).copy_(getattr(new, name))
        eh, edx, egrads = new.step("silu")
        enorm, eflat = torch.empty_like(norm), torch.empty_like(flat)
        gca.clip_grad_norm([g.view(-1) for g in egrads], 0.01, enorm, out=eflat)
        graph.replay()
        torch.cuda.synchronize()
        for got, want in ((h, eh), (dx, edx), (norm, enorm), (flat, eflat)):
            assert torch.equal(got, want)
