"""The activation operators together, as a training step uses them: norm, linear layer, backward
pass from the 8-bit checkpoint into the flat gradient, and the Top-k compression of that gradient."""
import numpy as np
import pytest
import torch

import gradient_compression_amd as gca
import oracle
from tests.gpu_helpers import assert_bitwise, log

pytestmark = pytest.mark.gpu

ROWS, COLS, OUT, EPS = 384, 256, 320, 1e-5


class Block:
    """y = norm(x + residual) @ W^T with a loss of sum(y * target); parameters w (norm) and W, their
    gradients segments of one flat buffer, 8-bit checkpoints in between."""

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.w = (1.0 + 0.2 * r(COLS)).cuda()
        self.W = (r(OUT, COLS) / COLS ** 0.5).cuda()
        self.x, self.res = r(ROWS, COLS).cuda(), r(ROWS, COLS).cuda()
        self.target = (r(ROWS, OUT) / ROWS).cuda()
        self.off = np.cumsum([0, COLS, OUT * COLS]).astype(np.int64)
        pitch, groups = gca.act_layout(COLS)
        self.codes = torch.empty(ROWS, pitch, dtype=torch.int8, device="cuda")
        self.exps = torch.empty(ROWS, groups, dtype=torch.uint8, device="cuda")
        self.rstd = torch.empty(ROWS, device="cuda")
        self.h, self.y = torch.empty_like(self.x), torch.empty_like(self.x)
        self.dx = torch.empty_like(self.x)

    def step(self, flat, accumulate=False):
        gca.rmsnorm(self.x, weight=self.w, eps=EPS, residual=self.res, h=self.h, y=self.y,
                    rstd=self.rstd, codes=self.codes, exps=self.exps)
        out = self.y @ self.W.t()
        loss = (out * self.target).sum()
        dy = self.target @ self.W
        a, b, c = (int(v) for v in self.off)
        gca.act_weight_grad(self.target, self.codes, self.exps, flat[b:c].view(OUT, COLS),
                            col_scale=self.w, accumulate=accumulate)
        gca.rmsnorm_backward(dy, self.codes, self.exps, self.rstd, self.dx, weight=self.w,
                             dweight=flat[a:b], accumulate=accumulate)
        return loss

    def loss64(self, x, w, W):
        h = x + self.res.double()
        z = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
        return ((z * w) @ W.t() * self.target.double()).sum()


def relative(a, b):
    return float((a.double() - b).norm() / b.norm())


def test_gradients_against_autograd_and_differences():
    blk = Block(0)
    flat = torch.empty(int(blk.off[-1]), device="cuda")
    blk.step(flat)
    x, w, W = (t.double().requires_grad_() for t in (blk.x, blk.w, blk.W))
    gx, gw, gW = torch.autograd.grad(blk.loss64(x, w, W), (x, w, W))
    # a code is off by at most half a unit 2^e, and 2^e < A / 63 with A the group's largest
    # magnitude: the kept rows are off by the root mean square of that, about 0.3 / 63 * A; the
    # largest of 32 normal values is below 4.5, so z is off by less than 2.2 percent of its size 1
    z = torch.empty(ROWS, COLS, device="cuda")
    gca.act_restore(blk.codes, blk.exps, z)
    h = blk.x.double() + blk.res.double()
    z64 = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
    kept = relative(z, z64)
    log(f"[block] kept rows {kept:.2e}")
    assert kept <= 0.022
    # gradients are linear in z (quadratic for x, whose second term is small): the same share, twice
    a, b, c = (int(v) for v in blk.off)
    for name, got, want in (("w", flat[a:b], gw), ("W", flat[b:c].view(OUT, COLS), gW),
                            ("x", blk.dx, gx)):
        r = relative(got, want)
        log(f"[block] gradient of {name}: {r:.2e}")
        assert r <= 2 * 0.022
    # against differences of the loss in 64 bits, along each gradient's own direction: the
    # directional derivative is the product with the true gradient
    for got, p, i in ((flat[a:b], w, 1), (flat[b:c].view(OUT, COLS), W, 2), (blk.dx, x, 0)):
        d = got.double() / got.double().norm()
        args = [x.detach(), w.detach(), W.detach()]
        t, vals = 1e-4, []
        for s in (t, -t):
            moved = list(args)
            moved[i] = moved[i] + s * d
            vals.append(float(blk.loss64(*moved)))
        slope = (vals[0] - vals[1]) / (2 * t)
        # the third derivative's share of a central difference is of order t^2
        assert abs(slope - float(got.double().norm())) <= 2 * 0.022 * float(got.double().norm()) + 1e-6


def test_flat_gradient_goes_through_the_compressor():
    blk = Block(1)
    n = int(blk.off[-1])
    flat = torch.empty(n, device="cuda")
    plan = gca.Plan(blk.off, ratio=0.01)
    e = torch.zeros(n, device="cuda")
    vals = torch.empty(plan.total_k, device="cuda")
    idx = torch.empty(plan.total_k, dtype=torch.int32, device="cuda")
    e_h = np.zeros(n, np.float32)
    for t in range(3):
        blk.x.mul_(1.0 + 0.1 * t)
        blk.step(flat)
        once = flat.clone()
        blk.step(flat, accumulate=True)      # two micro-batches of the same data
        assert torch.equal(flat, 2 * once)
        plan.compress(flat, e, vals, idx)
        torch.cuda.synchronize()
        want_v, want_i = oracle.topk_ef(flat.cpu().numpy(), e_h, blk.off, plan.k)
        assert_bitwise(idx, want_i, f"step {t} idx")
        assert_bitwise(vals, want_v, f"step {t} vals")
        assert_bitwise(e, e_h, f"step {t} residual")
    plan.close()
