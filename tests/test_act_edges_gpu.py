"""Calls of the activation operators at the edges of what their contract allows."""
from types import SimpleNamespace

import pytest
import torch

import gradient_compression_amd as gca
import oracle
from tests.gpu_helpers import assert_bitwise

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_stochastic_codes_of_values_far_below_their_group(dtype):
    """A draw of 0 rounds every value but 0 away from 0, also one whose quotient by the scale is below
    fp32's smallest number.  Seed 4 draws a 0 for row 20578, column 21 of rows of 32 columns."""
    rows, row, col = 20580, 20578, 21
    for small in (2.0 ** -133, -(2.0 ** -126), 2.0 ** -100, 0.0):
        for top in (126.75 * 2.0 ** 120, 127.0 * 2.0 ** 30, 3.0 * 2.0 ** -120):
            x = torch.zeros(rows, 32)
            x[row, col], x[row, col + 1] = small, top
            x = x.to(dtype)
            want_c, want_e = oracle.act_quant(x.float().numpy(), random=True, seed=4, step=0)
            if small != 0.0 and top > 1.0:
                assert want_c[row, col] == (1 if small > 0 else -1)
            codes = torch.empty(rows, 32, dtype=torch.int8, device="cuda")
            exps = torch.empty(rows, 1, dtype=torch.uint8, device="cuda")
            gca.act_quant(x.cuda(), codes, exps, stochastic=True, seed=4, step=0)
            assert_bitwise(exps, want_e, f"{small} beside {top} exponents")
            assert_bitwise(codes, want_c, f"{small} beside {top} codes")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_weight_gradient_of_no_rows_is_zero_whatever_the_scale(dtype):
    scale = torch.tensor([1.0, -2.0, float("inf"), float("nan"), -float("inf")], device="cuda").repeat(7)
    none = torch.empty(0, 4, dtype=dtype, device="cuda")
    codes = torch.empty(0, 64, dtype=torch.int8, device="cuda")
    exps = torch.empty(0, 2, dtype=torch.uint8, device="cuda")
    dw = torch.full((4, 35), 5.0, device="cuda")
    gca.act_weight_grad(none, codes, exps, dw, col_scale=scale)
    assert bool((dw == 0.0).all())
    dw.fill_(5.0)
    gca.act_weight_grad(none, codes, exps, dw, col_scale=scale, accumulate=True)
    assert bool((dw == 5.0).all())


class Buffers:
    """What a block's calls read and write, 40 x 96 and a layer of 24 outputs."""

    def __init__(self):
        gen = torch.Generator("cuda").manual_seed(3)
        self.x, self.res, self.dout = (torch.randn(40, n, generator=gen, device="cuda")
                                       for n in (96, 96, 24))
        self.w = torch.rand(96, generator=gen, device="cuda")
        self.h, self.y, self.dx = (torch.empty_like(self.x) for _ in range(3))
        self.rstd, self.dw = torch.empty(40, device="cuda"), torch.empty(96, device="cuda")
        self.codes = torch.empty(40, 96, dtype=torch.int8, device="cuda")
        self.exps = torch.empty(40, 3, dtype=torch.uint8, device="cuda")
        self.flat = torch.empty(2 + 24 * 96, device="cuda")
        self.dl = self.flat[1:-1].view(24, 96)

    def calls(self):
        """Each call with the names of what it writes."""
        return [
            (lambda: gca.rmsnorm(self.x, weight=self.w, residual=self.res, h=self.h, y=self.y,
                                 rstd=self.rstd, codes=self.codes, exps=self.exps),
             {"h", "y", "rstd", "codes", "exps"}),
            (lambda: gca.rmsnorm(self.x, residual=self.res, h=self.res, y=self.x), {"x", "res"}),
            (lambda: gca.act_quant(self.x, self.codes, self.exps), {"codes", "exps"}),
            (lambda: gca.act_restore(self.codes, self.exps, self.h), {"h"}),
            (lambda: gca.rmsnorm_backward(self.y, self.codes, self.exps, self.rstd, self.dx,
                                          weight=self.w, dres=self.h), {"dx"}),
            (lambda: gca.rmsnorm_backward(self.y, self.codes, self.exps, self.rstd, self.y,
                                          dweight=self.dw), {"y", "dw"}),
            (lambda: gca.act_weight_grad(self.dout, self.codes, self.exps, self.dl,
                                         col_scale=self.w), {"dl", "flat"}),
        ]


def test_written_tensors_raise_their_version_and_no_others():
    b = Buffers()
    for i, (call, written) in enumerate(b.calls()):
        before = {k: t._version for k, t in vars(b).items()}
        call()
        raised = {k for k, t in vars(b).items() if t._version != before[k]}
        assert raised == written, f"call {i}"
    with torch.inference_mode():       # such tensors have no version
        b = Buffers()
        for call, _ in b.calls():
            call()


@pytest.mark.parametrize("which", ["h", "x", "res", "dx", "dw", "dl"])
def test_autograd_notices_a_saved_tensor_that_a_call_overwrote(which):
    b = Buffers()
    w = torch.ones((), device="cuda", requires_grad=True)
    saved = torch.zeros_like(getattr(b, which))
    loss = (saved * w).sum()           # keeps `saved` for w's gradient
    setattr(b, which, saved)
    for call, written in b.calls():
        if which in written:
            call()
            break
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_outputs_are_constants_to_autograd():
    b = Buffers()
    b.x.requires_grad_()
    b.w.requires_grad_()
    gca.rmsnorm(b.x, weight=b.w, residual=b.res, h=b.h, y=b.y, rstd=b.rstd, codes=b.codes,
                exps=b.exps)
    assert not (b.h.requires_grad or b.y.requires_grad or b.rstd.requires_grad)
    (b.y * b.w).sum().backward()
    assert torch.equal(b.w.grad, b.y.sum(0)) and b.x.grad is None


def test_a_stream_of_another_device_is_refused():
    """The workspace would be allocated there, and the kernel would run there."""
    b = Buffers()
    other = SimpleNamespace(device_index=torch.cuda.current_device() + 1, cuda_stream=0)
    before = {k: t.clone() for k, t in vars(b).items()}
    for call in (lambda: gca.act_quant(b.x, b.codes, b.exps, stream=other),
                 lambda: gca.act_restore(b.codes, b.exps, b.h, stream=other),
                 lambda: gca.rmsnorm(b.x, y=b.y, stream=other),
                 lambda: gca.rmsnorm_backward(b.y, b.codes, b.exps, b.rstd, b.dx, dweight=b.dw,
                                              stream=other),
                 lambda: gca.act_weight_grad(b.dout, b.codes, b.exps, b.dl, stream=other)):
        with pytest.raises(ValueError, match="stream is on"):
            call()
    torch.cuda.synchronize()
    for k, t in vars(b).items():
        assert torch.equal(t.view(torch.uint8), before[k].view(torch.uint8)), k


@pytest.mark.parametrize("every", [2, 3])
def test_column_blocks_of_all_rows_and_of_every_second_or_third_row(every):
    """x in every row of a buffer, h and y beside it in every second or third row: pitches that
    differ, and no shared byte."""
    rows, cols = 5, 64
    wide = torch.full((rows * every, 3 * cols + 5), 7.0, device="cuda")
    x, h, y = wide[:rows, :cols], wide[::every, cols:2 * cols], wide[::every, 2 * cols + 5:]
    x.copy_(torch.randn(rows, cols, generator=torch.Generator("cuda").manual_seed(1), device="cuda"))
    want, untouched = torch.empty(rows, cols, device="cuda"), wide.clone()
    gca.rmsnorm(x.contiguous(), y=want)
    gca.rmsnorm(x, h=h, y=y)
    assert torch.equal(h, x) and torch.equal(y, want)
    gca.rmsnorm(y, y=x)                       # and the other way round
    gca.rmsnorm(want, y=h)
    assert torch.equal(x, h)
    for t in (x, h, y):
        t.fill_(0.0)
    for t in (untouched[:rows, :cols], untouched[::every, cols:2 * cols],
              untouched[::every, 2 * cols + 5:]):
        t.fill_(0.0)
    assert torch.equal(wide, untouched)
    with pytest.raises(gca.GCError):
        gca.rmsnorm(x, y=wide[::every, cols - 1:2 * cols - 1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,n_out,cols", [(70, 5, 33), (130, 100, 257), (300, 1000, 200), (200, 260, 3601)])
def test_what_lies_between_the_rows_does_not_reach_the_results(rows, n_out, cols, dtype):
    """Rows of every matrix in a buffer that is NaN between them; whole numbers, so sums are exact."""
    gen = torch.Generator("cuda").manual_seed(rows)

    def matrix(width, pad, most):
        wide = torch.full((rows, width + pad), float("nan"), dtype=dtype, device="cuda")
        m = wide[:, :width]
        m.copy_(torch.randint(-most, most + 1, (rows, width), generator=gen, device="cuda"))
        return m

    pitch, groups = gca.act_layout(cols)
    codes = torch.randint(-20, 21, (rows, pitch), generator=gen, device="cuda", dtype=torch.int8)
    codes[:, cols:] = 0
    exps = torch.full((rows, groups), 127, dtype=torch.uint8, device="cuda")
    for pad in (1, 8, 19):
        dout = matrix(n_out, pad, 30)
        dl = torch.empty(n_out, cols, device="cuda")
        gca.act_weight_grad(dout, codes, exps, dl)
        want = dout.float().t().contiguous() @ codes[:, :cols].float()
        assert torch.equal(dl, want)
        x, res, dres = (matrix(cols, pad, 9) for _ in range(3))
        outs = [torch.empty(rows, cols, dtype=dtype, device="cuda") for _ in range(4)]
        h, y, dx, dx2 = outs
        h2, y2 = torch.empty_like(h), torch.empty_like(y)
        c, e = torch.empty_like(codes), torch.empty_like(exps)
        rstd, dw, dw2 = (torch.empty(n, device="cuda") for n in (rows, cols, cols))
        gca.rmsnorm(x, residual=res, h=h, y=y, rstd=rstd, codes=c, exps=e)
        gca.rmsnorm(x.contiguous(), residual=res.contiguous(), h=h2, y=y2)
        gca.rmsnorm_backward(x, c, e, rstd, dx, dres=dres, dweight=dw)
        gca.rmsnorm_backward(x.contiguous(), c, e, rstd, dx2, dres=dres.contiguous(), dweight=dw2)
        for a, b in ((h, h2), (y, y2), (dx, dx2), (dw, dw2)):
            assert torch.equal(a, b) and not torch.isnan(a).any()
        c2, e2 = torch.empty_like(codes), torch.empty_like(exps)
        gca.act_quant(x, c, e)
        gca.act_quant(x.contiguous(), c2, e2)
        assert torch.equal(c, c2) and torch.equal(e, e2) and not bool((e == 255).any())
