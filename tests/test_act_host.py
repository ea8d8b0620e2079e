"""The activation operators' host side (no GPU): layouts, workspaces and every refusal of the C
ABI, and the binding's checks of its arguments.  The pointers are made up: each call here is
refused, or has nothing to do, before anything is launched."""
import ctypes

import pytest
import torch

import gradient_compression_amd as gca

BAD, UNSUPPORTED, OK = gca.GC_ERR_INVALID_ARG, gca.GC_ERR_UNSUPPORTED, gca.GC_OK
A, B, C, D, E, F, G, H = (0x10000000 * (i + 1) for i in range(8))   # far apart, 16-byte aligned


@pytest.mark.parametrize("cols,want", [(0, (0, 0)), (1, (32, 1)), (32, (32, 1)), (33, (64, 2)),
                                       (4096, (4096, 128)), (11008, (11008, 344))])
def test_layout(cols, want):
    assert gca.act_layout(cols) == want


def test_layout_refuses():
    L = gca.lib()
    assert L.gc_act_layout(-1, None, None) == BAD
    assert L.gc_act_layout(1 << 31, None, None) == UNSUPPORTED
    assert L.gc_act_layout(7, None, None) == OK


def quant(x=A, ld=64, dtype=1, rows=4, cols=64, rounding=0, codes=B, exps=C):
    return gca.lib().gc_act_quant(x, ld, dtype, rows, cols, rounding, 0, 0, codes, exps, None)


@pytest.mark.parametrize("case,want", [
    (dict(dtype=3), BAD), (dict(dtype=-1), BAD), (dict(rounding=2), BAD),
    (dict(rows=-1), BAD), (dict(cols=-1), BAD), (dict(ld=63), BAD),
    (dict(x=None), BAD), (dict(codes=None), BAD), (dict(exps=None), BAD),
    (dict(x=A + 1), BAD), (dict(x=A + 2, dtype=0), BAD), (dict(codes=B + 8), BAD),
    (dict(codes=A), BAD), (dict(exps=A + 100), BAD), (dict(exps=B + 255), BAD),
    (dict(rows=(1 << 25) + 1, cols=32), UNSUPPORTED),
    (dict(rows=1 << 25, cols=513, ld=513), UNSUPPORTED),
    (dict(cols=1 << 31, ld=1 << 31), UNSUPPORTED),
    (dict(cols=(1 << 27) + 1, ld=1 << 28), UNSUPPORTED),
    # odd pitches, the second buffer in front of the first, behind it, and inside a row
    (dict(ld=77, codes=A - 160), BAD), (dict(ld=77, exps=A + 77 * 2 - 8 + 1), BAD),
    (dict(ld=77, exps=A - 5), BAD),
    (dict(rows=0, x=None, codes=None, exps=None), OK),
    (dict(cols=0, x=None, codes=None, exps=None), OK),
    (dict(rows=0, ld=(1 << 63) - 1), OK), (dict(cols=0, ld=-(1 << 63)), OK),
    (dict(ld=(1 << 63) - 1), BAD), (dict(ld=-(1 << 63)), BAD),
    (dict(rows=(1 << 63) - 1), UNSUPPORTED), (dict(cols=(1 << 63) - 1), UNSUPPORTED),
])
def test_quant_refuses(case, want):
    assert quant(**case) == want


def restore(codes=B, exps=C, rows=4, cols=64, out=A, ld=64, dtype=1):
    return gca.lib().gc_act_restore(codes, exps, rows, cols, out, ld, dtype, None)


@pytest.mark.parametrize("case,want", [
    (dict(dtype=7), BAD), (dict(ld=10), BAD), (dict(out=None), BAD), (dict(codes=None), BAD),
    (dict(out=B), BAD), (dict(out=C - 2), BAD), (dict(rows=-3), BAD), (dict(out=A + 1), BAD),
    (dict(rows=0, out=None, codes=None, exps=None), OK),
])
def test_restore_refuses(case, want):
    assert restore(**case) == want


def norm(x=A, ld_x=64, res=B, ld_r=64, dtype=1, rows=4, cols=64, w=C, wd=0, eps=1e-5, h=D, ld_h=64,
         y=E, ld_y=64, rstd=F, codes=G, exps=H, rounding=0):
    return gca.lib().gc_rmsnorm(x, ld_x, res, ld_r, dtype, rows, cols, w, wd, eps, h, ld_h, y, ld_y,
                                rstd, codes, exps, rounding, 0, 0, None)


@pytest.mark.parametrize("case,want", [
    (dict(dtype=5), BAD), (dict(wd=5), BAD), (dict(eps=-1e-9), BAD), (dict(eps=float("nan")), BAD),
    (dict(eps=float("inf")), BAD), (dict(rounding=9), BAD), (dict(x=None), BAD),
    (dict(y=None, codes=None, exps=None), BAD), (dict(codes=None), BAD), (dict(exps=None), BAD),
    (dict(ld_x=63), BAD), (dict(ld_r=63), BAD), (dict(ld_h=63), BAD), (dict(ld_y=63), BAD),
    (dict(rstd=F + 2), BAD), (dict(w=C + 2), BAD), (dict(codes=G + 4), BAD),
    (dict(h=E), BAD),                            # two outputs in one place
    (dict(h=A, ld_h=72), BAD),                   # the same place with another pitch
    (dict(h=A + 2), BAD), (dict(y=C), BAD), (dict(rstd=A), BAD), (dict(codes=A), BAD),
    (dict(y=B + 128 * 3 + 126), BAD),            # shares the residual's last element
    # column blocks of one matrix that meet by one element, from either side
    (dict(ld_x=130, ld_y=130, y=A + 126), BAD), (dict(ld_x=130, ld_y=130, y=A - 126), BAD),
    (dict(ld_x=130, ld_y=130, y=A + 130 * 2 - 126), BAD),
    (dict(cols=32769, ld_x=40000, ld_r=40000, ld_h=40000, ld_y=40000), UNSUPPORTED),
    (dict(rows=1 << 26), UNSUPPORTED), (dict(rows=-1), BAD),
    (dict(rows=0), OK), (dict(cols=0), OK),
])
def test_norm_refuses(case, want):
    assert norm(**case) == want


def backward(dy=A, ld_dy=64, dtype=1, rows=4, cols=64, codes=B, exps=C, rstd=D, w=E, wd=0, res=F,
             ld_r=64, dx=G, ld_dx=64, dw=H, acc=0, ws=H + (1 << 20), n=1 << 20):
    return gca.lib().gc_rmsnorm_backward(dy, ld_dy, dtype, rows, cols, codes, exps, rstd, w, wd, res,
                                         ld_r, dx, ld_dx, dw, acc, ws, n, None)


@pytest.mark.parametrize("case,want", [
    (dict(dtype=3), BAD), (dict(wd=3), BAD), (dict(dy=None), BAD), (dict(dx=None), BAD),
    (dict(codes=None), BAD), (dict(exps=None), BAD), (dict(rstd=None), BAD), (dict(ws=None), BAD),
    (dict(n=gca.rmsnorm_backward_workspace(4, 64) - 1), BAD), (dict(ws=H + (1 << 20) + 8), BAD), (dict(dw=H + 2), BAD),
    (dict(ld_dx=63), BAD), (dict(dx=B), BAD), (dict(dx=A + 2), BAD), (dict(dx=F, ld_dx=128), BAD),
    (dict(dw=G), BAD), (dict(ws=A), BAD), (dict(ws=H), BAD), (dict(dw=D), BAD),
    (dict(cols=32769), UNSUPPORTED), (dict(rows=-1), BAD),
    (dict(cols=0, dy=None, dx=None), OK),
])
def test_norm_backward_refuses(case, want):
    assert backward(**case) == want


def wgrad(dy=A, ld=64, dtype=1, rows=4, n_out=64, cols=64, codes=B, exps=C, sc=D, sd=0, dw=E, acc=0,
          ws=F, n=1 << 24):
    return gca.lib().gc_act_weight_grad(dy, ld, dtype, rows, n_out, cols, codes, exps, sc, sd, dw, acc,
                                        ws, n, None)


@pytest.mark.parametrize("case,want", [
    (dict(dtype=3), BAD), (dict(sd=3), BAD), (dict(dy=None), BAD), (dict(codes=None), BAD),
    (dict(exps=None), BAD), (dict(dw=None), BAD), (dict(dw=E + 1), BAD), (dict(sc=D + 1), BAD),
    (dict(ld=63), BAD), (dict(rows=-1), BAD), (dict(n_out=-1), BAD), (dict(cols=-1), BAD),
    (dict(dw=A), BAD), (dict(dw=B), BAD), (dict(dw=D), BAD), (dict(ws=F + 4), BAD),
    (dict(n_out=1 << 20, ld=1 << 20, cols=1 << 11), UNSUPPORTED),
    (dict(n_out=(1 << 63) - 1), UNSUPPORTED), (dict(ld=(1 << 63) - 1), BAD), (dict(n=-1), BAD),
    (dict(n_out=0, dy=None, dw=None), OK), (dict(cols=0, dw=None), OK),
    (dict(rows=0, acc=1, dy=None, codes=None, exps=None, ws=None, n=0), OK),
])
def test_weight_grad_refuses(case, want):
    assert wgrad(**case) == want


def test_weight_grad_workspace_too_small():
    need = gca.act_weight_grad_workspace(4096, 64, 64, torch.bfloat16)
    assert need > 0     # one tile and a long sum: split over the rows
    assert wgrad(rows=4096, n=need - 1) == BAD
    assert wgrad(rows=4096, ws=None, n=need) == BAD


def test_workspaces():
    L = gca.lib()
    n = ctypes.c_int64()
    assert L.gc_act_weight_grad_workspace(4, 4, 4, 1, None) == BAD
    assert L.gc_act_weight_grad_workspace(4, 4, 4, 9, ctypes.byref(n)) == BAD
    assert L.gc_rmsnorm_backward_workspace(4, 4, None) == BAD
    assert gca.rmsnorm_backward_workspace(0, 100) == 0
    assert gca.rmsnorm_backward_workspace(1, 100) == 128 * 4
    for rows in (0, 1, 31, 1000, 16384):
        need = gca.act_weight_grad_workspace(rows, 100, 200, torch.float32)
        assert need % (100 * 200 * 4) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 32)
    codes, exps = torch.zeros(2, 32, dtype=torch.int8), torch.zeros(2, 1, dtype=torch.uint8)
    for call in (lambda: gca.act_quant(x, codes, exps), lambda: gca.act_restore(codes, exps, x),
                 lambda: gca.rmsnorm(x, y=x), lambda: gca.act_weight_grad(x, codes, exps, x),
                 lambda: gca.rmsnorm_backward(x, codes, exps, x[:, 0], x)):
        with pytest.raises(ValueError, match="must live on the GPU"):
            call()
    for call in (lambda: gca.act_quant(None, codes, exps), lambda: gca.rmsnorm([1.0])):
        with pytest.raises(TypeError):
            call()
