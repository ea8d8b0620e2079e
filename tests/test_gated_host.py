"""The gated block's host side (no GPU): workspaces and every refusal of the C ABI, and the binding's
checks.  The pointers are made up: each call here is refused, or has nothing to do, before anything is
launched."""
import ctypes

import pytest
import torch

import gradient_compression_amd as gca

BAD, UNSUPPORTED, OK = gca.GC_ERR_INVALID_ARG, gca.GC_ERR_UNSUPPORTED, gca.GC_OK
A, B, C, D, E, F, G, H, W = (0x10000000 * (i + 1) for i in range(9))   # far apart, 16-byte aligned


def forward(x=A, ld_x=64, dtype=1, rows=4, cols=64, wg=B, ld_wg=64, wu=C, ld_wu=64, n=32, act=0, h=D,
            ld_h=32, gate=E, ld_g=32, up=F, ld_u=32, ws=W, size=1 << 24):
    return gca.lib().gc_gated_linear(x, ld_x, dtype, rows, cols, wg, ld_wg, wu, ld_wu, n, act, h,
                                     ld_h, gate, ld_g, up, ld_u, ws, size, None)


@pytest.mark.parametrize("case,want", [
    (dict(dtype=3), BAD), (dict(dtype=-1), BAD), (dict(act=3), BAD), (dict(act=-1), BAD),
    (dict(rows=-1), BAD), (dict(cols=-1), BAD), (dict(n=-1), BAD),
    (dict(x=None), BAD), (dict(wg=None), BAD), (dict(wu=None), BAD), (dict(h=None), BAD),
    (dict(ld_x=63), BAD), (dict(ld_wg=63), BAD), (dict(ld_wu=63), BAD), (dict(ld_h=31), BAD),
    (dict(ld_g=31), BAD), (dict(ld_u=31), BAD), (dict(x=A + 1), BAD), (dict(wg=B + 1), BAD),
    (dict(h=D + 1), BAD), (dict(x=A + 2, dtype=0), BAD), (dict(ws=W + 8), BAD), (dict(size=-1), BAD),
    # outputs on inputs and on each other, whole or by one element
    (dict(h=A), BAD), (dict(h=B), BAD), (dict(gate=C), BAD), (dict(up=D), BAD), (dict(gate=F), BAD),
    (dict(h=A + 4 * 128 - 2), BAD), (dict(up=E + 4 * 64 - 2), BAD),
    (dict(gate=E, up=E + 64, ld_g=63, ld_u=63), BAD),
    (dict(rows=(1 << 25) + 1), UNSUPPORTED), (dict(n=(1 << 27) + 1, ld_h=1 << 28), UNSUPPORTED),
    (dict(cols=1 << 24, n=1 << 12, ld_x=1 << 24, ld_wg=1 << 24, ld_wu=1 << 24), UNSUPPORTED),
    (dict(rows=(1 << 63) - 1), UNSUPPORTED), (dict(n=(1 << 63) - 1), UNSUPPORTED),
    (dict(ld_x=(1 << 63) - 1), BAD),
    (dict(rows=0, x=None, h=None, gate=None, up=None), OK),
    (dict(n=0, wg=None, wu=None, h=None), OK),
])
def test_forward_refuses(case, want):
    assert forward(**case) == want


def backward(dh=A, ld=32, gate=B, ld_g=32, up=C, ld_u=32, dtype=1, rows=4, n=32, act=0, dg=D,
             ld_dg=32, du=E, ld_du=32, wg=F, ld_wg=64, wu=G, ld_wu=64, cols=64, dx=H, ld_dx=64, ws=W,
             size=1 << 24):
    return gca.lib().gc_gated_linear_backward(dh, ld, gate, ld_g, up, ld_u, dtype, rows, n, act, dg,
                                              ld_dg, du, ld_du, wg, ld_wg, wu, ld_wu, cols, dx, ld_dx,
                                              ws, size, None)


@pytest.mark.parametrize("case,want", [
    (dict(dtype=3), BAD), (dict(act=3), BAD), (dict(rows=-1), BAD), (dict(cols=-1), BAD),
    (dict(n=-1), BAD), (dict(dh=None), BAD), (dict(gate=None), BAD), (dict(up=None), BAD),
    (dict(dg=None), BAD), (dict(du=None), BAD), (dict(wg=None), BAD), (dict(wu=None), BAD),
    (dict(ld=31), BAD), (dict(ld_g=31), BAD), (dict(ld_u=31), BAD), (dict(ld_dg=31), BAD),
    (dict(ld_du=31), BAD), (dict(ld_wg=63), BAD), (dict(ld_wu=63), BAD), (dict(ld_dx=63), BAD),
    (dict(dg=D + 1), BAD), (dict(dx=H + 1), BAD), (dict(ws=W + 4), BAD), (dict(size=-1), BAD),
    (dict(dg=A, du=A), BAD), (dict(dg=B, du=B), BAD), (dict(dg=E), BAD),
    (dict(dg=B, ld_dg=40), BAD), (dict(dg=B + 2), BAD), (dict(du=A - 2), BAD),
    (dict(dx=A), BAD), (dict(dx=D), BAD), (dict(dx=F), BAD), (dict(dg=F), BAD), (dict(du=G), BAD),
    (dict(dx=None, dg=E), BAD), (dict(dx=None, dh=None, cols=-5), BAD),
    (dict(rows=(1 << 25) + 1), UNSUPPORTED), (dict(n=(1 << 63) - 1), UNSUPPORTED),
    (dict(cols=(1 << 63) - 1), UNSUPPORTED),
    (dict(n=1 << 12, cols=1 << 24), UNSUPPORTED),
    (dict(rows=0, dh=None, gate=None, up=None, dg=None, du=None, dx=None), OK),
])
def test_backward_refuses(case, want):
    assert backward(**case) == want


def test_workspaces():
    L = gca.lib()
    n = ctypes.c_int64()
    for f in (L.gc_gated_linear_workspace, L.gc_gated_linear_backward_workspace):
        assert f(4, 4, 4, 1, None) == BAD
        assert f(4, 4, 4, 9, ctypes.byref(n)) == BAD
        assert f(-4, 4, 4, 1, ctypes.byref(n)) == BAD
        assert f(1 << 26, 4, 4, 1, ctypes.byref(n)) == UNSUPPORTED
    for f in (gca.gated_linear_workspace, gca.gated_linear_backward_workspace):
        for rows in (0, 1, 16, 64, 300, 4096, 16384):
            for n, cols in ((0, 5), (5, 0), (7, 33), (1000, 4096), (11008, 4096)):
                for t in (torch.float32, torch.bfloat16, torch.float16):
                    assert f(rows, n, cols, t) >= 0
        with pytest.raises(gca.GCError):
            f(1, 1, 1, torch.int8)


def test_binding_refuses():
    x, w = torch.zeros(2, 32), torch.zeros(4, 32)
    h = torch.zeros(2, 4)
    for call in (lambda: gca.gated_linear(x, w, w, h),
                 lambda: gca.gated_linear_backward(h, h, h, h, h)):
        with pytest.raises(ValueError, match="must live on the GPU"):
            call()
    for call in (lambda: gca.gated_linear(None, w, w, h), lambda: gca.gated_linear([1.0], w, w, h),
                 lambda: gca.gated_linear_backward(None, h, h, h, h)):
        with pytest.raises(TypeError):
            call()
    assert sorted(gca.ACTIVATIONS.values()) == [0, 1, 2]
