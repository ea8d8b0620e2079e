"""The gated block's workspace where sums are split (no GPU): its size, and every refusal that keeps the parts
of the sums inside it.  The pointers are made up: each call is refused before anything is launched."""
import pytest
import torch

import gradient_compression_amd as gca

BAD = gca.GC_ERR_INVALID_ARG
A, B, C, D, E, F, G, H, W = (0x10000000 * (i + 1) for i in range(9))   # far apart, 16-byte aligned
FORWARD = [(64, 264, 2000, 1), (64, 264, 2000, 2), (300, 77, 4100, 1), (300, 77, 4100, 0)]
BACKWARD = [(512, 4096, 1024, 1), (512, 4096, 1024, 2), (300, 4100, 77, 0)]     # rows, n, cols, type
CODES = {0: torch.float32, 1: torch.bfloat16, 2: torch.float16}


def forward(rows, n, cols, dtype, ws, size, x=A, wg=B, wu=C, h=D, gate=E, up=F):
    return gca.lib().gc_gated_linear(x, cols, dtype, rows, cols, wg, cols, wu, cols, n, 0, h, n, gate, n,
                                     up, n, ws, size, None)


def backward(rows, n, cols, dtype, ws, size, dh=A, gate=B, up=C, dg=D, du=E, wg=F, wu=G, dx=H):
    return gca.lib().gc_gated_linear_backward(dh, n, gate, n, up, n, dtype, rows, n, 0, dg, n, du, n, wg,
                                              cols, wu, cols, cols, dx, cols, ws, size, None)


@pytest.mark.parametrize("call,shape", [(forward, s) for s in FORWARD] + [(backward, s) for s in BACKWARD],
                         ids=str)
def test_parts_of_sums_need_their_workspace(call, shape):
    rows, n, cols, dtype = shape
    size_of, part, names = (
        (gca.gated_linear_workspace, 2 * rows * n * 4, ("x", "wg", "wu", "h", "gate", "up"))
        if call is forward else
        (gca.gated_linear_backward_workspace, rows * cols * 4,
         ("dh", "gate", "up", "dg", "du", "wg", "wu", "dx")))
    need = size_of(rows, n, cols, CODES[dtype])
    assert need >= 2 * part and need % part == 0          # whole parts, at least two
    for ws, size in ((None, need), (None, 0), (W, need - 1), (W, 0), (W, -1), (W + 8, need), (W + 2, need)):
        assert call(*shape, ws, size) == BAD
    # a buffer over the workspace's first or last bytes
    for name in names:
        for at in (W, W + need - 16):
            assert call(*shape, W, need, **{name: at}) == BAD, (name, at - W)
            assert call(*shape, W, need + 4096, **{name: at}) == BAD, (name, at - W)
