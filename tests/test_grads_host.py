"""The host side of the norm and the clipping of many tensors (no GPU): workspaces and every refusal
of the C ABI, and the binding's checks.  The pointers are made up: each call here is refused before
anything is launched."""
import ctypes

import numpy as np
import pytest
import torch

import gradient_compression_amd as gca

BAD, UNSUPPORTED, OK = gca.GC_ERR_INVALID_ARG, gca.GC_ERR_UNSUPPORTED, gca.GC_OK
A, B, C, D, N, M, W = (0x10000000 * (i + 1) for i in range(7))


def arrays(ptrs, sizes, kinds):
    return (None if ptrs is None else np.array([p or 0 for p in ptrs], np.uint64),
            None if sizes is None else np.array(sizes, np.int64),
            None if kinds is None else np.array(kinds, np.int32))


def ptr(a):
    return None if a is None else a.ctypes.data


def norm(ptrs=(A, B), sizes=(100, 200), kinds=(0, 1), n=None, out=N, norms=M, ws=W, size=1 << 24):
    p, s, k = arrays(ptrs, sizes, kinds)
    n = len(sizes) if n is None else n
    return gca.lib().gc_grad_norm(ptr(p), ptr(s), ptr(k), n, out, norms, ws, size, None)


@pytest.mark.parametrize("case,want", [
    (dict(n=-1), BAD), (dict(ptrs=None), BAD), (dict(sizes=None, n=2), BAD), (dict(kinds=None), BAD),
    (dict(kinds=(0, 3)), BAD), (dict(kinds=(-1, 0)), BAD), (dict(sizes=(-1, 5)), BAD),
    (dict(ptrs=(A, None)), BAD), (dict(ptrs=(A + 2, B)), BAD), (dict(ptrs=(A, B + 1)), BAD),
    (dict(out=None), BAD), (dict(out=N + 2), BAD), (dict(norms=M + 2), BAD), (dict(ws=None), BAD),
    (dict(ws=W + 8), BAD), (dict(size=gca.grad_norm_workspace([100, 200]) - 1), BAD),
    # outputs in a tensor, in the workspace, in each other
    (dict(out=A + 396), BAD), (dict(out=B + 398), BAD), (dict(norms=A - 4), BAD), (dict(ws=A), BAD),
    (dict(ws=B - 16), BAD), (dict(out=W), BAD), (dict(out=M + 4), BAD), (dict(out=M + 8, norms=M, ws=M), BAD),
    (dict(sizes=((1 << 44) + 1, 5)), UNSUPPORTED), (dict(sizes=(1 << 44, 1)), UNSUPPORTED),
    (dict(sizes=((1 << 63) - 1, 5)), UNSUPPORTED), (dict(n=(1 << 20) + 1), UNSUPPORTED),
])
def test_norm_refuses(case, want):
    assert norm(**case) == want


def clip(ptrs=(A, B), sizes=(100, 200), kinds=(0, 1), n=None, out=(C, D), to=(0, 0), limit=1.0,
         norm=N, factors=M, count=3):
    p, s, k = arrays(ptrs, sizes, kinds)
    o, _, t = arrays(out, sizes, to)
    n = len(sizes) if n is None else n
    return gca.lib().gc_grad_clip(ptr(p), ptr(s), ptr(k), n, ptr(o), ptr(t), limit, norm, factors,
                                  count, None)


@pytest.mark.parametrize("case,want", [
    (dict(n=-1), BAD), (dict(ptrs=None), BAD), (dict(out=None), BAD), (dict(kinds=None), BAD),
    (dict(to=None), BAD), (dict(kinds=(0, 7)), BAD), (dict(to=(0, 7)), BAD), (dict(limit=-1.0), BAD),
    (dict(limit=float("nan")), BAD), (dict(limit=-float("inf")), BAD), (dict(norm=None), BAD),
    (dict(norm=N + 1), BAD), (dict(factors=M + 1), BAD), (dict(count=-1), BAD),
    (dict(ptrs=(None, B)), BAD), (dict(out=(C, None)), BAD), (dict(out=(C + 2, D)), BAD),
    (dict(count=(1 << 44) + 1), UNSUPPORTED),
    # an output in another's or another tensor's place, or over its own shifted or of another type
    (dict(out=(C, C)), BAD), (dict(out=(C, C + 396)), BAD), (dict(out=(B, D)), BAD),
    (dict(out=(C, A)), BAD), (dict(out=(A + 4, D)), BAD), (dict(out=(A - 4, D)), BAD),
    (dict(out=(A, B)), BAD), (dict(out=(C, B + 2), to=(0, 1)), BAD), (dict(out=(C, B), to=(0, 2)), BAD),
    (dict(out=(A, B), to=(0, 1), norm=A), BAD), (dict(norm=C), BAD), (dict(norm=M + 8), BAD),
    (dict(factors=C + 396), BAD), (dict(factors=A, count=1), BAD),
    # the same tensor twice, in place
    (dict(ptrs=(A, A), sizes=(100, 100), kinds=(0, 0), out=(A, A)), BAD),
    (dict(ptrs=(A, A + 40), sizes=(100, 100), kinds=(0, 0), out=(A, A + 40)), BAD),
    # a long tensor around a short one, whose output lies in the long one
    (dict(ptrs=(A, A + 100), sizes=(100, 5), kinds=(0, 0), out=(C, A + 100)), BAD),
    (dict(ptrs=(A, D), sizes=(100, 5), kinds=(0, 0), out=(A, A + 396)), BAD),
    (dict(sizes=(1 << 44, 1)), UNSUPPORTED),
    (dict(ptrs=(), sizes=(), kinds=(), out=(), to=(), factors=None), OK),
    (dict(ptrs=(None, None), sizes=(0, 0), out=(None, None), count=0), OK),
])
def test_clip_refuses(case, want):
    assert clip(**case) == want


def test_workspace():
    L, b = gca.lib(), ctypes.c_int64()
    assert L.gc_grad_norm_workspace(None, 0, None) == BAD
    assert L.gc_grad_norm_workspace(None, 1, ctypes.byref(b)) == BAD
    assert gca.grad_norm_workspace([]) == 0
    for sizes in ([0], [1], [0] * 1000, [1 << 30] * 300, list(range(5000))):
        chunks = sum(-(-n // 16384) for n in sizes)
        got = gca.grad_norm_workspace(sizes)
        assert 0 < got <= 8 * (min(chunks, 2048 * -(-len(sizes) // 240)) + 3 * len(sizes) + 1000)


def test_binding_refuses_host_tensors():
    t = torch.zeros(4)
    for call in (lambda: gca.grad_norm([t], t[:1]), lambda: gca.grad_clip([t], 1.0, t[:1]),
                 lambda: gca.clip_grad_norm([t], 1.0, t[:1])):
        with pytest.raises(ValueError, match="must live on the GPU"):
            call()
    with pytest.raises(TypeError):
        gca.grad_norm([t], None)
