"""Every refusal of the call that takes the norm over many tensors and clips them by it, on the host (no
GPU): both halves' arguments are looked at before either launches.  The pointers are made up."""
import numpy as np
import pytest

import gradient_compression_amd as gca

BAD, UNSUPPORTED = gca.GC_ERR_INVALID_ARG, gca.GC_ERR_UNSUPPORTED
A, B, C, D, N, M, W, F = (0x10000000 * (i + 1) for i in range(8))
NEED = gca.grad_norm_workspace([100, 200])


def joint(ptrs=(A, B), sizes=(100, 200), kinds=(0, 1), n=2, out=(C, D), to=(0, 0), limit=1.0, norm=N,
          norms=M, factors=F, count=3, ws=W, size=NEED):
    arrays = [None if v is None else np.array([p or 0 for p in v], t) for v, t in (
        (ptrs, np.uint64), (sizes, np.int64), (kinds, np.int32), (out, np.uint64), (to, np.int32))]
    p, s, k, o, t = (None if a is None else a.ctypes.data for a in arrays)
    return gca.lib().gc_clip_grad_norm(p, s, k, n, o, t, limit, norm, norms, factors, count, ws, size,
                                       None)


@pytest.mark.parametrize("case,want", [
    # as the norm refuses
    (dict(n=-1), BAD), (dict(ptrs=None), BAD), (dict(sizes=None), BAD), (dict(kinds=None), BAD),
    (dict(kinds=(0, 3)), BAD), (dict(sizes=(-1, 5)), BAD), (dict(ptrs=(A, None)), BAD),
    (dict(ptrs=(A, B + 1)), BAD), (dict(norm=None), BAD), (dict(norm=N + 2), BAD),
    (dict(norms=M + 2), BAD), (dict(ws=None), BAD), (dict(ws=W + 8), BAD), (dict(size=NEED - 1), BAD),
    (dict(norm=A + 396), BAD), (dict(norms=A - 4), BAD), (dict(ws=B - 16), BAD), (dict(norm=W), BAD),
    (dict(norm=W + NEED - 4), BAD), (dict(norms=W + NEED - 4), BAD), (dict(norm=M + 4), BAD),
    (dict(sizes=(1 << 44, 1)), UNSUPPORTED), (dict(n=(1 << 20) + 1), UNSUPPORTED),
    # as the scaling refuses
    (dict(out=None), BAD), (dict(to=None), BAD), (dict(to=(0, 7)), BAD), (dict(limit=-1.0), BAD),
    (dict(limit=float("nan")), BAD), (dict(factors=F + 1), BAD), (dict(count=-1), BAD),
    (dict(count=(1 << 44) + 1), UNSUPPORTED), (dict(out=(C, None)), BAD), (dict(out=(C + 2, D)), BAD),
    (dict(out=(C, C)), BAD), (dict(out=(B, D)), BAD), (dict(out=(A + 4, D)), BAD),
    (dict(out=(C, B), to=(0, 2)), BAD), (dict(out=(N, D)), BAD), (dict(out=(C, N - 796)), BAD),
    (dict(factors=N), BAD), (dict(factors=N - 8), BAD), (dict(factors=C + 396), BAD),
    (dict(factors=A + 396, count=1), BAD),
    (dict(ptrs=(A, A), sizes=(100, 100), kinds=(0, 0), out=(A, A)), BAD),
])
def test_either_half_s_refusals(case, want):
    assert joint(**case) == want
