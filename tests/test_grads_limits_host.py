"""The limits of the operators over many tensors where the running total of the sizes would pass 63 bits (no
GPU): every call here is refused before anything is launched."""
import ctypes

import numpy as np
import pytest

import gradient_compression_amd as gca

MOST = 1 << 44      # elements of a tensor, and of a call


@pytest.mark.parametrize("count", [2, 1 << 18, (1 << 19) - 1, 1 << 19, (1 << 19) + 1, 1 << 20])
@pytest.mark.parametrize("size", [MOST, MOST - 1, MOST // 2 + 1])
def test_more_elements_than_a_call_takes(count, size):
    """2^19 tensors of 2^44 elements are 2^63 in all, 2^20 of them 2^64: neither may pass for few."""
    L, need = gca.lib(), ctypes.c_int64(-7)
    sizes = np.full(count, size, np.int64)
    ptrs, kinds = np.full(count, 0x10000000, np.uint64), np.zeros(count, np.int32)
    at = [a.ctypes.data for a in (ptrs, sizes, kinds)]
    assert L.gc_grad_norm_workspace(at[1], count, ctypes.byref(need)) == gca.GC_ERR_UNSUPPORTED
    assert need.value == -7
    assert L.gc_grad_norm(*at, count, 0x20000000, None, 0x30000000, 1 << 40,
                          None) == gca.GC_ERR_UNSUPPORTED
    assert L.gc_grad_clip(*at, count, at[0], at[2], 1.0, 0x20000000, None, 0,
                          None) == gca.GC_ERR_UNSUPPORTED
    with pytest.raises(gca.GCError):
        gca.grad_norm_workspace(sizes)


def test_as_many_elements_as_a_call_takes():
    assert gca.grad_norm_workspace([MOST]) > 0
    assert gca.grad_norm_workspace([MOST // 2, 0, MOST // 2]) > 0
    assert gca.grad_norm_workspace(np.full(1 << 20, 1 << 24)) > 0
