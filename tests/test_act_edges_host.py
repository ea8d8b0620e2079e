"""Checks of the activation operators' binding that need no GPU."""
from types import SimpleNamespace

import pytest

import gradient_compression_amd as gca


def test_streams_are_of_the_current_device():
    assert gca._raw_stream(SimpleNamespace(device_index=3, cuda_stream=77), 3) == 77
    with pytest.raises(ValueError, match="stream is on cuda:1, the current device is cuda:0"):
        gca._raw_stream(SimpleNamespace(device_index=1, cuda_stream=77), 0)


A, BF16 = 0x10000000, 1     # a made-up pointer: each call is refused


@pytest.mark.parametrize("y,ld_x,ld_y", [
    # rows of x (64 columns of bf16) every 130 elements, rows of y every 260: meet by one element
    (A + 126, 130, 260), (A + 260 - 126, 130, 260), (A + 2 * 260 + 126, 130, 260),
    (A + 126, 260, 130), (A - 126, 130, 390), (A + 2 * 130 - 2, 130, 260),
    # no common pitch with room for both
    (A + 128, 130, 131), (A + 128, 192, 130),
])
def test_rows_that_meet_at_unlike_pitches_are_refused(y, ld_x, ld_y):
    rc = gca.lib().gc_rmsnorm(A, ld_x, None, 0, BF16, 4, 64, None, 0, 1e-5, None, 0, y, ld_y,
                              None, None, None, 0, 0, 0, None)
    assert rc == gca.GC_ERR_INVALID_ARG
