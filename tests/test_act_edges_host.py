"""Checks of the activation operators' binding that need no GPU."""
from types import SimpleNamespace

import pytest

import gradient_compression_amd as gca


def test_streams_are_of_the_current_device():
    assert gca._raw_stream(SimpleNamespace(device_index=3, cuda_stream=77), 3) == 77
    with pytest.raises(ValueError, match="stream is on cuda:1, the current device is cuda:0"):
        gca._raw_stream(SimpleNamespace(device_index=1, cuda_stream=77), 0)
