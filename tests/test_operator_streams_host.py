"""A stream of another device than the tensors' is refused: the call would
otherwise allocate there and launch on the tensors' device's current stream."""
import types

import pytest
import torch

import fp8_scaled_quantization_scale_amd as fm


def test_stream_of_another_device_is_refused():
    stream = types.SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(fm.Fp8Error, match="the stream is on cuda:1, the tensors on cuda:0"):
        fm._scope(torch.device("cuda", 0), stream)
