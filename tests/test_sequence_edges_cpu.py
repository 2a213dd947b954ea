"""Host checks of the sequence operators' edges (no GPU): what is refused before any HIP call."""
from types import SimpleNamespace

import pytest
import torch

import depthwise_convolution_gconv_amd as gc
from depthwise_convolution_gconv_amd import _sequence as S


def test_stream_of_another_device():
    stream = SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(gc.GconvError, match="stream is on cuda:1, the tensors are on device 0"):
        S._on_stream(stream, SimpleNamespace(get_device=lambda: 0), None)
    z = torch.zeros
    for call in (lambda: gc.rms_norm(z(2, 8), z(8), stream=stream),
                 lambda: gc.linear_attention(z(1, 2, 1, 8), z(1, 2, 1, 8), z(1, 2, 1, 8), z(1), stream=stream),
                 lambda: gc.dwconv1d_causal_step(z(1, 8), z(8, 1, 4), None, z(1, 3, 8), stream=stream)):
        with pytest.raises(gc.GconvError, match="GPU tensor"):
            call()
