"""Host checks of the sequence operators' edges (no GPU): what is refused before any HIP call."""
import os
import subprocess
import sys
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


def test_import_without_a_gpu_build_of_torch():
    # The private names that the calls take the device and the stream from exist in GPU builds only.
    code = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import depthwise_convolution_gconv_amd as gc
assert gc.gconv_out_shape((1, 4, 5, 5), (4, 1, 3, 3), groups=4) == (1, 4, 3, 3)
for call in (lambda z: gc.rms_norm(z(2, 8), z(8)), lambda z: gc.dwconv1d_causal(z(1, 2, 8), z(8, 1, 4))):
    try:
        call(torch.zeros)
    except gc.GconvError as e:
        assert "GPU tensor" in str(e)
    else:
        raise AssertionError("not refused")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
