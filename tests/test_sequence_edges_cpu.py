"""Host checks of the sequence operators' edges (no GPU): what is refused before any HIP call."""
import ctypes
import os
import subprocess
import sys
from types import SimpleNamespace

import pytest
import torch

import depthwise_convolution_gconv_amd as gc
from depthwise_convolution_gconv_amd import _sequence as S

UNSUPPORTED = 3


def arr(*v):
    return (ctypes.c_int64 * len(v))(*v)


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


# A launch takes fewer than 2^32 threads; what needs more is refused before anything is enqueued.
FAR = [(i + 1) << 58 for i in range(10)]      # made-up addresses, never dereferenced


def test_attention_refuses_more_threads_than_a_launch_takes():
    L = S._library()

    def attn(shape, dtype, state=0):
        strides = arr(*(0, 0, 0) * 4)
        return L.gconv_linear_attention(*FAR[:4], arr(*shape), strides, FAR[4], 1.0, 0, state, 0, dtype, FAR[5], 1 << 40, None)

    def bwd(shape, dtype):
        return L.gconv_linear_attention_backward(*FAR[:7], arr(*shape), arr(*(0, 0, 0) * 7), FAR[7], 1.0, 0, 0, 0, 0, dtype,
                                                 FAR[8], 1 << 50, None)

    n = ctypes.c_size_t()
    for shape, dtype, backward in (((1 << 23, 1, 1, 1, 256, 256), 2, 0),     # 2^23 workgroups of 512 threads
                                   ((1 << 23, 1, 1, 1, 64, 256), 2, 0),      # two column tiles of 256 threads
                                   ((1 << 23, 1, 1, 1, 256, 256), 0, 0),
                                   ((5600000, 1, 1, 1, 128, 128), 2, 1),     # three walks of 256 threads
                                   ((5600000, 1, 1, 2, 128, 64), 2, 1)):     # two walks of 256
        run = bwd if backward else attn
        assert run(shape, dtype) == UNSUPPORTED and "threads" in gc.gconv_last_error()
        assert L.gconv_linear_attention_workspace(arr(*shape), dtype, backward, ctypes.byref(n)) == UNSUPPORTED
    # The state of sequences without a token: 256 x 256 of each of 2^23 heads.
    assert attn((1 << 23, 0, 1, 1, 256, 256), 2, FAR[6]) == UNSUPPORTED
    # One head less than 2^32 threads need is taken.
    assert L.gconv_linear_attention_workspace(arr((1 << 23) - 8, 1, 1, 1, 256, 256), 2, 0, ctypes.byref(n)) == 0


def test_conv_refuses_more_threads_than_a_launch_takes():
    L = S._library()

    def conv(B, T, C, K, dtype=1):
        return L.gconv_dw1d_causal(FAR[0], FAR[1], 0, FAR[2], 0, 0, 0, arr(B, T, C, K), arr(T * C, C), 0, dtype, None)

    def bwd(B, T, C, K):
        return L.gconv_dw1d_causal_backward(FAR[0], FAR[1], 0, FAR[2], 0, 0, FAR[3], FAR[4], 0, 0, 0, arr(B, T, C, K),
                                            arr(T * C, C, T * C, C), 0, 1, FAR[5], 1 << 50, None)

    def step(B, C, K):
        return L.gconv_dw1d_causal_step(FAR[0], FAR[1], 0, FAR[2], FAR[3], FAR[4], arr(B, C, K, 5), C, 0, 1, None)

    for call in (lambda: conv(1 << 24, 1, 1, 4), lambda: conv(1 << 24, 1, 1, 9), lambda: conv(1 << 12, 1 << 18, 64, 5),
                 lambda: bwd(1 << 24, 1, 1, 4), lambda: bwd(1, 1, 1 << 23, 64), lambda: step(1 << 24, 1, 4),
                 lambda: step(1 << 23, 1025, 4)):
        assert call() == UNSUPPORTED and "threads" in gc.gconv_last_error()
