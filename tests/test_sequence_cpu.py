"""Host checks of the sequence operators (no GPU): every call here is refused, or has
nothing to do, before any HIP call.  Addresses are made up and never dereferenced."""
import ctypes

import pytest
import torch

import depthwise_convolution_gconv_amd as gc
from depthwise_convolution_gconv_amd import _binding as B
from depthwise_convolution_gconv_amd import _sequence as S

OK, ARG, SHAPE, UNSUPPORTED = 0, 1, 2, 3
A = [(i + 1) << 40 for i in range(16)]     # far apart


def arr(*v):
    return (ctypes.c_int64 * len(v))(*v)


def attn(shape=(2, 100, 2, 4, 64, 32), strides=None, ptrs=None, decay=A[8], s0=0, sf=0, lengths=0, dtype=2, ws=A[9],
         ws_bytes=1 << 40):
    Bn, T, Hk, H, Dk, Dv = shape
    st = strides or (T * Hk * Dk, Hk * Dk, Dk) * 2 + (T * H * Dv, H * Dv, Dv) * 2
    p = ptrs or A[:4]
    return S._library().gconv_linear_attention(*p, arr(*shape), arr(*st), decay, 1.0, s0, sf, lengths, dtype, ws, ws_bytes,
                                               None)


def test_linear_attention_refusals():
    assert attn((2, 100, 3, 4, 64, 32)) == SHAPE                     # heads do not divide
    assert attn((2, 100, 2, 4, 257, 32)) == UNSUPPORTED              # columns of a head
    assert attn((2, 100, 2, 4, 64, 257)) == UNSUPPORTED
    for bad in ((-1, 100, 2, 4, 64, 32), (2, -1, 2, 4, 64, 32), (2, 100, 0, 4, 64, 32), (2, 100, 2, 4, 0, 32)):
        assert attn(bad) == ARG
    assert attn((1 << 24, 100, 2, 4, 64, 32)) == UNSUPPORTED
    assert attn(dtype=7) == ARG and attn(decay=0) == ARG
    assert attn(ptrs=[0, A[1], A[2], A[3]]) == ARG and attn(ptrs=[A[0], A[1], A[2], 0]) == ARG
    assert attn(strides=(-1,) * 12) == ARG
    assert attn(ptrs=[A[0], A[1], A[2], A[2] + 64]) == ARG           # o inside v
    assert "overlaps" in gc.gconv_last_error()
    assert attn(sf=A[0] + 8) == ARG and attn(s0=A[5], sf=A[5]) == ARG
    assert attn((1, 4096, 1, 1, 64, 64), ws=A[0]) == ARG             # the workspace over q
    assert attn(ws=A[9] + 4) == ARG and attn((1, 4096, 1, 1, 64, 64), ws=0) == ARG
    assert attn((1, 4096, 1, 1, 64, 64), ws_bytes=16) == ARG
    assert "needed" in gc.gconv_last_error()


def test_linear_attention_workspace():
    n = ctypes.c_size_t()
    f = S._library().gconv_linear_attention_workspace
    assert f(arr(1, 4096, 1, 1, 64, 64), 2, 0, ctypes.byref(n)) == OK and n.value % (64 * 64 * 4) == 0 and n.value > 0
    assert gc.linear_attention_workspace((1, 4096, 1, 1, 64, 64), torch.bfloat16) == n.value
    # Gradients of a key head that serves two value heads: fp32 shares beside the states.
    assert gc.linear_attention_workspace((1, 4096, 1, 2, 64, 64), torch.bfloat16, True) >= 4096 * 2 * 64 * 4
    assert gc.linear_attention_workspace((0, 10, 1, 1, 64, 64), torch.float32) == 0
    assert f(arr(1, 1, 1, 1, 300, 64), 2, 0, ctypes.byref(n)) == UNSUPPORTED
    assert f(arr(1, 1, 1, 1, 64, 64), 9, 0, ctypes.byref(n)) == ARG
    with pytest.raises(gc.GconvError):
        gc.linear_attention_workspace((1, 1, 2, 3, 64, 64), torch.float32)


def test_nothing_to_do():
    assert attn((0, 100, 2, 4, 64, 32), ptrs=[0] * 4) == OK and gc.gconv_last_kernel() == ""
    assert attn((2, 0, 2, 4, 64, 32), ptrs=[0] * 4) == OK            # no token and no state asked for
    assert step(shape=(0, 1, 2, 8, 8, 4)) == OK
    assert norm(rows=0) == OK
    assert conv((0, 5, 8, 4)) == OK and conv((2, 0, 8, 4)) == OK
    assert conv_step((0, 8, 4, 3)) == OK


def bwd(shape=(2, 100, 2, 4, 64, 32), ptrs=None, dinitial=0, ws_bytes=1 << 40):
    Bn, T, Hk, H, Dk, Dv = shape
    k3, v3 = (T * Hk * Dk, Hk * Dk, Dk), (T * H * Dv, H * Dv, Dv)
    p = ptrs or A[:7]
    return S._library().gconv_linear_attention_backward(*p, arr(*shape), arr(*(k3 * 2 + v3 * 2 + k3 * 2 + v3)), A[8], 1.0, 0,
                                                        0, dinitial, 0, 2, A[9], ws_bytes, None)


def test_linear_attention_backward_refusals():
    assert bwd((2, 100, 3, 4, 64, 32)) == SHAPE
    assert bwd(ptrs=[0] + A[1:7]) == ARG and bwd(ptrs=A[:6] + [0]) == ARG
    assert bwd(ptrs=A[:4] + [A[4], A[4] + 2, A[6]]) == ARG           # dk over dq
    assert bwd(dinitial=A[1]) == ARG
    assert bwd(ws_bytes=0) == ARG


def step(shape=(2, 1, 2, 8, 8, 4), ptrs=None, slots=A[6], decay=A[5], strides=(8, 8, 8, 8, 16, 8, 16, 8), dtype=0):
    p = ptrs or A[:5]
    return S._library().gconv_linear_attention_step(*p, arr(*shape), arr(*strides), decay, 1.0, slots, dtype, None)


def test_linear_attention_step_refusals():
    assert step((2, 2, 3, 8, 8, 4)) == SHAPE
    assert step((5, 1, 2, 8, 8, 4), slots=0) == SHAPE                # fewer states than sequences
    assert step((2, 1, 2, 8, 8, -1)) == ARG and step(decay=0) == ARG and step(dtype=3) == ARG
    assert step(ptrs=A[:4] + [0]) == ARG and step(ptrs=A[:4] + [A[3]]) == ARG
    assert step((2, 1, 2, 300, 8, 4)) == UNSUPPORTED


def norm(rows=4, C=100, x=A[0], res=0, w=A[2], y=A[3], h=0, strides=(100, 100), eps=1e-6, dtype=2):
    return S._library().gconv_rms_norm(x, res, w, y, h, rows, C, arr(*strides), eps, dtype, None)


def norm8(block=0, C=100, scales=A[5]):
    return S._library().gconv_rms_norm_e4m3(A[0], 0, A[2], A[3], scales, 0, 4, C, arr(C, C), 1e-6, block, 2, None)


def test_rms_norm_refusals():
    assert norm(rows=-1) == ARG and norm(C=0) == ARG and norm(eps=-1.0) == ARG and norm(eps=float("nan")) == ARG
    assert norm(C=(1 << 24) + 1) == UNSUPPORTED and norm(dtype=4) == ARG
    assert norm(x=0) == ARG and norm(y=0) == ARG and norm(w=0) == ARG
    assert norm(h=A[6]) == ARG and norm(res=A[1]) == ARG             # h goes with a residual
    assert norm(y=A[0]) == ARG and norm(res=A[1], h=A[1]) == ARG     # in place
    for block in (-1, 1, 16, 96, 512):
        assert norm8(block) == UNSUPPORTED
    assert norm8(scales=0) == ARG and norm8(scales=A[3]) == ARG
    f = S._library().gconv_rms_norm_backward
    args = lambda ws, dx=A[4]: (A[0], A[1], A[2], 0, dx, A[5], 4, 100, arr(100, 100, 0), 1e-6, 2, A[6], ws, None)  # noqa: E731
    assert f(*args(8)) == ARG and f(*args(1 << 30, dx=A[1])) == ARG


def conv(shape=(2, 10, 8, 4), x=A[0], w=A[1], y=A[3], s0=0, sf=0, strides=None, act=1, dtype=1):
    st = strides or (shape[1] * shape[2], shape[2])
    return S._library().gconv_dw1d_causal(x, w, 0, y, s0, sf, 0, arr(*shape), arr(*st), act, dtype, None)


def conv_step(shape=(2, 8, 4, 3), state=A[4], slots=A[5]):
    return S._library().gconv_dw1d_causal_step(A[0], A[1], 0, state, A[3], slots, arr(*shape), shape[1], 1, 1, None)


def test_dwconv1d_causal_refusals():
    assert conv((2, 10, 8, 65)) == UNSUPPORTED and conv((2, 10, 8, 0)) == ARG and conv((2, 10, 0, 4)) == ARG
    assert conv((2, -1, 8, 4)) == ARG and conv(act=2) == ARG and conv(dtype=5) == ARG
    assert conv(x=0) == ARG and conv(w=0) == ARG and conv(y=A[0] + 16) == ARG
    assert conv(strides=(-8, 8)) == ARG and conv(s0=A[6], sf=A[6]) == ARG
    assert conv_step((4, 8, 4, 3), slots=0) == SHAPE and conv_step(state=A[3]) == ARG and conv_step(state=0) == ARG
    assert conv_step((2, 8, 4, -1)) == ARG
    f = S._library().gconv_dw1d_causal_backward
    args = lambda ws, ds=0, dx=A[5]: (A[0], A[1], 0, A[2], 0, 0, dx, A[6], 0, ds, 0, arr(2, 10, 8, 4), arr(80, 8, 80, 8), 0,  # noqa: E731
                                      1, A[8], ws, None)
    assert f(*args(8)) == ARG and f(*args(1 << 30, ds=A[9])) == ARG and f(*args(1 << 30, dx=A[2])) == ARG


def test_binding_refusals():
    z = torch.zeros
    with pytest.raises(gc.GconvError, match="GPU tensor"):
        gc.linear_attention(z(1, 2, 1, 8), z(1, 2, 1, 8), z(1, 2, 1, 8), z(1))
    with pytest.raises(gc.GconvError, match="GPU tensor"):
        gc.rms_norm(z(2, 8), z(8))
    with pytest.raises(gc.GconvError, match="GPU tensor"):
        gc.dwconv1d_causal(z(1, 2, 8), z(8, 1, 4))
    with pytest.raises(gc.GconvError, match="unsupported dtype"):
        gc.rms_norm(z(2, 8, dtype=torch.float64), z(8, dtype=torch.float64))


def test_row_strides():
    x = torch.zeros(6, 4, 10)
    assert S._rows("x", x, x) == 10
    assert S._rows("x", x[..., :7], x[..., :7]) == 10
    assert S._rows("x", x[:, 0], x[:, 0]) == 40
    assert S._rows("x", x[2:3, :, 1:5], x[2:3, :, 1:5]) == 10
    assert S._rows("x", x[0, 0], x[0, 0]) == 10
    with pytest.raises(gc.GconvError, match="one stride"):
        S._rows("x", x[:, :3], x[:, :3])
    with pytest.raises(gc.GconvError, match="contiguous"):
        S._rows("x", x[..., ::2], x[..., ::2])
