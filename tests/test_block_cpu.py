"""Host checks of the recurrent block's operators (no GPU): every call here is refused, or has
nothing to do, before any HIP call.  Addresses are made up and never dereferenced."""
import ctypes

import pytest
import torch

import depthwise_convolution_gconv_amd as gc
from depthwise_convolution_gconv_amd import _block as S

OK, ARG, SHAPE, UNSUPPORTED = 0, 1, 2, 3
A = [(i + 1) << 40 for i in range(20)]     # far apart


def arr(*v):
    return (ctypes.c_int64 * len(v))(*v)


def rec(shape=(2, 100, 64), strides=None, ptrs=None, decay=A[8], s0=0, sf=0, lengths=0, dtype=2, ws=A[9], ws_bytes=1 << 40):
    B, T, C = shape
    x, r, i, h = ptrs or A[:4]
    st = strides or (T * C, C) * 3
    return S._library().gconv_gated_recurrence(x, r, i, decay, h, arr(*shape), arr(*st), s0, sf, lengths, dtype, ws, ws_bytes, None)


def rec_bwd(shape=(2, 100, 64), strides=None, ptrs=None, dlog=A[10], s0=0, dfinal=0, dinitial=0, dtype=2, ws=A[9], ws_bytes=1 << 40):
    B, T, C = shape
    p = ptrs or A[:8]      # x, r, i, h, dh, dx, dr, di
    st = strides or (T * C, C) * 5
    return S._library().gconv_gated_recurrence_backward(*p[:3], A[8], *p[3:], dlog, arr(*shape), arr(*st), s0, dfinal, dinitial, 0,
                                                        dtype, ws, ws_bytes, None)


def rec_step(shape=(2, 64, 4), strides=(64, 64, 64), ptrs=None, slots=A[6], decay=A[8], dtype=0):
    x, r, i, state, h = ptrs or A[:5]
    return S._library().gconv_gated_recurrence_step(x, r, i, decay, state, h, arr(*shape), arr(*strides), slots, dtype, None)


def test_gated_recurrence_refusals():
    for bad in ((-1, 100, 64), (2, -1, 64), (2, 100, 0)):
        assert rec(bad) == ARG and rec_bwd(bad) == ARG
    assert rec((2, 2 ** 31 - 1, 64)) == UNSUPPORTED and rec((2, 100, 2 ** 30)) == UNSUPPORTED
    assert rec(dtype=5) == ARG and rec(decay=0) == ARG and rec_bwd(dlog=0) == ARG
    for i in range(4):
        assert rec(ptrs=[0 if j == i else A[j] for j in range(4)]) == ARG
    for i in range(8):
        assert rec_bwd(ptrs=[0 if j == i else A[j] for j in range(8)]) == ARG
    assert rec(strides=(-1,) * 6) == ARG and rec(strides=(1 << 61,) + (64,) * 5) == UNSUPPORTED
    assert rec(strides=(6400, 1 << 30) * 3) == UNSUPPORTED           # a tile past 32-bit offsets
    assert rec(ptrs=[A[0], A[1], A[2], A[2] + 64]) == ARG            # h inside i
    assert "overlaps" in gc.gconv_last_error()
    assert rec(sf=A[0] + 8) == ARG and rec(s0=A[5], sf=A[5]) == ARG
    assert rec_bwd(ptrs=A[:5] + [A[5], A[5] + 2, A[7]]) == ARG       # dr over dx
    assert rec_bwd(dinitial=A[11]) == ARG                            # without an initial state
    assert rec_bwd(s0=A[11], dinitial=A[11]) == ARG
    assert rec_bwd(ws_bytes=0) == ARG and "needed" in gc.gconv_last_error()
    assert rec_bwd(ws=A[9] + 4) == ARG and rec_bwd(ws=0) == ARG
    long = (1, 200000, 64)                                           # cut into segments
    assert rec(long, ws=0) == ARG and rec(long, ws_bytes=16) == ARG and rec(long, ws=A[3] + 1024) == ARG


def test_gated_recurrence_workspace():
    w = gc.gated_recurrence_workspace
    assert w((1, 10, 64), torch.float32) == 0 and w((0, 10, 64), torch.float32) == 0
    n = w((1, 200000, 64), torch.bfloat16)
    assert n >= 2 * 8 * 64 and n % 256 == 0
    assert w((4, 100, 64), torch.bfloat16, True) >= 4 * 4 * 64
    for bad in ((1, -1, 4), (1, 1, 0)):
        with pytest.raises(gc.GconvError):
            w(bad, torch.float32)


def test_gated_recurrence_step_refusals():
    assert rec_step((5, 64, 4), slots=0) == SHAPE                    # fewer states than sequences
    assert rec_step((2, 64, -1)) == ARG and rec_step((2, 0, 4)) == ARG and rec_step(decay=0) == ARG and rec_step(dtype=3) == ARG
    for i in range(5):
        assert rec_step(ptrs=[0 if j == i else A[j] for j in range(5)]) == ARG
    assert rec_step(ptrs=A[:4] + [A[3] + 64]) == ARG                 # h over the states
    assert rec_step(strides=(-1, 64, 64)) == ARG and rec_step(strides=(64, 64, 1 << 61)) == UNSUPPORTED
    assert rec_step((1 << 20, 1 << 13, 4), strides=(1 << 13,) * 3) == UNSUPPORTED      # more threads than a launch takes


def norm(shape=(2, 100, 64, 4), strides=None, x=A[0], w=A[1], b=A[2], y=A[3], stats=A[4], lengths=0, eps=1e-5, act=0, dtype=2, ws=A[5],
         ws_bytes=1 << 40):
    st = strides or (shape[1] * shape[2], shape[2])
    return S._library().gconv_group_norm(x, w, b, y, stats, arr(*shape), arr(*st), lengths, eps, act, dtype, ws, ws_bytes, None)


def norm_bwd(shape=(2, 100, 64, 4), strides=None, ptrs=None, act=0, dtype=2, ws=A[9], ws_bytes=1 << 40):
    p = ptrs or A[:8]      # dy, x, w, b, stats, dx, dw, db
    st = strides or (shape[1] * shape[2], shape[2]) * 2
    return S._library().gconv_group_norm_backward(*p, arr(*shape), arr(*st), 0, act, dtype, ws, ws_bytes, None)


def test_group_norm_refusals():
    assert norm((2, 100, 64, 5)) == SHAPE and norm_bwd((2, 100, 64, 5)) == SHAPE
    for bad in ((-1, 100, 64, 4), (2, -1, 64, 4), (2, 100, 0, 1), (2, 100, 64, 0), (2, 100, 64, -4)):
        assert norm(bad) == ARG and norm_bwd(bad) == ARG
    assert norm((1, 1, 1 << 21, 1)) == UNSUPPORTED and norm((2, 2 ** 31 - 1, 64, 4)) == UNSUPPORTED
    assert norm(act=2) == ARG and norm(dtype=9) == ARG and norm(eps=-1.0) == ARG and norm(eps=float("nan")) == ARG
    assert norm(x=0) == ARG and norm(w=0) == ARG and norm(y=0) == ARG
    assert norm(strides=(-1, 64)) == ARG and norm(strides=(1 << 62, 64)) == UNSUPPORTED
    assert norm(strides=(6400, 1 << 31)) == UNSUPPORTED              # positions past 32-bit offsets
    assert norm(y=A[0]) == ARG and norm(y=A[0] + 128) == ARG and norm(stats=A[3] + 4) == ARG      # in place
    for i in (0, 1, 2, 4, 5, 6):
        assert norm_bwd(ptrs=[0 if j == i else A[j] for j in range(8)]) == ARG
    assert norm_bwd(ptrs=A[:3] + [0] + A[4:8]) == ARG and norm_bwd(ptrs=A[:7] + [0]) == ARG       # db goes with a bias
    assert norm_bwd(ptrs=A[:5] + [A[1], A[6], A[7]]) == ARG          # dx over x
    assert norm_bwd(ws_bytes=0) == ARG and norm_bwd(ws=A[9] + 8) == ARG
    big = (1, 100000, 64, 4)                                         # chunks
    assert norm(big, ws=0) == ARG and norm(big, ws_bytes=8) == ARG


def test_group_norm_workspace():
    w = gc.group_norm_workspace
    assert w((4, 1, 64, 4), torch.bfloat16) == 0
    assert w((1, 100000, 64, 4), torch.bfloat16) >= 8 * 4
    assert w((4, 1, 64, 4), torch.bfloat16, True) >= 8 * 64
    with pytest.raises(gc.GconvError):
        w((1, 1, 64, 3), torch.float32)


def quant(rows=4, K=100, stride=100, x=A[0], q=A[1], scales=A[2], dtype=2):
    return S._library().gconv_quantize_int8(x, q, scales, rows, K, stride, dtype, None)


def mm(shape=(4, 32, 100), q=A[0], s=A[1], w=A[2], ws=A[3], b=A[4], y=A[5], dtype=2):
    return S._library().gconv_matmul_int8(q, s, w, ws, b, y, arr(*shape), dtype, None)


def test_int8_refusals():
    assert quant(rows=-1) == ARG and quant(K=0) == ARG and quant(dtype=4) == ARG and quant(stride=-1) == ARG
    assert quant(x=0) == ARG and quant(q=0) == ARG and quant(scales=0) == ARG
    assert quant(q=A[0] + 16) == ARG and quant(scales=A[1] + 4) == ARG
    assert quant(rows=1 << 25) == UNSUPPORTED and quant(K=1 << 31, stride=1 << 31) == UNSUPPORTED
    for bad in ((-1, 32, 100), (4, 0, 100), (4, 32, 0)):
        assert mm(bad) == ARG
    assert mm((4, 32, 131072)) == UNSUPPORTED and "32 bits" in gc.gconv_last_error()
    assert mm((2 ** 31 - 1, 32, 1)) == UNSUPPORTED and mm((4, 2 ** 31 - 1, 1)) == UNSUPPORTED
    assert mm(dtype=3) == ARG
    for name in ("q", "s", "w", "ws", "y"):
        assert mm(**{name: 0}) == ARG
    assert mm(y=A[2] + 64) == ARG and mm(y=A[4]) == ARG              # over the weights, over the bias


def test_nothing_to_do():
    assert rec((0, 100, 64), ptrs=[0] * 4) == OK and gc.gconv_last_kernel() == ""
    assert rec((2, 0, 64), ptrs=[0] * 4) == OK                       # no token and no state asked for
    assert rec_step((0, 64, 3)) == OK
    assert norm((0, 5, 8, 2), x=0, y=0) == OK and norm((2, 0, 8, 2), x=0, y=0, stats=0) == OK
    assert quant(rows=0, x=0, q=0, scales=0) == OK and mm((0, 32, 100), q=0, y=0) == OK


def test_python_refuses_before_the_library():
    x = torch.zeros(2, 3, 8)
    for call in (lambda: gc.gated_recurrence(x, x, x, torch.zeros(8)), lambda: gc.group_norm(x, 2, torch.ones(8)),
                 lambda: gc.quantize_int8(x), lambda: gc.gated_recurrence_step(x[0], x[0], x[0], torch.zeros(8), x[0]),
                 lambda: gc.matmul_int8(x.to(torch.int8), x[..., :1], x[0].to(torch.int8), torch.ones(3))):
        with pytest.raises(gc.GconvError):        # not GPU tensors
            call()
    with pytest.raises(gc.GconvError):
        gc.quantize_int8(x.to(torch.int32))
    with pytest.raises(gc.GconvError):
        gc.matmul_int8(x.to(torch.int8), x[..., :1], x[0].to(torch.int8), torch.ones(3), dtype=torch.float64)


def test_gated_recurrence_backward_channels():
    """The sum over log_decay's shares takes 64 threads a channel: with 2^26 - 15 channels and more a launch of
    2^32 threads, which HIP would cut short."""
    for C in (2 ** 26 - 15, 2 ** 26 - 1):
        for shape in ((1, 1, C), (0, 1, C), (1, 0, C)):
            assert rec_bwd(shape) == UNSUPPORTED, shape


def test_group_norm_workspace_beside_its_tensors():
    """Gradients of groups wider than a workgroup: 8 bytes a part of a group and sample, and partial sums of dw and
    db in up to 2048 rows or a sixteenth of x in 16 bits."""
    w = gc.group_norm_workspace
    for dtype in (torch.float32, torch.bfloat16):
        for P, C in ((1, 16384), (3, 1031), (20, 20000), (100, 16384)):
            for N in (2000, 16384, 1000000):
                assert w((N, P, C, 1), dtype, True) <= 8 * C * max(2048, N * P // 64 + 1) + 8 * N * 32 + 512, (N, P, C)
