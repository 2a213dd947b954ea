"""Operators of a recurrent mixing block in libgconv.so: the gated linear recurrence, group
norm with an activation over channels-last tensors, and the product in 8-bit integers.

Argument checks and marshalling only, in the manner of the other sequence operators: the
caller's current device and stream, or `stream`; outputs and workspaces from torch.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from ._binding import DTYPES, _check, _i32, _i64, _i64p, _vp, lib
from ._sequence import (ACTIVATIONS, _array, _bad, _device, _dtype, _f32, _like, _on_stream, _ptr, _raw_stream, _rows,
                        _size, _view, _whole, _workspace)

_fns = None


def _library():
    """The entry points with their argument types set."""
    global _fns
    if _fns is None:
        L = lib()
        sizep = ctypes.POINTER(_size)
        for name, args in {
            "gconv_gated_recurrence_workspace": [_i64p, _i32, _i32, sizep],
            "gconv_gated_recurrence": [_vp] * 5 + [_i64p, _i64p] + [_vp] * 3 + [_i32, _vp, _size, _vp],
            "gconv_gated_recurrence_backward": [_vp] * 10 + [_i64p, _i64p] + [_vp] * 4 + [_i32, _vp, _size, _vp],
            "gconv_gated_recurrence_step": [_vp] * 6 + [_i64p, _i64p, _vp, _i32, _vp],
            "gconv_group_norm_workspace": [_i64p, _i32, _i32, sizep],
            "gconv_group_norm": [_vp] * 5 + [_i64p, _i64p, _vp, _f32, _i32, _i32, _vp, _size, _vp],
            "gconv_group_norm_backward": [_vp] * 8 + [_i64p, _i64p, _vp, _i32, _i32, _vp, _size, _vp],
            "gconv_quantize_int8": [_vp] * 3 + [_i64, _i64, _i64, _i32, _vp],
            "gconv_matmul_int8": [_vp] * 6 + [_i64p, _i32, _vp],
        }.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = _i32
        _fns = L
    return _fns


# ---------------------------------------------------------------- gated recurrence

def _gated_args(x, r, i, log_decay, lengths, dims):
    dt = _dtype("x", x)
    if x.dim() != dims:
        _bad("x, r and i must be [B, T, C]" if dims == 3 else "x, r and i must be [B, C]")
    dtype, dev, shape = x.dtype, x.get_device(), x.shape
    st = (*_view("x", x, dtype, dev, shape)[:-1], *_view("r", r, dtype, dev, shape)[:-1],
          *_view("i", i, dtype, dev, shape)[:-1])
    g = _whole("log_decay", log_decay, torch.float32, dev, (shape[-1],))
    if not g and shape[-1]:
        _bad("log_decay is needed")
    return dt, dev, st, g, _whole("lengths", lengths, torch.int32, dev, (shape[0],))


def gated_recurrence_workspace(shape, dtype: torch.dtype, backward: bool = False) -> int:
    """Workspace bytes of gated_recurrence (or its backward) for shape (B, T, C)."""
    n = _size(0)
    _check(_library().gconv_gated_recurrence_workspace(_array(*shape), DTYPES[dtype], int(backward), ctypes.byref(n)))
    return n.value


def gated_recurrence(x, r, i, log_decay, initial_state=None, lengths=None, return_state: bool = False, stream=None):
    """Gated linear recurrence over whole prompts, each channel by itself.

        a_t = exp(log_decay * sigmoid(r_t)),   h_t = a_t h_(t-1) + sqrt(1 - a_t^2) sigmoid(i_t) x_t

    x and the logits r, i of its gates [B, T, C], any strides but contiguous channels; log_decay
    fp32 [C], finite and <= 0.  initial_state: fp32 [B, C].  lengths: int32 [B], the tokens of each
    sequence that exist; the outputs of the others are zero.  Returns h [B, T, C], or (h, state)
    with the fp32 state after each sequence's last token, which gated_recurrence_step carries on
    from.

    Gates, sums and states are fp32.  A value that is not finite reaches its own and later tokens
    of its channel only; an infinity may count as NaN in later ones."""
    if stream is not None:
        return _on_stream(stream, x, gated_recurrence, x, r, i, log_decay, initial_state, lengths, return_state)
    dt, dev, strides, g, n = _gated_args(x, r, i, log_decay, lengths, 3)
    B, T, C = x.shape
    s0 = _whole("initial_state", initial_state, torch.float32, dev, (B, C))
    sh = _array(B, T, C)
    need = _size(0)
    L = _library()
    _check(L.gconv_gated_recurrence_workspace(sh, dt, 0, ctypes.byref(need)))
    if _device() != dev:
        with torch.cuda.device(dev):
            return gated_recurrence(x, r, i, log_decay, initial_state, lengths, return_state)
    h = _like(x)
    st = x.new_empty((B, C), dtype=torch.float32) if return_state else None
    ws = _workspace(need.value, x)
    _check(L.gconv_gated_recurrence(x.data_ptr(), r.data_ptr(), i.data_ptr(), g, h.data_ptr(), sh, _array(*strides), s0,
                                    _ptr(st), n, dt, _ptr(ws), need.value, _raw_stream(dev)))
    return (h, st) if return_state else h


def gated_recurrence_backward(x, r, i, log_decay, h, dh, initial_state=None, lengths=None, dstate=None, stream=None):
    """(dx, dr, di, dlog_decay, dinitial) of gated_recurrence from its output h, the gradient dh of
    that and dstate (fp32 [B, C], or None: zero) of its final state.  The states before each token
    are taken from h as it was rounded.  dlog_decay is fp32 [C]; dinitial is None without an
    initial_state.  Where 1 - a^2 is zero or below 2^-126 (log_decay next to zero, or a gate that
    underflows) the root is taken as zero, without a derivative."""
    if stream is not None:
        return _on_stream(stream, x, gated_recurrence_backward, x, r, i, log_decay, h, dh, initial_state, lengths, dstate)
    dt, dev, strides, g, n = _gated_args(x, r, i, log_decay, lengths, 3)
    B, T, C = x.shape
    strides += (*_view("h", h, x.dtype, dev, x.shape)[:2], *_view("dh", dh, x.dtype, dev, x.shape)[:2])
    s0 = _whole("initial_state", initial_state, torch.float32, dev, (B, C))
    sf = _whole("dstate", dstate, torch.float32, dev, (B, C))
    sh = _array(B, T, C)
    need = _size(0)
    L = _library()
    _check(L.gconv_gated_recurrence_workspace(sh, dt, 1, ctypes.byref(need)))
    if _device() != dev:
        with torch.cuda.device(dev):
            return gated_recurrence_backward(x, r, i, log_decay, h, dh, initial_state, lengths, dstate)
    dx, dr, di = _like(x), _like(r), _like(i)
    dg = torch.empty_like(log_decay)
    ds = x.new_empty((B, C), dtype=torch.float32) if initial_state is not None else None
    ws = _workspace(need.value, x)
    _check(L.gconv_gated_recurrence_backward(
        x.data_ptr(), r.data_ptr(), i.data_ptr(), g, h.data_ptr(), dh.data_ptr(), dx.data_ptr(), dr.data_ptr(),
        di.data_ptr(), dg.data_ptr(), sh, _array(*strides), s0, sf, _ptr(ds), n, dt, _ptr(ws), need.value,
        _raw_stream(dev)))
    return dx, dr, di, dg, ds


def gated_recurrence_step(x, r, i, log_decay, state, slots=None, stream=None):
    """The next token of each sequence: x, r, i [B, C]; state fp32 [n, C] is updated in place.
    slots: int32 [B], the row of `state` that each sequence owns, each row at most once (default:
    row b); a slot outside [0, n) leaves the pool alone and gives a zero output.  Returns h [B, C]."""
    if stream is not None:
        return _on_stream(stream, x, gated_recurrence_step, x, r, i, log_decay, state, slots)
    dt, dev, strides, g, _ = _gated_args(x, r, i, log_decay, None, 2)
    B, C = x.shape
    if state.dim() != 2:
        _bad("state must be [n, C]")
    sp = _whole("state", state, torch.float32, dev, (state.shape[0], C))
    sl = _whole("slots", slots, torch.int32, dev, (B,))
    if _device() != dev:
        with torch.cuda.device(dev):
            return gated_recurrence_step(x, r, i, log_decay, state, slots)
    h = _like(x)
    _check(_library().gconv_gated_recurrence_step(x.data_ptr(), r.data_ptr(), i.data_ptr(), g, sp, h.data_ptr(),
                                                  _array(B, C, state.shape[0]), _array(*strides), sl, dt,
                                                  _raw_stream(dev)))
    return h


# ---------------------------------------------------------------- group norm

def _positions(name: str, t: torch.Tensor, ref: torch.Tensor):
    """Strides of a [N, ..., C] tensor's samples and positions, whose axes must lie at one stride."""
    st = _view(name, t, ref.dtype, ref.get_device(), ref.shape)
    if t.dim() == 2:
        return st[0], 0
    if t.dim() == 3:
        return st[0], st[1]
    step = None          # from the last position axis on: each longer axis goes on where the shorter ones end
    for n, s in reversed(list(zip(t.shape[1:-1], st[1:-1]))):
        if n == 1:
            continue
        if step is None:
            first = step = s
        elif s != step and t.numel():
            _bad(f"{name}: its positions must lie at one stride")
        step = s * n
    return st[0], 0 if step is None else first


def _norm_args(x, groups, weight, bias, activation, lengths):
    dt = _dtype("x", x)
    if x.dim() < 2 or x.shape[-1] < 1:
        _bad("x must be [N, ..., C] with C >= 1")
    if activation not in ACTIVATIONS:
        _bad(f"unknown activation {activation!r}")
    dev, N, C = x.get_device(), x.shape[0], x.shape[-1]
    P = 1
    for n in x.shape[1:-1]:
        P *= n
    w = _whole("weight", weight, x.dtype, dev, (C,))
    if not w:
        _bad("weight is needed")
    return (dt, dev, (N, P, C, int(groups)), _positions("x", x, x), w, _whole("bias", bias, x.dtype, dev, (C,)),
            ACTIVATIONS[activation], _whole("lengths", lengths, torch.int32, dev, (N,)))


def group_norm_workspace(shape, dtype: torch.dtype, backward: bool = False) -> int:
    """Workspace bytes of group_norm (or its backward) for shape (N, P, C, G), P positions a sample."""
    n = _size(0)
    _check(_library().gconv_group_norm_workspace(_array(*shape), DTYPES[dtype], int(backward), ctypes.byref(n)))
    return n.value


def group_norm(x, groups: int, weight, bias=None, eps: float = 1e-5, activation: Optional[str] = None, lengths=None,
               return_stats: bool = False, stream=None):
    """Group norm with an activation over channels-last x [N, ..., C]: y = act(weight * (x - mean) /
    sqrt(var + eps) + bias), mean and (biased) variance over a sample's positions and the C / groups
    channels of a group.  x [N, C] is normed row by row (a token's heads, say).

    x may be a view whose positions lie at one stride, with contiguous channels.  activation: None
    or "silu".  lengths: int32 [N], the positions of each sample that exist, in order; the outputs
    of the others are zero.  Returns y, or (y, stats) with stats fp32 [N, groups, 2], the mean and
    1 / sqrt(var + eps), which group_norm_backward takes.  A sample without positions has mean 0
    and variance 0."""
    if stream is not None:
        return _on_stream(stream, x, group_norm, x, groups, weight, bias, eps, activation, lengths, return_stats)
    dt, dev, shape, strides, w, b, act, n = _norm_args(x, groups, weight, bias, activation, lengths)
    sh = _array(*shape)
    need = _size(0)
    L = _library()
    _check(L.gconv_group_norm_workspace(sh, dt, 0, ctypes.byref(need)))
    if _device() != dev:
        with torch.cuda.device(dev):
            return group_norm(x, groups, weight, bias, eps, activation, lengths, return_stats)
    y = _like(x)
    stats = x.new_empty((shape[0], shape[3], 2), dtype=torch.float32) if return_stats else None
    ws = _workspace(need.value, x)
    _check(L.gconv_group_norm(x.data_ptr(), w, b, y.data_ptr(), _ptr(stats), sh, _array(*strides), n, eps, act, dt,
                              _ptr(ws), need.value, _raw_stream(dev)))
    return (y, stats) if return_stats else y


def group_norm_backward(dy, x, groups: int, weight, bias, stats, activation: Optional[str] = None, lengths=None,
                        stream=None):
    """(dx, dw, db) of group_norm from the gradient dy of its output and the stats that it returned.
    db is None without a bias.  A sample without positions adds nothing, whatever its stats are."""
    if stream is not None:
        return _on_stream(stream, x, group_norm_backward, dy, x, groups, weight, bias, stats, activation, lengths)
    dt, dev, shape, strides, w, b, act, n = _norm_args(x, groups, weight, bias, activation, lengths)
    ds = _positions("dy", dy, x)
    sh = _array(*shape)
    need = _size(0)
    L = _library()
    _check(L.gconv_group_norm_workspace(sh, dt, 1, ctypes.byref(need)))
    st = _whole("stats", stats, torch.float32, dev, (shape[0], shape[3], 2))
    if _device() != dev:
        with torch.cuda.device(dev):
            return group_norm_backward(dy, x, groups, weight, bias, stats, activation, lengths)
    dx, dw = _like(x), _like(weight)
    db = _like(bias) if bias is not None else None
    ws = _workspace(need.value, x)
    _check(L.gconv_group_norm_backward(dy.data_ptr(), x.data_ptr(), w, b, st, dx.data_ptr(), dw.data_ptr(), _ptr(db), sh,
                                       _array(*ds, *strides), n, act, dt, _ptr(ws), need.value, _raw_stream(dev)))
    return dx, dw, db


# ---------------------------------------------------------------- product in 8-bit integers

def quantize_int8(x, stream=None):
    """Rows of x [..., K] as 8-bit integers: (q int8 [..., K], scales fp32 [..., 1]) with
    scale = max(max|row|, 2^-100) / 127 and q = x / scale, each quotient fp32's own, rounded to
    the nearest integer (ties to even); x is about q * scale.  x's rows may lie at any one stride.
    A value that is not finite makes its row's scale that, and q without meaning."""
    if stream is not None:
        return _on_stream(stream, x, quantize_int8, x)
    dt = _dtype("x", x)
    if x.dim() < 1 or x.shape[-1] < 1:
        _bad("x must be [..., K] with K >= 1")
    K, dev = x.shape[-1], x.get_device()
    if _device() != dev:
        with torch.cuda.device(dev):
            return quantize_int8(x)
    xs = _rows("x", x, x)
    q = x.new_empty(x.shape, dtype=torch.int8)
    scales = x.new_empty((*x.shape[:-1], 1), dtype=torch.float32)
    _check(_library().gconv_quantize_int8(x.data_ptr(), q.data_ptr(), scales.data_ptr(), x.numel() // K, K, xs, dt,
                                          _raw_stream(dev)))
    return q, scales


def matmul_int8(q, scales, weight, weight_scales, bias=None, dtype: torch.dtype = torch.bfloat16, stream=None):
    """y[..., n] = (sum_k q[..., k] * weight[n, k]) * scales * weight_scales[n] + bias[n] in `dtype`
    (float32, float16 or bfloat16).

    q int8 [..., K] and scales fp32 [..., 1] as quantize_int8 gives them; weight int8 [N, K],
    weight_scales fp32 [N] or [N, 1] (quantize_int8 of the weights gives both); bias [N] in `dtype`.  All
    contiguous, K at most 131071.  The sum is exact.  It is rounded to fp32, its product with the
    token's scale too, and that times the channel's scale plus the bias once (a fused multiply and
    add); the result is rounded to the dtype."""
    if stream is not None:
        return _on_stream(stream, q, matmul_int8, q, scales, weight, weight_scales, bias, dtype)
    dt = DTYPES.get(dtype)
    if dt is None:
        _bad(f"unsupported output dtype {dtype}")
    if q.dtype is not torch.int8 or not q.is_cuda:
        _bad("q must be an int8 GPU tensor")
    if q.dim() < 1 or weight.dim() != 2 or q.shape[-1] < 1:
        _bad("q must be [..., K] and weight [N, K] with K >= 1")
    K, N, dev = q.shape[-1], weight.shape[0], q.get_device()
    qp = _whole("q", q, torch.int8, dev, q.shape)
    sp = _whole("scales", scales, torch.float32, dev, (*q.shape[:-1], 1))
    w = _whole("weight", weight, torch.int8, dev, (N, K))
    ws = _whole("weight_scales", weight_scales.view(N) if weight_scales.dim() == 2 and weight_scales.numel() == N
                and weight_scales.is_contiguous() else weight_scales, torch.float32, dev, (N,))
    b = _whole("bias", bias, dtype, dev, (N,))
    if _device() != dev:
        with torch.cuda.device(dev):
            return matmul_int8(q, scales, weight, weight_scales, bias, dtype)
    y = q.new_empty((*q.shape[:-1], N), dtype=dtype)
    _check(_library().gconv_matmul_int8(qp, sp, w, ws, b, y.data_ptr(), _array(q.numel() // K, N, K), dt,
                                        _raw_stream(dev)))
    return y
