"""Sequence operators of libgconv.so: linear attention with a decay for each head, RMS
norm with the residual's addition (16/32-bit or e4m3 output), and the causal depthwise
conv1d that carries its state.

Like the convolution binding: argument checks and marshalling only, on the caller's
current device and stream, outputs and workspaces from torch.  Every function takes
`stream` (default: the current stream of the tensors' device).  With another one the call
runs as under torch.cuda.stream(stream): its outputs and workspace are that stream's
memory, and the outputs may also be used on the caller's current stream, once that waits
for the other.  That the inputs are ready on `stream`, and kept, is the caller's to see to.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from ._binding import (DTYPES, ERR_INVALID_ARG, ERR_SHAPE, GconvError, _check, _i32, _i64, _i64p, _vp, lib)

ACTIVATIONS = {None: 0, "silu": 1}
_f32 = ctypes.c_float
_size = ctypes.c_size_t

_fns = None


def _library():
    """The entry points with their argument types set."""
    global _fns
    if _fns is None:
        L = lib()
        sizep = ctypes.POINTER(_size)
        for name, args in {
            "gconv_linear_attention_workspace": [_i64p, _i32, _i32, sizep],
            "gconv_linear_attention": [_vp] * 4 + [_i64p, _i64p, _vp, _f32] + [_vp] * 3 + [_i32, _vp, _size, _vp],
            "gconv_linear_attention_backward": [_vp] * 7 + [_i64p, _i64p, _vp, _f32] + [_vp] * 4 + [_i32, _vp, _size, _vp],
            "gconv_linear_attention_step": [_vp] * 5 + [_i64p, _i64p, _vp, _f32, _vp, _i32, _vp],
            "gconv_rms_norm": [_vp] * 5 + [_i64, _i64, _i64p, _f32, _i32, _vp],
            "gconv_rms_norm_e4m3": [_vp] * 6 + [_i64, _i64, _i64p, _f32, _i32, _i32, _vp],
            "gconv_rms_norm_backward_workspace": [_i64, _i64, _i32, sizep],
            "gconv_rms_norm_backward": [_vp] * 6 + [_i64, _i64, _i64p, _f32, _i32, _vp, _size, _vp],
            "gconv_dw1d_causal": [_vp] * 7 + [_i64p, _i64p, _i32, _i32, _vp],
            "gconv_dw1d_causal_backward_workspace": [_i64p, _i32, sizep],
            "gconv_dw1d_causal_backward": [_vp] * 11 + [_i64p, _i64p, _i32, _i32, _vp, _size, _vp],
            "gconv_dw1d_causal_step": [_vp] * 6 + [_i64p, _i64, _i32, _i32, _vp],
        }.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = _i32
        _fns = L
    return _fns


@functools.lru_cache(maxsize=4096)
def _array(*values):
    """Sizes or strides for the C entry points; those of a serving loop's calls repeat."""
    return (_i64 * len(values))(*values)


def _bad(text: str, status: int = ERR_INVALID_ARG):
    raise GconvError(status, text)


def _dtype(name: str, t: torch.Tensor) -> int:
    d = DTYPES.get(t.dtype)
    if d is None:
        _bad(f"{name}: unsupported dtype {t.dtype}")
    if not t.is_cuda:
        _bad(f"{name} must be a GPU tensor")
    return d


def _view(name: str, t: torch.Tensor, dtype, dev: int, shape):
    """Strides of a tensor of that dtype, device and shape whose last axis is contiguous."""
    if t.dtype is not dtype or t.get_device() != dev:
        _bad(f"{name} must match the dtype and device of the other tensors")
    if t.shape != shape:
        _bad(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}", ERR_SHAPE)
    st = t.stride()
    if st[-1] != 1 and t.shape[-1] > 1 and t.numel():
        _bad(f"{name}: the last axis must be contiguous")
    return st


def _whole(name: str, t: Optional[torch.Tensor], dtype, dev: int, shape) -> int:
    """Address of a contiguous tensor of that dtype, device and shape (0 for None)."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.get_device() != dev:
        _bad(f"{name} must be a {dtype} tensor on device {dev}")
    if t.shape != shape:
        _bad(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}", ERR_SHAPE)
    if not t.is_contiguous():
        _bad(f"{name} must be contiguous")
    return t.data_ptr()


# The current device and stream without their Python objects, which cost more than the rest of a
# single-token call's checks.  Builds of torch without a GPU lack them, and have no tensor that a
# call would get as far with.
_device = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _on_stream(stream, ref: torch.Tensor, fn, *args):
    """fn(*args) as the work of `stream`: what it allocates is the stream's own memory (a block
    that the current stream has freed may still be in use there), and the current stream's use
    of its outputs counts too when they are freed."""
    dev = ref.get_device()
    if dev < 0:
        return fn(*args)      # refuses them
    if stream.device.index != dev:
        _bad(f"stream is on {stream.device}, the tensors are on device {dev}")
    here = torch.cuda.current_stream(dev)
    with torch.cuda.stream(stream):
        out = fn(*args)
    if here != stream:
        for t in out if isinstance(out, tuple) else (out,):
            if t is not None:
                t.record_stream(here)
    return out


def _workspace(need: int, ref: torch.Tensor) -> Optional[torch.Tensor]:
    return ref.new_empty(need, dtype=torch.uint8) if need else None


def _like(t: torch.Tensor) -> torch.Tensor:
    """A contiguous tensor of t's shape and dtype."""
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def _ptr(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


# ---------------------------------------------------------------- linear attention

def _attn_args(q, k, v, log_decay, lengths):
    dt = _dtype("q", q)
    if q.dim() != 4 or v.dim() != 4:
        _bad("q and k must be [B, T, Hk, Dk], v [B, T, H, Dv]")
    B, T, Hk, Dk = q.shape
    H, Dv = v.shape[2], v.shape[3]
    dtype, dev = q.dtype, q.get_device()
    st = (*_view("q", q, dtype, dev, q.shape)[:3], *_view("k", k, dtype, dev, q.shape)[:3],
          *_view("v", v, dtype, dev, (B, T, H, Dv))[:3])
    g = _whole("log_decay", log_decay, torch.float32, dev, (H,))
    n = _whole("lengths", lengths, torch.int32, dev, (B,))
    return dt, (B, T, Hk, H, Dk, Dv), st, g, n


def linear_attention_workspace(shape, dtype: torch.dtype, backward: bool = False) -> int:
    """Workspace bytes of linear_attention (or its backward) for shape (B, T, Hk, H, Dk, Dv)."""
    n = _size(0)
    _check(_library().gconv_linear_attention_workspace(_array(*shape), DTYPES[dtype], int(backward),
                                                       ctypes.byref(n)))
    return n.value


def linear_attention(q, k, v, log_decay, scale: Optional[float] = None, initial_state=None, lengths=None,
                     return_state: bool = False, stream=None):
    """Linear attention with a decay for each head over whole prompts.

        S_t = exp(log_decay[h]) S_(t-1) + k_t v_t^T,   o_t = scale * q_t S_t

    q, k [B, T, Hk, Dk], v [B, T, H, Dv] with H a multiple of Hk (each key head serves
    H / Hk value heads), any strides but a contiguous last axis; log_decay fp32 [H];
    scale defaults to Dk**-0.5.  initial_state: fp32 [B, H, Dk, Dv].  lengths: int32 [B],
    the tokens of each sequence that exist; the outputs of the others are zero.
    Returns o [B, T, H, Dv], or (o, state) with the fp32 state after each sequence's last
    token, which linear_attention_step carries on from.

    Sums and states are fp32; scores, and the state where a query meets it, enter their second
    product with 16 bits for 16-bit inputs and 24 for fp32.
    A value that is not finite reaches its own and later tokens only; an infinity counts as NaN."""
    if stream is not None:
        return _on_stream(stream, q, linear_attention, q, k, v, log_decay, scale, initial_state, lengths, return_state)
    dt, shape, strides, g, n = _attn_args(q, k, v, log_decay, lengths)
    B, T, Hk, H, Dk, Dv = shape
    dev = q.get_device()
    s0 = _whole("initial_state", initial_state, torch.float32, dev, (B, H, Dk, Dv))
    sh = _array(*shape)
    need = _size(0)
    L = _library()
    _check(L.gconv_linear_attention_workspace(sh, dt, 0, ctypes.byref(need)))
    if _device() != dev:
        with torch.cuda.device(dev):
            return linear_attention(q, k, v, log_decay, scale, initial_state, lengths, return_state)
    o = _like(v)
    st = q.new_empty((B, H, Dk, Dv), dtype=torch.float32) if return_state else None
    ws = _workspace(need.value, q)
    _check(L.gconv_linear_attention(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), sh,
        _array(*strides, *o.stride()[:3]), g,
        Dk ** -0.5 if scale is None else scale, s0, _ptr(st), n, dt, _ptr(ws), need.value, _raw_stream(dev)))
    return (o, st) if return_state else o


def linear_attention_backward(q, k, v, log_decay, do, scale: Optional[float] = None, initial_state=None,
                              lengths=None, dstate=None, stream=None):
    """(dq, dk, dv, dinitial) of linear_attention from the gradients `do` of its output and
    `dstate` (fp32, or None: zero) of its final state.  dinitial is None without an
    initial_state.  log_decay is a constant: it gets no gradient.  Precision as forward; a value
    that is not finite reaches the tokens that the formulas name (of q and do: its own and
    earlier ones)."""
    if stream is not None:
        return _on_stream(stream, q, linear_attention_backward, q, k, v, log_decay, do, scale, initial_state, lengths, dstate)
    dt, shape, strides, g, n = _attn_args(q, k, v, log_decay, lengths)
    B, T, Hk, H, Dk, Dv = shape
    dev = q.get_device()
    strides += _view("do", do, q.dtype, dev, (B, T, H, Dv))[:3]
    s0 = _whole("initial_state", initial_state, torch.float32, dev, (B, H, Dk, Dv))
    sf = _whole("dstate", dstate, torch.float32, dev, (B, H, Dk, Dv))
    sh = _array(*shape)
    need = _size(0)
    L = _library()
    _check(L.gconv_linear_attention_workspace(sh, dt, 1, ctypes.byref(need)))
    if _device() != dev:
        with torch.cuda.device(dev):
            return linear_attention_backward(q, k, v, log_decay, do, scale, initial_state, lengths, dstate)
    dq, dk, dv = _like(q), _like(k), _like(v)
    ds = q.new_empty((B, H, Dk, Dv), dtype=torch.float32) if initial_state is not None else None
    ws = _workspace(need.value, q)
    _check(L.gconv_linear_attention_backward(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), do.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), sh,
        _array(*strides, *dq.stride()[:3], *dk.stride()[:3], *dv.stride()[:3]), g, Dk ** -0.5 if scale is None else scale, s0, sf,
        _ptr(ds), n, dt, _ptr(ws), need.value, _raw_stream(dev)))
    return dq, dk, dv, ds


def linear_attention_step(q, k, v, log_decay, state, scale: Optional[float] = None, slots=None, stream=None):
    """The next token of each sequence: q, k [B, Hk, Dk], v [B, H, Dv]; state fp32
    [n, H, Dk, Dv] is updated in place.  slots: int32 [B], the row of `state` that each
    sequence owns, each row at most once (default: row b); a slot outside [0, n) leaves
    the pool alone and gives a zero output.  Returns o [B, H, Dv]."""
    if stream is not None:
        return _on_stream(stream, q, linear_attention_step, q, k, v, log_decay, state, scale, slots)
    dt = _dtype("q", q)
    if q.dim() != 3 or v.dim() != 3 or state.dim() != 4:
        _bad("q and k must be [B, Hk, Dk], v [B, H, Dv], state [n, H, Dk, Dv]")
    B, Hk, Dk = q.shape
    H, Dv = v.shape[1], v.shape[2]
    dtype, dev = q.dtype, q.get_device()
    strides = (*_view("q", q, dtype, dev, q.shape)[:2], *_view("k", k, dtype, dev, q.shape)[:2],
               *_view("v", v, dtype, dev, (B, H, Dv))[:2])
    g = _whole("log_decay", log_decay, torch.float32, dev, (H,))
    sp = _whole("state", state, torch.float32, dev, (state.shape[0], H, Dk, Dv))
    sl = _whole("slots", slots, torch.int32, dev, (B,))
    if _device() != dev:
        with torch.cuda.device(dev):
            return linear_attention_step(q, k, v, log_decay, state, scale, slots)
    o = _like(v)
    _check(_library().gconv_linear_attention_step(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), sp, _array(B, Hk, H, Dk, Dv, state.shape[0]),
        _array(*strides, *o.stride()[:2]), g,
        Dk ** -0.5 if scale is None else scale, sl, dt, _raw_stream(dev)))
    return o


# ---------------------------------------------------------------- RMS norm

def _rows(name: str, t: torch.Tensor, ref: torch.Tensor) -> int:
    """The one stride that leads from row to row of t's last axis."""
    _view(name, t, ref.dtype, ref.get_device(), ref.shape)
    if t.dim() == 2:
        return t.stride(0)
    if t.dim() == 1 or t.numel() == 0 or t.is_contiguous():
        return t.shape[-1]
    step = None          # from the last row axis on: each longer axis goes on where the shorter ones end
    for n, s in reversed(list(zip(t.shape[:-1], t.stride()[:-1]))):
        if n == 1:
            continue
        if step is None:
            row = step = s
        elif s != step:
            _bad(f"{name}: its rows must lie at one stride")
        step = s * n
    return t.shape[-1] if step is None else row


def _norm(x, weight, residual, eps, q8, block):
    dt = _dtype("x", x)
    if x.dim() < 1 or x.shape[-1] < 1:
        _bad("x must be [..., C] with C >= 1")
    C = x.shape[-1]
    rows = x.numel() // C
    dev = x.get_device()
    if _device() != dev:
        with torch.cuda.device(dev):
            return _norm(x, weight, residual, eps, q8, block)
    xs = _rows("x", x, x)
    w = _whole("weight", weight, x.dtype, dev, (C,))
    if not w:
        _bad("weight is needed")
    if residual is not None:
        rs = _rows("residual", residual, x)
        h = _like(x)
    else:
        rs, h = 0, None
    L = _library()
    if not q8:
        y = _like(x)
        _check(L.gconv_rms_norm(x.data_ptr(), _ptr(residual), w, y.data_ptr(), _ptr(h), rows, C, _array(xs, rs), eps,
                                dt, _raw_stream(dev)))
        return y, h
    y = x.new_empty(x.shape, dtype=torch.float8_e4m3fn)
    nb = -(-C // block) if block > 0 else 1
    scales = x.new_empty((*x.shape[:-1], nb), dtype=torch.float32)
    _check(L.gconv_rms_norm_e4m3(x.data_ptr(), _ptr(residual), w, y.data_ptr(), scales.data_ptr(), _ptr(h), rows, C,
                                 _array(xs, rs), eps, block, dt, _raw_stream(dev)))
    return y, scales, h


def rms_norm(x, weight, residual=None, eps: float = 1e-6, stream=None):
    """y = weight * h / sqrt(mean(h^2) + eps) over the last axis of x [..., C], where h is x,
    or x + residual rounded to the dtype.  Returns y, or (y, h) with a residual."""
    if stream is not None:
        return _on_stream(stream, x, rms_norm, x, weight, residual, eps)
    y, h = _norm(x, weight, residual, eps, False, 0)
    return y if residual is None else (y, h)


def rms_norm_e4m3(x, weight, residual=None, eps: float = 1e-6, block: int = 0, stream=None):
    """rms_norm with its output as e4m3 values q (float8_e4m3fn [..., C]) and fp32 scales,
    y = q * scale: one scale for a row (block 0, scales [..., 1]) or for each `block`
    columns (32, 64, 128 or 256; scales [..., ceil(C / block)]).
    Returns (q, scales), or (q, scales, h) with a residual."""
    if stream is not None:
        return _on_stream(stream, x, rms_norm_e4m3, x, weight, residual, eps, block)
    y, scales, h = _norm(x, weight, residual, eps, True, int(block))
    return (y, scales) if residual is None else (y, scales, h)


def rms_norm_backward(dy, h, weight, eps: float = 1e-6, dh=None, stream=None):
    """(dx, dw) of rms_norm: dx is the gradient of x and of residual alike, from the gradient
    dy of y, the normed rows h (x itself without a residual) and the gradient dh of the h
    output (or None)."""
    if stream is not None:
        return _on_stream(stream, h, rms_norm_backward, dy, h, weight, eps, dh)
    dt = _dtype("h", h)
    if h.dim() < 1 or h.shape[-1] < 1:
        _bad("h must be [..., C] with C >= 1")
    C = h.shape[-1]
    rows = h.numel() // C
    dev = h.get_device()
    L = _library()
    need = _size(0)
    _check(L.gconv_rms_norm_backward_workspace(rows, C, dt, ctypes.byref(need)))
    if _device() != dev:
        with torch.cuda.device(dev):
            return rms_norm_backward(dy, h, weight, eps, dh)
    w = _whole("weight", weight, h.dtype, dev, (C,))
    if not w:
        _bad("weight is needed")
    ys, hs = _rows("dy", dy, h), _rows("h", h, h)
    es = _rows("dh", dh, h) if dh is not None else 0
    dx, dw = _like(h), _like(weight)
    ws = _workspace(need.value, h)
    _check(L.gconv_rms_norm_backward(dy.data_ptr(), h.data_ptr(), w, _ptr(dh), dx.data_ptr(), dw.data_ptr(), rows,
                                     C, _array(ys, hs, es), eps, dt, _ptr(ws), need.value, _raw_stream(dev)))
    return dx, dw


# ---------------------------------------------------------------- causal depthwise conv1d

def _conv_args(x, weight, bias, activation, dims):
    dt = _dtype("x", x)
    if x.dim() != dims or weight.dim() != 3:
        _bad(f"x must be {dims}-D with channels last and weight [C, 1, K]")
    C, K = x.shape[-1], weight.shape[2]
    if activation not in ACTIVATIONS:
        _bad(f"unknown activation {activation!r}")
    dtype, dev = x.dtype, x.get_device()
    _view("x", x, dtype, dev, x.shape)
    w = _whole("weight", weight, dtype, dev, (C, 1, K))
    b = _whole("bias", bias, dtype, dev, (C,))
    return dt, C, K, w, b, ACTIVATIONS[activation]


def dwconv1d_causal(x, weight, bias=None, activation: Optional[str] = None, initial_state=None, lengths=None,
                    return_state: bool = False, stream=None):
    """Causal depthwise conv1d over x [B, T, C] (any strides, channels contiguous) with weight
    [C, 1, K]: y[t] = act(bias + sum_k weight[k] * xs[t - (K-1) + k]), where the K-1 inputs
    before the first token come from initial_state [B, K-1, C] (default: zeros).
    activation: None or "silu".  lengths: int32 [B]; the outputs past them are zero.
    Returns y, or (y, state) with the last K-1 inputs of each sequence, which
    dwconv1d_causal_step carries on from."""
    if stream is not None:
        return _on_stream(stream, x, dwconv1d_causal, x, weight, bias, activation, initial_state, lengths, return_state)
    dt, C, K, w, b, act = _conv_args(x, weight, bias, activation, 3)
    B, T, _ = x.shape
    dev = x.get_device()
    s0 = _whole("initial_state", initial_state, x.dtype, dev, (B, K - 1, C))
    n = _whole("lengths", lengths, torch.int32, dev, (B,))
    if _device() != dev:
        with torch.cuda.device(dev):
            return dwconv1d_causal(x, weight, bias, activation, initial_state, lengths, return_state)
    y = _like(x)
    st = x.new_empty((B, K - 1, C)) if return_state else None
    _check(_library().gconv_dw1d_causal(x.data_ptr(), w, b, y.data_ptr(), s0, _ptr(st), n, _array(B, T, C, K),
                                        _array(*x.stride()[:2]), act, dt, _raw_stream(dev)))
    return (y, st) if return_state else y


def dwconv1d_causal_backward(x, weight, bias, dy, activation: Optional[str] = None, initial_state=None, lengths=None,
                             dstate=None, stream=None):
    """(dx, dw, db, dinitial) of dwconv1d_causal from the gradients dy of its output and
    dstate (or None: zero) of its final state.  db is None without a bias, dinitial
    without an initial_state."""
    if stream is not None:
        return _on_stream(stream, x, dwconv1d_causal_backward, x, weight, bias, dy, activation, initial_state, lengths, dstate)
    dt, C, K, w, b, act = _conv_args(x, weight, bias, activation, 3)
    B, T, _ = x.shape
    dev = x.get_device()
    _view("dy", dy, x.dtype, dev, x.shape)
    s0 = _whole("initial_state", initial_state, x.dtype, dev, (B, K - 1, C))
    sf = _whole("dstate", dstate, x.dtype, dev, (B, K - 1, C))
    n = _whole("lengths", lengths, torch.int32, dev, (B,))
    L = _library()
    sh = _array(B, T, C, K)
    need = _size(0)
    _check(L.gconv_dw1d_causal_backward_workspace(sh, dt, ctypes.byref(need)))
    if _device() != dev:
        with torch.cuda.device(dev):
            return dwconv1d_causal_backward(x, weight, bias, dy, activation, initial_state, lengths, dstate)
    dx, dw = _like(x), _like(weight)
    db = _like(bias) if bias is not None else None
    ds = x.new_empty((B, K - 1, C)) if initial_state is not None else None
    ws = _workspace(need.value, x)
    _check(L.gconv_dw1d_causal_backward(x.data_ptr(), w, b, dy.data_ptr(), s0, sf, dx.data_ptr(), dw.data_ptr(),
                                        _ptr(db), _ptr(ds), n, sh, _array(*x.stride()[:2], *dy.stride()[:2]),
                                        act, dt, _ptr(ws), need.value, _raw_stream(dev)))
    return dx, dw, db, ds


def dwconv1d_causal_step(x, weight, bias, state, activation: Optional[str] = None, slots=None, stream=None):
    """The next token of each sequence: x [B, C]; state [n, K-1, C] moves up by one row in
    place.  slots as for linear_attention_step.  Returns y [B, C]."""
    if stream is not None:
        return _on_stream(stream, x, dwconv1d_causal_step, x, weight, bias, state, activation, slots)
    dt, C, K, w, b, act = _conv_args(x, weight, bias, activation, 2)
    B = x.shape[0]
    dev = x.get_device()
    if state.dim() != 3:
        _bad("state must be [n, K-1, C]")
    sp = _whole("state", state, x.dtype, dev, (state.shape[0], K - 1, C))
    sl = _whole("slots", slots, torch.int32, dev, (B,))
    if _device() != dev:
        with torch.cuda.device(dev):
            return dwconv1d_causal_step(x, weight, bias, state, activation, slots)
    y = _like(x)
    _check(_library().gconv_dw1d_causal_step(x.data_ptr(), w, b, sp, y.data_ptr(), sl,
                                             _array(B, C, K, state.shape[0]), x.stride(0), act, dt, _raw_stream(dev)))
    return y
