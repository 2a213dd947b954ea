"""GPU parity of the product in 8-bit integers and of its quantiser.

The quantiser's scale and quotients are fp32's own, so that its outputs are compared bit for bit:
a quotient of two fp32 numbers taken in 64 bits and rounded to fp32 is fp32's.  The integer sum is
exact.  Its conversion to fp32, two products and an addition are off by u = 2^-24 each of the
intermediate result; the output is rounded once more.
"""
import pytest
import torch

import depthwise_convolution_gconv_amd as gc

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24


def rounding(dtype, r):
    f = torch.finfo(dtype)
    return (f.eps / 2 * r.abs()).clamp(min=f.eps * f.smallest_normal / 2)


def near(name, y, r, bound):
    y = y.detach().double().cpu()
    assert y.shape == r.shape, (name, y.shape, r.shape)
    assert torch.isfinite(y).all(), name
    over = (y - r).abs() - bound
    assert float(over.max()) <= 0, f"{name}: over its bound by {float(over.max()):.3e} at {int(over.argmax())} of {tuple(r.shape)}"


def quantized(x):
    x = x.double().cpu()
    scale = (x.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -100) / 127.0).float()
    return torch.round((x / scale.double()).float()).to(torch.int8), scale


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (2, 8), (70, 129), (5, 1000), (4, 1025), (3, 4096), (2, 4100), (2, 16384),
                                 (1, 33333), (300, 64)])
def test_quantize(M, K, dt):
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(M, K, generator=gen) * torch.exp(3 * torch.randn(M, 1, generator=gen))
    x = x.to(DT[dt])
    x[0] = 0
    if M > 2:      # quotients on the border between two integers
        x[1] = torch.arange(K).remainder(255) - 127
        x[2] = (torch.arange(K).remainder(255) - 127) * 0.5
    print("quantize", M, K, dt, flush=True)
    q, s = gc.quantize_int8(x.cuda())
    torch.cuda.synchronize()
    rq, rs = quantized(x)
    assert torch.equal(s.cpu(), rs) and torch.equal(q.cpu(), rq)
    assert int(q.abs().max()) <= 127


def test_quantize_views_and_axes():
    gen = torch.Generator().manual_seed(2)
    x = torch.randn(3, 5, 41, generator=gen).to(torch.bfloat16).cuda()
    for v in (x[..., 1:40], x[:, 2], x[0, 0], x[:1]):
        q, s = gc.quantize_int8(v)
        rq, rs = quantized(v)
        assert torch.equal(q.cpu(), rq) and torch.equal(s.cpu(), rs) and s.shape == (*v.shape[:-1], 1)
    with pytest.raises(gc.GconvError):
        gc.quantize_int8(x.transpose(0, 1))
    assert gc.quantize_int8(x[:0])[0].shape == (0, 5, 41)


def test_quantize_values_that_are_not_finite():
    x = torch.ones(4, 100).cuda()
    x[1, 50], x[2, 99] = float("nan"), float("-inf")
    q, s = gc.quantize_int8(x)
    assert torch.isnan(s[1, 0]) and torch.isinf(s[2, 0]) and torch.equal(s[0], s[3]) and bool((q[0] == 127).all())
    y = gc.matmul_int8(q, s, torch.ones(3, 100, dtype=torch.int8).cuda(), torch.ones(3).cuda(), dtype=torch.float32)
    assert torch.isfinite(y[0]).all() and torch.equal(y[0], y[3])


SHAPES = [  # M, N, K
    (1, 1, 1), (1, 16, 64), (1, 100, 4096), (2, 33, 63), (16, 40, 1350), (17, 64, 512), (33, 130, 129), (63, 17, 1000),
    (64, 8200, 256), (1, 8208, 100), (65, 64, 128), (65, 65, 16), (100, 130, 144), (333, 410, 1350), (130, 200, 15),
    (128, 128, 2048), (300, 500, 1), (257, 4100, 272), (1000, 2100, 100), (1800, 2200, 384), (4097, 4099, 64), (4000, 4096, 160),
]


def operands(M, N, K, seed, top=False):
    gen = torch.Generator().manual_seed(seed)
    lo, hi = (-128, -127) if top else (-128, 128)
    q = torch.randint(lo, hi, (M, K), generator=gen, dtype=torch.int8)
    w = torch.randint(lo, hi, (N, K), generator=gen, dtype=torch.int8)
    return q.cuda(), (0.5 + torch.rand(M, 1, generator=gen)).cuda() * 0.01, w.cuda(), (0.5 + torch.rand(N, generator=gen)).cuda() * 0.01


def check(q, s, w, ws, b, dtype):
    y = gc.matmul_int8(q, s, w, ws, b, dtype)
    torch.cuda.synchronize()
    total = (q.double() @ w.double().t()).cpu()
    r = total * s.double().cpu() * ws.double().cpu()
    off = 3 * U * r.abs()
    if b is not None:
        r = r + b.double().cpu()
        off = off + U * r.abs()
    near("y", y, r, rounding(dtype, r) + off * (1 + torch.finfo(dtype).eps))
    return y


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda c: "x".join(map(str, c)))
def test_matmul(shape, dt):
    M, N, K = shape
    q, s, w, ws = operands(M, N, K, 1)
    print("int8", shape, dt, flush=True)
    b = None if K % 2 else (torch.randn(N, generator=torch.Generator().manual_seed(2)) * 0.1).to(DT[dt]).cuda()
    y = check(q, s, w, ws, b, DT[dt])
    assert torch.equal(y, gc.matmul_int8(q, s, w, ws.view(N, 1), b, DT[dt]))


def test_rows_at_any_address_and_leading_axes():
    """The same product from operands that start on no 16-byte border, which take another path."""
    for M, N, K in ((3, 40, 128), (70, 90, 128), (300, 1000, 256)):
        q, s, w, ws = operands(M, N, K, 3)
        odd = lambda t: torch.cat([t.new_zeros(5), t.reshape(-1)])[5:].view_as(t)  # noqa: E731
        want = gc.matmul_int8(q, s, w, ws, dtype=torch.float32)
        assert torch.equal(gc.matmul_int8(odd(q), s, odd(w), ws, dtype=torch.float32), want)
    q, s, w, ws = operands(24, 20, 32, 4)
    y = gc.matmul_int8(q.view(2, 3, 4, 32), s.view(2, 3, 4, 1), w, ws)
    assert torch.equal(y.view(24, 20), gc.matmul_int8(q, s, w, ws)) and y.dtype is torch.bfloat16
    assert gc.matmul_int8(q[0], s[0], w, ws).shape == (20,)
    assert gc.matmul_int8(q[:0], s[:0], w, ws).shape == (0, 20)


@pytest.mark.parametrize("M", [2, 70])
def test_the_largest_sums(M):
    """-128 times -128 over the largest K: 2^31 - 2^14 fits, and no sum saturates."""
    q, s, w, ws = operands(M, 20, 131071, 5, top=True)
    assert int(q.max()) == -128
    check(q, s, w, ws, None, torch.float32)


def test_quantised_linear_layer():
    """Tokens and weights quantised, multiplied: off by half a step of each operand."""
    gen = torch.Generator().manual_seed(6)
    x, w = torch.randn(200, 300, generator=gen).to(torch.bfloat16).cuda(), torch.randn(150, 300, generator=gen).cuda()
    (q, s), (wq, ws) = gc.quantize_int8(x), gc.quantize_int8(w)
    y = gc.matmul_int8(q, s, wq, ws, dtype=torch.float32).double()
    xd, wd = x.double(), w.double()
    half = 0.5 * (1 + 1e-6)
    bound = half * (s.double() * wd.abs().sum(1) + ws.double().view(-1) * xd.abs().sum(1, keepdim=True)) + 0.25 * 300 * 1.01 * s.double() * ws.double().view(-1)
    r = xd @ wd.t()
    assert bool(((y - r).abs() <= bound + 1e-5 * r.abs()).all())
