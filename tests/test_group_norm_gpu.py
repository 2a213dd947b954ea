"""GPU parity of group norm with an activation (channels last) and of its gradients against the
definition in 64 bits on the CPU.

Tolerances, fixed from the arithmetic before the first run.  u = 2^-24.  A sum over a group has at
most 128 additions in a thread, 16 and 6 in a wave, and over chunks as many as lanes take and 6:
ADD = 300 u of the sum of magnitudes.  So a mean is off by ADD mean|x|; squares about a thread's
own mean, joined exactly, are off by ADD of their sum, and the root of the variance by half of that
and 4u.  silu's slope is at most 1.1; its sigmoid is off by (6 + 1.5 |z|) u.  Outputs are rounded
once.  Gradients come from automatic differentiation of the definition.
"""
import pytest
import torch

import depthwise_convolution_gconv_amd as gc

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24
ADD = 300 * U
EPS = 1e-5


def rounding(dtype, r):
    f = torch.finfo(dtype)
    return (f.eps / 2 * r.abs()).clamp(min=f.eps * f.smallest_normal / 2)


def near(name, y, r, bound):
    y = y.detach().double().cpu()
    assert y.shape == r.shape, (name, y.shape, r.shape)
    assert torch.isfinite(y).all(), name
    if y.numel():
        over = (y - r).abs() - bound
        assert float(over.max()) <= 0, f"{name}: over its bound by {float(over.max()):.3e} at {int(over.argmax())} of {tuple(r.shape)}"


def live_of(lengths, N, P):
    if lengths is None:
        return torch.ones(N, P, 1, 1, dtype=torch.float64)
    return (torch.arange(P)[None] < torch.tensor(lengths)[:, None]).double().view(N, P, 1, 1)


def definition(x, w, b, G, silu, live):
    """(y, mean, rstd, hat, z) of x [N, P, C], fp64, differentiable."""
    N, P, C = x.shape
    v = x.view(N, P, G, C // G)
    m = (live.sum((1, 2, 3), keepdim=True) * (C // G)).clamp(min=1)
    mean = (v * live).sum((1, 3), keepdim=True) / m
    rstd = (((v - mean) * live).square().sum((1, 3), keepdim=True) / m + EPS).rsqrt()
    hat = (v - mean) * rstd
    z = hat * w.view(G, -1) + (b.view(G, -1) if b is not None else 0.0)
    y = (z * torch.sigmoid(z) if silu else z) * live
    return y.reshape(N, P, C), mean, rstd, hat, z


def inputs(N, P, C, dtype, layout, seed, offset=1.5):
    gen = torch.Generator().manual_seed(seed)
    size, at = torch.exp(0.5 * torch.randn(C, generator=gen)), offset * torch.randn(C, generator=gen)
    x = (torch.randn(N, P, C, generator=gen) * size + at).to(dtype)
    if layout == "wide":         # channels out of wider rows, at an odd offset
        t = torch.zeros(N, P, C + 7, dtype=dtype)
        t[..., 3:C + 3] = x
        x = t.cuda()[..., 3:C + 3]
    elif layout == "swapped":    # [P, N, C] in memory
        x = x.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    else:
        x = x.cuda()
    w = (1 + 0.2 * torch.randn(C, generator=gen)).to(dtype).cuda()
    b = (0.3 * torch.randn(C, generator=gen)).to(dtype).cuda()
    return x, w, b


def d(t):
    return None if t is None else t.detach().double().cpu()


CASES = [  # N, P, C, G, silu, bias, lengths, layout
    (1, 1, 1, 1, True, True, None, "plain"),
    (3, 1, 96, 4, True, True, None, "plain"),
    (70, 1, 1024, 8, True, True, None, "wide"),        # rows by themselves: a token's heads
    (5, 1, 77, 7, False, False, None, "plain"),        # 11 channels a group, nothing but scalar loads
    (2, 49, 32, 32, True, True, None, "plain"),        # a channel is a group
    (2, 50, 24, 4, True, True, [0, 50], "plain"),
    (2, 196, 60, 5, False, True, [1, 195], "swapped"),
    (1, 784, 128, 2, True, True, None, "wide"),
    (4, 300, 512, 32, True, True, [300, 7, 0, 299], "plain"),
    (2, 1025, 72, 3, True, False, None, "swapped"),
    (1, 4096, 64, 2, True, True, None, "plain"),       # the whole sample in registers
    (2, 5000, 48, 4, True, True, [5000, 1234], "wide"),
    (2, 20001, 32, 4, True, True, None, "plain"),      # chunks of positions
    (1, 9000, 20, 2, False, True, [4097], "plain"),
    (2, 3, 5000, 1, True, True, None, "plain"),        # a group wider than a workgroup
    (1, 70, 2062, 2, True, True, [33], "plain"),
    (300, 2, 64, 4, True, True, None, "plain"),
    (1100, 3, 1030, 1, True, True, None, "plain"),    # too wide, and enough samples for one chunk each
    (40, 17000, 3, 1, False, True, None, "plain"),
]


def ids(c):
    return "x".join(map(str, c[:4]))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=ids)
def test_group_norm(case, dt):
    N, P, C, G, silu, bias, lengths, layout = case
    dtype, act = DT[dt], "silu" if silu else None
    x, w, b = inputs(N, P, C, dtype, layout, 1)
    b = b if bias else None
    ln = torch.tensor(lengths, dtype=torch.int32).cuda() if lengths else None
    print("group norm", case, dt, flush=True)
    y, stats = gc.group_norm(x, G, w, b, EPS, act, ln, return_stats=True)
    torch.cuda.synchronize()
    live = live_of(lengths, N, P)
    ry, mean, rstd, hat, z = definition(d(x), d(w), d(b), G, silu, live)
    m = (live.sum((1, 2, 3), keepdim=True) * (C // G)).clamp(min=1)
    mean_off = ADD * (d(x).view(N, P, G, -1).abs() * live).sum((1, 3), keepdim=True) / m + U * mean.abs()
    near("mean", stats[..., 0], mean.view(N, G), mean_off.view(N, G))
    near("rstd", stats[..., 1], rstd.view(N, G), ((ADD / 2 + 4 * U) * rstd).view(N, G))
    zoff = d(w).abs().view(G, -1) * (hat.abs() * (ADD / 2 + 8 * U) + rstd * mean_off) + 4 * U * z.abs()
    off = zoff if not silu else 1.1 * zoff + z.abs() * (8 + 1.5 * z.abs()) * U
    near("y", y, ry, (rounding(dtype, ry) + (off * live).reshape(N, P, C) * (1 + torch.finfo(dtype).eps)))
    assert torch.equal(y, gc.group_norm(x, G, w, b, EPS, act, ln))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=ids)
def test_group_norm_backward(case, dt):
    N, P, C, G, silu, bias, lengths, layout = case
    dtype, act = DT[dt], "silu" if silu else None
    x, w, b = inputs(N, P, C, dtype, layout, 2)
    b = b if bias else None
    dy = torch.randn(N, P, C, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    ln = torch.tensor(lengths, dtype=torch.int32).cuda() if lengths else None
    live = live_of(lengths, N, P)
    X, W = d(x).requires_grad_(), d(w).requires_grad_()
    Bs = d(b).requires_grad_() if bias else None
    ry, mean, rstd, hat, z = definition(X, W, Bs, G, silu, live)
    wanted = torch.autograd.grad((ry * d(dy)).sum(), [X, W] + ([Bs] if bias else []))
    stats = torch.stack([mean, rstd], -1).view(N, G, 2).float().cuda()
    print("group norm backward", case, dt, flush=True)
    dx, dw, db = gc.group_norm_backward(dy, x, G, w, b, stats, act, ln)
    torch.cuda.synchronize()
    mean, rstd, hat, z = (t.detach() for t in (mean, rstd, hat, z))
    A = d(dy).abs().view(N, P, G, -1) * live
    wa = d(w).abs().view(G, -1)
    hoff = 4 * U * hat.abs() + U * rstd * mean.abs()
    if silu:   # the slope s + z s (1 - s) is at most 1.1, its own slope at most 1/2
        dz, dzoff = 1.1 * A, A * (0.5 * (wa * hoff + 4 * U * z.abs()) + (24 + 4 * z.abs()) * U)
    else:
        dz, dzoff = A, 2 * U * A
    m = (live.sum((1, 2, 3), keepdim=True) * (C // G)).clamp(min=1)
    over = lambda t: t.sum((1, 3), keepdim=True) / m  # noqa: E731
    s1, s1off = over(wa * dz), over(wa * (dzoff + 2 * U * dz)) + ADD * over(wa * dz)
    t2, t2off = dz * hat.abs(), dzoff * hat.abs() + dz * hoff + 3 * U * dz * hat.abs()
    s2, s2off = over(wa * t2), over(wa * t2off) + ADD * over(wa * t2)
    off = rstd * (wa * dzoff + s1off + hat.abs() * s2off + hoff * s2 + 6 * U * (wa * dz + s1 + hat.abs() * s2)) * live
    near("dx", dx, wanted[0], rounding(dtype, wanted[0]) + off.reshape(N, P, C) * (1 + torch.finfo(dtype).eps))
    rows = ADD + (N / 16 + 20) * U
    cols = lambda t: t.sum((0, 1)).reshape(C)  # noqa: E731
    near("dw", dw, wanted[1], rounding(dtype, wanted[1]) + (cols(t2off) + rows * cols(t2)) * (1 + torch.finfo(dtype).eps))
    if bias:
        near("db", db, wanted[2], rounding(dtype, wanted[2]) + (cols(dzoff) + rows * cols(dz)) * (1 + torch.finfo(dtype).eps))
    else:
        assert db is None
    again = gc.group_norm_backward(dy, x, G, w, b, stats, act, ln)
    assert all(p is None or torch.equal(p, q) for p, q in zip((dx, dw, db), again))


def test_gradients_against_differences():
    N, P, C, G = 2, 60, 12, 3
    x, w, b = inputs(N, P, C, torch.float32, "plain", 5)
    r = torch.randn(N, P, C, generator=torch.Generator().manual_seed(6))
    live = live_of([60, 31], N, P)
    ln = torch.tensor([60, 31], dtype=torch.int32).cuda()
    _, stats = gc.group_norm(x, G, w, b, EPS, "silu", ln, return_stats=True)
    grads = gc.group_norm_backward(r.cuda(), x, G, w, b, stats, "silu", ln)
    args = [d(x), d(w), d(b)]
    f = lambda q: float((definition(*q, G, True, live)[0] * r.double()).sum())  # noqa: E731
    for k, g in enumerate(grads):
        v = torch.randn(args[k].shape, generator=torch.Generator().manual_seed(7 + k)).double()
        hi, lo = ([q + s * 1e-5 * v if j == k else q for j, q in enumerate(args)] for s in (1, -1))
        want, got = (f(hi) - f(lo)) / 2e-5, float((d(g) * v).sum())
        assert abs(want - got) <= 1e-5 * float((d(g) * v).abs().sum()) + 1e-6 * abs(want), (k, want, got)


@pytest.mark.parametrize("shape", [(2, 7, 9, 48), (3, 48), (2, 3, 2, 5, 16)])
def test_positions_of_any_number_of_axes(shape):
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(*shape, generator=gen).cuda()
    w, b = torch.ones(shape[-1]).cuda(), torch.zeros(shape[-1]).cuda()
    flat = x.reshape(shape[0], -1, shape[-1])
    assert torch.equal(gc.group_norm(x, 4, w, b), gc.group_norm(flat, 4, w, b).view(shape))
    if len(shape) == 4:
        wide = torch.zeros(2, 7, 9, 50).cuda()
        wide[..., 1:49] = x
        assert torch.equal(gc.group_norm(wide[..., 1:49], 4, w, b), gc.group_norm(x, 4, w, b))
        with pytest.raises(gc.GconvError):
            gc.group_norm(x.transpose(1, 2), 4, w, b)


@pytest.mark.parametrize("P", [40, 20001])
def test_values_that_are_not_finite(P):
    """Padding reaches nothing; a NaN reaches its sample's group only."""
    x, w, b = inputs(2, P, 32, torch.bfloat16, "plain", 8)
    dy = torch.randn(2, P, 32, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    n = torch.tensor([P - 9, P], dtype=torch.int32).cuda()
    y, st = gc.group_norm(x, 4, w, b, lengths=n, return_stats=True)
    back = gc.group_norm_backward(dy, x, 4, w, b, st, lengths=n)
    x[0, P - 9:] = float("nan")
    dy[0, P - 9:] = float("inf")
    y2, st2 = gc.group_norm(x, 4, w, b, lengths=n, return_stats=True)
    assert torch.equal(y, y2) and torch.equal(st, st2) and not y2[0, P - 9:].any()
    assert all(torch.equal(p, q) for p, q in zip(back, gc.group_norm_backward(dy, x, 4, w, b, st2, lengths=n)))
    x[1, 3, 9] = float("nan")
    y3 = gc.group_norm(x, 4, w, b, lengths=n)
    assert torch.isnan(y3[1, :, 8:16]).all()
    y3[1, :, 8:16] = y2[1, :, 8:16]
    assert torch.equal(y3, y2)


def test_an_offset_much_larger_than_the_spread():
    """Values near 4096 with a spread of 1: the variance keeps its digits."""
    gen = torch.Generator().manual_seed(1)
    for P in (600, 30000):
        x = (4096 + torch.randn(2, P, 16, generator=gen)).cuda()
        w, b = torch.ones(16).cuda(), torch.zeros(16).cuda()
        _, st = gc.group_norm(x, 2, w, b, EPS, return_stats=True)
        _, mean, rstd, _, _ = definition(d(x), d(w), d(b), 2, False, live_of(None, 2, P))
        # The threads' own means are off by 128 u of 4096, which enters squared: 1e-9 of the variance.
        near("rstd", st[..., 1], rstd.view(2, 2), ((ADD / 2 + 4 * U + 1e-8) * rstd).view(2, 2))


def test_nothing_to_do():
    w = torch.ones(8).cuda()
    e = torch.zeros(0, 5, 8).cuda()
    assert gc.group_norm(e, 2, w).shape == e.shape
    dx, dw, db = gc.group_norm_backward(e, e, 2, w, w, torch.zeros(0, 2, 2).cuda())
    assert dx.shape == e.shape and not dw.any() and not db.any()
    e = torch.zeros(3, 0, 8).cuda()
    y, st = gc.group_norm(e, 2, w, eps=0.25, return_stats=True)
    assert y.shape == e.shape and torch.equal(st, torch.tensor([0.0, 2.0]).cuda().expand(3, 2, 2))
    assert not gc.group_norm_backward(e, e, 2, w, None, st)[1].any()
