"""GPU parity of the gated linear recurrence (prompts, gradients, single tokens) against its
definition in 64 bits on the CPU.

Tolerances, fixed from the arithmetic before the first run.  u = 2^-24 is fp32's half step.
The hardware's exponential, reciprocal and root are off by at most 2u of their value; an
exponential's argument z, scaled by log2 e, is off by 1.5 u of it, which is 1.5 |z| u of the
result.  So a sigmoid of z is off by (6 + 1.5 |z|) u, la = log_decay sigmoid(r) by two more, a
by |la| of that plus 3u, the root of 1 - a^2 by as much as la and 8u, and u_t by all of these:
at most (24 + 1.5 |r| + 1.5 |i|) u of itself.  An error in a at token t enters with the state
before it, and from there on is carried like the state: ERR below is that recurrence, with one
more u for each multiplication and addition.  Joining runs adds one rounding for each level of
the join (6) and tile: 16 u of a sum of magnitudes.  Outputs are rounded once.
"""
import pytest
import torch

import depthwise_convolution_gconv_amd as gc

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


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


def definition(x, r, i, g, s0, lengths):
    """Token by token in fp64, differentiable: (h [B, T, C], state [B, C])."""
    B, T, C = x.shape
    S = s0 if s0 is not None else torch.zeros(B, C, dtype=torch.float64)
    a = torch.exp(g * torch.sigmoid(r))
    add = torch.sqrt(-torch.expm1(2 * g * torch.sigmoid(r))) * torch.sigmoid(i) * x
    out = []
    for t in range(T):
        live = torch.tensor([t < n for n in lengths]).view(B, 1)
        S = torch.where(live, a[:, t] * S + add[:, t], S)
        out.append(torch.where(live, S, torch.zeros((), dtype=torch.float64)))
    return torch.stack(out, 1) if out else torch.zeros(B, 0, C, dtype=torch.float64), S


def carried(a, add, err_a, err_add, first, first_err=0.0, reverse=False):
    """Magnitudes of a recurrence and the bound ERR on its error, along axis 1."""
    B, T, C = a.shape
    H, E = first.abs(), first.abs() * 0 + first_err
    mags, errs = [], []
    for t in (range(T - 1, -1, -1) if reverse else range(T)):
        E = a[:, t] * E + a[:, t] * H * (err_a[:, t] + 2 * U) + add[:, t] * (err_add[:, t] + U)
        H = a[:, t] * H + add[:, t]
        mags.append(H)
        errs.append(E + 16 * U * H)
    if reverse:
        mags, errs = mags[::-1], errs[::-1]
    return torch.stack(mags, 1), torch.stack(errs, 1)


def inputs(B, T, C, dtype, state, layout, seed=1, decay="spread"):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    if layout == "fused":      # views of one projection, an odd number of columns apart
        x, r, i = (rnd(B, T, 3 * C + 3).to(dtype).cuda()[..., 1:]).split([C, C, C, 2], dim=-1)[:3]
    elif layout == "time":     # [T, B, C] in memory
        x, r, i = (rnd(T, B, C).to(dtype).cuda().transpose(0, 1) for _ in range(3))
    else:
        x, r, i = (rnd(B, T, C).to(dtype).cuda() for _ in range(3))
    g = (2 * torch.log1p(-(2.0 ** (-1.5 - 10 * torch.rand(C, generator=gen))))).cuda() if decay == "spread" else torch.full((C,), float(decay)).cuda()
    s0 = (2 * rnd(B, C)).cuda() if state else None
    return x, r, i, g, s0


def d(t):
    return None if t is None else t.detach().double().cpu()


CASES = [  # B, T, C, state, lengths, layout
    (1, 1, 1, False, None, "plain"),
    (2, 5, 1, True, [5, 0], "plain"),
    (1, 1, 64, True, None, "plain"),
    (3, 2, 2, True, [0, 1, 2], "plain"),
    (2, 31, 33, True, None, "fused"),
    (2, 128, 32, False, None, "plain"),
    (2, 129, 47, True, [129, 127], "time"),
    (1, 255, 3, False, None, "fused"),
    (1, 256, 96, True, None, "plain"),
    (3, 257, 65, True, [257, 256, 1], "fused"),
    (2, 513, 40, True, [300, 513], "time"),
    (1, 1537, 34, True, None, "plain"),           # several segments
    (2, 2500, 31, True, [2500, 1111], "fused"),   # segments past a sequence's end, odd rows
    (1, 3000, 1, True, None, "plain"),
    (5, 700, 2000, False, [700, 0, 699, 1, 350], "plain"),
]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[:3])))
def test_gated_recurrence(case, dt):
    B, T, C, state, lengths, layout = case
    dtype = DT[dt]
    x, r, i, g, s0 = inputs(B, T, C, dtype, state, layout)
    ln = torch.tensor(lengths, dtype=torch.int32).cuda() if lengths else None
    print("gated", case, dt, flush=True)
    h, st = gc.gated_recurrence(x, r, i, g, initial_state=s0, lengths=ln, return_state=True)
    torch.cuda.synchronize()
    n = lengths or [T] * B
    X, R, I, Gd, S0 = d(x), d(r), d(i), d(g), d(s0)
    rh, rs = definition(X, R, I, Gd, S0, n)
    sr = torch.sigmoid(R)
    la = (Gd * sr).abs()
    live = (torch.arange(T)[None] < torch.tensor(n)[:, None])[..., None]
    a = torch.where(live, torch.exp(-la), 1.0)
    add = torch.where(live, torch.sqrt(-torch.expm1(-2 * la)) * torch.sigmoid(I) * X.abs(), 0.0)
    err_a = torch.where(live, (la * (9 + 1.5 * R.abs()) + 3) * U, 0.0)
    _, err = carried(a, add, err_a, (24 + 1.5 * R.abs() + 1.5 * I.abs()) * U, S0 if S0 is not None else torch.zeros(B, C).double())
    near("h", h, rh, rounding(dtype, rh) + err * (1 + half_step(dtype)))
    near("state", st, rs, err[:, -1])
    assert torch.equal(h, gc.gated_recurrence(x, r, i, g, initial_state=s0, lengths=ln))
    if lengths:
        for b, m in enumerate(lengths):
            assert not h[b, m:].any()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[:3])))
def test_gated_recurrence_backward(case, dt):
    B, T, C, state, lengths, layout = case
    dtype = DT[dt]
    x, r, i, g, s0 = inputs(B, T, C, dtype, state, layout, seed=2)
    gen = torch.Generator().manual_seed(3)
    dh = torch.randn(B, T, C, generator=gen).to(dtype).cuda()
    dst = torch.randn(B, C, generator=gen).cuda() if state else None
    ln = torch.tensor(lengths, dtype=torch.int32).cuda() if lengths else None
    n = lengths or [T] * B
    print("gated backward", case, dt, flush=True)
    X, R, I, Gd = (d(t).requires_grad_() for t in (x, r, i, g))
    S0 = d(s0).requires_grad_() if state else None
    rh, rs = definition(X, R, I, Gd, S0, n)
    h = rh.detach().to(dtype).cuda()
    out = gc.gated_recurrence_backward(x, r, i, g, h, dh, initial_state=s0, lengths=ln, dstate=dst)
    torch.cuda.synchronize()
    loss = (rh * d(dh)).sum() + ((rs * d(dst)).sum() if state else 0.0)
    wanted = torch.autograd.grad(loss, [X, R, I, Gd] + ([S0] if state else []), allow_unused=True)
    X, R, I, Gd, rh = (t.detach() for t in (X, R, I, Gd, rh))
    live = (torch.arange(T)[None] < torch.tensor(n)[:, None])[..., None]
    zero = torch.zeros((), dtype=torch.float64)
    sr, si = torch.sigmoid(R), torch.sigmoid(I)
    la = Gd.abs() * sr
    a, root = torch.where(live, torch.exp(-la), 1.0), torch.sqrt(-torch.expm1(-2 * la))
    err_a = torch.where(live, (la * (9 + 1.5 * R.abs()) + 3) * U, zero)
    # c_t = a_t (dh_t + c_(t+1)): magnitudes and errors of c, then of G_t = dh_t + c_(t+1).
    end = d(dst).abs() if state else torch.zeros(B, C).double()
    mag = torch.where(live, d(dh).abs(), zero)
    cm, ce = carried(a, a * mag, err_a, err_a + 2 * U, end, reverse=True)
    G = mag + torch.cat([cm[:, 1:], end[:, None]], 1)
    GE = torch.cat([ce[:, 1:], 0 * end[:, None]], 1) + U * G
    G, GE = torch.where(live, G, zero), torch.where(live, GE, zero)
    K = (40 + 3 * R.abs() + 3 * I.abs()) * U
    prev = torch.cat([(d(s0) if state else torch.zeros(B, C).double())[:, None], rh[:, :-1]], 1).abs()
    # The states are handed in as they were rounded.
    given = torch.cat([torch.zeros(B, 1, C).double(), rounding(dtype, rh[:, :-1])], 1) if T else prev
    f = a * (prev + a / root * si * X.abs())
    fE = K * f + a * given
    one = lambda s, z: (1 - s) + (12 + 3 * z.abs()) * U / K  # noqa: E731 -- 1 - sigmoid and the error of the difference
    err = [GE * root * si + G * root * si * K,
           (GE * f + G * fE) * la * (1 - sr) + G * f * la * one(sr, R) * K,
           GE * root * si * (1 - si) * X.abs() + G * root * si * one(si, I) * X.abs() * K]
    shapes = ("dx", "dr", "di")
    for name, got, want, e in zip(shapes, out, wanted, err):
        want = want if want is not None else torch.zeros_like(X)
        near(name, got, want, rounding(dtype, want) + e * (1 + half_step(dtype)))
    terms = (GE * f + G * fE) * sr + G * f * sr * K
    near("dlog_decay", out[3], wanted[3] if wanted[3] is not None else torch.zeros(C).double(),
         terms.sum((0, 1)) + (16 + T / 64 + B) * U * (G * f * sr).sum((0, 1)))
    if state:
        near("dinitial", out[4], wanted[4], ce[:, 0] if T else 0 * end)
    else:
        assert out[4] is None
    again = gc.gated_recurrence_backward(x, r, i, g, h, dh, initial_state=s0, lengths=ln, dstate=dst)
    assert all(p is None or torch.equal(p, q) for p, q in zip(out, again))


def test_gradients_against_differences():
    """Central differences of the definition along random directions, against the kernel's gradients."""
    B, T, C = 2, 150, 8
    x, r, i, g, s0 = inputs(B, T, C, torch.float32, True, "plain", seed=5)
    w = torch.randn(B, T, C, generator=torch.Generator().manual_seed(6))
    h = gc.gated_recurrence(x, r, i, g, initial_state=s0)
    grads = gc.gated_recurrence_backward(x, r, i, g, h, w.cuda(), initial_state=s0)
    args = [d(t) for t in (x, r, i, g, s0)]
    f = lambda q: float((definition(*q, [T] * B)[0] * w.double()).sum())  # noqa: E731
    for k, gk in enumerate(grads):
        v = torch.randn(args[k].shape, generator=torch.Generator().manual_seed(7 + k)).double()
        e = 1e-5 if k != 3 else 1e-7      # a small log_decay stays negative
        hi, lo = ([q + s * e * v if j == k else q for j, q in enumerate(args)] for s in (1, -1))
        want, got = (f(hi) - f(lo)) / (2 * e), float((d(gk) * v).sum())
        scale = float((d(gk) * v).abs().sum())
        # Differences: e^2 of the third derivative and 2^-52 / e of the loss; gradients: fp32's own error.
        assert abs(want - got) <= 1e-5 * scale + 1e-4 * abs(want), (k, want, got)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,C,slots", [(1, 1, None), (3, 33, None), (4, 257, [6, 0, 3, 9]), (2, 64, [-1, 5])])
def test_step_carries_on(B, C, slots, dt):
    dtype = DT[dt]
    x, r, i, g, _ = inputs(B, 4, C, dtype, False, "fused", seed=4)
    pool = torch.randn(7 if slots else B, C, generator=torch.Generator().manual_seed(1)).cuda()
    rows = torch.tensor(slots, dtype=torch.int32).cuda() if slots else None
    own = slots or list(range(B))
    there = [0 <= s < pool.shape[0] for s in own]
    first = torch.stack([pool[s] if ok else torch.zeros_like(pool[0]) for s, ok in zip(own, there)])
    was = pool.clone()
    want, last = gc.gated_recurrence(x, r, i, g, initial_state=first, return_state=True)
    for t in range(4):
        print("step", B, C, slots, dt, t, flush=True)
        h = gc.gated_recurrence_step(x[:, t], r[:, t], i[:, t], g, pool, slots=rows)
        for b, ok in enumerate(there):
            if ok:      # the same operations, joined in another order
                assert torch.allclose(h[b].float(), want[b, t].float(), rtol=2 * half_step(dtype), atol=1e-5)
            else:
                assert not h[b].any()
    for b, (s, ok) in enumerate(zip(own, there)):
        if ok:
            assert torch.allclose(pool[s], last[b], rtol=1e-5, atol=1e-5)
    for s in set(range(pool.shape[0])) - set(own):
        assert torch.equal(pool[s], was[s])


@pytest.mark.parametrize("T", [40, 1600])
def test_values_that_are_not_finite(T):
    """Padding never reaches anything; a NaN reaches its own and later tokens of its channel."""
    x, r, i, g, s0 = inputs(2, T, 40, torch.bfloat16, True, "plain", seed=8)
    n = torch.tensor([T - 9, T], dtype=torch.int32).cuda()
    dh = torch.randn(2, T, 40, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    h, st = gc.gated_recurrence(x, r, i, g, initial_state=s0, lengths=n, return_state=True)
    back = gc.gated_recurrence_backward(x, r, i, g, h, dh, initial_state=s0, lengths=n)
    for t in (x, r, i, dh):
        t[0, T - 9:] = float("nan")
    h2, st2 = gc.gated_recurrence(x, r, i, g, initial_state=s0, lengths=n, return_state=True)
    h[0, T - 9:] = float("nan")
    back2 = gc.gated_recurrence_backward(x, r, i, g, h, dh, initial_state=s0, lengths=n)
    assert torch.equal(st, st2) and torch.equal(h[1], h2[1]) and torch.equal(h[0, :T - 9], h2[0, :T - 9]) and not h2[0, T - 9:].any()
    assert all(torch.equal(a, b) for a, b in zip(back, back2))
    for k, t in enumerate((x, r, i)):
        keep = t[1, 17, 5].clone()
        t[1, 17, 5] = float("nan")
        bad = gc.gated_recurrence(x, r, i, g, initial_state=s0, lengths=n)
        assert torch.isnan(bad[1, 17:, 5]).all() and not torch.isnan(bad[1, :17, 5]).any()
        bad[1, :, 5] = h2[1, :, 5]
        assert torch.equal(bad, h2), k
        t[1, 17, 5] = keep


def test_log_decay_of_zero_and_gates_at_their_ends():
    """a = 1 and 1 - a^2 = 0: the state stays, no gradient is infinite."""
    x, r, i, g, s0 = inputs(1, 300, 6, torch.float32, True, "plain", seed=9)
    g[:2] = 0.0
    r[..., 2] = -200.0      # sigmoid underflows
    r[..., 3] = 200.0
    i[..., 4] = -200.0
    h, st = gc.gated_recurrence(x, r, i, g, initial_state=s0, return_state=True)
    assert torch.equal(st[0, :3], s0[0, :3]) and torch.equal(h[0, :, :3], s0[:, :3].expand(300, 3))
    back = gc.gated_recurrence_backward(x, r, i, g, h, torch.ones_like(x), initial_state=s0)
    assert all(torch.isfinite(t).all() for t in back)
    assert not back[0][..., :3].any() and torch.equal(back[4][0, :3], torch.full((3,), 300.0).cuda())


def test_nothing_to_do_and_no_token():
    x = torch.zeros(2, 0, 5).cuda()
    g = torch.full((5,), -0.1).cuda()
    s0 = torch.randn(2, 5).cuda()
    h, st = gc.gated_recurrence(x, x, x, g, initial_state=s0, return_state=True)
    assert h.shape == (2, 0, 5) and torch.equal(st, s0)
    assert not gc.gated_recurrence(x, x, x, g, return_state=True)[1].any()
    out = gc.gated_recurrence_backward(x, x, x, g, h, x, initial_state=s0, dstate=s0)
    assert not out[3].any() and torch.equal(out[4], s0)
    e = torch.zeros(0, 7, 5).cuda()
    out = gc.gated_recurrence_backward(e, e, e, g, e, e)
    assert out[0].shape == e.shape and not out[3].any()
    assert gc.gated_recurrence(e, e, e, g).shape == e.shape
    assert gc.gated_recurrence_step(e[:, 0], e[:, 0], e[:, 0], g, s0).shape == (0, 5)
