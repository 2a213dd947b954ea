"""GPU parity of the sequence operators against their definitions in 64 bits on the CPU:
linear attention (prompts, gradients, single tokens), RMS norm (same dtype, e4m3,
gradients), causal depthwise conv1d (prompts, gradients, single tokens).

Tolerances, fixed from the arithmetic.  u = finfo(dtype).eps / 2 is the relative error of
one rounding (half of the constant step among subnormals).  An output is rounded once.  Sums are fp32: n additions and the
factors of a term are off by at most (n + 8) 2^-24 of the sum of the terms' magnitudes A
(the same operation on absolute values).  16-bit attention may round a score and a state
to the dtype before its second product, each u of A.  Gradients come from automatic
differentiation of the definitions, which shares no formula with the kernels.
"""
import pytest
import torch

import depthwise_convolution_gconv_amd as gc

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rounding(dtype, r):
    """Error of rounding r to dtype: half a step, which below the smallest normal stays what it is there."""
    f = torch.finfo(dtype)
    return (f.eps / 2 * r.abs()).clamp(min=f.eps * f.smallest_normal / 2)


def near(name, y, r, bound):
    """|y - r| <= bound, elementwise."""
    y = y.detach().double().cpu()
    assert y.shape == r.shape, (name, y.shape, r.shape)
    assert torch.isfinite(y).all(), name
    over = (y - r).abs() - bound
    worst = float(over.max()) if over.numel() else -1.0
    assert worst <= 0, f"{name}: over its bound by {worst:.3e} at {int(over.argmax())} of {tuple(r.shape)}"


def near_norm(name, y, r, rel):
    """2-norm of the error over the result's, where there are enough values for it."""
    if r.numel() >= 512 and float(r.norm()) > 0:
        e = float((y.detach().double().cpu() - r).norm() / r.norm())
        print(f"{name}: 2-norm error {e:.2e} (bound {rel:.2e})", flush=True)
        assert e <= rel, (name, e, rel)


# ---------------------------------------------------------------- linear attention

def attn_def(q, k, v, g, scale, s0, lengths):
    """Token by token, fp64, differentiable; tokens past a sequence's length do not exist."""
    B, T, Hk, Dk = q.shape
    H, Dv = v.shape[2], v.shape[3]
    r = H // Hk
    lam = torch.exp(g.double()).view(1, H, 1, 1)
    S = s0 if s0 is not None else torch.zeros(B, H, Dk, Dv, dtype=torch.float64)
    out = []
    for t in range(T):
        live = torch.tensor([t < n for n in lengths]).view(B, 1, 1, 1)
        kk, qq = k[:, t].repeat_interleave(r, 1), q[:, t].repeat_interleave(r, 1)
        new = lam * S + kk.unsqueeze(3) * v[:, t].unsqueeze(2)
        S = torch.where(live, new, S)
        o = scale * (qq.unsqueeze(3) * S).sum(2)
        out.append(torch.where(live[..., 0], o, torch.zeros((), dtype=torch.float64)))
    o = torch.stack(out, 1) if out else torch.zeros(B, 0, H, Dv, dtype=torch.float64)
    return o, S


def attn_inputs(B, T, Hk, H, Dk, Dv, dtype, seed, state, layout="plain", decay="spread"):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    if layout == "fused":        # views of one projection, an odd number of columns apart
        x = rnd(B, T, 2 * Hk * Dk + H * Dv + 3).to(dtype).cuda()[..., 1:]
        q, k, v, _ = x.split([Hk * Dk, Hk * Dk, H * Dv, 2], dim=-1)
        q, k, v = q.unflatten(-1, (Hk, Dk)), k.unflatten(-1, (Hk, Dk)), v.unflatten(-1, (H, Dv))
    elif layout == "heads":      # [B, H, T, D] in memory
        q, k = (rnd(B, Hk, T, Dk).to(dtype).cuda().transpose(1, 2) for _ in range(2))
        v = rnd(B, H, T, Dv).to(dtype).cuda().transpose(1, 2)
    else:
        q, k, v = rnd(B, T, Hk, Dk).to(dtype).cuda(), rnd(B, T, Hk, Dk).to(dtype).cuda(), rnd(B, T, H, Dv).to(dtype).cuda()
    g = -(2.0 ** torch.linspace(-1, -9, H)) if decay == "spread" else torch.full((H,), float(decay))
    s0 = rnd(B, H, Dk, Dv).cuda() * 3 if state else None
    return q, k, v, g.cuda(), s0


def bounds(dtype, T, D):
    """(output: factors of |r| and of A; state: factor of A)."""
    sums = (64 + D + 8 + T / 8) * U32
    if dtype == torch.float32:
        return half_step(dtype), sums, sums
    return half_step(dtype), 2.02 * half_step(dtype) + sums, sums


ATTN = [  # B, T, Hk, H, Dk, Dv, state, lengths, layout
    (1, 1, 1, 1, 1, 1, False, None, "plain"),
    (1, 1, 2, 2, 64, 64, True, None, "plain"),
    (2, 2, 1, 3, 8, 9, True, [0, 1], "plain"),
    (2, 63, 2, 2, 64, 64, False, None, "fused"),
    (1, 64, 2, 4, 64, 128, True, None, "heads"),
    (2, 65, 1, 1, 128, 128, True, [65, 64], "plain"),
    (3, 130, 2, 6, 96, 80, True, [0, 129, 57], "fused"),
    (1, 200, 1, 2, 37, 201, False, None, "fused"),
    (1, 129, 1, 1, 256, 256, True, None, "plain"),
    (2, 100, 1, 2, 255, 33, False, [100, 3], "heads"),
    (1, 1000, 1, 1, 128, 64, True, None, "plain"),      # several segments
    (2, 777, 1, 2, 40, 128, True, [777, 300], "fused"),  # segments that end inside and before a sequence's end
    (1, 700, 3, 3, 128, 128, False, None, "fused"),
    (9, 70, 4, 32, 64, 64, True, None, "plain"),         # enough heads for one segment
]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", ATTN, ids=lambda c: "x".join(map(str, c[:6])))
def test_linear_attention(case, dt):
    B, T, Hk, H, Dk, Dv, state, lengths, layout = case
    print("attn", case, dt, flush=True)
    q, k, v, g, s0 = attn_inputs(B, T, Hk, H, Dk, Dv, DT[dt], 1, state, layout)
    n = lengths if lengths is not None else [T] * B
    ln = torch.tensor(lengths, dtype=torch.int32).cuda() if lengths is not None else None
    scale = Dk ** -0.5
    o, s = gc.linear_attention(q, k, v, g, initial_state=s0, lengths=ln, return_state=True)
    torch.cuda.synchronize()
    d = lambda t: None if t is None else t.double().cpu()  # noqa: E731
    ro, rs = attn_def(d(q), d(k), d(v), g.cpu(), scale, d(s0), n)
    a = lambda t: None if t is None else t.double().cpu().abs()  # noqa: E731
    ao, as_ = attn_def(a(q), a(k), a(v), g.cpu(), scale, a(s0), n)
    f, fa, fs = bounds(DT[dt], T, Dk)
    near("o", o, ro, rounding(DT[dt], ro) + fa * ao)
    near("state", s, rs, fs * as_)
    near_norm("o", o, ro, 2 * f if dt != "f32" else 1e-6)
    near_norm("state", s, rs, 1e-6)
    assert torch.equal(o, gc.linear_attention(q, k, v, g, initial_state=s0, lengths=ln))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", ATTN, ids=lambda c: "x".join(map(str, c[:6])))
def test_linear_attention_backward(case, dt):
    B, T, Hk, H, Dk, Dv, state, lengths, layout = case
    print("attn_bwd", case, dt, flush=True)
    q, k, v, g, s0 = attn_inputs(B, T, Hk, H, Dk, Dv, DT[dt], 2, state, layout)
    n = lengths if lengths is not None else [T] * B
    ln = torch.tensor(lengths, dtype=torch.int32).cuda() if lengths is not None else None
    gen = torch.Generator().manual_seed(3)
    do = torch.randn(B, T, H, Dv, generator=gen).to(DT[dt]).cuda()
    ds = torch.randn(B, H, Dk, Dv, generator=gen).cuda() if state else None
    scale = 0.7 * Dk ** -0.5
    got = gc.linear_attention_backward(q, k, v, g, do, scale=scale, initial_state=s0, lengths=ln, dstate=ds)
    torch.cuda.synchronize()

    def grads(fn):
        leaves = [fn(t).requires_grad_() for t in (q, k, v)] + ([fn(s0).requires_grad_()] if state else [])
        o, s = attn_def(*leaves[:3], g.cpu(), scale, leaves[3] if state else None, n)
        loss = (o * fn(do)).sum() + ((s * fn(ds)).sum() if state else 0.0)
        return torch.autograd.grad(loss, leaves)

    ref, mag = grads(lambda t: t.double().cpu()), grads(lambda t: t.double().cpu().abs())
    f, fa, fs = bounds(DT[dt], T, max(Dk, Dv) + H // Hk)
    for name, y, r, m in zip(("dq", "dk", "dv"), got, ref, mag):
        near(name, y, r, rounding(DT[dt], r) + fa * m)
        near_norm(name, y, r, 2 * f if dt != "f32" else 1e-6)
    if state:
        near("dstate", got[3], ref[3], fs * mag[3])
        near_norm("dstate", got[3], ref[3], 1e-6)
    else:
        assert got[3] is None


def test_linear_attention_gradient_against_differences():
    # The loss is linear in each input, so a central difference is exact but for rounding.
    B, T, Hk, H, Dk, Dv = 1, 150, 1, 2, 32, 48
    q, k, v, g, s0 = attn_inputs(B, T, Hk, H, Dk, Dv, torch.float32, 4, True)
    gen = torch.Generator().manual_seed(5)
    do, ds = torch.randn(B, T, H, Dv, generator=gen).cuda(), torch.randn(B, H, Dk, Dv, generator=gen).cuda()
    grads = gc.linear_attention_backward(q, k, v, g, do, initial_state=s0, dstate=ds)

    def loss(q, k, v, s0):
        o, s = gc.linear_attention(q, k, v, g, initial_state=s0, return_state=True)
        return float((o.double() * do).sum() + (s.double() * ds).sum())

    ins = [q, k, v, s0]
    for i, gr in enumerate(grads):
        step = torch.randn(ins[i].shape, generator=gen).cuda()
        up, down = list(ins), list(ins)
        up[i], down[i] = ins[i] + step, ins[i] - step
        diff = (loss(*up) - loss(*down)) / 2
        want = float((gr.double() * step).sum())
        # Rounding: 2^-24 of the loss's terms, about 300 additions deep.
        size = float((do.abs().sum() + ds.abs().sum()) * 40)
        assert abs(diff - want) <= 300 * U32 * size, (i, diff, want)


def test_padding_tokens_do_not_reach_anything():
    # NaN and infinities past a sequence's length, in every input.
    B, T, H, D = 2, 100, 2, 64
    q, k, v, g, s0 = attn_inputs(B, T, H, H, D, D, torch.bfloat16, 6, True)
    ln = torch.tensor([70, 0], dtype=torch.int32).cuda()
    do = torch.randn(B, T, H, D, device="cuda").to(torch.bfloat16)
    clean = gc.linear_attention(q, k, v, g, initial_state=s0, lengths=ln, return_state=True)
    cleang = gc.linear_attention_backward(q, k, v, g, do, initial_state=s0, lengths=ln)
    for t in (q, k, v, do):
        t[0, 70:] = float("nan")
        t[1] = float("inf")
    for a, b in zip(clean, gc.linear_attention(q, k, v, g, initial_state=s0, lengths=ln, return_state=True)):
        assert torch.equal(a, b)
    for a, b in zip(cleang, gc.linear_attention_backward(q, k, v, g, do, initial_state=s0, lengths=ln)):
        assert torch.equal(a, b)
    assert (clean[0][0, 70:] == 0).all() and (clean[0][1] == 0).all() and torch.equal(clean[1][1], s0[1])


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("decay", ["0.0", "-inf", "-30.0", "-1e-6"])
def test_decays_at_the_ends_of_their_range(decay, dt):
    B, T, H, D = 1, 150, 2, 64
    q, k, v, g, s0 = attn_inputs(B, T, H, H, D, D, DT[dt], 7, True, decay=decay)
    o, s = gc.linear_attention(q, k, v, g, initial_state=s0, return_state=True)
    d = lambda t: t.double().cpu()  # noqa: E731
    ro, rs = attn_def(d(q), d(k), d(v), g.cpu(), D ** -0.5, d(s0), [T])
    ao, as_ = attn_def(d(q).abs(), d(k).abs(), d(v).abs(), g.cpu(), D ** -0.5, d(s0).abs(), [T])
    f, fa, fs = bounds(DT[dt], T, D)
    near("o", o, ro, rounding(DT[dt], ro) + fa * ao)
    near("state", s, rs, fs * as_)


def test_wide_ranges_in_fp16():
    # Scores and states far beyond fp16's largest value (and below its smallest), outputs inside it.
    for kq, kv in ((300.0, 1e-3), (1e-3, 300.0), (200.0, 1.0)):
        q, k, v, g, _ = attn_inputs(1, 150, 1, 1, 64, 64, torch.float16, 8, False)
        q, k, v = (q.float() * kq).half(), (k.float() * kq).half(), (v.float() * kv).half()
        scale = 1.0 / (kq * kq * kv)
        o, s = gc.linear_attention(q, k, v, g, scale=scale, return_state=True)
        d = lambda t: t.double().cpu()  # noqa: E731
        ro, rs = attn_def(d(q), d(k), d(v), g.cpu(), scale, None, [150])
        ao, as_ = attn_def(d(q).abs(), d(k).abs(), d(v).abs(), g.cpu(), scale, None, [150])
        f, fa, fs = bounds(torch.float16, 150, 64)
        near("o", o, ro, rounding(torch.float16, ro) + fa * ao)
        near("state", s, rs, fs * as_)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", [(1, 1, 1, 1, 1), (1, 8, 8, 64, 64), (3, 2, 6, 37, 81), (5, 1, 2, 128, 128),
                                  (2, 1, 1, 256, 256), (4, 3, 3, 9, 200)], ids=str)
@pytest.mark.parametrize("pool", [False, True])
def test_linear_attention_step(case, dt, pool):
    B, Hk, H, Dk, Dv = case
    print("attn_step", case, dt, pool, flush=True)
    gen = torch.Generator().manual_seed(9)
    x = torch.randn(B, 2 * Hk * Dk + H * Dv, generator=gen).to(DT[dt]).cuda()
    q, k, v = x.split([Hk * Dk, Hk * Dk, H * Dv], -1)
    q, k, v = q.unflatten(-1, (Hk, Dk)), k.unflatten(-1, (Hk, Dk)), v.unflatten(-1, (H, Dv))
    n = B + 3 if pool else B
    state = torch.randn(n, H, Dk, Dv, generator=gen).cuda()
    old = state.clone()
    g = (-torch.rand(H, generator=gen)).cuda()
    rows = torch.randperm(n, generator=gen)[:B].int() if pool else torch.arange(B).int()
    if pool and B > 1:
        rows[0], rows[1] = -1, n      # no state
    o = gc.linear_attention_step(q, k, v, g, state, slots=rows.cuda() if pool else None)
    torch.cuda.synchronize()
    r = H // Hk
    d = lambda t: t.double().cpu()  # noqa: E731
    want, ro, ao = d(old), torch.zeros(B, H, Dv, dtype=torch.float64), torch.zeros(B, H, Dv, dtype=torch.float64)
    mag = want.abs()
    for b in range(B):
        if not 0 <= int(rows[b]) < n:
            continue
        kk, qq = d(k[b]).repeat_interleave(r, 0), d(q[b]).repeat_interleave(r, 0)
        lam = torch.exp(d(g)).view(H, 1, 1)
        want[rows[b]] = lam * want[rows[b]] + kk[:, :, None] * d(v[b])[:, None, :]
        mag[rows[b]] = lam * mag[rows[b]] + kk.abs()[:, :, None] * d(v[b]).abs()[:, None, :]
        ro[b] = Dk ** -0.5 * (qq[:, :, None] * want[rows[b]]).sum(1)
        ao[b] = Dk ** -0.5 * (qq.abs()[:, :, None] * mag[rows[b]]).sum(1)
    near("state", state, want, 8 * U32 * mag)
    near("o", o, ro, rounding(DT[dt], ro) + (Dk + 16) * U32 * ao)
    gone = [b for b in range(B) if not 0 <= int(rows[b]) < n]
    assert (o[gone] == 0).all()


def test_steps_carry_on_from_a_prompt():
    B, T, Hk, H, Dk, Dv, extra = 2, 70, 1, 2, 64, 64, 5
    q, k, v, g, _ = attn_inputs(B, T + extra, Hk, H, Dk, Dv, torch.float32, 10, False)
    whole = gc.linear_attention(q, k, v, g)
    o, s = gc.linear_attention(q[:, :T], k[:, :T], v[:, :T], g, return_state=True)
    for t in range(T, T + extra):
        o1 = gc.linear_attention_step(q[:, t], k[:, t], v[:, t], g, s)
        near("step", o1, whole[:, t].double().cpu(), 2e-5 * whole.abs().max().item())
    near("prompt", o, whole[:, :T].double().cpu(), 2e-5 * whole.abs().max().item())


def test_state_rows_past_two_to_the_31():
    # 300000 states of 1 x 96 x 96 floats: the last ones start beyond 2^31 elements (11 GB).
    n, D = 300000, 96
    state = torch.empty(n, 1, D, D, dtype=torch.float32, device="cuda")
    state[-2:] = 1.0
    q, k, v = (torch.ones(2, 1, D, device="cuda") for _ in range(3))
    g = torch.zeros(1, device="cuda")
    o = gc.linear_attention_step(q, k, v, g, state, scale=1.0, slots=torch.tensor([n - 1, n - 2], dtype=torch.int32).cuda())
    assert (state[-2:] == 2.0).all() and (o == 2.0 * D).all()


# ---------------------------------------------------------------- RMS norm

NORM = [(1, 1), (3, 7), (2, 128), (5, 129), (1, 512), (4, 513), (3, 2048), (2, 2049), (1, 4096), (3, 5000), (2, 8192),
        (2, 16384), (2, 16385), (1, 20001), (17, 640)]


def norm_inputs(rows, C, dtype, seed, strided):
    gen = torch.Generator().manual_seed(seed)
    big = 1.0 + 20.0 * (torch.rand(C, generator=gen) < 0.02).float()
    wide = torch.randn(rows, C + (5 if strided else 0), generator=gen).to(dtype).cuda()
    x = wide[:, 3:3 + C] if strided else wide
    r = (torch.randn(rows, C, generator=gen) * big).to(dtype).cuda()
    w = (1.0 + 0.1 * torch.randn(C, generator=gen)).to(dtype).cuda()
    return x, r, w


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,C", NORM)
@pytest.mark.parametrize("residual", [False, True])
def test_rms_norm(rows, C, dt, residual):
    print("norm", rows, C, dt, residual, flush=True)
    x, r, w = norm_inputs(rows, C, DT[dt], 11, strided=residual)
    eps = 1e-5
    if residual:
        y, h = gc.rms_norm(x, w, residual=r, eps=eps)
        assert torch.equal(h.cpu(), (x.cpu().float() + r.cpu().float()).to(DT[dt]))
        hd = h.cpu().double()
    else:
        y = gc.rms_norm(x, w, eps=eps)
        hd = x.cpu().double()
    ref = w.cpu().double() * hd / torch.sqrt(hd.pow(2).mean(-1, keepdim=True) + eps)
    # Squares' sum: 16 additions a thread and 10 levels; then a root, a quotient and two products.
    near("y", y, ref, rounding(DT[dt], ref) + 48 * U32 * ref.abs())


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,C", NORM)
@pytest.mark.parametrize("block", [0, 32, 64, 128, 256])
def test_rms_norm_e4m3(rows, C, dt, block):
    print("norm e4m3", rows, C, dt, block, flush=True)
    x, r, w = norm_inputs(rows, C, DT[dt], 12, strided=False)
    if rows > 2:
        x[1], r[1] = 0, 0
    q, s, h = gc.rms_norm_e4m3(x, w, residual=r, block=block)
    assert q.dtype == torch.float8_e4m3fn and torch.equal(h, (x.float() + r.float()).to(DT[dt]))
    hd = h.cpu().double()
    y = w.cpu().double() * hd / torch.sqrt(hd.pow(2).mean(-1, keepdim=True) + 1e-6)
    blk = block or C
    nb = -(-C // blk)
    top = torch.nn.functional.pad(y, (0, nb * blk - C)).view(rows, nb, blk).abs().amax(-1).clamp(min=2.0 ** -100) / 448
    assert s.shape == (rows, nb)
    near("scales", s, top, 50 * U32 * top)
    scale = s.cpu().double().repeat_interleave(blk, 1)[:, :C]
    # One rounding to 4 significant bits (2^-9 among the subnormals, with 2^-6 the smallest normal).
    near("q", q.float() * 1.0, y / scale, (2.0 ** -4 * (y / scale).abs()).clamp(min=2.0 ** -10) + 50 * U32 * (y / scale).abs())


def test_rms_norm_nan_and_infinity():
    x = torch.randn(4, 300, device="cuda").to(torch.bfloat16)
    w = torch.ones(300, device="cuda", dtype=torch.bfloat16)
    x[1, 7], x[2, 299] = float("nan"), float("inf")
    y = gc.rms_norm(x, w)
    assert torch.isfinite(y[[0, 3]].float()).all() and torch.isnan(y[1]).all()
    assert torch.isnan(y[2, 299]) and (y[2, :299] == 0).all()
    q, s = gc.rms_norm_e4m3(x, w, block=64)
    assert torch.isnan(s[1]).all() and torch.isnan(s[2, 4]) and (q.float()[2, :256] == 0).all()
    assert torch.isfinite(q[[0, 3]].float()).all() and torch.isfinite(s[[0, 3]]).all()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,C", NORM + [(3000, 100), (2500, 300)])
@pytest.mark.parametrize("residual", [False, True])
def test_rms_norm_backward(rows, C, dt, residual):
    print("norm_bwd", rows, C, dt, residual, flush=True)
    dy, h, w = norm_inputs(rows, C, DT[dt], 13, strided=residual)
    dh = torch.randn(rows, C, generator=torch.Generator().manual_seed(14)).to(DT[dt]).cuda() if residual else None
    dx, dw = gc.rms_norm_backward(dy, h, w, eps=1e-5, dh=dh)
    hd, wd = h.cpu().double().requires_grad_(), w.cpu().double().requires_grad_()
    y = wd * hd / torch.sqrt(hd.pow(2).mean(-1, keepdim=True) + 1e-5)
    loss = (y * dy.cpu().double()).sum() + ((hd * dh.cpu().double()).sum() if residual else 0.0)
    rx, rw = torch.autograd.grad(loss, (hd, wd))
    hd = hd.detach()
    r = 1.0 / torch.sqrt(hd.pow(2).mean(-1, keepdim=True) + 1e-5)
    a = (wd.detach() * dy.cpu().double()).abs()
    mag = r * (a + hd.abs() * (r * r * (a * hd.abs()).mean(-1, keepdim=True))) + (dh.cpu().double().abs() if residual else 0.0)
    near("dx", dx, rx, rounding(DT[dt], rx) + 64 * U32 * mag)
    # A column's sum over the rows: (rows / 1024 + 100) additions.
    near("dw", dw, rw, rounding(DT[dt], rw) + (rows / 1024 + 160) * U32 * (dy.cpu().double() * hd * r).abs().sum(0))


def test_rms_norm_gradient_against_differences():
    x, _, w = norm_inputs(4, 96, torch.float32, 15, False)
    gen = torch.Generator().manual_seed(16)
    dy, step = torch.randn(4, 96, generator=gen).cuda(), torch.randn(4, 96, generator=gen).cuda()
    dx, dw = gc.rms_norm_backward(dy, x, w)
    e = 2.0 ** -6
    loss = lambda t, ww: float((gc.rms_norm(t, ww).double() * dy).sum())  # noqa: E731
    diff = (loss(x + e * step, w) - loss(x - e * step, w)) / (2 * e)
    # Third derivatives of a norm of about one, times e^2, over 4 x 96 values; and fp32's rounding over e.
    assert abs(diff - float((dx.double() * step).sum())) <= 384 * (e * e + 16 * U32 / e)
    ws = torch.randn(96, generator=gen).cuda()
    diff = (loss(x, w + ws) - loss(x, w - ws)) / 2
    assert abs(diff - float((dw.double() * ws).sum())) <= 384 * 64 * U32


# ---------------------------------------------------------------- causal conv

def conv_def(x, w, b, act, s0, lengths):
    B, T, C = x.shape
    K = w.shape[2]
    st = s0 if s0 is not None else torch.zeros(B, K - 1, C, dtype=torch.float64)
    xs = torch.cat([st, x], 1)
    z = torch.zeros(B, T, C, dtype=torch.float64) + (b if b is not None else 0.0)
    for j in range(K):
        z = z + xs[:, j:j + T] * w[:, 0, j]
    y = z * torch.sigmoid(z) if act else z
    live = torch.tensor([[t < n for t in range(T)] for n in lengths], dtype=torch.bool).view(B, T, 1)
    y = torch.where(live, y, torch.zeros((), dtype=torch.float64))
    return y, torch.stack([xs[i, n:n + K - 1] for i, n in enumerate(lengths)])


CONV = [  # B, T, C, K, bias, silu, state, lengths, strided
    (1, 1, 1, 1, False, False, False, None, False),
    (2, 5, 9, 1, True, True, False, [5, 2], False),
    (1, 1, 40, 4, True, True, True, None, False),
    (2, 2, 13, 4, True, False, True, [0, 2], True),
    (2, 33, 200, 2, False, True, True, [33, 1], True),
    (3, 100, 65, 3, True, True, False, [0, 100, 50], False),
    (1, 300, 136, 4, True, True, True, None, True),
    (2, 70, 2100, 4, True, True, False, None, False),
    (2, 64, 64, 5, True, True, True, [64, 63], False),
    (1, 65, 70, 8, False, True, False, None, True),
    (2, 130, 33, 15, True, False, True, [130, 7], False),
    (2, 200, 96, 31, True, True, True, [200, 128], True),
    (1, 20, 31, 31, True, True, False, None, False),
    (1, 3, 10, 64, True, True, True, None, False),
    (1, 150, 66, 64, False, True, False, [149], False),
]


def conv_inputs(B, T, C, K, bias, state, strided, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    wide = torch.randn(B, T, C + (3 if strided else 0), generator=gen).to(dtype).cuda()
    x = wide[..., 1:1 + C] if strided else wide
    w = (torch.randn(C, 1, K, generator=gen) * K ** -0.5).to(dtype).cuda()
    b = torch.randn(C, generator=gen).to(dtype).cuda() if bias else None
    s0 = torch.randn(B, K - 1, C, generator=gen).to(dtype).cuda() if state else None
    return x, w, b, s0


def dbl(t):
    return None if t is None else t.double().cpu()


def mag_(t):
    return None if t is None else t.double().cpu().abs()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", CONV, ids=lambda c: "x".join(map(str, c[:4])))
def test_dwconv1d_causal(case, dt):
    B, T, C, K, bias, act, state, lengths, strided = case
    print("conv", case, dt, flush=True)
    x, w, b, s0 = conv_inputs(B, T, C, K, bias, state, strided, DT[dt], 17)
    n = lengths if lengths is not None else [T] * B
    ln = torch.tensor(lengths, dtype=torch.int32).cuda() if lengths is not None else None
    if lengths is not None:
        for i, m in enumerate(lengths):
            x[i, m:] = float("nan")
    y, s = gc.dwconv1d_causal(x, w, b, "silu" if act else None, s0, ln, return_state=True)
    xd = torch.nan_to_num(dbl(x))
    ry, rs = conv_def(xd, dbl(w), dbl(b), act, dbl(s0), n)
    az, _ = conv_def(xd.abs(), mag_(w), mag_(b), False, mag_(s0), n)
    # |act'| <= 1.1; the 16-bit activation adds 2^-21 (|z| + 8) / 16 of the value.
    extra = 2.0 ** -20 * (1 + az) * ry.abs() if act and dt != "f32" else 4 * U32 * (1 + az) * ry.abs()
    near("y", y, ry, rounding(DT[dt], ry) + 1.1 * (K + 4) * U32 * az + extra)
    assert torch.equal(s.double().cpu(), rs)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", CONV, ids=lambda c: "x".join(map(str, c[:4])))
def test_dwconv1d_causal_backward(case, dt):
    B, T, C, K, bias, act, state, lengths, strided = case
    print("conv_bwd", case, dt, flush=True)
    x, w, b, s0 = conv_inputs(B, T, C, K, bias, state, strided, DT[dt], 18)
    n = lengths if lengths is not None else [T] * B
    ln = torch.tensor(lengths, dtype=torch.int32).cuda() if lengths is not None else None
    gen = torch.Generator().manual_seed(19)
    dy = torch.randn(B, T, C, generator=gen).to(DT[dt]).cuda()
    ds = torch.randn(B, K - 1, C, generator=gen).to(DT[dt]).cuda() if state else None
    if lengths is not None:
        for i, m in enumerate(lengths):
            x[i, m:] = float("nan")
            dy[i, m:] = float("inf")
    got = gc.dwconv1d_causal_backward(x, w, b, dy, "silu" if act else None, s0, ln, ds)
    torch.cuda.synchronize()
    live = torch.tensor([[t < m for t in range(T)] for m in n], dtype=torch.bool).view(B, T, 1)
    xd = torch.where(live, dbl(x), 0.0)
    dyd = torch.where(live, dbl(dy), 0.0)
    ins = [xd, dbl(w), dbl(b), dbl(s0)]
    leaves = [t.requires_grad_() for t in ins if t is not None]
    y, s = conv_def(ins[0], ins[1], ins[2], act, ins[3], n)
    loss = (y * dyd).sum() + ((s * dbl(ds)).sum() if state else 0.0)
    grads = iter(torch.autograd.grad(loss, leaves, allow_unused=True))
    ref = [None if t is None else next(grads) for t in ins]
    # Magnitudes: dz <= 1.1 |dy| (plus the error of z through act'', at most 1/2 of it), then the plain sums.
    az, _ = conv_def(xd.detach().abs(), mag_(w), mag_(b), False, mag_(s0), n)
    dz = (1.1 * dyd.abs()).detach()
    lost = dz * ((K + 8) * U32 * az + (2.0 ** -19 * (1 + az) if act and dt != "f32" else 8 * U32 * (1 + az)))
    st = mag_(s0) if state else torch.zeros(B, K - 1, C, dtype=torch.float64)
    xs = torch.cat([st, xd.detach().abs()], 1)
    wm = mag_(w)[:, 0]

    def spread(d):
        out = torch.zeros(B, T + K - 1, C, dtype=torch.float64)
        for j in range(K):
            out[:, j:j + T] += d * wm[:, j]
        return out

    fx = spread(dz) * (K + 6) * U32 + spread(lost)
    if state:
        for i, m in enumerate(n):
            fx[i, m:m + K - 1] += mag_(ds)[i] * 4 * U32
    near("dx", got[0], ref[0], rounding(DT[dt], ref[0]) + fx[:, K - 1:])
    terms = 64 + B * (T + K) / 64
    fw = torch.stack([((dz * terms * U32 + lost) * xs[:, j:j + T]).sum((0, 1)) for j in range(K)], -1).unsqueeze(1)
    near("dw", got[1], ref[1], rounding(DT[dt], ref[1]) + fw)
    if bias:
        near("db", got[2], ref[2], rounding(DT[dt], ref[2]) + (dz * terms * U32 + lost).sum((0, 1)))
    else:
        assert got[2] is None
    if state:
        rs0 = ref[3] if ref[3] is not None else torch.zeros(B, K - 1, C, dtype=torch.float64)
        near("dinitial", got[3], rs0, rounding(DT[dt], rs0) + fx[:, :K - 1])
    else:
        assert got[3] is None


def test_dwconv1d_causal_gradient_against_differences():
    x, w, b, s0 = conv_inputs(2, 40, 24, 4, True, True, False, torch.float32, 20)
    gen = torch.Generator().manual_seed(21)
    dy, ds = torch.randn(2, 40, 24, generator=gen).cuda(), torch.randn(2, 3, 24, generator=gen).cuda()
    grads = gc.dwconv1d_causal_backward(x, w, b, dy, "silu", s0, None, ds)

    def loss(x, w, b, s0):
        y, s = gc.dwconv1d_causal(x, w, b, "silu", s0, return_state=True)
        return float((y.double() * dy).sum() + (s.double() * ds).sum())

    e, ins = 2.0 ** -6, [x, w, b, s0]
    for i, gr in enumerate(grads):
        step = torch.randn(ins[i].shape, generator=gen).cuda()
        up, down = list(ins), list(ins)
        up[i], down[i] = ins[i] + e * step, ins[i] - e * step
        diff = (loss(*up) - loss(*down)) / (2 * e)
        # silu''' <= 0.6 and steps of z of a few e, over 2 x 40 x 24 outputs.
        assert abs(diff - float((gr.double() * step).sum())) <= 1920 * (4 * e * e + 16 * U32 / e), i


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", [(1, 1, 1, False), (1, 5, 2, True), (3, 1030, 4, True), (2, 64, 31, False), (2, 7, 64, True)],
                         ids=str)
@pytest.mark.parametrize("pool", [False, True])
def test_dwconv1d_causal_step(case, dt, pool):
    B, C, K, act = case
    print("conv_step", case, dt, pool, flush=True)
    gen = torch.Generator().manual_seed(22)
    x = torch.randn(B, C + 2, generator=gen).to(DT[dt]).cuda()[:, 1:1 + C]
    w = (torch.randn(C, 1, K, generator=gen) * K ** -0.5).to(DT[dt]).cuda()
    b = torch.randn(C, generator=gen).to(DT[dt]).cuda()
    n = B + 2 if pool else B
    state = torch.randn(n, K - 1, C, generator=gen).to(DT[dt]).cuda()
    old = state.clone()
    rows = torch.randperm(n, generator=gen)[:B].int() if pool else torch.arange(B).int()
    if pool and B > 1:
        rows[0] = -5
    y = gc.dwconv1d_causal_step(x, w, b, state, "silu" if act else None, slots=rows.cuda() if pool else None)
    torch.cuda.synchronize()
    want, ry, az = dbl(old), torch.zeros(B, C, dtype=torch.float64), torch.zeros(B, C, dtype=torch.float64)
    for i in range(B):
        if not 0 <= int(rows[i]) < n:
            continue
        xs = torch.cat([want[rows[i]], dbl(x[i:i + 1])], 0)
        z = dbl(b) + (xs * dbl(w)[:, 0].t()).sum(0)
        az[i] = mag_(b) + (xs.abs() * mag_(w)[:, 0].t()).sum(0)
        ry[i] = z * torch.sigmoid(z) if act else z
        want[rows[i]] = xs[1:]
    assert torch.equal(dbl(state), want)
    near("y", y, ry, rounding(DT[dt], ry) + 1.1 * (K + 4) * U32 * az + 2.0 ** -20 * (1 + az) * ry.abs())


# ---------------------------------------------------------------- empty calls, streams, graphs

def test_empty_sequences_and_batches():
    g = torch.zeros(2, device="cuda")
    z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    s0 = torch.randn(3, 2, 8, 8, device="cuda")
    o, s = gc.linear_attention(z(3, 0, 2, 8), z(3, 0, 2, 8), z(3, 0, 2, 8), g, initial_state=s0, return_state=True)
    assert o.shape == (3, 0, 2, 8) and torch.equal(s, s0)
    o, s = gc.linear_attention(z(3, 0, 2, 8), z(3, 0, 2, 8), z(3, 0, 2, 8), g, return_state=True)
    assert (s == 0).all()
    d = gc.linear_attention_backward(z(3, 0, 2, 8), z(3, 0, 2, 8), z(3, 0, 2, 8), g, z(3, 0, 2, 8), initial_state=s0, dstate=s0)
    assert torch.equal(d[3], s0)
    o, s = gc.linear_attention(z(0, 5, 2, 8), z(0, 5, 2, 8), z(0, 5, 2, 8), g, return_state=True)
    assert o.shape == (0, 5, 2, 8) and s.shape == (0, 2, 8, 8)
    assert gc.linear_attention_step(z(0, 2, 8), z(0, 2, 8), z(0, 2, 8), g, s0).shape == (0, 2, 8)
    assert gc.rms_norm(z(0, 16), z(16)).shape == (0, 16)
    dx, dw = gc.rms_norm_backward(z(0, 16), z(0, 16), z(16))
    assert dx.shape == (0, 16) and (dw == 0).all()
    c0 = torch.randn(2, 3, 16, device="cuda")
    y, s = gc.dwconv1d_causal(z(2, 0, 16), z(16, 1, 4), None, None, c0, return_state=True)
    assert y.shape == (2, 0, 16) and torch.equal(s, c0)
    dx, dw, db, ds = gc.dwconv1d_causal_backward(z(2, 0, 16), z(16, 1, 4), z(16), z(2, 0, 16), None, c0, None, c0)
    assert torch.equal(ds, c0) and (dw == 0).all() and (db == 0).all()
    assert gc.dwconv1d_causal(z(0, 4, 16), z(16, 1, 4)).shape == (0, 4, 16)


def test_side_stream_and_repeatability():
    q, k, v, g, s0 = attn_inputs(1, 500, 2, 4, 64, 64, torch.bfloat16, 23, True)
    do = torch.randn_like(v)
    side = torch.cuda.Stream()
    want = gc.linear_attention(q, k, v, g, initial_state=s0, return_state=True)
    wantg = gc.linear_attention_backward(q, k, v, g, do, initial_state=s0)
    x, r, w = norm_inputs(2000, 640, torch.bfloat16, 24, False)
    wantn = gc.rms_norm_backward(x, r, w)
    torch.cuda.synchronize()
    got = gc.linear_attention(q, k, v, g, initial_state=s0, return_state=True, stream=side)
    gotg = gc.linear_attention_backward(q, k, v, g, do, initial_state=s0, stream=side)
    gotn = gc.rms_norm_backward(x, r, w, stream=side)
    side.synchronize()
    for a, b in zip((*want, *wantg, *wantn), (*got, *gotg, *gotn)):
        assert torch.equal(a, b)


def test_graph_replays():
    # A prompt's pass, its gradients and a token, captured and replayed with other inputs.
    q, k, v, g, s0 = attn_inputs(1, 400, 2, 4, 64, 64, torch.bfloat16, 25, True)
    do = torch.randn_like(v)
    x, r, w = norm_inputs(300, 256, torch.bfloat16, 26, False)
    cx, cw, cb, cs = conv_inputs(2, 90, 48, 4, True, True, False, torch.bfloat16, 27)

    def work():
        o, s = gc.linear_attention(q, k, v, g, initial_state=s0, return_state=True)
        d = gc.linear_attention_backward(q, k, v, g, do, initial_state=s0, dstate=s)
        o1 = gc.linear_attention_step(q[:, -1], k[:, -1], v[:, -1], g, s)
        y, h = gc.rms_norm(x, w, residual=r)
        n = gc.rms_norm_backward(y, h, w)
        c, st = gc.dwconv1d_causal(cx, cw, cb, "silu", cs, return_state=True)
        e = gc.dwconv1d_causal_backward(cx, cw, cb, c, "silu", cs)
        c1 = gc.dwconv1d_causal_step(cx[:, 0], cw, cb, st, "silu")
        return [o, s, *d, o1, y, h, *n, c, st, *e, c1]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work()
    for i in range(4):
        for t in (q, k, v, do, x, r, cx):
            t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(100 + i)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        for j, (a, b) in enumerate(zip(got, work())):
            assert torch.equal(a, b), (i, j)
