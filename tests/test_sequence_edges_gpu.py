"""Edges of the sequence operators: precision of scores and states, borders of roundings, slow
decays, non-finite values, streams and sizes near the largest ones.

u = 2^-24 is the relative error of one fp32 rounding; the other tolerances stand beside their
tests, counted from the roundings that a result passes.
"""
import pytest
import torch

import depthwise_convolution_gconv_amd as gc
from test_sequence_gpu import DT, U32, attn_def, attn_inputs, bounds, near, near_norm, rounding

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- precision of scores and states

@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_scores_and_states_are_finer_than_the_outputs(dt):
    # Few positive terms, so that one rounding of a score or a state shows in the output.  Scores, and
    # the state where a query meets it, have 16 bits (2^-16 of a term), sums fp32; the output is
    # rounded once, the gradients of k and v meet one state more.
    B, T, Dk, Dv = 3000, 3, 2, 4
    gen = torch.Generator().manual_seed(1)
    pos = lambda *s: 1.0 + torch.rand(*s, generator=gen)  # noqa: E731
    q, k, v, do = (pos(B, T, 1, d).to(DT[dt]).cuda() for d in (Dk, Dk, Dv, Dv))
    s0, ds = pos(B, 1, Dk, Dv).cuda(), pos(B, 1, Dk, Dv).cuda()
    g = torch.full((1,), -0.1).cuda()
    o, s = gc.linear_attention(q, k, v, g, scale=0.75, initial_state=s0, return_state=True)
    got = gc.linear_attention_backward(q, k, v, g, do, scale=0.75, initial_state=s0, dstate=ds)
    leaves = [t.double().cpu().requires_grad_() for t in (q, k, v, s0)]
    ro, rs = attn_def(*leaves[:3], g.cpu(), 0.75, leaves[3], [T] * B)
    ref = torch.autograd.grad((ro * do.double().cpu()).sum() + (rs * ds.double().cpu()).sum(), leaves)
    for name, y, r in zip(("o", "dq", "dk", "dv"), (o, *got), (ro.detach(), *ref)):
        near(name, y, r, rounding(DT[dt], r) + (1.02 * 2.0 ** -16 + (T + Dv + 24) * U32) * r)
    near("state", s, rs.detach(), (T + 8) * U32 * rs.detach())
    near("dinitial", got[3], ref[3], (T + 8) * U32 * ref[3])


def test_bf16_error_is_that_of_the_outputs_rounding():
    # Terms of either sign: errors of 2^-16 of a term stay 2^-16 of the sum, beside a rounding whose
    # 2-norm is above 2^-10 of it; together less than a tenth more.
    B, T, H, D = 2, 300, 2, 64
    q, k, v, g, s0 = attn_inputs(B, T, H, H, D, D, torch.bfloat16, 2, True)
    do = torch.randn(B, T, H, D, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    o = gc.linear_attention(q, k, v, g, initial_state=s0)
    got = gc.linear_attention_backward(q, k, v, g, do, initial_state=s0)
    leaves = [t.double().cpu().requires_grad_() for t in (q, k, v)]
    ro, _ = attn_def(*leaves, g.cpu(), D ** -0.5, s0.double().cpu(), [T] * B)
    ref = torch.autograd.grad((ro * do.double().cpu()).sum(), leaves)
    for name, y, r in zip(("o", "dq", "dk", "dv"), (o, *got), (ro.detach(), *ref)):
        own = float((r.bfloat16().double() - r).norm())
        assert float((y.double().cpu() - r).norm()) <= 1.1 * own, name


# ---------------------------------------------------------------- e4m3

@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("C", [64, 300, 2000, 5000, 20001])
@pytest.mark.parametrize("block", [0, 32, 64, 256])
def test_e4m3_is_the_quotient(C, block, dt):
    # Few distinct values: with 448 in every scale's columns many quotients lie on a border between
    # two e4m3 numbers.  All values are exact in every dtype and so are the sums of their squares
    # (below 2^24), so the fp32 norm of the same rows has the same y, and q = e4m3(y / scale) bit for bit.
    gen = torch.Generator().manual_seed(4)
    x = torch.zeros(200, C)
    x[:, :40] = torch.randint(-112, 113, (200, 40), generator=gen).float() * 4
    x[:, 3], x[:, 33] = 448.0, -448.0
    w = torch.ones(C)
    y = gc.rms_norm(x.cuda(), w.cuda())
    q, s = gc.rms_norm_e4m3(x.to(DT[dt]).cuda(), w.to(DT[dt]).cuda(), block=block)
    blk = block or C
    nb = -(-C // blk)
    top = torch.nn.functional.pad(y.cpu(), (0, nb * blk - C)).view(200, nb, blk).abs().amax(-1)
    want = top.clamp(min=2.0 ** -100) / 448.0
    assert torch.equal(s.cpu(), want)
    want = (y.cpu() / want.repeat_interleave(blk, 1)[:, :C]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    assert torch.equal(q.float().cpu(), want.float())


# ---------------------------------------------------------------- the longest sequences

@pytest.fixture
def much_memory():
    """Gives tens of GB back to the device after the test."""
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def test_last_segment_of_the_longest_sequence(much_memory):
    # The largest T, where the last segment's rounded-up end passes 2^31.  All inputs are one value
    # at stride 0 and the decay is 1/2, so every sum is 2 but near its start, all of it exact.
    T = 2 ** 31 - 1 - 4096
    one = torch.ones(1, 1, 1, 1, dtype=torch.bfloat16, device="cuda").expand(1, T, 1, 1)
    g = torch.full((1,), 0.5, dtype=torch.float64).log().float().cuda()
    o, s = gc.linear_attention(one, one, one, g, scale=1.0, return_state=True)
    assert o.flatten()[:3].tolist() == [1.0, 1.5, 1.75]
    assert abs(float(s) - 2.0) <= 16 * U32
    assert bool((o.view(-1)[16:] == 2.0).all())
    del o
    dq, dk, dv, _ = gc.linear_attention_backward(one, one, one, g, one, scale=1.0)
    assert dq.flatten()[:3].tolist() == [1.0, 1.5, 1.75] and bool((dq.view(-1)[16:] == 2.0).all())
    for d in (dk, dv):
        assert d.flatten()[-3:].tolist() == [1.75, 1.5, 1.0] and bool((d.view(-1)[:-16] == 2.0).all())


# ---------------------------------------------------------------- other streams

def stream_calls():
    """Every entry point as a function of the stream it is given, with its inputs ready."""
    q, k, v, g, s0 = attn_inputs(1, 500, 2, 4, 64, 64, torch.bfloat16, 5, True)
    do, r = torch.randn_like(v), torch.randn(2000, 640, device="cuda").bfloat16()
    x, w = torch.randn(2000, 640, device="cuda").bfloat16(), torch.ones(640, device="cuda", dtype=torch.bfloat16)
    cx, cw = torch.randn(2, 400, 640, device="cuda").bfloat16(), torch.randn(640, 1, 4, device="cuda").bfloat16()
    cs = torch.randn(2, 3, 640, device="cuda").bfloat16()

    def fresh(t):
        t = t.clone()
        torch.cuda.synchronize()
        return t

    calls = {
        "attn": lambda st: gc.linear_attention(q, k, v, g, initial_state=s0, return_state=True, stream=st),
        "attn_bwd": lambda st: gc.linear_attention_backward(q, k, v, g, do, initial_state=s0, stream=st),
        "attn_step": lambda st: gc.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], g, fresh(s0), stream=st),
        "norm": lambda st: gc.rms_norm(x, w, residual=r, stream=st),
        "norm_e4m3": lambda st: [t.view(torch.uint8) for t in gc.rms_norm_e4m3(x, w, residual=r, block=64, stream=st)],
        "norm_bwd": lambda st: gc.rms_norm_backward(x, r, w, stream=st),
        "conv": lambda st: gc.dwconv1d_causal(cx, cw, None, "silu", cs, return_state=True, stream=st),
        "conv_bwd": lambda st: gc.dwconv1d_causal_backward(cx, cw, None, cx, "silu", cs, stream=st),
        "conv_step": lambda st: gc.dwconv1d_causal_step(cx[:, 0], cw, None, fresh(cs), "silu", stream=st),
    }
    torch.cuda.synchronize()
    return calls


@pytest.mark.parametrize("name", ["attn", "attn_bwd", "norm", "norm_bwd", "conv", "conv_bwd"])
def test_a_side_stream_leaves_memory_alone_that_the_current_one_still_reads(name):
    # The current stream has freed blocks of every size the call needs, and reads them late.
    call = stream_calls()[name]
    want = [t.clone() for t in call(None) if t is not None]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    sizes = {1 << 20, 12 << 20} | {t.numel() * t.element_size() for t in want}
    kept = [torch.randint(0, 255, (n,), dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    expect = [t.clone() for t in kept]
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)
    late = [t.clone() for t in kept]      # after the sleep
    del kept
    got = call(side)
    side.synchronize()
    torch.cuda.synchronize()
    for a, b in zip(late, expect):
        assert torch.equal(a, b)
    for a, b in zip(want, [t for t in got if t is not None]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", ["attn", "attn_bwd", "norm", "norm_bwd", "conv", "conv_bwd"])
def test_outputs_of_a_side_stream_are_kept_for_the_current_one(name):
    # The current stream waits for the side one and reads the outputs late; they are freed before
    # that, and the side stream makes the next outputs at once.
    call, side = stream_calls()[name], torch.cuda.Stream()
    want = [t.clone() for t in call(None) if t is not None]
    torch.cuda.synchronize()
    got = [t for t in call(side) if t is not None]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(50_000_000)
    late = [t.clone() for t in got]
    del got
    with torch.cuda.stream(side):
        junk = [torch.full_like(t, 3.0) for t in want for _ in range(3)]
    call(side)
    torch.cuda.synchronize()
    for a, b in zip(want, late):
        assert torch.equal(a, b)
    del junk


def test_every_entry_point_takes_a_stream():
    side = torch.cuda.Stream()
    for name, call in stream_calls().items():
        want = call(None)
        torch.cuda.synchronize()
        got = call(side)
        side.synchronize()
        torch.cuda.synchronize()
        for a, b in zip(want if isinstance(want, (tuple, list)) else (want,), got if isinstance(got, (tuple, list)) else (got,)):
            assert (a is None and b is None) or torch.equal(a, b), name


# ---------------------------------------------------------------- slow decays

@pytest.mark.parametrize("H,segments", [(768, 1), (96, 8), (85, 9), (1, 512)])
@pytest.mark.parametrize("decay", [-1e-6, -3e-7, -4e-8, 3e-7])
def test_a_state_fades_over_many_tokens(H, segments, decay):
    # Keys of zero leave the initial state to fade: lam^T S_0, and lam^(t+1) S_0 as outputs, with no
    # sum in them.  A segment rounds its state's scale and its product (2 u), a join of two segments
    # the power, the product and the sum (3 u), an output the two powers, the product of the scales,
    # the state's parts, and its own value (8 u).
    T = 65536
    shape = (1, T, H, H, 1, 1)
    assert gc.linear_attention_workspace(shape, torch.float32) in ((0,) if segments == 1 else
                                                                   (4 * H * segments, -(-4 * H * segments // 256) * 256))
    one, zero = (torch.full((1, 1, 1, 1), x, device="cuda").expand(1, T, H, 1) for x in (1.0, 0.0))
    g = torch.full((H,), decay).cuda()
    s0 = 1.0 + torch.rand(1, H, 1, 1, generator=torch.Generator().manual_seed(6)).cuda()
    o, s = gc.linear_attention(one, zero, zero, g, scale=1.0, initial_state=s0, return_state=True)
    gd, joins = g.double(), min(segments, 8)
    want = s0.double() * torch.exp(gd * T).view(1, H, 1, 1)
    assert float(((s - want).abs() / want).max()) <= (4 + 3 * joins) * U32
    t = torch.arange(1, T + 1, device="cuda", dtype=torch.float64).view(1, T, 1, 1)
    want = s0.double().view(1, 1, H, 1) * torch.exp(gd.view(1, 1, H, 1) * t)
    assert float(((o - want).abs() / want).max()) <= (12 + 3 * joins) * U32


# ---------------------------------------------------------------- values that are not finite

# Where a value of an input that is not finite shows: in the outputs' rows before its token, its
# own, and later ones; in its own column or in all.  What the rows do not name stays bit for bit.
REACH = {
    ("q", "o"): ("own", "all"), ("k", "o"): ("own later", "all"), ("v", "o"): ("own later", "col"),
    ("q", "dk"): ("before own", "col"), ("q", "dv"): ("before own", "all"),
    ("k", "dq"): ("own later", "col"), ("k", "dv"): ("own", "all"),
    ("v", "dq"): ("own later", "all"), ("v", "dk"): ("own", "all"),
    ("do", "dq"): ("own", "all"), ("do", "dk"): ("before own", "all"), ("do", "dv"): ("before own", "col"),
}


@pytest.mark.parametrize("value", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("T,token,D", [(100, 50, 64), (100, 63, 33), (700, 130, 128), (2600, 2111, 40)])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_values_that_are_not_finite_reach_no_token_they_must_not(dt, T, token, D, value):
    q, k, v, g, s0 = attn_inputs(1, T, 1, 1, D, D, DT[dt], 7, True, decay="-0.01")
    do = torch.randn(1, T, 1, D, generator=torch.Generator().manual_seed(8)).to(DT[dt]).cuda()
    ins = {"q": q, "k": k, "v": v, "do": do}

    def run():
        o, s = gc.linear_attention(q, k, v, g, initial_state=s0, return_state=True)
        dq, dk, dv, ds = gc.linear_attention_backward(q, k, v, g, do, initial_state=s0)
        return {"o": o, "dq": dq, "dk": dk, "dv": dv}, s, ds

    clean, clean_s, clean_ds = run()
    col = D - 2
    for name, t in ins.items():
        kept = t[0, token, 0, col].clone()
        t[0, token, 0, col] = float(value)
        got, s, ds = run()
        t[0, token, 0, col] = kept
        for out, y in got.items():
            rows, cols = REACH.get((name, out), ("", ""))
            hit = torch.zeros(T, D, dtype=torch.bool, device="cuda")
            c = slice(col, col + 1) if cols == "col" else slice(0, D)
            for part, r in (("before", slice(0, token)), ("own", slice(token, token + 1)), ("later", slice(token + 1, T))):
                if part in rows:
                    hit[r, c] = True
            y, ref = y[0, :, 0], clean[out][0, :, 0]
            assert torch.equal(y[~hit], ref[~hit]), (name, out)
            assert not torch.isfinite(y[hit]).any(), (name, out)
        # The state: a row of it for k, a column for v; the initial state's gradient likewise for q and do.
        for y, ref, row, column in ((s[0, 0], clean_s[0, 0], "k", "v"), (ds[0, 0], clean_ds[0, 0], "q", "do")):
            hit = torch.zeros(D, D, dtype=torch.bool, device="cuda")
            if name == row:
                hit[col] = True
            if name == column:
                hit[:, col] = True
            assert torch.equal(y[~hit], ref[~hit]) and not torch.isfinite(y[hit]).any(), name


def test_shares_of_value_heads_past_a_launch(much_memory):
    # 2^24 tokens of 256 columns are 2^32 threads for the sum over two value heads: two launches.
    # All inputs are one value at stride 0 and the decay is 1/2, so a head's share is 2 but near an end.
    T, D = 2 ** 24, 256
    one = lambda h, d: torch.ones(1, 1, 1, 1, dtype=torch.bfloat16, device="cuda").expand(1, T, h, d)  # noqa: E731
    g = torch.full((2,), 0.5, dtype=torch.float64).log().float().cuda()
    dense = torch.ones(1, 1, 1, D, dtype=torch.bfloat16, device="cuda").expand(1, T, 1, D)
    dq, dk, dv, _ = gc.linear_attention_backward(dense, dense, one(2, 1), g, one(2, 1), scale=1.0)
    assert bool((dq[0, 16:] == 4.0).all()) and bool((dk[0, :-16] == 4.0).all())
    assert bool((dq[0, 0] == 2.0).all()) and bool((dk[0, -1] == 2.0).all())
    assert bool((dv[0, :-16] == 2.0 * D).all())


def test_norm_of_more_rows_than_a_launch_takes(much_memory):
    # 16 rows of one column share a workgroup: 2^28 rows are 2^32 threads.  A row of one value has
    # itself as its norm: y is its sign, h twice the value, and the scale of 448 is |y| / 448.
    rows = 2 ** 28 + 5
    x = torch.ones(rows, 1, dtype=torch.float16, device="cuda")
    x[::3] = -1.5
    x[-1] = 0.0
    w = torch.ones(1, dtype=torch.float16, device="cuda")
    y, h = gc.rms_norm(x, w, residual=x)
    assert torch.equal(y, x.sign()) and torch.equal(h, 2 * x)
    del y, h
    q, s, h = gc.rms_norm_e4m3(x, w, residual=x)
    assert torch.equal(h, 2 * x)
    del h
    sign = x.sign()
    assert torch.equal(q.to(torch.float16), 448.0 * sign)
    # The root and the quotient are one rounding each, eps 1e-6 / 8 of a value of 2 at most.
    assert bool(((s[:-1] * 448.0 - 1.0).abs() <= 1.3e-7 + 6 * U32).all()) and float(s[-1]) == float(torch.tensor(2.0 ** -100) / 448.0)


def test_norm_gradient_of_more_rows_and_columns_than_a_launch_takes(much_memory):
    # Rows past 16384 columns take 1024 threads each: 2^22 rows are 2^32 threads (dx of 137 GB, from
    # one row at stride 0).
    rows, C = 2 ** 22 + 3, 16385
    w = torch.ones(C, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator().manual_seed(9)
    dy, h = (torch.randn(1, C, generator=gen).bfloat16().cuda() for _ in range(2))
    first, _ = gc.rms_norm_backward(dy, h, w)
    if torch.cuda.mem_get_info()[0] > 160 << 30:
        dx, _ = gc.rms_norm_backward(dy.expand(rows, C), h.expand(rows, C), w)
        for r in range(0, rows, 1 << 19):
            assert bool((dx[r:r + (1 << 19)] == first).all()), r
        del dx
        torch.cuda.empty_cache()
    # 2^22 columns in 1024 rows of partial sums are 2^32 threads.
    rows, C = 1024, 2 ** 22
    one = torch.ones(1, 1, dtype=torch.bfloat16, device="cuda").expand(1, C).contiguous()
    dx, dw = gc.rms_norm_backward(one.expand(rows, C), one.expand(rows, C), one[0])
    assert bool((dw == 1024.0).all()) and bool((dx.abs() <= 2e-6).all())


# ---------------------------------------------------------------- joined segments

def grads_def(leaves, g, scale, n, do, ds):
    o, s = attn_def(*leaves[:3], g, scale, leaves[3], n)
    return [o.detach(), s.detach(), *torch.autograd.grad((o * do).sum() + (s * ds).sum(), leaves)]


SEGMENTS = [  # B, T, H, Dk, Dv, lengths, segments: to eight the walks add the states up, past that a scan does
    (1, 300, 1, 32, 32, None, 2),
    (1, 1000, 1, 64, 64, None, 8),
    (1, 1000, 2, 48, 96, [997], 8),
    (1, 1100, 1, 64, 64, None, 9),
    (2, 1150, 1, 40, 128, [1150, 500], 9),      # one ends segments before the last
    (1, 2500, 1, 33, 20, [2449], 20),
]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", SEGMENTS, ids=lambda c: "x".join(map(str, c[:5])) + f"-{c[6]}")
def test_segments_with_a_visible_carry(case, dt):
    # A decay of -1e-3 leaves nine tenths of a state after a segment of 128 tokens.  Tolerances as in
    # test_sequence_gpu.py.
    B, T, H, Dk, Dv, lengths, segments = case
    q, k, v, g, s0 = attn_inputs(B, T, H, H, Dk, Dv, DT[dt], 31, True, decay="-0.001")
    n = lengths if lengths is not None else [T] * B
    ln = torch.tensor(lengths, dtype=torch.int32).cuda() if lengths is not None else None
    gen = torch.Generator().manual_seed(32)
    do, ds = torch.randn(B, T, H, Dv, generator=gen).to(DT[dt]).cuda(), torch.randn(B, H, Dk, Dv, generator=gen).cuda()
    one = -(-4 * B * H * segments * Dk * Dv // 256) * 256
    shape = (B, T, H, H, Dk, Dv)
    assert gc.linear_attention_workspace(shape, DT[dt]) == one
    assert gc.linear_attention_workspace(shape, DT[dt], backward=True) == 3 * one
    o, s = gc.linear_attention(q, k, v, g, initial_state=s0, lengths=ln, return_state=True)
    got = gc.linear_attention_backward(q, k, v, g, do, initial_state=s0, lengths=ln, dstate=ds)
    torch.cuda.synchronize()
    ref, mag = (grads_def([fn(t).requires_grad_() for t in (q, k, v, s0)], g.cpu(), Dk ** -0.5, n, fn(do), fn(ds))
                for fn in (lambda t: t.double().cpu(), lambda t: t.double().cpu().abs()))
    f, fa, fs = bounds(DT[dt], T, max(Dk, Dv) + 1)
    for name, y, r, m in zip(("o", "state", "dq", "dk", "dv", "dinitial"), (o, s, *got), ref, mag):
        if y.dtype == torch.float32:
            near(name, y, r, fs * m + (rounding(DT[dt], r) if dt == "f32" else 0.0))
            near_norm(name, y, r, 1e-6)
        else:
            near(name, y, r, rounding(DT[dt], r) + fa * m)
            near_norm(name, y, r, 2 * f)


# ---------------------------------------------------------------- lengths, strides, threads

def test_lengths_outside_their_range():
    # Below 0 as 0, above T as T.
    lengths, meant = (torch.tensor(x, dtype=torch.int32).cuda() for x in ([-5, 40, 1000, -2 ** 31, 2 ** 31 - 1],
                                                                       [0, 40, 70, 0, 70]))
    q, k, v, g, s0 = attn_inputs(5, 70, 1, 2, 40, 24, torch.bfloat16, 33, True)
    x, w, c0 = torch.randn(5, 70, 48, device="cuda"), torch.randn(48, 1, 4, device="cuda"), torch.randn(5, 3, 48, device="cuda")
    x9, w9, c9 = x, torch.randn(48, 1, 9, device="cuda"), torch.randn(5, 8, 48, device="cuda")

    def run(ln):
        return [*gc.linear_attention(q, k, v, g, initial_state=s0, lengths=ln, return_state=True),
                *gc.linear_attention_backward(q, k, v, g, v, initial_state=s0, lengths=ln),
                *gc.dwconv1d_causal(x, w, None, "silu", c0, ln, return_state=True),
                *gc.dwconv1d_causal_backward(x, w, w[:, 0, 0].contiguous(), x, "silu", c0, ln, c0),
                *gc.dwconv1d_causal(x9, w9, None, None, c9, ln, return_state=True),
                *gc.dwconv1d_causal_backward(x9, w9, w[:, 0, 0].contiguous(), x9, None, c9, ln, c9)]

    for i, (a, b) in enumerate(zip(run(lengths), run(meant))):
        assert torch.equal(a, b), i


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_strided_gradients_of_outputs(dt):
    # Views of wider tensors against their copies, bit for bit: the same arithmetic on the same values.
    gen = torch.Generator().manual_seed(34)
    rnd = lambda *s: torch.randn(*s, generator=gen).to(DT[dt]).cuda()  # noqa: E731
    q, k, v, g, s0 = attn_inputs(2, 90, 2, 4, 40, 37, DT[dt], 35, True)
    for do in (rnd(2, 90, 4, 40)[..., 1:38], rnd(2, 4, 90, 37).transpose(1, 2), rnd(2, 1, 4, 37).expand(2, 90, 4, 37)):
        a = gc.linear_attention_backward(q, k, v, g, do, initial_state=s0)
        b = gc.linear_attention_backward(q, k, v, g, do.contiguous(), initial_state=s0)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    for K in (3, 9):
        x, w, b0 = rnd(2, 90, 48), rnd(48, 1, K), rnd(48)
        for dy in (rnd(2, 90, 53)[..., 2:50], rnd(90, 2, 48).transpose(0, 1), rnd(2, 1, 48).expand(2, 90, 48)):
            a = gc.dwconv1d_causal_backward(x, w, b0, dy, "silu")[:3]
            b = gc.dwconv1d_causal_backward(x, w, b0, dy.contiguous(), "silu")[:3]
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    for C in (37, 600, 3000, 9000, 17000):
        dy, h, dh = (rnd(6, C + 5)[:, i:i + C] for i in (1, 2, 3))
        w = rnd(C)
        a = gc.rms_norm_backward(dy, h, w, dh=dh)
        b = gc.rms_norm_backward(dy.contiguous(), h.contiguous(), w, dh=dh.contiguous())
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_host_threads():
    # Each on a stream of its own, with calls that are refused in between: results and error texts
    # are the thread's own.
    import threading

    sizes, out, errors = (96, 160), {}, []

    def inputs(i):
        q, k, v, g, s0 = attn_inputs(1, 300 + 50 * i, 1, 2, 64, 64, torch.bfloat16, 36 + i, True)
        x = torch.randn(500, sizes[i], generator=torch.Generator().manual_seed(38 + i)).bfloat16().cuda()
        return q, k, v, g, s0, x, torch.ones(sizes[i], device="cuda", dtype=torch.bfloat16)

    def run(q, k, v, g, s0, x, w):
        return [*gc.linear_attention(q, k, v, g, initial_state=s0, return_state=True),
                *gc.linear_attention_backward(q, k, v, g, v, initial_state=s0),
                *gc.rms_norm(x, w, residual=x), *gc.rms_norm_backward(x, x, w)]

    ins = [inputs(i) for i in range(2)]
    want = [run(*ins[i]) for i in range(2)]
    torch.cuda.synchronize()

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    out[i] = run(*ins[i])
                    with pytest.raises(gc.GconvError, match=f"{i + 17} columns a scale"):
                        gc.rms_norm_e4m3(ins[i][5], ins[i][6], block=i + 17)
                torch.cuda.current_stream().synchronize()
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(out[i], want[i]))
