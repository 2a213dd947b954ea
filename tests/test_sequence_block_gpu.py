"""The mixing block made of the sequence operators, and linear attention over enough tokens
that a scan joins its segments.

Tolerances of linear attention as in test_sequence_gpu.py.  The block is compared in fp32: its
operators sum in fp32 and round nothing else, so that against the same block in 64 bits each
stage adds a relative 2-norm error of a few 2^-24 times the depth of its sums (width 96, heads
of 32, 150 tokens: below 300 2^-24 = 1.8e-5 for each), and five stages with gains near one stay
below 2e-4 forward and, twice as many stages, 4e-4 backward.
"""
import pytest
import torch

import depthwise_convolution_gconv_amd as gc
from depthwise_convolution_gconv_amd.sequence_block import SequenceBlock
from test_sequence_gpu import DT, attn_def, attn_inputs, bounds, near, rounding

pytestmark = pytest.mark.gpu


def off(y, r):
    y = y.detach().double().cpu()
    assert y.shape == r.shape and torch.isfinite(y).all()
    return float((y - r).norm() / r.norm())


LONG = [  # B, T, Hk, H, Dk, Dv, lengths: ten segments, which a scan joins; the last eight, which the walks add up
    (1, 2600, 1, 1, 64, 64, None),
    (2, 2500, 1, 1, 48, 96, [2500, 1300]),     # one sequence ends segments before the last
    (1, 2400, 1, 2, 128, 40, [2370]),
]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", LONG, ids=lambda c: "x".join(map(str, c[:6])))
def test_many_segments(case, dt):
    B, T, Hk, H, Dk, Dv, lengths = case
    print("long", case, dt, flush=True)
    q, k, v, g, s0 = attn_inputs(B, T, Hk, H, Dk, Dv, DT[dt], 11, True)
    n = lengths if lengths is not None else [T] * B
    ln = torch.tensor(lengths, dtype=torch.int32).cuda() if lengths is not None else None
    gen = torch.Generator().manual_seed(12)
    do = torch.randn(B, T, H, Dv, generator=gen).to(DT[dt]).cuda()
    ds = torch.randn(B, H, Dk, Dv, generator=gen).cuda()
    scale = Dk ** -0.5
    assert gc.linear_attention_workspace((B, T, Hk, H, Dk, Dv), DT[dt]) >= 8 * 4 * B * H * Dk * Dv
    o, s = gc.linear_attention(q, k, v, g, initial_state=s0, lengths=ln, return_state=True)
    got = gc.linear_attention_backward(q, k, v, g, do, initial_state=s0, lengths=ln, dstate=ds)
    torch.cuda.synchronize()

    def run(fn):
        leaves = [fn(t).requires_grad_() for t in (q, k, v, s0)]
        ro, rs = attn_def(*leaves[:3], g.cpu(), scale, leaves[3], n)
        loss = (ro * fn(do)).sum() + (rs * fn(ds)).sum()
        return [ro.detach(), rs.detach(), *torch.autograd.grad(loss, leaves)]

    ref, mag = run(lambda t: t.double().cpu()), run(lambda t: t.double().cpu().abs())
    f, fa, fs = bounds(DT[dt], T, max(Dk, Dv) + H // Hk)
    for name, y, r, m in zip(("o", "state", "dq", "dk", "dv", "dinitial"), (o, s, *got), ref, mag):
        if y.dtype == torch.float32:
            near(name, y, r, fs * m + (rounding(DT[dt], r) if dt == "f32" else 0.0))
        else:
            near(name, y, r, rounding(DT[dt], r) + fa * m)


@pytest.mark.parametrize("decay", ["0.001", "-0.02", "-3.0"])
def test_scale_of_the_state(decay):
    # Growing, slowly and quickly fading states: the walk keeps the state's scale apart.
    B, T, H, D = 1, 2600, 1, 32
    q, k, v, g, s0 = attn_inputs(B, T, H, H, D, D, torch.float32, 13, True, decay=decay)
    for tokens in (100, T):      # one segment, many
        o, s = gc.linear_attention(q[:, :tokens], k[:, :tokens], v[:, :tokens], g, initial_state=s0, return_state=True)
        d = lambda t: t.double().cpu()  # noqa: E731
        a = lambda t: t.double().cpu().abs()  # noqa: E731
        args = lambda f: (f(q[:, :tokens]), f(k[:, :tokens]), f(v[:, :tokens]), g.cpu(), D ** -0.5, f(s0), [tokens])  # noqa: E731
        (ro, rs), (ao, as_) = attn_def(*args(d)), attn_def(*args(a))
        f, fa, fs = bounds(torch.float32, tokens, D)
        near("o", o, ro, rounding(torch.float32, ro) + fa * ao)
        near("state", s, rs, fs * as_)


def test_infinite_keys_reach_no_earlier_token():
    q, k, v, g, _ = attn_inputs(1, 100, 1, 1, 64, 64, torch.bfloat16, 14, False)
    clean = gc.linear_attention(q, k, v, g)
    k[0, 50, 0, 3] = float("inf")
    o = gc.linear_attention(q, k, v, g)
    assert torch.equal(o[:, :50], clean[:, :50]) and not torch.isfinite(o[0, 50]).all()


# ---------------------------------------------------------------- the block

def block_def(b, x, r):
    """The block token by token in 64 bits, differentiable in the weights `b` and x, r."""
    h = x + r
    y = b["norm"] * h / torch.sqrt(h.pow(2).mean(-1, keepdim=True) + 1e-6)
    p = y @ b["w_in"].t()
    xs = torch.nn.functional.pad(p, (0, 0, b["taps"] - 1, 0))
    z = b["conv_b"] + sum(xs[:, j:j + p.shape[1]] * b["conv_w"][:, 0, j] for j in range(b["taps"]))
    u = (z * torch.sigmoid(z)).split(b["heads"] * b["dim"], dim=-1)
    q, k, v = (t.unflatten(-1, (b["heads"], b["dim"])) for t in u)
    o, s = attn_def(q, k, v, b["log_decay"], b["dim"] ** -0.5, None, [x.shape[1]] * x.shape[0])
    return o.flatten(-2) @ b["w_out"].t(), h, s


def block64(block):
    d = {n: getattr(block, n).double().cpu() for n in ("norm", "w_in", "conv_w", "conv_b", "w_out", "log_decay")}
    return dict(d, heads=block.heads, dim=block.dim, taps=block.taps)


def test_block_against_its_definition():
    block = SequenceBlock(96, 3, 32, dtype=torch.float32)
    gen = torch.Generator().manual_seed(2)
    x, r, dout, dh = (torch.randn(2, 150, 96, generator=gen).cuda() for _ in range(4))
    out, h, kept = block.forward(x, r)
    dx, grads = block.backward(dout, dh, kept)
    out2, h2, states = block.prompt(x, r)
    assert torch.equal(out, out2) and torch.equal(h, h2)
    b = block64(block)
    names = ("norm", "w_in", "conv_w", "conv_b", "w_out")
    xd, rd = x.double().cpu().requires_grad_(), r.double().cpu()
    for n in names:
        b[n].requires_grad_()
    ro, rh, rs = block_def(b, xd, rd)
    ref = torch.autograd.grad((ro * dout.double().cpu()).sum() + (rh * dh.double().cpu()).sum(), [xd] + [b[n] for n in names])
    assert off(out, ro.detach()) < 2e-4 and off(states[1], rs.detach()) < 2e-4
    assert off(dx, ref[0]) < 4e-4
    for n, t in zip(names, ref[1:]):
        assert off(grads[n], t) < 4e-4, n


def test_tokens_carry_on_from_prompts():
    block = SequenceBlock(96, 3, 32, dtype=torch.float32)
    gen = torch.Generator().manual_seed(3)
    B, T = 3, 40
    x, r = torch.randn(B, T + 4, 96, generator=gen).cuda(), torch.randn(B, T + 4, 96, generator=gen).cuda()
    lengths = [40, 13, 0]
    _, _, states = block.prompt(x[:, :T].contiguous(), r[:, :T].contiguous(), torch.tensor(lengths, dtype=torch.int32).cuda())
    pools, slots = block.pools(5), torch.tensor([4, 1, 3], dtype=torch.int32).cuda()
    for pool, state in zip(pools, states):
        pool[slots.long()] = state
    rows = torch.arange(B)
    for i in range(4):
        at = torch.tensor(lengths) + i
        out, _ = block.token(x[rows, at], r[rows, at], pools, slots)
        for j, n in enumerate(lengths):
            ro, _, _ = block_def(block64(block), x[j:j + 1, :n + i + 1].double().cpu(), r[j:j + 1, :n + i + 1].double().cpu())
            assert off(out[j], ro[0, -1]) < 2e-4
    assert (pools[1][0] == 0).all() and (pools[1][2] == 0).all()


def test_step_of_training_replays_in_a_graph():
    block = SequenceBlock(64, 2, 32, dtype=torch.bfloat16)
    x, r, dout, dh = (torch.randn(2, 600, 64, device="cuda").bfloat16() for _ in range(4))

    def step():
        out, h, kept = block.forward(x, r)
        dx, grads = block.backward(dout, dh, kept)
        return [out, h, dx, *grads.values()]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for i in range(3):
        x.copy_(torch.randn(2, 600, 64, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        for y, z in zip(kept, step()):
            assert torch.equal(y, z), i
