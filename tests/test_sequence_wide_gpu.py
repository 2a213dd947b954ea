"""Linear attention of heads wider than 128 columns on both sides (eight waves a workgroup in 16
bits), with row ends inside a load, shared key heads and several segments.  Tolerances as in
test_sequence_gpu.py."""
import pytest
import torch

import depthwise_convolution_gconv_amd as gc
from test_sequence_gpu import DT, attn_def, attn_inputs, bounds, near, rounding

pytestmark = pytest.mark.gpu

WIDE = [  # B, T, Hk, H, Dk, Dv, lengths, layout
    (2, 300, 1, 2, 198, 170, [300, 170], "fused"),
    (1, 40, 2, 2, 129, 256, None, "heads"),
    (1, 150, 1, 1, 250, 129, [0], "plain"),
]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", WIDE, ids=lambda c: "x".join(map(str, c[:6])))
def test_wide_heads(case, dt):
    B, T, Hk, H, Dk, Dv, lengths, layout = case
    print("wide", case, dt, flush=True)
    q, k, v, g, s0 = attn_inputs(B, T, Hk, H, Dk, Dv, DT[dt], 21, True, layout)
    n = lengths if lengths is not None else [T] * B
    ln = torch.tensor(lengths, dtype=torch.int32).cuda() if lengths is not None else None
    gen = torch.Generator().manual_seed(22)
    do = torch.randn(B, T, H, Dv, generator=gen).to(DT[dt]).cuda()
    ds = torch.randn(B, H, Dk, Dv, generator=gen).cuda()
    o, s = gc.linear_attention(q, k, v, g, initial_state=s0, lengths=ln, return_state=True)
    got = gc.linear_attention_backward(q, k, v, g, do, initial_state=s0, lengths=ln, dstate=ds)
    torch.cuda.synchronize()

    def run(fn):
        leaves = [fn(t).requires_grad_() for t in (q, k, v, s0)]
        ro, rs = attn_def(*leaves[:3], g.cpu(), Dk ** -0.5, leaves[3], n)
        loss = (ro * fn(do)).sum() + (rs * fn(ds)).sum()
        return [ro.detach(), rs.detach(), *torch.autograd.grad(loss, leaves)]

    ref, mag = run(lambda t: t.double().cpu()), run(lambda t: t.double().cpu().abs())
    f, fa, fs = bounds(DT[dt], T, max(Dk, Dv) + H // Hk)
    for name, y, r, m in zip(("o", "state", "dq", "dk", "dv", "dinitial"), (o, s, *got), ref, mag):
        if y.dtype == torch.float32:
            near(name, y, r, fs * m + (rounding(DT[dt], r) if dt == "f32" else 0.0))
        else:
            near(name, y, r, rounding(DT[dt], r) + fa * m)
