"""Gradients of the gated recurrence where 1 - a^2 is next to nothing: gates that almost underflow, and
decays that are hardly there, against the definition in 64 bits.

Below 2^-126, fp32's smallest normal number, 1 - a^2 counts as zero and its root as having no derivative,
so there the root's terms may be left out (`dropped`; a factor of two about the border is the kernel's own);
a sigmoid below 2^-126 may be zero (`tiny`).  Everything else has the errors of test_gated_recurrence_gpu.py:
a token's factors are off by at most (40 + 3 |r| + 3 |i|) u, here 320 u, one minus a sigmoid of at most 2 by
(6 + 3) u of 0.88 in 0.12, 70 u more, and each token of a carry by (9 + 1.5 |r|) |la| u + 5 u, at most 20 u
for the ordinary tokens (|r| <= 2, |la| < 1) as for the others (la next to zero)."""
import pytest
import torch

import depthwise_convolution_gconv_amd as gc
from test_gated_recurrence_gpu import DT, U, d, half_step, near, rounding

pytestmark = pytest.mark.gpu

DECAYS = (-7e-4, -1e-3, -0.01, -0.1, -1.0, -1e-30, -1e-37, -2e-38, -1e-38, -1e-40)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T", [1, 82, 700, 3000])       # one tile, several, segments
def test_one_minus_a_squared_next_to_zero(T, dt):
    dtype, B, C = DT[dt], 2, 4 * len(DECAYS)
    gen = torch.Generator().manual_seed(1)
    rnd = lambda: torch.randn(B, T, C, generator=gen).clamp(-2, 2)  # noqa: E731
    x, r, i, dh = rnd(), rnd(), rnd(), rnd()
    # Every second token's gate almost underflows: logits from -80 to -90.
    r[:, ::2] = -80.0 - 10.0 * torch.rand(B, (T + 1) // 2, C, generator=gen)
    r[:, 4::10, 20:] = -20.0
    x, r, i, dh = (t.to(dtype).cuda() for t in (x, r, i, dh))
    g = torch.tensor(DECAYS).repeat_interleave(4).cuda()
    s0 = torch.randn(B, C, generator=gen).cuda()
    h = gc.gated_recurrence(x, r, i, g, initial_state=s0)
    print("next to zero", T, dt, flush=True)
    got = gc.gated_recurrence_backward(x, r, i, g, h, dh, initial_state=s0)
    torch.cuda.synchronize()
    for name, t in zip(("dx", "dr", "di", "dlog_decay", "dinitial"), got):
        assert torch.isfinite(t).all(), f"{name}: {int((~torch.isfinite(t)).sum())} of {t.numel()} values are not finite"

    X, R, I, G, S, DH, H = d(x), d(r), d(i), d(g), d(s0), d(dh), d(h)
    sr, si = torch.sigmoid(R), torch.sigmoid(I)
    la = G * sr
    a, m = torch.exp(la), -torch.expm1(2 * la)
    s, prev = m.sqrt(), torch.cat([S[:, None], H[:, :-1]], 1)
    grad, size = torch.zeros(B, T, C).double(), torch.zeros(B, T, C).double()
    c, cm = torch.zeros(B, C).double(), torch.zeros(B, C).double()
    for t in range(T - 1, -1, -1):
        grad[:, t], size[:, t] = DH[:, t] + c, DH[:, t].abs() + cm
        c, cm = a[:, t] * grad[:, t], a[:, t] * size[:, t]
    e, tiny = (20 * T + 500) * U, 2.0 ** -125
    dropped = (m < 2.0 ** -125).double()
    term = a / s * si * X
    f, fm, fdrop = a * (prev - term), a * (prev.abs() + term.abs()), a * term.abs() * dropped + tiny * a * prev.abs() / sr
    out = 1 + half_step(dtype)
    for name, k, want, mag, drop in (
            ("dx", 0, grad * s * si, size * s * si, dropped * size * s * si),
            ("dr", 1, grad * f * la * (1 - sr), size * fm * -la, size * fdrop * -la),
            ("di", 2, grad * s * si * (1 - si) * X, size * s * si * X.abs(), dropped * size * s * si * X.abs())):
        near(name, got[k], want, rounding(dtype, want) + (e * mag + drop) * out)
    # An addition more for each run of 2 to 4 tokens, tile and sequence: within e.
    near("dlog_decay", got[3], (grad * f * sr).sum((0, 1)), ((2 * e * size * fm + size * fdrop) * sr).sum((0, 1)))
    near("dinitial", got[4], c, e * cm)
