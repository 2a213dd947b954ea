"""Group norm with eps = 0 over batches in which samples without positions stand: their 1 / sqrt(var + eps)
is infinite, and they add nothing to the gradients of the others."""
import pytest
import torch

import depthwise_convolution_gconv_amd as gc
from test_group_norm_gpu import DT

pytestmark = pytest.mark.gpu

CASES = [  # N, P, C, G, lengths
    (3, 1, 96, 4, [1, 0, 1]),                           # rows by themselves
    (2500, 1, 64, 2, [k % 3 // 2 for k in range(2500)]),
    (3, 40, 64, 4, [0, 40, 17]),                        # whole samples in registers
    (600, 40, 64, 4, [k % 41 for k in range(600)]),
    (2, 20001, 32, 4, [20001, 0]),                      # chunks of positions
    (3, 20001, 32, 4, [0, 9, 20001]),                   # chunks behind a sample's end
    (3, 5, 1031, 1, [5, 0, 2]),                         # a group wider than a workgroup
    (3100, 2, 1031, 1, [k % 3 for k in range(3100)]),   # samples one after the other
    (4, 700, 16, 1, [0, 0, 0, 0]),                      # nothing at all
]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[:4])))
def test_samples_without_positions_and_no_eps(case, silu, dt):
    N, P, C, G, lengths = case
    act = "silu" if silu else None
    gen = torch.Generator().manual_seed(1)
    x, dy = (torch.randn(N, P, C, generator=gen).to(DT[dt]).cuda() for _ in range(2))
    w, b = (torch.randn(C, generator=gen).to(DT[dt]).cuda() for _ in range(2))
    ln = torch.tensor(lengths, dtype=torch.int32).cuda()
    print("no eps", case[:4], silu, dt, flush=True)
    y, stats = gc.group_norm(x, G, w, b, 0.0, act, ln, return_stats=True)
    got = gc.group_norm_backward(dy, x, G, w, b, stats, act, ln)
    torch.cuda.synchronize()
    none = ln == 0
    assert torch.isinf(stats[none][..., 1]).all() and not stats[none][..., 0].any() and torch.isfinite(stats[~none]).all()
    assert torch.isfinite(y).all() and not y[none].any() and not got[0][none].any()
    for name, t in zip(("dx", "dw", "db"), got):
        assert torch.isfinite(t).all(), f"{name}: {int((~torch.isfinite(t)).sum())} of {t.numel()} values are not finite"
    # What the statistics of a sample without positions are changes no bit.
    other = stats.clone()
    other[none] = torch.tensor([3.0, 2.0]).cuda()
    assert all(torch.equal(p, q) for p, q in zip(got, gc.group_norm_backward(dy, x, G, w, b, other, act, ln)))
    # And they are the gradients without such samples, whose sums come in another order.
    if not bool(none.all()):
        few = gc.group_norm_backward(dy[~none], x[~none], G, w, b, stats[~none], act, ln[~none])
        half = torch.finfo(DT[dt]).eps / 2
        for p, q in ((got[0][~none], few[0]), got[1:2] + few[1:2], got[2:] + few[2:]):
            assert float((p.double() - q.double()).norm()) <= (2 * half + 1e-5) * float(q.double().norm())
