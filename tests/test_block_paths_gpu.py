"""The recurrent block's operators on the kernels that their other tests run for one tile, one stage or one
chunk only, or compare with themselves: stripes of every width over several tiles, tiles of the 8-bit product
over many stages of K, groups wider than a workgroup in batches, tokens and statistics against the
definition.  Checked as in the operators' own tests."""
import pytest
import torch

import depthwise_convolution_gconv_amd as gc
import test_gated_recurrence_gpu as rec
import test_group_norm_gpu as gn
import test_int8_gpu as i8

pytestmark = pytest.mark.gpu

U = 2.0 ** -24

# 127 channels in fp32 and 254 in 16 bits are 64 lanes of 8 bytes; with them stripes of ...
REC = [  # B, T, C, state, lengths, layout
    (14, 1100, 254, True, None, "plain"),                                # 4 lanes over tiles of 512 tokens
    (30, 600, 254, True, [600 - 31 * k % 601 for k in range(30)], "fused"),       # 8 lanes, 256 tokens
    (60, 300, 254, True, [300 - 7 * k % 301 for k in range(60)], "fused"),        # 16 lanes, 128 tokens
    (100, 300, 254, False, None, "plain"),                               # 32 lanes, 64 tokens
    (14, 1100, 127, True, None, "plain"),
    (30, 600, 127, True, [600 - 31 * k % 601 for k in range(30)], "fused"),
    (60, 300, 127, True, [300 - 7 * k % 301 for k in range(60)], "fused"),
    (100, 300, 127, False, None, "plain"),
]
GN = [  # N, P, C, G, silu, bias, lengths, layout
    (600, 3, 1031, 1, True, True, None, "plain"),                        # one chunk a sample, two parts a group
    (3, 5, 16400, 1, True, True, [5, 0, 3], "wide"),                     # several parts in every type
    (2100, 1, 1031, 1, False, True, None, "plain"),                      # more samples than rows of partial sums
    (1500, 3, 1031, 1, True, False, [k % 4 for k in range(1500)], "swapped"),
    (1300, 2, 2062, 2, True, True, [2 - k % 3 for k in range(1300)], "plain"),
    (1, 1, 8192, 1, True, True, None, "plain"),
    (3100, 2, 1031, 1, True, True, [k % 3 for k in range(3100)], "wide"),         # ranges of samples, empty ones in them
    (4103, 1, 1033, 1, True, False, [k % 5 // 4 for k in range(4103)], "plain"),
]
I8 = [  # M, N, K: stages past the first ring, with rests of K, rows and channels
    (3790, 3810, 1296),      # 225 tiles of 256
    (1790, 2040, 1296),      # 224 tiles of 128
    (1800, 2050, 1001),      # 255 unaligned tiles of 128
    (300, 400, 2000), (300, 400, 2003), (20, 9000, 1296), (25, 300, 2003),
]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", REC, ids=lambda c: "x".join(map(str, c[:3])))
def test_stripes_over_several_tiles(case, dt):
    rec.test_gated_recurrence(case, dt)
    rec.test_gated_recurrence_backward(case, dt)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,C,slots", [(1, 1, None), (5, 131, None), (70, 257, list(range(100, 30, -1))), (4, 64, [7, -1, 0, 200])])
def test_tokens_against_the_definition(B, C, slots, dt):
    dtype, T = rec.DT[dt], 5
    x, r, i, g, _ = rec.inputs(B, T, C, dtype, False, "fused", seed=11)
    pool = 2 * torch.randn(200 if slots else B, C, generator=torch.Generator().manual_seed(1)).cuda()
    was = pool.clone()
    rows = torch.tensor(slots, dtype=torch.int32).cuda() if slots else None
    own = slots or list(range(B))
    there = [0 <= s < pool.shape[0] for s in own]
    first = torch.stack([was[s] if ok else torch.zeros_like(was[0]) for s, ok in zip(own, there)]).double().cpu()
    n = [T if ok else 0 for ok in there]
    X, R, I, G = (rec.d(t) for t in (x, r, i, g))
    rh, rs = rec.definition(X, R, I, G, first, n)
    la = (G * torch.sigmoid(R)).abs()
    live = torch.tensor(there).view(B, 1, 1)
    a = torch.where(live, torch.exp(-la), 1.0)
    add = torch.where(live, torch.sqrt(-torch.expm1(-2 * la)) * torch.sigmoid(I) * X.abs(), 0.0)
    err_a = torch.where(live, (la * (9 + 1.5 * R.abs()) + 3) * U, 0.0)
    _, err = rec.carried(a, add, err_a, (24 + 1.5 * R.abs() + 1.5 * I.abs()) * U, first)
    for t in range(T):
        print("token", B, C, dt, t, flush=True)
        h = gc.gated_recurrence_step(x[:, t], r[:, t], i[:, t], g, pool, slots=rows)
        rec.near("h", h, rh[:, t], rec.rounding(dtype, rh[:, t]) + err[:, t] * (1 + rec.half_step(dtype)) * live[:, 0])
    for b, (s, ok) in enumerate(zip(own, there)):
        if ok:
            rec.near("state", pool[s], rs[b], err[b, -1])
    untouched = sorted(set(range(pool.shape[0])) - set(own))
    assert torch.equal(pool[untouched], was[untouched])


def test_most_channels_of_a_gradient():
    """One token of 2^26 - 16 channels, the most that the sum of log_decay's shares takes: every channel's gradients
    are the same closed form (r = i = 0, log_decay = -1/2: a = exp(-1/4))."""
    C = 2 ** 26 - 16
    x, r = torch.ones(1, 1, C, device="cuda").bfloat16(), torch.zeros(1, 1, C, device="cuda").bfloat16()
    g = torch.full((C,), -0.5, device="cuda")
    s0 = torch.full((1, C), 3.0, device="cuda")
    # (of one token only the first state is read, not h)
    dx, dr, di, dg, ds = gc.gated_recurrence_backward(x, r, r, g, x, x, initial_state=s0)
    a = torch.tensor(-0.25, dtype=torch.float64).exp()
    s = (-torch.expm1(torch.tensor(-0.5, dtype=torch.float64))).sqrt()
    dla = a * 3 - a * a / s * 0.5
    half = rec.half_step(torch.bfloat16)
    # A few fp32 roundings (at most 40 u of the terms, which cancel to no less than half), and bf16's own.
    for name, got, want, off in (("dx", dx, s / 2, half), ("dr", dr, dla * -0.5 / 4, half), ("di", di, s / 4, half),
                                 ("dlog_decay", dg, dla / 2, 0), ("dinitial", ds, a, 0)):
        lo, hi = float(got.min()), float(got.max())
        assert lo == hi and abs(lo - float(want)) <= (off + 80 * U) * abs(float(want)), (name, lo, hi, float(want))
    with pytest.raises(gc.GconvError):
        one = torch.zeros(1, 1, C + 1, device="cuda").bfloat16()
        gc.gated_recurrence_backward(one, one, one, torch.zeros(C + 1, device="cuda"), one, one)
    del x, r, g, s0, dx, dr, di, dg, ds, got, one
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", GN, ids=lambda c: "x".join(map(str, c[:4])))
def test_groups_wider_than_a_workgroup(case, dt):
    gn.test_group_norm(case, dt)
    gn.test_group_norm_backward(case, dt)


def test_statistics_of_most_positions():
    """1 and 3 over 2^31 - 65537 positions: the means of threads and chunks are 2 exactly and their squares whole
    numbers below 2^24, so what is rounded is a lane's sum over 8 chunks and 6 joins, the number of elements
    and a division: at most 20 u of the mean and, with a root more, 24 u of 1 / sqrt(var)."""
    P = 2 ** 31 - 1 - 65536
    x = torch.tensor([1.0, 3.0], device="cuda").bfloat16().expand(1, P, 2)
    w = torch.ones(2, device="cuda").bfloat16()
    y, st = gc.group_norm(x, 1, w, None, eps=0.0, return_stats=True)
    assert abs(float(st[0, 0, 0]) - 2) <= 20 * U * 2 and abs(float(st[0, 0, 1]) - 1) <= 24 * U
    flat = y.view(-1, 2)
    assert bool((flat[:, 0] == -1).all()) and bool((flat[:, 1] == 1).all())
    del x, y, flat
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", I8, ids=lambda c: "x".join(map(str, c)))
def test_product_over_many_stages(shape, dt):
    i8.test_matmul(shape, dt)
