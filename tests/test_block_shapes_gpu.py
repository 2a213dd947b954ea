"""The recurrent block's operators where their launches take another shape: short prompts over many
channels, sequences in many segments, single positions in their thousands, samples that fill a
workgroup's registers, tiles on both sides of each choice.  Checked as in the operators' own tests."""
import pytest

import test_gated_recurrence_gpu as rec
import test_group_norm_gpu as gn
import test_int8_gpu as i8

pytestmark = pytest.mark.gpu

REC = [  # B, T, C, state, lengths, layout
    (10, 2, 700, True, None, "plain"),
    (16, 40, 514, True, [40 - k for k in range(16)], "fused"),       # wide stripes, tiles one after the other
    (3, 200, 66, False, [200, 0, 131], "time"),                      # one tile of a narrow stripe
    (40, 90, 260, True, None, "plain"),
    (1, 9000, 70, True, None, "plain"),                              # segments in tens
    (2, 12000, 6, True, [12000, 7001], "time"),
    (1, 257, 260, True, None, "plain"),
]
GN = [  # N, P, C, G, silu, bias, lengths, layout
    (20000, 1, 64, 4, True, True, [k % 3 // 2 for k in range(20000)], "plain"),   # samples one after the other
    (17001, 1, 33, 3, False, True, None, "plain"),
    (2500, 1, 128, 32, True, True, None, "wide"),                    # groups of one vector
    (1100, 2, 40, 20, True, True, [k % 3 for k in range(1100)], "plain"),
    (3, 1000, 64, 1, True, True, [1000, 999, 0], "plain"),           # a workgroup's registers
    (2, 60, 410, 5, True, True, None, "swapped"),                    # groups of 41 vectors
]
I8 = [  # M, N, K
    (17, 8300, 64), (32, 8100, 48), (33, 130, 64), (1400, 2000, 128), (1700, 2050, 100), (3700, 4000, 64),
]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", REC, ids=lambda c: "x".join(map(str, c[:3])))
def test_recurrence_shapes(case, dt):
    rec.test_gated_recurrence(case, dt)
    rec.test_gated_recurrence_backward(case, dt)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", GN, ids=lambda c: "x".join(map(str, c[:4])))
def test_group_norm_shapes(case, dt):
    gn.test_group_norm(case, dt)
    gn.test_group_norm_backward(case, dt)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", I8, ids=lambda c: "x".join(map(str, c)))
def test_matmul_shapes(shape, dt):
    i8.test_matmul(shape, dt)
