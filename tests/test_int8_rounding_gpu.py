"""The 8-bit product's roundings, bit for bit: the exact sum to fp32, its product with the token's scale to fp32,
and the product of that with the channel's scale plus the bias once to fp32, as a fused multiply and add; then to
the dtype.  Biases next to minus the product make every other order of roundings visible."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import depthwise_convolution_gconv_amd as gc
from test_int8_gpu import DT, operands

pytestmark = pytest.mark.gpu


def to_f32(exact):
    """A fraction rounded once to fp32: to odd in 64 bits first, so that the second rounding sees no false tie."""
    v = np.float64(float(exact))
    if Fraction(float(v)) != exact:
        if abs(Fraction(float(v))) > abs(exact):
            v = np.nextafter(v, np.float64(0.0))
        v = (np.array(v).view(np.int64) | 1).view(np.float64)[()]
    return np.float32(v)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 40, 4096), (16, 24, 100), (30, 20, 333), (40, 33, 1350), (70, 20, 1024)])
def test_each_rounding(M, N, K, dt):
    dtype = DT[dt]
    q, s, w, ws = operands(M, N, K, 12)
    total = (q.double() @ w.double().t()).cpu()
    scaled = (total.float().double() * s.double().cpu()).float()       # products of two fp32 numbers are exact in 64 bits
    gen = torch.Generator().manual_seed(13)
    near = -(scaled.double() * ws.double().cpu())[torch.randint(0, M, (N,), generator=gen), torch.arange(N)]
    for bias in (None, near.to(dtype)):
        print("roundings", M, N, K, dt, bias is not None, flush=True)
        y = gc.matmul_int8(q, s, w, ws, None if bias is None else bias.cuda(), dtype).cpu()
        want = np.empty((M, N), np.float32)
        left, right = scaled.tolist(), ws.cpu().tolist()
        add = [0.0] * N if bias is None else bias.float().tolist()
        for m in range(M):
            for n in range(N):
                want[m, n] = to_f32(Fraction(left[m][n]) * Fraction(right[n]) + Fraction(add[n]))
        assert torch.equal(y, torch.from_numpy(want).to(dtype))
