"""Scales at the low end of their range: every key counts alike, and out is the mean of the values."""
import math

import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu

F64, BF16 = torch.float64, torch.bfloat16
# p rounded for the product, the mean rounded once: each 2^-8; the sums 2^-10, as elsewhere
U, E = 2.0 ** -8 * 1.01, 2.0 ** -10


@pytest.fixture(scope="module")
def fp8():
    import fp8_precision_amd
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    return fp8_precision_amd


@pytest.mark.parametrize("scale", [1e-30, 1e-37, 1e-38, 1e-40, 2.0 ** -149])
@pytest.mark.parametrize("nq,nk,hq,hk", [(1, 20000, 8, 2), (90, 3000, 2, 1), (300, 300, 4, 4), (3, 2, 1, 1)])
def test_a_vanishing_scale(fp8, scale, nq, nk, hq, hk):
    say("attention, scale", scale, nq, nk, hq, hk)
    g = torch.Generator().manual_seed(nk)
    q, k, v, dout = (torch.randn(*s, generator=g).to(BF16).cuda() for s in ((nq, hq, 64), (nk, hk, 64), (nk, hk, 64), (nq, hq, 64)))
    out, lse = fp8.attention(q, k, v, scale=scale)
    wide = v.to(F64).repeat_interleave(hq // hk, 1)
    mean = wide.mean(0)
    assert ((out.to(F64) - mean).abs() <= U * mean.abs() + (U + E) * wide.abs().mean(0)).all()
    assert ((lse - math.log(nk)).abs() <= 2.0 ** -18 * math.log(nk)).all()
    _, _, dv = fp8.attention_backward(dout, q, k, v, out, lse, scale=scale)
    want = dout.to(F64).unflatten(1, (hk, -1)).sum((0, 2)) / nk
    room = dout.to(F64).abs().unflatten(1, (hk, -1)).sum((0, 2)) / nk
    assert ((dv.to(F64) - want).abs() <= U * want.abs() + (U + E) * room).all()
