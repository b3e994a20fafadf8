"""Queries that see nothing (causal, with fewer keys than queries): whatever they and their output's
gradient hold, they reach neither the other rows nor the keys, bit for bit."""
import itertools

import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def fp8():
    import fp8_precision_amd
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    return fp8_precision_amd


CASES = [([5], [3], 2, 1, 64), ([200], [64], 2, 2, 128), ([37, 130, 1, 64], [101, 77, 1, 300], 12, 4, 64),
         ([1000, 40, 7], [513, 0, 2], 4, 1, 104), ([700], [129], 8, 8, 128), ([1500], [20], 2, 2, 128)]


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[1]}-{c[4]}")
def test_rows_that_see_nothing(fp8, case, value):
    lq, lk, hq, hk, d = case
    say("attention, rows that see nothing", *case, value)
    g = torch.Generator().manual_seed(sum(lq))
    new = lambda n, h: torch.randn(n, h, d, generator=g).to(BF16).cuda()
    q, k, v, dout = new(sum(lq), hq), new(sum(lk), hk), new(sum(lk), hk), new(sum(lq), hq)
    cu_q, cu_k = (torch.tensor([0] + list(itertools.accumulate(n)), dtype=torch.int32, device="cuda") for n in (lq, lk))
    blind = torch.cat([torch.arange(a) < a - b for a, b in zip(lq, lk)]).cuda()
    assert blind.any() and not blind.all()
    results = []
    for fill in (0.0, value):
        q2, dout2 = q.clone(), dout.clone()
        q2[blind], dout2[blind] = fill, fill
        out, lse = fp8.attention(q2, k, v, cu_q, cu_k, causal=True)
        results.append((out, lse) + fp8.attention_backward(dout2, q2, k, v, out, lse, cu_q, cu_k, causal=True))
    for a, b in zip(*results):
        assert torch.equal(a, b)
    out, lse, dq, dk, dv = results[1]
    assert not out[blind].any() and torch.isneginf(lse[:, blind]).all() and not dq[blind].any()
    assert torch.isfinite(dk.float()).all() and torch.isfinite(dv.float()).all() and dv.any()
