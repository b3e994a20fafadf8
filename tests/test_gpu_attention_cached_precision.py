"""Cached attention of few rows holds its probabilities to twice bf16's precision in the product
with the values: sequences of up to 16 rows (queries times the heads that share a key head), and
of up to 32 where the call can have none of more.

Tolerance, elementwise: with A the largest sum of a score's magnitudes, n keys and d the head
dimension, a score is off by at most 4 d 2^-24 A (sums of exact products, whose accumulator may
truncate) and its exponent's two roundings by 2^-22 A; the exponential by 2^-22; the sum over the keys by n 2^-24,
the products' by 8 n 2^-24 (twice as many terms); p as two bf16 by 2^-8 2^-8.  The scores' and
exponentials' errors are in p and in the sum.  out is rounded once, by 2^-8 of itself.
The same with p rounded to one bf16 does not hold, which each case says of its own oracle.
"""
import pytest
import torch

import kv_cache_reference as ref
import test_gpu_attention_cached as cached
from gpu_util import say

pytestmark = pytest.mark.gpu
BF16, F64 = torch.bfloat16, torch.float64


@pytest.fixture(scope="module")
def fp8():
    import fp8_precision_amd
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    return fp8_precision_amd


CASES = [
    # new tokens, held before, hq, hk, d, page, causal, blocks of the table without a page, bounds
    ([1] * 6, [1, 2, 4, 9, 30, 100], 16, 1, 64, 16, True, 0, False),      # each head by one workgroup
    ([1] * 6, [1, 2, 4, 9, 30, 100], 16, 2, 128, 16, True, 90, False),    # in shares
    ([5, 0, 3, 1], [2, 50, 0, 7], 3, 1, 72, 16, True, 90, True),
    ([16], [200], 2, 2, 64, 32, False, 40, False),                        # split and joined
    ([3] * 4, [0, 1, 6, 20], 10, 1, 128, 16, True, 0, False),             # 30 rows
    ([4] * 4, [3, 1, 6, 40], 16, 2, 64, 16, True, 90, False),             # 32
    ([20, 2, 10], [2, 1, 6], 1, 1, 64, 16, True, 90, True),               # 32 in the call
    ([1, 300], [4, 0], 4, 4, 64, 16, True, 0, True),                      # one row among tiles: the first alone
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_probabilities(fp8, case):
    news, past, hq, hk, d, page, causal, spare, bounded = CASES[case]
    say("precision", CASES[case])
    pool, table, lengths = cached.setup(news, past, hk, d, page, 90 + case, spare=spare)
    q = torch.randn(sum(news), hq, d, generator=torch.Generator().manual_seed(case)).to(BF16).cuda()
    scale = d ** -0.5
    out, _ = fp8.attention_cached(q, ref.on_gpu(fp8, pool), table.cuda(), torch.tensor(lengths, dtype=torch.int32).cuda(),
                                  cu=ref.bounds(news) if bounded else None, causal=causal, scale=scale)
    first = worse = 0
    for b, n in enumerate(news):
        rows = slice(first, first + n)
        first += n
        if n == 0 or n * hq // hk > 32:
            continue
        held = lengths[b]
        k, v = (ref.read(pool, table[b:b + 1], [held], [held], x).cuda() for x in "kv")
        i, j = torch.arange(n, device="cuda")[:, None], torch.arange(held, device="cuda")[None, :]
        seen = (j <= i + held - n) if causal else torch.ones(n, held, dtype=torch.bool, device="cuda")
        for h in range(hq):
            x, y, z = q[rows, h].to(F64), k[:, h // (hq // hk)], v[:, h // (hq // hk)]
            s = (x @ y.t() * scale).masked_fill(~seen, -float("inf"))
            p = torch.exp(s - s.amax(1, keepdim=True))
            total = p.sum(1, keepdim=True)
            o, slack = p @ z / total, p @ z.abs() / total
            most = (x.abs() @ y.abs().t()).max().item() * scale
            e = 4 * d * 2.0 ** -24 * most + 2.0 ** -22 * most + 2.0 ** -22
            bound = 2.0 ** -8 * o.abs() + (2 * e + 9 * held * 2.0 ** -24 + 2.0 ** -16) * 1.01 * slack + 1e-30
            bad = (out[rows, h].to(F64) - o).abs() > bound
            assert not bad.any(), (b, h, int(bad.sum()))
            once = p.to(torch.float32).to(BF16).to(F64) @ z / total
            worse += int(((once.to(torch.float32).to(BF16).to(F64) - o).abs() > bound).sum())
    assert worse > 0


@pytest.mark.parametrize("news", [[1, 1], [40, 1]])
def test_largest_scale(fp8, news):
    """Queries of zeros: every score is 0 whatever the scale, out the mean of the values."""
    say("largest scale", news)
    pool, table, lengths = cached.setup(news, [20, 50], 1, 64, 16, 7)
    q = torch.zeros(sum(news), 2, 64, dtype=BF16, device="cuda")
    n = torch.tensor(lengths, dtype=torch.int32).cuda()
    out, lse = fp8.attention_cached(q, ref.on_gpu(fp8, pool), table.cuda(), n, cu=ref.bounds(news), causal=False, scale=2.3e38)
    cached.check(q, out, lse, pool, table, lengths, news, False, 1.0)
