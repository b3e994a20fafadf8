"""Cached attention whose last round of tiles is split, with every number of heads to a tile's
row, against float64 (tolerances of test_gpu_attention_cached.py): no row is left unwritten."""
import pytest
import torch

import kv_cache_reference as ref
import test_gpu_attention_cached as cached
from gpu_util import say

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def fp8():
    import fp8_precision_amd
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    return fp8_precision_amd


CASES = [
    # new tokens, held before, hq, hk, d, page, causal
    ([2048], [6144], 40, 40, 128, 64, True),             # 16 tiles of 40 heads: the whole units end inside one
    ([1664], [2000], 40, 40, 64, 64, False),             # 13 tiles
    ([1408], [2100], 48, 24, 64, 64, False),             # 22 of 24 heads, two queries to a key
    ([1664, 1, 5], [2000, 700, 90], 40, 40, 64, 32, False),    # among sequences of few rows
    ([700, 1300, 1000], [3100, 2900, 3500], 24, 24, 64, 128, True),
    ([1250], [2400], 56, 56, 72, 64, False),
    ([1408], [2100], 25, 25, 64, 64, False),             # no multiple of 8
    ([2048], [1900], 33, 33, 8, 16, False),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_no_row_is_left(fp8, case):
    news, past, hq, hk, d, page, causal = CASES[case]
    say("tiles", CASES[case])
    pool, table, lengths = cached.setup(news, past, hk, d, page, 70 + case)
    q = torch.randn(sum(news), hq, d, generator=torch.Generator().manual_seed(case)).to(BF16).cuda()
    n = torch.tensor(lengths, dtype=torch.int32).cuda()
    cache, table_gpu = ref.on_gpu(fp8, pool), table.cuda()
    for cu in [ref.bounds(news)] + [None] * (len(news) == 1):
        out = torch.full(q.shape, float("nan"), dtype=BF16, device="cuda")
        lse = torch.full((hq, sum(news)), float("nan"), device="cuda")
        top = torch.zeros(1, device="cuda")
        fp8.attention_cached(q, cache, table_gpu, n, cu=cu, causal=causal, out=out, lse=lse, absmax=top)
        assert not torch.isnan(out).any() and not torch.isnan(lse).any()
        cached.check(q, out, lse, pool, table, lengths, news, causal, d ** -0.5)
        assert top.item() == out.float().abs().max().item()
