"""Norms of more rows than one launch holds (its threads are counted in 32 bits): the rows at the
launches' ends give what they give in a small tensor, bit for bit."""
import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
THREADS = 1 << 32


@pytest.fixture(scope="module")
def fp8():
    import fp8_precision_amd
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    return fp8_precision_amd


def random(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(BF16).cuda()


def check(fp8, rows, cols, border, rms, add):
    """Rows of zeros but for some at the ends and around row `border`."""
    at = torch.cat([torch.arange(40), torch.arange(border - 40, border + 40), torch.arange(rows - 40, rows)]).unique()
    assert 0 <= at.min() and at.max() < rows
    at = at.cuda()
    some, a, w = random(len(at), cols), random(len(at), cols, seed=1), random(cols, seed=2)
    bias = None if rms else random(cols, seed=3)
    x = torch.zeros(rows, cols, dtype=BF16, device="cuda")
    x[at] = some
    more = None
    if add:
        more = torch.zeros_like(x)
        more[at] = a
    top, top2 = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
    y, s, mean, rstd = fp8.norm(x, w, bias, add=more, rms=rms, absmax=top)
    want = fp8.norm(some, w, bias, add=a if add else None, rms=rms, absmax=top2)
    assert torch.equal(y[at], want[0]) and torch.equal(s[at], want[1]) and torch.equal(rstd[at], want[3])
    assert rms or torch.equal(mean[at], want[2])
    # a row of zeros: 1 / sqrt(eps), and the bias
    rest = torch.randint(0, rows, (100000,), device="cuda", generator=torch.Generator("cuda").manual_seed(4))
    rest = rest[~torch.isin(rest, at)]
    zero = fp8.norm(torch.zeros(1, cols, dtype=BF16, device="cuda"), w, bias, rms=rms)
    assert (rstd[rest] == zero[3]).all() and (y[rest] == zero[0]).all() and not s[rest].any()
    assert top.item() == max(top2.item(), zero[0].float().abs().max().item())


def test_narrow_rows(fp8):
    say("norm, 2^28 rows of 8")
    check(fp8, (1 << 28) + 101, 8, (THREADS - 1) // 256 * 16, rms=False, add=True)


def test_rows_of_a_workgroup_each(fp8):
    say("norm, 2^25 rows of 513")
    check(fp8, (1 << 25) + 101, 513, (THREADS - 1) // 128, rms=True, add=False)
