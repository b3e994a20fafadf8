"""The rounding of dloss is in none of the gradients: a dloss midway between two bf16 values, whose
own rounding would put 2^-8 into every gradient alike, over the tilings of few and of many tokens."""
import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu

F64, BF16 = torch.float64, torch.bfloat16


@pytest.fixture(scope="module")
def fp8():
    import fp8_precision_amd
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    return fp8_precision_amd


# tiles of 64, 128 and 256 rows, halves, several pieces of the reduction of dx, dweight's split
@pytest.mark.parametrize("T,V,D", [(1, 4096, 128), (17, 8192, 256), (100, 4096, 128), (300, 9001, 320), (1023, 4096, 64),
                                   (8000, 4096, 64)])
@pytest.mark.parametrize("steps", [1, 3])
def test_dloss_between_two_bf16_values(fp8, T, V, D, steps):
    """The results' own rounding has an rms of at most 2^-8 / sqrt 3 (uniform in the last place,
    at the shortest mantissa); g's, where a target's p - 1 rounds to -1, is p: about 1 / V at
    these logits, below e / V.  With dloss in g its rounding adds nearly 2^-8: the test says
    so of g rounded whole, on the same inputs, in 64 bits."""
    say("loss backward, a mean", T, V, D, steps)
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, D, generator=g).to(BF16).cuda()
    w = (torch.randn(V, D, generator=g) * 0.1 * D ** -0.5).to(BF16).cuda()
    t = torch.randint(0, V, (T,), generator=g).cuda()
    d = (1 + 2.0 ** -8) * 2.0 ** -(10 + torch.arange(T) % steps).float().cuda()
    assert ((d.to(BF16).to(F64) / d.to(F64) - 1).abs() > 0.99 * 2.0 ** -8).all()
    _, lse = fp8.linear_cross_entropy(x, w, t)
    got = fp8.linear_cross_entropy_backward(d, x, w, t, lse)
    p = torch.softmax(x.to(F64) @ w.to(F64).t(), 1)
    p[torch.arange(T, device="cuda"), t] -= 1
    exact = p * d.to(F64)[:, None]
    whole = exact.to(BF16).to(F64)
    bound = 2.0 ** -8 / 3 ** 0.5 + 2.72 / V
    for a, want, other in zip(got, (exact @ w.to(F64), exact.t() @ x.to(F64)), (whole @ w.to(F64), whole.t() @ x.to(F64))):
        off = lambda y: float((y.to(F64) - want).norm() / want.norm())
        assert off(other.to(BF16)) > bound, "these inputs would not show it"
        assert off(a) <= bound
