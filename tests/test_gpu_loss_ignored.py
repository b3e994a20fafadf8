"""Tokens without a target: whatever their hidden states are, the gradients are those of a batch
in which they are zero, bit for bit."""
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


# one and several tiles of rows, whole and half ones; dweight's sum split over the tokens; a
# vocabulary of several pieces; a last step of few tokens
SHAPES = [(3, 50, 16), (40, 700, 64), (64, 3000, 264), (65, 300, 72), (300, 9001, 320), (1001, 2100, 1600), (5000, 300, 136),
          (8039, 1246, 272), (9000, 8500, 64), (2049, 40, 8)]


def make(T, V, D, share=0.2):
    g = torch.Generator().manual_seed(T + V)
    x = torch.randn(T, D, generator=g).to(BF16).cuda()
    w = (torch.randn(V, D, generator=g) * D ** -0.5).to(BF16).cuda()
    t = torch.randint(0, V, (T,), generator=g)
    gone = torch.rand(T, generator=g) < share
    gone[-1], gone[0] = True, False
    t[gone] = torch.tensor([-100, -1, V, 1 << 40])[torch.randint(0, 4, (int(gone.sum()),), generator=g)]
    return x, w, t.cuda(), gone.cuda(), torch.randn(T, generator=g).abs().cuda() / T


@pytest.mark.parametrize("T,V,D", SHAPES)
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 3.0])
def test_hidden_states_of_tokens_without_a_target(fp8, T, V, D, value):
    say("loss backward, ignored tokens", T, V, D, value)
    x, w, t, gone, d = make(T, V, D)
    clean, other = x.clone(), x.clone()
    clean[gone], other[gone] = 0.0, value
    _, lse = fp8.linear_cross_entropy(clean, w, t)
    loss2, lse2 = fp8.linear_cross_entropy(other, w, t)
    assert torch.equal(lse2[~gone], lse[~gone]) and (loss2[gone] == 0).all()
    dx, dw = fp8.linear_cross_entropy_backward(d, clean, w, t, lse)
    dx2, dw2 = fp8.linear_cross_entropy_backward(d, other, w, t, lse2)
    assert torch.isfinite(dw.float()).all() and dw.any()
    assert torch.equal(dw2, dw) and torch.equal(dx2, dx) and not dx2[gone].any()


@pytest.mark.parametrize("T,V,D", SHAPES)
@pytest.mark.parametrize("value", [float("nan"), float("-inf"), -3e38, 2.0])
def test_dloss_of_tokens_without_a_target(fp8, T, V, D, value):
    """It is no measure of the others' gradients, which are held as fractions of the largest."""
    say("loss backward, dloss of ignored tokens", T, V, D, value)
    x, w, t, gone, d = make(T, V, D)
    clean, other = d.clone(), d.clone()
    clean[gone], other[gone] = 0.0, value
    _, lse = fp8.linear_cross_entropy(x, w, t)
    want = fp8.linear_cross_entropy_backward(clean, x, w, t, lse)
    for a, b in zip(fp8.linear_cross_entropy_backward(other, x, w, t, lse), want):
        assert b.any() and torch.equal(a, b)
