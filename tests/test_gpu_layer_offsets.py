"""Norm, attention and loss on tensors whose elements lie more than 2^31 apart: the far rows
give what the same rows give in a small tensor, bit for bit where the sums are the same.

Tolerances elsewhere: a sum of 64 terms in another order is off by 64 2^-24 of its magnitudes
(1e-4 covers terms up to 25 times the sum); a logit by 2048 2^-24 of its own (below 1); the
gradients carry g's rounding and their own (2^-8 each)."""
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


def random(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(BF16).cuda()


def test_norm_of_many_rows(fp8):
    say("norm, more than 2^31 elements")
    rows, cols, n = 140_000, 16_384, 64
    x = torch.zeros(rows, cols, dtype=BF16, device="cuda")
    x[-n:] = random(n, cols)
    w, dy = random(cols, seed=1), torch.zeros_like(x)
    dy[-n:] = random(n, cols, seed=2)
    y, _, _, rstd = fp8.norm(x, w)
    y2, _, _, rstd2 = fp8.norm(x[-n:].clone(), w)
    assert torch.equal(y[-n:], y2) and torch.equal(rstd[-n:], rstd2) and not y[:-n].any()
    del y
    dx, dw, _ = fp8.norm_backward(dy, x, w, None, rstd)
    dx2, dw2, _ = fp8.norm_backward(dy[-n:].clone(), x[-n:].clone(), w, None, rstd2)
    assert torch.equal(dx[-n:], dx2)
    assert torch.allclose(dw, dw2, rtol=1e-4, atol=1e-4)      # the rows are added in another order


@pytest.mark.parametrize("nq", [3, 1100])
def test_attention_on_far_apart_tokens(fp8, nq):
    say("attention, tokens 4 MB apart", nq)
    nk, d, step = 1100, 128, 1 << 21
    q, dout = random(nq, 2, d), random(nq, 2, d, seed=1)
    far = [torch.empty(nk, step, dtype=BF16, device="cuda")[:, :d].unflatten(1, (1, d)) for _ in range(2)]
    for i, t in enumerate(far):
        t.copy_(random(nk, 1, d, seed=2 + i))
    near = [t.contiguous() for t in far]
    out, lse = fp8.attention(q, *far, causal=True)
    out2, lse2 = fp8.attention(q, *near, causal=True)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    want = fp8.attention_backward(dout, q, *near, out, lse, causal=True)
    # the gradients are written over tensors laid out like k and v
    to = [torch.empty(nk, step, dtype=BF16, device="cuda")[:, :d].unflatten(1, (1, d)) for _ in range(2)]
    got = fp8.attention_backward(dout, q, *far, out, lse, causal=True, dk=to[0], dv=to[1])
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [3, 200])
def test_loss_over_a_weight_of_more_than_2_31_elements(fp8, T):
    say("loss, large weight", T)
    V, D, n = 1_060_000, 2048, 512
    w = torch.zeros(V, D, dtype=BF16, device="cuda")
    w[-n:] = random(n, D) * 0.05
    x = random(T, D, seed=1)
    t = V - 1 - torch.arange(T, device="cuda") % n
    z = x.double() @ w[-n:].double().t()
    lse64 = torch.logsumexp(torch.cat([z, torch.full((T, 1), 0.0, device="cuda").double() + torch.log(torch.tensor(float(V - n)).double())], 1), 1)
    loss, lse = fp8.linear_cross_entropy(x, w, t)
    hit = z[torch.arange(T, device="cuda"), t - (V - n)]
    assert ((lse.double() - lse64).abs() <= 1e-4).all() and ((loss.double() - (lse64 - hit)).abs() <= 2e-4).all()
    dx, dw = fp8.linear_cross_entropy_backward(torch.ones(T, device="cuda"), x, w, t, lse)
    g = torch.exp(z - lse64[:, None])
    g[torch.arange(T, device="cuda"), t - (V - n)] -= 1
    for got, want in ((dx, g @ w[-n:].double()), (dw[-n:], g.t() @ x.double())):
        assert float((got.double() - want).norm() / want.norm()) <= 2.0 ** -7
    assert float(dw[:16].double().sub(torch.exp(-lse64) @ x.double()).norm()) <= 2.0 ** -7 * 4 * float((torch.exp(-lse64) @ x.double()).norm())
