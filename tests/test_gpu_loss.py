"""Cross entropy of a linear head, forward and backward, against a float64 evaluation.

Tolerances, from the roundings (u = 2^-8, bf16's unit):
 - a logit is an fp32 sum of dim exact products: off by at most dim 2^-24 of its sum of
   magnitudes a; lse is off by no more than the largest such error plus the fp32 sum of
   exponentials (2^-18 covers blocks, lanes and the joins) and its own size 2^-22;
 - g is rounded once (u) and carries p's relative error (the logit's plus 2^-18);
 - dx and dweight are fp32 sums of g's products, rounded once (u).
"""
import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu

F64, BF16 = torch.float64, torch.bfloat16
U = 2.0 ** -8 * 1.01


@pytest.fixture(scope="module")
def fp8():
    import fp8_precision_amd
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    return fp8_precision_amd


def make(T, V, D, seed, sigma=None):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, D, generator=g).to(BF16).cuda()
    w = (torch.randn(V, D, generator=g) * (sigma or D ** -0.5 * 1.5)).to(BF16).cuda()
    t = torch.randint(0, V, (T,), generator=g)
    t[torch.rand(T, generator=g) < 0.1] = -100
    if T > 3:
        t[0], t[1], t[2] = V - 1, 0, V          # the vocabulary's ends, and one past it
    d = torch.randn(T, generator=g).abs() / T
    return x, w, t.cuda(), d.cuda()


def reference(x, w, t, d):
    z = x.to(F64) @ w.to(F64).t()
    size = x.to(F64).abs() @ w.to(F64).abs().t()
    lse = torch.logsumexp(z, 1)
    has = (t >= 0) & (t < w.shape[0])
    hot = torch.zeros_like(z)
    hot[has, t[has]] = 1
    p = torch.exp(z - lse[:, None])
    g = (p - hot) * (d.to(F64) * has)[:, None]
    zerr = size * x.shape[1] * 2.0 ** -24
    return z, lse, has, hot, p, g, zerr


SHAPES = [(1, 1, 8), (1, 1000, 64), (2, 7, 72), (16, 3001, 256), (64, 256, 128), (65, 257, 136), (128, 512, 64),
          (129, 511, 200), (200, 5000, 320), (256, 1024, 512), (257, 1025, 520), (300, 9001, 1600), (777, 2111, 1000),
          (1100, 4096, 64), (5, 40007, 72)]


@pytest.mark.parametrize("T,V,D", SHAPES)
def test_forward(fp8, T, V, D):
    say("loss forward", T, V, D)
    x, w, t, d = make(T, V, D, T + V + D)
    loss, lse = fp8.linear_cross_entropy(x, w, t)
    z, lse64, has, hot, p, g, zerr = reference(x, w, t, d)
    tol = zerr.amax(1) + 2.0 ** -18 + lse64.abs() * 2.0 ** -22
    assert ((lse.to(F64) - lse64).abs() <= tol).all()
    want = torch.where(has, lse64 - (z * hot).sum(1), 0.0)
    assert ((loss.to(F64) - want).abs() <= 2 * tol + 2.0 ** -22 * (z * hot).sum(1).abs()).all()
    assert (loss[~has] == 0).all()


def check_gradients(x, w, t, d, dx, dw):
    z, lse64, has, hot, p, g, zerr = reference(x, w, t, d)
    gerr = U * g.abs() + p * (d.to(F64) * has)[:, None] * (2 * zerr.amax(1, keepdim=True) + 2.0 ** -16)
    a, b = x.to(F64), w.to(F64)
    for got, want, slack, size in ((dx, g @ b, gerr @ b.abs(), g.abs() @ b.abs()),
                                   (dw, g.t() @ a, gerr.t() @ a.abs(), g.t().abs() @ a.abs())):
        n = max(x.shape[0], w.shape[0])
        bad = (got.to(F64) - want).abs() > U * want.abs() + slack + size * n * 2.0 ** -24 + 1e-37
        assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())


@pytest.mark.parametrize("T,V,D", SHAPES)
def test_backward(fp8, T, V, D):
    say("loss backward", T, V, D)
    x, w, t, d = make(T, V, D, T + 3 * V + D)
    _, lse = fp8.linear_cross_entropy(x, w, t)
    dx, dw = fp8.linear_cross_entropy_backward(d, x, w, t, lse)
    check_gradients(x, w, t, d, dx, dw)


@pytest.mark.parametrize("T,V,D", [(9000, 8500, 64), (17000, 5001, 72)])
def test_backward_in_several_pieces(fp8, T, V, D):
    """More columns than one piece of the vocabulary holds at this many tokens."""
    say("loss backward, pieces", T, V, D)
    x, w, t, d = make(T, V, D, 5)
    loss, lse = fp8.linear_cross_entropy(x, w, t)
    dx, dw = fp8.linear_cross_entropy_backward(d, x, w, t, lse)
    check_gradients(x, w, t, d, dx, dw)


@pytest.mark.parametrize("T,V,D", [(5000, 300, 136), (2049, 1, 8), (4096, 256, 264), (1500, 1700, 1032)])
def test_backward_of_a_small_vocabulary(fp8, T, V, D):
    """dweight's sum over the tokens is split over workgroups."""
    test_backward(fp8, T, V, D)


@pytest.mark.parametrize("T,V,D", [(255, 2048, 256), (17, 4096, 128), (1023, 1000, 64)])
def test_a_mean_is_not_rounded_into_every_gradient(fp8, T, V, D):
    """1 / T next to the middle between two bf16 values: as a factor of g it would be off by
    2^-8 for every token alike.  The roundings left are the results' own (an rms of at
    most 2^-8 / sqrt 3, uniform in the last place) and g's, where a target's p - 1 rounds to
    -1 (p, about 1 / V at these logits, up to e^1 of it)."""
    x, w, t, d = make(T, V, D, 3, sigma=0.1 * D ** -0.5)
    d = torch.full_like(d, 1.0 / T)
    _, lse = fp8.linear_cross_entropy(x, w, t)
    dx, dw = fp8.linear_cross_entropy_backward(d, x, w, t, lse)
    *_, g, _ = reference(x, w, t, d)
    for got, want in ((dx, g @ w.to(F64)), (dw, g.t() @ x.to(F64))):
        off = float((got.to(F64) - want).norm() / want.norm())
        assert off <= 2.0 ** -8 / 3 ** 0.5 + 2.72 / V, off


def test_gradient_against_differences(fp8):
    T, V, D = 3, 11, 8
    x, w, t, d = make(T, V, D, 4, sigma=1.0)
    t[1] = -100
    _, lse = fp8.linear_cross_entropy(x, w, t)
    grads = fp8.linear_cross_entropy_backward(d, x, w, t, lse)

    def total(x, w):
        z = x @ w.t()
        has = t >= 0
        return ((torch.logsumexp(z, 1) - z.gather(1, t.clamp(min=0)[:, None])[:, 0]) * d.to(F64) * has).sum()

    base = [x.to(F64), w.to(F64)]
    for which, got in enumerate(grads):
        want = torch.zeros_like(base[which])
        for i in range(want.numel()):
            val = []
            for sign in (1, -1):
                moved = [b.clone() for b in base]
                moved[which].view(-1)[i] += sign * 1e-6
                val.append(total(*moved))
            want.view(-1)[i] = (val[0] - val[1]) / 2e-6
        # g and the result rounded to bf16: two roundings of 2^-8
        assert torch.linalg.norm(got.to(F64) - want) <= 0.01 * torch.linalg.norm(want), which


def test_no_target_at_all_and_rows_that_are_not_finite(fp8):
    T, V, D = 70, 300, 64
    x, w, t, d = make(T, V, D, 8)
    t[:] = -1
    loss, lse = fp8.linear_cross_entropy(x, w, t)
    dx, dw = fp8.linear_cross_entropy_backward(d, x, w, t, lse)
    assert (loss == 0).all() and (dx == 0).all() and (dw == 0).all() and torch.isfinite(lse).all()
    # a token without a target may be anything: its gradient row is zero, its logits its own
    x, w, t, d = make(T, V, D, 8)
    clean = fp8.linear_cross_entropy(x, w, t)
    t[5] = -100
    x2 = x.clone()
    x2[5] = float("nan")
    loss, lse = fp8.linear_cross_entropy(x2, w, t)
    others = torch.arange(T, device="cuda") != 5
    assert loss[5] == 0 and torch.equal(loss[others], clean[0][others]) and torch.equal(lse[others], clean[1][others])
    dx, _ = fp8.linear_cross_entropy_backward(d, x2, w, t, lse)
    assert (dx[5] == 0).all() and torch.isfinite(dx.float()).all()


def test_large_logits(fp8):
    """Logits in the hundreds: the maximum is taken out before the exponential."""
    T, V, D = 40, 700, 64
    x, w, t, d = make(T, V, D, 9, sigma=20.0)
    loss, lse = fp8.linear_cross_entropy(x, w, t)
    z, lse64, has, hot, p, g, zerr = reference(x, w, t, d)
    assert torch.isfinite(loss).all()
    assert ((lse.to(F64) - lse64).abs() <= zerr.amax(1) + 2.0 ** -18 + lse64.abs() * 2.0 ** -22).all()


def test_same_bytes_every_time_and_on_another_stream(fp8):
    x, w, t, d = make(500, 3000, 512, 10)

    def run():
        loss, lse = fp8.linear_cross_entropy(x, w, t)
        return (loss, lse) + fp8.linear_cross_entropy_backward(d, x, w, t, lse)

    first = run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        second = run()
    side.synchronize()
    for a, b in zip(first, second):
        assert torch.equal(a, b)


def test_refusals(fp8):
    x, w, t, d = make(8, 32, 64, 1)
    loss, lse = fp8.linear_cross_entropy(x, w, t)
    with pytest.raises(TypeError):
        fp8.linear_cross_entropy(x.float(), w, t)
    with pytest.raises(TypeError):
        fp8.linear_cross_entropy(x, w, t.int())
    with pytest.raises(ValueError):
        fp8.linear_cross_entropy(x, w[:, :32].contiguous(), t)
    with pytest.raises(ValueError):
        fp8.linear_cross_entropy(x, w, t[:4])
    with pytest.raises(ValueError):
        fp8.linear_cross_entropy(x[:, :32], w[:, :32], t)
    with pytest.raises(fp8.Fp8Error, match="multiple of 8"):
        fp8.linear_cross_entropy(x[:, :60].contiguous(), w[:, :60].contiguous(), t)
    with pytest.raises(fp8.Fp8Error, match="positive"):
        fp8.linear_cross_entropy(x[:0], w, t[:0])
    with pytest.raises(fp8.Fp8Error, match="overlapping"):
        fp8.linear_cross_entropy_backward(d, x, w, t, lse, dx=x)
    with pytest.raises(fp8.Fp8Error, match="overlapping"):
        fp8.linear_cross_entropy(x, w, t, loss=loss, lse=loss)
