"""A single packed token sliced from a head-major tensor, whose heads lie far apart: the same
bytes as from a contiguous one, which the other tests hold to float64."""
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


def sliced(heads, length, d, at, seed):
    """Token `at` of a head-major [heads, length, d] tensor of random values, as [1, heads, d]."""
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    whole = torch.randn(heads, length, d, generator=g, device="cuda", dtype=torch.float32).to(BF16)
    return whole[:, at:at + 1].transpose(0, 1)


def random(*shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(BF16).cuda()


# strides between heads of 1 MB, 8.4 MB and 16.8 MB
@pytest.mark.parametrize("heads,length,d", [(32, 4096, 128), (32, 32768, 128), (16, 131072, 64)])
@pytest.mark.parametrize("single", ["q", "k", "both"])
def test_one_token_with_heads_far_apart(fp8, heads, length, d, single):
    say("attention, one token", heads, length, d, single)
    n = 100
    far = lambda seed: sliced(heads, length, d, length - 1, seed)
    q, dout = (far(1), far(2)) if single != "k" else (random(n, heads, d, seed=1), random(n, heads, d, seed=2))
    k, v = (far(3), far(4)) if single != "q" else (random(n, heads, d, seed=3), random(n, heads, d, seed=4))
    near = [t.contiguous() for t in (q, k, v, dout)]
    out, lse = fp8.attention(q, k, v)
    want_out, want_lse = fp8.attention(*near[:3])
    assert torch.equal(out, want_out) and torch.equal(lse, want_lse)
    got = fp8.attention_backward(dout, q, k, v, out, lse)
    want = fp8.attention_backward(near[3], *near[:3], out, lse)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_outputs_of_one_token_with_heads_far_apart(fp8):
    """The results of single tokens written into head-major tensors; nothing else there changes."""
    heads, length, d, at = 8, 65536, 128, 70
    say("attention, outputs of one token", heads, length, d)
    q, k, v, dout = (random(1, heads, d, seed=i) for i in range(4))
    whole = [torch.full((heads, length, d), 3.0, dtype=BF16, device="cuda") for _ in range(4)]
    out, dq, dk, dv = (t[:, at:at + 1].transpose(0, 1) for t in whole)
    _, lse = fp8.attention(q, k, v, out=out)
    o, z = fp8.attention(q, k, v)
    fp8.attention_backward(dout, q, k, v, o, z, dq=dq, dk=dk, dv=dv)
    want = (o,) + fp8.attention_backward(dout, q, k, v, o, z)
    assert torch.equal(lse, z)
    for t, part, w in zip(whole, (out, dq, dk, dv), want):
        assert torch.equal(part, w)
        part.fill_(3.0)
        assert (t == 3.0).all()
