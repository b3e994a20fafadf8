"""Attention of more tiles than one launch holds (its threads are counted in 32 bits): sequences of
one token, whose output is their value and whose value's gradient is the output's."""
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


def inputs(batch, heads, d, count):
    g = torch.Generator("cuda").manual_seed(batch)
    # heads outermost: a token's heads may lie far apart, tokens may not
    new = lambda: torch.empty(heads, batch, d, dtype=BF16, device="cuda").normal_(generator=g).transpose(0, 1)
    return torch.arange(batch + 1, dtype=torch.int32, device="cuda"), [new() for _ in range(count)]


def test_forward(fp8):
    batch, heads, d = 256, 65536, 8
    assert (batch // 128 + batch) * heads * 256 > THREADS
    say("attention forward", batch, heads, d)
    cu, (q, k, v) = inputs(batch, heads, d, 3)
    out = torch.full_like(v, 30.0)
    lse = torch.full((heads, batch), 1e9, device="cuda")
    fp8.attention(q, k, v, cu, cu, causal=True, out=out, lse=lse)
    assert torch.equal(out, v)
    s = (q.float() * k.float()).sum(2).t() * d ** -0.5
    # eight products of at most 25 each, and lse's own size: 2^-16 is 8 fp32 units of 32
    assert float((lse - s).abs().max()) <= 2.0 ** -16


def test_backward(fp8):
    batch, heads, d = 128, 65536, 128
    assert batch * heads * 512 >= THREADS
    say("attention backward", batch, heads, d)
    cu, (q, k, v, dout) = inputs(batch, heads, d, 4)
    out, lse = fp8.attention(q, k, v, cu, cu, out=torch.empty_like(v))
    dq, dk, dv = (torch.full_like(t, 30.0) for t in (q, k, v))
    top = torch.zeros(1, device="cuda")
    fp8.attention_backward(dout, q, k, v, out, lse, cu, cu, absmax=top, dq=dq, dk=dk, dv=dv)
    assert torch.equal(dv, dout) and top.item() == dout.abs().max().item()
    for some in (slice(0, 64), slice(32768, 32832), slice(heads - 64, heads)):
        part = [t[:, some] for t in (dout, q, k, v, out)]
        want = fp8.attention_backward(*part, lse[some].contiguous(), cu, cu)
        for a, b in zip((dq, dk, dv), want):
            assert torch.equal(a[:, some], b)
    # every row was written: p (dp - delta) of a single key is what rounding leaves of zero
    assert dq.abs().max().item() < 1e-2 and dk.abs().max().item() < 1e-2
