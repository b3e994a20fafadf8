"""q, k, v and their gradients as interleaved slices of one tensor: the same bytes as apart."""
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


def slices(t, layout):
    """The [tokens, heads, d] slices of a tensor whose slice axis is the given one."""
    axis = layout.index("s")
    order = [layout.replace("s", "").index(c) for c in "thd"]
    return [t.select(axis, i).permute(order) for i in range(t.shape[axis])]


@pytest.mark.parametrize("tokens", [1, 70, 300])
@pytest.mark.parametrize("layout", ["thsd", "tshd", "hstd", "sthd"])
def test_gradients_are_written_where_their_operands_lie(fp8, layout, tokens):
    say("attention, interleaved", layout, tokens)
    sizes = dict(t=tokens, h=6, d=64, s=4)
    g = torch.Generator().manual_seed(tokens)
    whole = torch.randn([sizes[c] for c in layout], generator=g).to(BF16).cuda()
    q, k, v, out = slices(whole, layout)
    dout = torch.randn(tokens, 6, 64, generator=g).to(BF16).cuda()
    near = [t.contiguous() for t in (q, k, v)]
    want, want_lse = fp8.attention(*near, causal=True)
    _, lse = fp8.attention(q, k, v, causal=True, out=out)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    for a, b in zip((q, k, v), near):
        assert torch.equal(a, b)
    to = torch.full_like(whole, 3.0)
    dq, dk, dv, rest = slices(to, layout)
    fp8.attention_backward(dout, q, k, v, out, lse, causal=True, dq=dq, dk=dk, dv=dv)
    for a, b in zip((dq, dk, dv), fp8.attention_backward(dout, *near, want, want_lse, causal=True)):
        assert torch.equal(a, b)
    assert (rest == 3.0).all()


def test_a_shared_element_is_refused(fp8):
    t, h, d = 20, 3, 64
    q, k, v, dout = (torch.randn(t, h, d, device="cuda").to(BF16) for _ in range(4))
    out, lse = fp8.attention(q, k, v)
    flat = torch.zeros(3 * t * h * d + 64, dtype=BF16, device="cuda")
    at = lambda off: flat.as_strided((t, h, d), (3 * h * d, 3 * d, 1), off)
    for off in (0, 8, d - 8):
        with pytest.raises(fp8.Fp8Error, match="overlapping"):
            fp8.attention_backward(dout, q, k, v, out, lse, dk=at(0), dv=at(off))
