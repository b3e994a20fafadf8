"""Norm, attention and loss, forward and backward, captured in a HIP graph: every replay,
with garbage in the outputs, eager work and synchronisations in between, gives the eager
calls' bytes again."""
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


@pytest.mark.parametrize("lengths,vocab", [([200, 1, 311], 3001), ([1, 5], 40007), ([2100], 260)])
def test_replays(fp8, lengths, vocab):
    say("layer graph", lengths, vocab)
    T, heads, hk, d = sum(lengths), 4, 2, 64
    D = heads * d
    g = torch.Generator().manual_seed(T)
    bf = lambda *s, sd=1.0: (torch.randn(s, generator=g) * sd).to(BF16).cuda()
    stream, add, weight, dy, head = bf(T, D), bf(T, D), bf(D), bf(T, D, sd=0.1), bf(vocab, D, sd=0.05)
    qkv, dout = bf(T, heads + 2 * hk, d), bf(T, heads, d, sd=0.1)
    target = torch.randint(0, vocab, (T,), generator=g).cuda()
    dloss = torch.full((T,), 1.0 / T).cuda()
    cu = torch.tensor([0] + torch.tensor(lengths).cumsum(0).tolist(), dtype=torch.int32).cuda()
    # keys many times as many as queries: split over the keys, and joined
    far = bf(4096, 2 * hk, d)
    few = bf(3, heads, d)
    stats = torch.empty(4, device="cuda")

    def step():
        stats.zero_()
        q, k, v = qkv[:, :heads], qkv[:, heads:heads + hk], qkv[:, heads + hk:]
        y, s, _, rstd = fp8.norm(stream, weight, add=add, absmax=stats[0:1])
        dx, dw, _ = fp8.norm_backward(dy, s, weight, None, rstd, dres=dy)
        o, lse = fp8.attention(q, k, v, cu, cu, causal=True, absmax=stats[1:2])
        grads = fp8.attention_backward(dout, q, k, v, o, lse, cu, cu, causal=True, absmax=stats[2:3])
        o2, lse2 = fp8.attention(few, far[:, :hk], far[:, hk:])
        grads2 = fp8.attention_backward(dout[:1].expand(3, heads, d).contiguous(), few, far[:, :hk], far[:, hk:], o2, lse2)
        loss, z = fp8.linear_cross_entropy(y, head, target)
        lx, lw = fp8.linear_cross_entropy_backward(dloss, y, head, target, z)
        return [stats, y, s, rstd, dx, dw, o, lse, *grads, o2, lse2, *grads2, loss, z, lx, lw]

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    torch.cuda.synchronize()
    for rep in range(4):
        say("replay", rep)
        for t in got:
            t.fill_(float("nan"))
        fp8.absmax(stream)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)), (rep, i)
