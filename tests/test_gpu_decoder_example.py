"""examples/decoder_step.py: the gradients of its step against torch's autograd on the same
decoder in float32, and its loss over a few steps.

The step's linears are FP8: E4M3 rounds to 4 significant bits (relative error up to 2^-4,
rms about 2^-5.3 = 0.026) and E5M2 gradients to 3 (rms 0.05).  A weight's gradient meets both once
at its own linear and what the linears behind it have left: with four of them, a relative
Frobenius error of 0.2 leaves a factor of two.  The head and the last norm lie behind
the forward's errors alone.
"""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def reference(w, sizes, x, lens, target):
    """Loss and gradients in float32 by autograd (on the CPU)."""
    p = {n: t.float().cpu().requires_grad_() for n, t in w.items()}
    x = x.float().cpu().requires_grad_()
    rms = lambda t, n: t * torch.rsqrt((t * t).mean(1, keepdim=True) + 1e-5) * p[n]
    hd, hq, hk = sizes.head_dim, sizes.heads, sizes.kv_heads
    qkv = rms(x, "norm1") @ p["qkv"].t()
    q, k, v = (t.unflatten(1, (-1, hd)) for t in qkv.split([sizes.d, hk * hd, hk * hd], 1))
    outs, at = [], 0
    for n in lens:
        a, b, c = (t[at:at + n].transpose(0, 1) for t in (q, k, v))
        b, c = b.repeat_interleave(hq // hk, 0), c.repeat_interleave(hq // hk, 0)
        s = (a @ b.transpose(1, 2)) * hd ** -0.5
        s = s.masked_fill(torch.ones(n, n).triu(1) > 0, -float("inf"))
        outs.append((torch.softmax(s, 2) @ c).transpose(0, 1))
        at += n
    x2 = x + torch.cat(outs).flatten(1) @ p["o"].t()
    gate, up = (rms(x2, "norm2") @ p["gate_up"].t()).chunk(2, 1)
    x3 = x2 + (torch.nn.functional.silu(gate) * up) @ p["down"].t()
    z = rms(x3, "norm3") @ p["head"].t()
    loss = torch.nn.functional.cross_entropy(z, target.cpu(), ignore_index=-100)
    loss.backward()
    return loss.item(), {**{n: t.grad for n, t in p.items()}, "x": x.grad}


def test_step_against_autograd():
    import decoder_step as ex
    sizes = ex.Sizes(d=256, ffn=384, heads=4, kv_heads=2, vocab=701)
    lens = [100, 1, 27, 128]
    w = ex.init(sizes, 1)
    x, cu, target = ex.batch(sizes, lens, 2)
    print("[case] decoder step", sizes, flush=True)
    loss, g = ex.step(w, sizes, x, cu, target)
    want, ref = reference(w, sizes, x, lens, target)
    assert abs(loss.item() - want) <= 0.02 * want
    for name, t in ref.items():
        err = (torch.linalg.norm(g[name].float().cpu().view_as(t) - t) / torch.linalg.norm(t)).item()
        assert err <= (0.1 if name in ("head", "norm3") else 0.2), (name, err)


def test_loss_falls():
    import decoder_step as ex
    sizes = ex.Sizes(d=256, ffn=384, heads=4, kv_heads=2, vocab=701)
    w = ex.init(sizes, 3)
    x, cu, target = ex.batch(sizes, [128, 128], 4)
    losses = []
    for _ in range(5):
        loss, g = ex.step(w, sizes, x, cu, target)
        losses.append(loss.item())
        for name, t in w.items():
            t.copy_(t.float() - 0.5 * g[name].float().view_as(t))
    assert losses[-1] < losses[0] - 0.05, losses
