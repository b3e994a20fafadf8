#!/usr/bin/env python3
"""A training step of a small decoder, put together from the library's calls.

One block and a language head on packed sequences: norm -> QKV (FP8) -> causal attention
-> output projection (FP8) -> norm with the residual sum -> gate/up (FP8) -> SwiGLU
requantised -> down (FP8) -> norm with the residual sum -> linear cross entropy, forward
and backward.  What each call hands to the next is what it needs there: the norms and
the attention leave the absmax of their outputs for the quantisation that follows, the
attention reads q, k and v as slices of the projection's output and writes their
gradients as slices of its gradient, and no logits are stored.

Usage: python examples/decoder_step.py [--steps 8]
"""
from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fp8_precision_amd as fp8  # noqa: E402

BF16 = torch.bfloat16


@dataclass
class Sizes:
    d: int = 512
    ffn: int = 1024
    heads: int = 8
    kv_heads: int = 2
    vocab: int = 5003

    @property
    def head_dim(self):
        return self.d // self.heads

    @property
    def qkv(self):
        return (self.heads + 2 * self.kv_heads) * self.head_dim


def init(sizes: Sizes, seed: int = 0, device="cuda") -> dict:
    """bf16 weights: linears N(0, 1 / inputs), norms 1."""
    g = torch.Generator().manual_seed(seed)
    w = lambda n, k: (torch.randn(n, k, generator=g) * k ** -0.5).to(BF16).to(device)
    one = lambda: torch.ones(sizes.d, dtype=BF16, device=device)
    return {"norm1": one(), "qkv": w(sizes.qkv, sizes.d), "o": w(sizes.d, sizes.d), "norm2": one(),
            "gate_up": w(2 * sizes.ffn, sizes.d), "down": w(sizes.d, sizes.ffn), "norm3": one(),
            "head": w(sizes.vocab, sizes.d)}


class Linear:
    """y = x w^T in FP8 with just-in-time scales, and its gradients."""

    def __init__(self, x, w, amax=None):
        """x bf16 [tokens, in] with the statistic that its producer took, or None."""
        stats = torch.empty(2, device=x.device)
        fp8.absmax_clear(stats)
        if amax is None:
            amax = stats[0:1]
            fp8.absmax_accumulate_many([x, w], [amax, stats[1:2]])
        else:
            fp8.absmax(w, out=stats[1:2], accumulate=True)
        (self.xq, wq), (self.xqt, self.wqt), _, (self.ix, self.iw) = fp8.quantize_many(
            [x, w], fp8.E4M3, [amax, stats[1:2]], want_qt=True, qt_later=True)
        self.y = fp8.gemm_fwd(self.xq, wq, self.ix, self.iw)

    def backward(self, dy, amax=None):
        """(dx, dw) of dy bf16 [tokens, out]."""
        amax = fp8.absmax(dy) if amax is None else amax
        dyq, dyqt, _, idy = fp8.quantize(dy, fp8.E5M2, amax, want_qt=True)
        return fp8.gemm_backward(dyq, dyqt, fp8.E5M2, self.wqt, self.xqt, idy, self.iw, self.ix)


def step(w: dict, sizes: Sizes, x, cu, target):
    """Mean loss of the tokens with a target, and the gradients of every weight and of x.
    x bf16 [tokens, d] (tokens a multiple of 128), cu int32 bounds of the sequences."""
    tokens, dev = x.shape[0], x.device
    stat = torch.empty(5, device=dev)
    fp8.absmax_clear(stat)
    s = [stat[i:i + 1] for i in range(5)]
    cut = lambda t: [y.unflatten(1, (-1, sizes.head_dim)) for y in
                     t.split([sizes.d] + 2 * [sizes.kv_heads * sizes.head_dim], 1)]

    # forward
    y1, _, _, r1 = fp8.norm(x, w["norm1"], absmax=s[0])
    qkv = Linear(y1, w["qkv"], s[0])
    q, k, v = cut(qkv.y)
    att, lse = fp8.attention(q, k, v, cu, cu, causal=True, absmax=s[1])
    o = Linear(att.flatten(1), w["o"], s[1])
    y2, x2, _, r2 = fp8.norm(x, w["norm2"], add=o.y, absmax=s[2])
    gu = Linear(y2, w["gate_up"], s[2])
    hq, hqt, _, ih = fp8.swiglu_requant(gu.y, want_hqt=True)
    dq8, dqt8, _, idown = fp8.quantize(w["down"], fp8.E4M3, fp8.absmax(w["down"]), want_qt=True)
    down = fp8.gemm_fwd(hq, dq8, ih, idown)
    y3, x3, _, r3 = fp8.norm(x2, w["norm3"], add=down)
    loss, logit_lse = fp8.linear_cross_entropy(y3, w["head"], target)

    # backward: dx3 is the gradient of x3 = x2 + down, and so on down the stream
    g = {}
    count = ((target >= 0) & (target < sizes.vocab)).sum().clamp(min=1)
    dloss = (1.0 / count).expand(tokens).contiguous()
    dy3, g["head"] = fp8.linear_cross_entropy_backward(dloss, y3, w["head"], target, logit_lse)
    dx3, g["norm3"], _ = fp8.norm_backward(dy3, x3, w["norm3"], None, r3)
    dyq, dyqt, _, idy = fp8.quantize(dx3, fp8.E5M2, fp8.absmax(dx3), want_qt=True)
    dh, g["down"] = fp8.gemm_backward(dyq, dyqt, fp8.E5M2, dqt8, hqt, idy, idown, ih)
    guq, guqt, _, _, igu = fp8.swiglu_backward(gu.y, dh, want_qt=True)
    dy2, g["gate_up"] = fp8.gemm_backward(guq, guqt, fp8.E5M2, gu.wqt, gu.xqt, igu, gu.iw, gu.ix)
    dx2, g["norm2"], _ = fp8.norm_backward(dy2, x2, w["norm2"], None, r2, dres=dx3)
    datt, g["o"] = o.backward(dx2)
    dqkv = torch.empty_like(qkv.y)
    dq, dk, dv = cut(dqkv)
    fp8.attention_backward(datt.unflatten(1, (-1, sizes.head_dim)), q, k, v, att, lse, cu, cu, causal=True,
                           absmax=s[3], dq=dq, dk=dk, dv=dv)
    dy1, g["qkv"] = qkv.backward(dqkv, s[3])
    g["x"], g["norm1"], _ = fp8.norm_backward(dy1, x, w["norm1"], None, r1, dres=dx2)
    return loss.sum() / count, g


def batch(sizes: Sizes, lens, seed: int = 0, device="cuda"):
    """Embedded tokens, sequence bounds, and the next token as target (none for a last one)."""
    g = torch.Generator().manual_seed(seed)
    tokens = sum(lens)
    x = torch.randn(tokens, sizes.d, generator=g).to(BF16).to(device)
    target = torch.randint(0, sizes.vocab, (tokens,), generator=g)
    ends = torch.tensor(lens).cumsum(0)
    target[ends[torch.tensor(lens) > 0] - 1] = -100
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), ends]).to(torch.int32).to(device)
    return x, cu, target.to(device)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=8)
    args = ap.parse_args()
    sizes = Sizes()
    w = init(sizes)
    x, cu, target = batch(sizes, [300, 1, 211, 512])
    for i in range(args.steps):
        loss, g = step(w, sizes, x, cu, target)
        for name, t in w.items():                          # plain gradient descent on the bf16 weights
            t.copy_(t.float() - 0.5 * g[name].float().view_as(t))
        print(f"step {i}: loss {loss.item():.4f}", flush=True)


if __name__ == "__main__":
    main()
