"""Attention over packed sequences, forward and backward, against a float64 evaluation.

Tolerances, elementwise, from the roundings (u = 2^-8, bf16's unit):
 - scores are fp32 sums of exact products and p is off by at most e = 2^-11 relative
   (d 2^-24 of the sum of magnitudes of a score, which for these inputs is below 40,
   plus the exponential and the sum over the keys);
 - out and dv are sums with p rounded once (u) and are rounded once themselves (u);
 - ds = p (dp - delta) is rounded once (u) and carries p's e and fp32 errors of dp and
   delta (2^-16 of their sums of magnitudes); dq and dk are sums of it, rounded once;
 - delta is the sum of p dp.  Over more than 128 keys it may be taken as dout . out, and
   then carries out's two roundings (u of |dout| . |out| and of |dout| . sum p |v|).
The backward call is checked for the lse that it is given, and the whole gradient
against differences.
"""
import itertools

import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu

F64, BF16 = torch.float64, torch.bfloat16
U, E = 2.0 ** -8 * 1.01, 2.0 ** -11


@pytest.fixture(scope="module")
def fp8():
    import fp8_precision_amd
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    return fp8_precision_amd


def bounds(lens):
    return torch.tensor([0] + list(itertools.accumulate(lens)), dtype=torch.int32, device="cuda")


def make(lq, lk, hq, hk, d, seed, fused=False):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g).to(BF16).cuda()
    tq, tk = sum(lq), sum(lk)
    if fused:
        x = n(tq, (hq + 2 * hk) * d)
        q, k, v = (y.unflatten(1, (-1, d)) for y in x.split([hq * d, hk * d, hk * d], 1))
    else:
        q, k, v = n(tq, hq, d), n(tk, hk, d), n(tk, hk, d)
    return q, k, v, n(tq, hq, d)


def visible(nq, nk, causal):
    i, j = torch.arange(nq, device="cuda")[:, None], torch.arange(nk, device="cuda")[None, :]
    return (j <= i + nk - nq) if causal else torch.ones(nq, nk, dtype=torch.bool, device="cuda")


def pieces(lq, lk, hq):
    q0 = k0 = 0
    for a, b in zip(lq, lk):
        for h in range(hq):
            yield slice(q0, q0 + a), slice(k0, k0 + b), h
        q0, k0 = q0 + a, k0 + b


def check_forward(q, k, v, out, lse, lq, lk, causal, scale):
    group = q.shape[1] // k.shape[1]
    for qs, ks, h in pieces(lq, lk, q.shape[1]):
        a, b, c = q[qs, h].to(F64), k[ks, h // group].to(F64), v[ks, h // group].to(F64)
        seen = visible(len(a), len(b), causal)
        s = (a @ b.t() * scale).masked_fill(~seen, -float("inf"))
        z = torch.logsumexp(s, 1) if len(b) else torch.full((len(a),), -float("inf"), dtype=F64, device="cuda")
        p = torch.where(seen, torch.exp(s - torch.where(z.isinf(), 0.0, z)[:, None]), 0.0)
        o = p @ c
        got = out[qs, h].to(F64)
        assert ((got - o).abs() <= U * o.abs() + (U + 2 * E) * (p @ c.abs()) + 1e-30).all()
        empty = ~seen.any(1)
        assert (got[empty] == 0).all() and torch.isneginf(lse[h, qs][empty]).all()
        assert ((lse[h, qs].to(F64) - z)[~empty].abs() <= E + 2.0 ** -22 * z[~empty].abs()).all()


def check_backward(dout, q, k, v, out, lse, dq, dk, dv, lq, lk, causal, scale):
    group = q.shape[1] // k.shape[1]
    want = {n: torch.zeros(t.shape, dtype=F64, device="cuda") for n, t in (("dq", q), ("dk", k), ("dv", v))}
    slack = {n: torch.zeros_like(t) for n, t in want.items()}
    for qs, ks, h in pieces(lq, lk, q.shape[1]):
        kh = h // group
        a, b, c, g, o = (t.to(F64) for t in (q[qs, h], k[ks, kh], v[ks, kh], dout[qs, h], out[qs, h]))
        seen = visible(len(a), len(b), causal)
        z = lse[h, qs].to(F64)[:, None]
        p = torch.where(seen, torch.exp(a @ b.t() * scale - torch.where(z.isinf(), 0.0, z)), 0.0)
        dp = g @ c.t()
        delta = (p * dp).sum(1, keepdim=True)
        ds = p * (dp - delta)
        err = (U + E) * ds.abs() + p * 2.0 ** -16 * (g.abs() @ c.abs().t() + (g * o).abs().sum(1, keepdim=True))
        if len(b) > 128:
            err = err + p * U * (g.abs() * (o.abs() + p @ c.abs())).sum(1, keepdim=True)
        want["dv"][ks, kh] += p.t() @ g
        slack["dv"][ks, kh] += (U + 2 * E) * (p.t() @ g.abs())
        want["dq"][qs, h] = scale * (ds @ b)
        slack["dq"][qs, h] = scale * (err @ b.abs()) + E * scale * (ds.abs() @ b.abs())
        want["dk"][ks, kh] += scale * (ds.t() @ a)
        slack["dk"][ks, kh] += scale * (err.t() @ a.abs()) + E * scale * (ds.abs().t() @ a.abs())
    for n, got in (("dq", dq), ("dk", dk), ("dv", dv)):
        bad = (got.to(F64) - want[n]).abs() > U * want[n].abs() + slack[n] + 1e-30
        assert not bad.any(), (n, int(bad.sum()), bad.nonzero()[:4].tolist())


CASES = [
    # lq, lk, hq, hk, d, causal
    ([1], [1], 1, 1, 128, True),
    ([1], [700], 8, 2, 128, True),                      # a single token against a long context
    ([5], [3], 2, 1, 64, True),                         # the first two queries see nothing
    ([128], [128], 2, 2, 128, True),
    ([129], [129], 3, 1, 128, True),
    ([200], [64], 2, 2, 64, True),                      # whole tiles of queries see nothing
    ([64], [513], 4, 2, 64, False),
    ([257, 0, 1, 33], [257, 0, 1, 33], 5, 5, 128, True),
    ([31, 40, 7, 300], [0, 90, 600, 1], 4, 1, 80, True),     # an empty key side
    ([0, 40, 0], [10, 50, 0], 2, 2, 32, False),
    ([31, 40, 7], [1, 90, 333], 6, 2, 8, False),
    ([700, 321], [700, 321], 16, 2, 104, True),
    ([2000], [2000], 8, 8, 128, True),
    ([1000], [1500], 8, 1, 64, True),
    ([300, 17] * 40, [300, 17] * 40, 2, 1, 64, True),   # more than 64 sequences
    # few queries on many keys: the keys split over workgroups and joined
    ([1], [5001], 4, 2, 128, True),
    ([90], [3000], 2, 1, 80, False),
    ([3, 100, 40], [2500, 90, 0], 4, 4, 64, True),      # some splits, and some sequences, have nothing to do
    ([130], [8000], 1, 1, 128, True),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{c[0][0]}-{c[1][0]}-{c[2]}h{c[3]}-d{c[4]}-{'c' if c[5] else 'f'}")
def test_forward_and_backward(fp8, case):
    lq, lk, hq, hk, d, causal = case
    say("attention", *case)
    q, k, v, dout = make(lq, lk, hq, hk, d, sum(lq) + 7 * d)
    cu_q, cu_k = bounds(lq), bounds(lk)
    scale = d ** -0.5
    top = torch.zeros(1, device="cuda")
    out, lse = fp8.attention(q, k, v, cu_q, cu_k, causal=causal, absmax=top)
    assert top.item() == out.float().abs().max().item()
    check_forward(q, k, v, out, lse, lq, lk, causal, scale)
    top.zero_()
    dq, dk, dv = fp8.attention_backward(dout, q, k, v, out, lse, cu_q, cu_k, causal=causal, absmax=top)
    assert top.item() == max(t.float().abs().max().item() for t in (dq, dk, dv))
    check_backward(dout, q, k, v, out, lse, dq, dk, dv, lq, lk, causal, scale)


# Few queries: the heads that share a key head share tiles, whose rows then are queries of
# several heads; with many keys, split over them.
FEW = [([1] * 70, [37 * i % 130 for i in range(70)], 10, 2, 128, True), ([1, 3, 2], [5000, 0, 4097], 8, 1, 128, True),
       ([2, 64, 0, 61], [1, 300, 5, 40], 12, 4, 64, True), ([1], [20000], 40, 8, 128, False),
       ([5, 130, 1], [700, 130, 9], 6, 2, 72, False), ([63, 1, 40], [10, 2000, 41], 14, 2, 40, True),
       ([1, 1], [1, 0], 200, 1, 8, True)]


@pytest.mark.parametrize("case", FEW, ids=lambda c: f"{len(c[0])}x{c[0][0]}-{c[1][0]}-{c[2]}h{c[3]}-d{c[4]}")
def test_few_queries(fp8, case):
    test_forward_and_backward(fp8, case)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hk,d", [(4, 4, 128), (10, 2, 64), (6, 1, 40)])
def test_gradients_of_short_sequences_carry_their_own_rounding_alone(fp8, hq, hk, d, causal):
    """At most 128 keys: the error's norm is that of one rounding, at most 2^-8 / sqrt 3 of the
    gradient's (uniform in the last place, at the shortest mantissa), and 2^-14 for the rest."""
    lens = [128, 37, 5, 1, 64, 100]
    q, k, v, dout = make(lens, lens, hq, hk, d, 11)
    cu = bounds(lens)
    out, lse = fp8.attention(q, k, v, cu, cu, causal=causal)
    got = fp8.attention_backward(dout, q, k, v, out, lse, cu, cu, causal=causal)
    want = [torch.zeros(t.shape, dtype=F64, device="cuda") for t in (q, k, v)]
    scale = d ** -0.5
    for qs, ks, h in pieces(lens, lens, hq):
        a, b, c, g = (t.to(F64) for t in (q[qs, h], k[ks, h * hk // hq], v[ks, h * hk // hq], dout[qs, h]))
        s = (a @ b.t() * scale).masked_fill(~visible(len(a), len(b), causal), -float("inf"))
        p = torch.softmax(s, 1)
        dp = g @ c.t()
        ds = p * (dp - (p * dp).sum(1, keepdim=True)) * scale
        want[0][qs, h] = ds @ b
        want[1][ks, h * hk // hq] += ds.t() @ a
        want[2][ks, h * hk // hq] += p.t() @ g
    for x, y in zip(got, want):
        assert float((x.to(F64) - y).norm() / y.norm()) <= 2.0 ** -8 / 3 ** 0.5 + 2.0 ** -14


def test_slices_of_one_projection(fp8):
    """q, k, v as slices of one tensor, and the gradients written as slices of one."""
    lens, hq, hk, d = [70, 200], 10, 2, 128
    q, k, v, dout = make(lens, lens, hq, hk, d, 3, fused=True)
    assert not q.is_contiguous()
    cu = bounds(lens)
    out, lse = fp8.attention(q, k, v, cu, cu, causal=True, scale=0.07)
    check_forward(q, k, v, out, lse, lens, lens, True, 0.07)
    whole = torch.full((sum(lens), (hq + 2 * hk) * d), 7.0, dtype=BF16, device="cuda")
    dq, dk, dv = (y.unflatten(1, (-1, d)) for y in whole.split([hq * d, hk * d, hk * d], 1))
    fp8.attention_backward(dout, q, k, v, out, lse, cu, cu, causal=True, scale=0.07, dq=dq, dk=dk, dv=dv)
    check_backward(dout, q, k, v, out, lse, dq, dk, dv, lens, lens, True, 0.07)
    plain = fp8.attention_backward(dout, q.contiguous(), k.contiguous(), v.contiguous(), out, lse, cu, cu, causal=True,
                                   scale=0.07)
    for a, b in zip((dq, dk, dv), plain):
        assert torch.equal(a, b)


def test_heads_outermost_and_shared_by_expansion(fp8):
    """Head-major tensors, and one key head expanded to several by a zero stride."""
    n, h, d = 150, 4, 64
    q, k, v, dout = make([n], [n], h, 1, d, 11)
    q2 = q.transpose(0, 1).contiguous().transpose(0, 1)
    out2 = torch.empty(h, n, d, dtype=BF16, device="cuda").transpose(0, 1)
    out, lse = fp8.attention(q, k, v, causal=True)
    a, b = fp8.attention(q2, k.expand(n, h, d), v.expand(n, h, d), causal=True, out=out2)
    assert torch.equal(a, out) and torch.equal(b, lse)
    grads = fp8.attention_backward(dout, q, k, v, out, lse, causal=True)
    more = fp8.attention_backward(dout, q2, k.expand(n, h, d), v.expand(n, h, d), a, b, causal=True)
    assert torch.equal(grads[0], more[0])
    for shared, each in zip(grads[1:], more[1:]):
        assert torch.allclose(shared.float(), each.float().sum(1, keepdim=True), rtol=0.05, atol=0.05)


def test_rows_outside_every_sequence_are_left_alone(fp8):
    """Bounds that cover part of the tokens: the rest is neither read nor written."""
    d, h = 64, 2
    q, k, v, dout = make([300], [300], h, h, d, 5)
    for t in (q, k, v, dout):
        t[:20] = float("nan")
        t[180:] = float("nan")
    cu = torch.tensor([20, 120, 180], dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 3.0)
    lse = torch.full((h, 300), 5.0, device="cuda")
    fp8.attention(q, k, v, cu, cu, causal=True, out=out, lse=lse)
    grads = [torch.full_like(q, 3.0) for _ in range(3)]
    fp8.attention_backward(dout, q, k, v, out, lse, cu, cu, causal=True, dq=grads[0], dk=grads[1], dv=grads[2])
    ins = [t[20:180].contiguous() for t in (q, k, v, dout)]
    cu0 = torch.tensor([0, 100, 160], dtype=torch.int32, device="cuda")
    o, z = fp8.attention(*ins[:3], cu0, cu0, causal=True)
    want = fp8.attention_backward(ins[3], *ins[:3], o, z, cu0, cu0, causal=True)
    assert torch.equal(out[20:180], o) and torch.equal(lse[:, 20:180], z)
    assert (out[:20] == 3).all() and (out[180:] == 3).all() and (lse[:, :20] == 5).all() and (lse[:, 180:] == 5).all()
    for t, w in zip(grads, want):
        assert torch.equal(t[20:180], w) and (t[:20] == 3).all() and (t[180:] == 3).all()


def test_rows_outside_every_sequence_are_left_alone_by_split_work(fp8):
    d, h = 64, 1
    q, k, v, dout = make([60], [4000], h, h, d, 15)
    cu_q, cu_k = (torch.tensor(b, dtype=torch.int32, device="cuda") for b in ([10, 50], [100, 3900]))
    out, lse = torch.full_like(q, 3.0), torch.full((h, 60), 5.0, device="cuda")
    fp8.attention(q, k, v, cu_q, cu_k, out=out, lse=lse)
    grads = [torch.full_like(t, 3.0) for t in (q, k, v)]
    fp8.attention_backward(dout, q, k, v, out, lse, cu_q, cu_k, dq=grads[0], dk=grads[1], dv=grads[2])
    qs, ks = slice(10, 50), slice(100, 3900)
    check_forward(q[qs], k[ks], v[ks], out[qs], lse[:, qs], [40], [3800], False, d ** -0.5)
    check_backward(dout[qs], q[qs], k[ks], v[ks], out[qs], lse[:, qs], grads[0][qs], grads[1][ks], grads[2][ks], [40],
                   [3800], False, d ** -0.5)
    for t, keep in ((out, qs), (grads[0], qs), (grads[1], ks), (grads[2], ks)):
        rest = torch.ones(len(t), dtype=torch.bool, device="cuda")
        rest[keep] = False
        assert (t[rest] == 3).all()
    assert (lse[:, :10] == 5).all() and (lse[:, 50:] == 5).all()


def test_bounds_out_of_range_are_held_to_the_tensor(fp8):
    d, h = 64, 1
    q, k, v, dout = make([100], [100], h, h, d, 6)
    wild = torch.tensor([-50, 1000], dtype=torch.int32, device="cuda")
    out, lse = fp8.attention(q, k, v, wild, wild, causal=True)
    o, z = fp8.attention(q, k, v, causal=True)
    assert torch.equal(out, o) and torch.equal(lse, z)
    for a, b in zip(fp8.attention_backward(dout, q, k, v, o, z, wild, wild, causal=True),
                    fp8.attention_backward(dout, q, k, v, o, z, causal=True)):
        assert torch.equal(a, b)


def test_a_masked_key_that_is_not_finite_stays_masked(fp8):
    """Scores of unseen keys are dropped by a comparison, not by adding a number."""
    n, d = 96, 64
    q, k, v, dout = make([n], [n], 1, 1, d, 8)
    o, z = fp8.attention(q[:90], k[:90], v[:90], causal=True)
    k2 = k.clone()
    k2[90:] = float("nan")
    out, lse = fp8.attention(q, k2, v, causal=True)
    assert torch.equal(out[:90], o) and torch.equal(lse[:, :90], z)
    assert torch.isnan(out[90:].float()).all()


def test_large_scores(fp8):
    """Scores in the thousands, and a row whose maximum moves by far between tiles."""
    n, d = 300, 128
    q, k, v, dout = make([n], [n], 2, 2, d, 9)
    q, k = q * 16, k * 16
    k[200:] *= 4
    out, lse = fp8.attention(q, k, v, causal=False)
    s = torch.einsum("ihd,jhd->hij", q.to(F64), k.to(F64)) * d ** -0.5
    o = torch.einsum("hij,jhd->ihd", torch.softmax(s, 2), v.to(F64))
    z = torch.logsumexp(s, 2)
    # a score of several thousand is off by up to 128 * 2^-24 of its sum of magnitudes
    assert ((lse.to(F64) - z).abs() <= 2.0 ** -17 * s.abs().amax(2) + 1e-3).all()
    assert torch.isfinite(out.float()).all()
    assert torch.linalg.norm(out.to(F64) - o) <= 0.02 * torch.linalg.norm(o)


def test_gradient_against_differences(fp8):
    """dq, dk, dv against central differences of the float64 forward."""
    lq, lk, d = [6, 4], [9, 3], 8
    q, k, v, dout = make(lq, lk, 2, 1, d, 12)
    cu_q, cu_k = bounds(lq), bounds(lk)
    out, lse = fp8.attention(q, k, v, cu_q, cu_k, causal=True)
    grads = fp8.attention_backward(dout, q, k, v, out, lse, cu_q, cu_k, causal=True)

    def loss(q, k, v):
        t = 0.0
        for qs, ks, h in pieces(lq, lk, 2):
            seen = visible(qs.stop - qs.start, ks.stop - ks.start, True)
            s = (q[qs, h] @ k[ks, 0].t() * d ** -0.5).masked_fill(~seen, -float("inf"))
            p = torch.where(seen.any(1, keepdim=True), torch.softmax(s, 1), 0.0)
            t = t + (torch.where(seen, p, 0.0) @ v[ks, 0] * dout[qs, h].to(F64)).sum()
        return t

    base = [t.to(F64) for t in (q, k, v)]
    for which, got in enumerate(grads):
        want = torch.zeros_like(base[which])
        for i in range(want.numel()):
            val = []
            for sign in (1, -1):
                moved = [t.clone() for t in base]
                moved[which].view(-1)[i] += sign * 1e-6
                val.append(loss(*moved))
            want.view(-1)[i] = (val[0] - val[1]) / 2e-6
        # bf16 out, p and ds: three roundings of 2^-8 on sums of a few terms of order 1
        assert torch.linalg.norm(got.to(F64) - want) <= 0.02 * torch.linalg.norm(want), which


def test_same_bytes_every_time_and_on_another_stream(fp8):
    lens = [900, 300]
    q, k, v, dout = make(lens, lens, 8, 2, 128, 13)
    cu = bounds(lens)

    def run():
        out, lse = fp8.attention(q, k, v, cu, cu, causal=True)
        return (out, lse) + fp8.attention_backward(dout, q, k, v, out, lse, cu, cu, causal=True)

    first = run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        second = run()
    side.synchronize()
    for a, b in zip(first, second):
        assert torch.equal(a, b)


def test_refusals(fp8):
    q, k, v, dout = make([16], [16], 4, 2, 64, 1)
    out, lse = fp8.attention(q, k, v)
    with pytest.raises(TypeError):
        fp8.attention(q.float(), k, v)
    with pytest.raises(ValueError):
        fp8.attention(q, k[:, :, :32], v[:, :, :32])
    with pytest.raises(ValueError):
        fp8.attention(q.transpose(1, 2), k, v)
    with pytest.raises(ValueError):
        fp8.attention(q, k, v, cu_q=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        fp8.attention(q, k, v, cu_q=torch.zeros(2, dtype=torch.int64, device="cuda"), cu_k=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(fp8.Fp8Error, match="multiple of heads_k"):
        fp8.attention(q[:, :3], k, v)
    with pytest.raises(fp8.Fp8Error, match="scale"):
        fp8.attention(q, k, v, scale=0.0)
    with pytest.raises(fp8.Fp8Error, match="positive"):
        fp8.attention(q[:0], k, v)
    with pytest.raises(fp8.Fp8Error, match="head_dim"):
        fp8.attention(*(torch.zeros(4, 2, 136, dtype=BF16, device="cuda") for _ in range(3)))
    with pytest.raises(fp8.Fp8Error, match="overlapping"):
        fp8.attention(q, k, v, out=q)
    with pytest.raises(fp8.Fp8Error, match="overlaps itself"):
        fp8.attention(q, k, v, out=torch.zeros(16, 1, 64, dtype=BF16, device="cuda").expand(16, 4, 64))
    with pytest.raises(fp8.Fp8Error, match="closer than head_dim"):
        fp8.attention(q, torch.zeros(1, 2, 64, dtype=BF16, device="cuda").expand(16, 2, 64), v)
    odd = torch.zeros(16 * 4 * 68, dtype=BF16, device="cuda").view(16, 4, 68)[:, :, :64]
    with pytest.raises(fp8.Fp8Error, match="multiples of 8"):
        fp8.attention(odd, k, v)
    with pytest.raises(fp8.Fp8Error, match="overlapping"):
        fp8.attention_backward(dout, q, k, v, out, lse, dq=dout)
    with pytest.raises(fp8.Fp8Error, match="overlapping"):
        fp8.attention_backward(dout, q, k, v, out, lse, dk=torch.empty_like(k), dv=k)
