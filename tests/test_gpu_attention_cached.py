"""Attention over the paged 8-bit cache against a float64 evaluation of what the codes stand for.

Tolerances, elementwise, from the roundings (u = 2^-8, bf16's unit): keys and values are
exact in bf16; scores are fp32 sums of exact products and p is off by at most e = 2^-11
relative (128 2^-24 of a score's sum of magnitudes, below 40 here, plus the exponential and
the sum over the keys); out is a sum with p rounded once (u) and is rounded once itself (u).
"""
import pytest
import torch

import kv_cache_reference as ref
from gpu_util import say

pytestmark = pytest.mark.gpu
BF16, F64 = torch.bfloat16, torch.float64
U, E = 2.0 ** -8 * 1.01, 2.0 ** -11


@pytest.fixture(scope="module")
def fp8():
    import fp8_precision_amd
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    return fp8_precision_amd


def setup(news, past, hk, d, page, seed, spare=0):
    """A pool whose slots that no sequence holds are random codes, NaNs among them; the held ones finite."""
    lengths = [a + b for a, b in zip(news, past)]
    pages = sum(-(-max(n, 0) // page) for n in lengths) + 2
    table = ref.make_table(lengths, page, pages, seed, spare)
    g = torch.Generator().manual_seed(seed)
    pool = ref.make_pool(pages, hk, page, d, seed)
    for name in "kv":
        for b, n in enumerate(lengths):
            for i in range(-(-n // page)):
                at, rows = int(table[b, i]), min(page, n - i * page)
                x = torch.randn(hk, rows, d, generator=g)
                e = ref.least_exponent(x.to(F64))
                pool[name][at, :, :rows] = ref.nearest(x.to(F64) * 2.0 ** -e)
                pool[name + "_scale"][at] = e + 127 + (at % 3 - 1)
    return pool, table, lengths


def check(q, out, lse, pool, table, lengths, news, causal, scale):
    hk, page = pool["k"].shape[1], pool["k"].shape[2]
    group = q.shape[1] // hk
    total = ref.held(lengths, table, page)
    first = 0
    for b, n in enumerate(news):
        if n == 0:
            continue
        one, held = table[b:b + 1], total[b]
        k, v = (ref.read(pool, one, [held], [held], x).cuda() for x in "kv")
        rows = slice(first, first + n)
        first += n
        i, j = torch.arange(n, device="cuda")[:, None], torch.arange(held, device="cuda")[None, :]
        seen = (j <= i + max(lengths[b], 0) - n) if causal else torch.ones(n, held, dtype=torch.bool, device="cuda")
        empty = ~seen.any(1)
        for h in range(q.shape[1]):
            s = (q[rows, h].to(F64) @ k[:, h // group].t() * scale).masked_fill(~seen, -float("inf"))
            z = torch.logsumexp(s, 1) if held else torch.full((n,), -float("inf"), dtype=F64, device="cuda")
            p = torch.exp(s - torch.where(z.isinf(), 0.0, z)[:, None])
            o, slack = p @ v[:, h // group], p @ v[:, h // group].abs()
            got = out[rows, h].to(F64)
            bad = (got - o).abs() > U * o.abs() + (U + 2 * E) * slack + 1e-30
            assert not bad.any(), (b, h, int(bad.sum()), bad.nonzero()[:4].tolist())
            assert (got[empty] == 0).all() and torch.isneginf(lse[h, rows][empty]).all()
            assert ((lse[h, rows].to(F64) - z)[~empty].abs() <= E + 2.0 ** -22 * z[~empty].abs()).all(), (b, h)


CASES = [
    # new tokens, held before, hq, hk, d, page, causal
    ([1], [0], 1, 1, 128, 64, True), ([1], [1], 8, 1, 64, 16, True), ([1], [700], 8, 2, 128, 64, True),
    ([1], [5000], 5, 1, 128, 128, True), ([1, 1, 1], [63, 64, 15], 4, 4, 128, 64, True),
    ([1] * 33, [37 * i % 400 for i in range(33)], 10, 2, 128, 32, True),
    ([5, 0, 3, 1], [100, 50, 0, 333], 12, 4, 64, 16, True), ([7, 2], [0, 600], 6, 3, 72, 16, True),
    ([17, 1], [300, 5], 16, 1, 128, 64, True), ([4, 4], [31, 200], 4, 2, 40, 32, False),
    ([130, 1, 64], [70, 900, 0], 4, 2, 128, 64, True), ([257], [0], 3, 3, 128, 16, True),
    ([65, 40, 1, 0, 300], [0, 90, 600, 5, 1], 5, 1, 80, 32, True), ([200], [313], 8, 8, 64, 128, False),
    ([31, 40, 7], [1, 90, 333], 6, 2, 8, 16, True), ([9], [3], 40, 8, 120, 64, True),
    ([40], [968], 8, 1, 64, 16, True),                   # few tiles, split: the last step part of one
    ([1100], [3000], 64, 8, 128, 64, True),              # 552 tiles: those behind the first 512 are split
    ([6] * 3, [40, 2000, 300], 5, 1, 128, 64, True),     # 30 rows, in shares where all have as many
    ([4] * 5, [0, 5000, 77, 1, 900], 16, 2, 72, 32, False),
    ([1] * 300, [i % 50 for i in range(300)], 2, 1, 64, 16, True), ([600, 1, 500], [1500, 3000, 0], 10, 2, 128, 64, True),
    ([40], [568], 8, 1, 64, 16, True),                   # split from 10 steps on, and from 16 with more tiles: the last part of one
    ([520], [488], 16, 16, 64, 16, True),
    ([6] * 3, [40, 800, 300], 5, 1, 128, 64, True),      # 30 rows, each head by one workgroup where all have as many
    ([8] * 2, [0, 100], 8, 2, 72, 16, False),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_float64(fp8, case):
    news, past, hq, hk, d, page, causal = CASES[case]
    say("attention_cached", CASES[case])
    pool, table, lengths = setup(news, past, hk, d, page, case, spare=case % 3)
    q = torch.randn(sum(news), hq, d, generator=torch.Generator().manual_seed(case)).to(BF16).cuda()
    top = torch.full((1,), 0.25, device="cuda")
    n = torch.tensor(lengths, dtype=torch.int32).cuda()
    cache = ref.on_gpu(fp8, pool)
    out, lse = fp8.attention_cached(q, cache, table.cuda(), n, cu=ref.bounds(news), causal=causal, absmax=top)
    check(q, out, lse, pool, table, lengths, news, causal, d ** -0.5)
    assert top.item() == max(0.25, out.float().abs().max().item())
    if len(set(news)) == 1:                               # the same work without bounds: the same rows
        out2, lse2 = fp8.attention_cached(q, cache, table.cuda(), n, causal=causal, scale=d ** -0.5)
        check(q, out2, lse2, pool, table, lengths, news, causal, d ** -0.5)
    again, lse3 = fp8.attention_cached(q, cache, table.cuda(), n, cu=ref.bounds(news), causal=causal)
    assert torch.equal(again, out) and torch.equal(lse3, lse)


UNEVEN = [
    # few tiles, each sequence's split as its own length has it: 1 to 16 parts a tile, then 2, 3 and none
    ([122, 38, 1, 425, 2, 2], [36, 1997, 105, 0, 3990, 488], 1, 1, 128, 64, True),
    ([44, 5, 137, 2, 1], [1923, 2, 270, 13, 11], 64, 8, 104, 64, True),
    ([900, 533, 53], [6260, 3769, 1086], 36, 18, 64, 128, True),
    ([17, 129], [69000, 0], 1, 1, 64, 128, False),       # as many parts as there can be
    ([2000, 3], [-900, 40], 1, 1, 64, 16, True),         # the middle query of the longest sees nothing
    ([18] * 70, [3] * 69 + [5000], 1, 1, 64, 32, True),  # more sequences than a wave has lanes
]


@pytest.mark.parametrize("case", range(len(UNEVEN)))
def test_uneven_tiles(fp8, case):
    news, past, hq, hk, d, page, causal = UNEVEN[case]
    say("uneven", UNEVEN[case])
    pool, table, lengths = setup(news, past, hk, d, page, 50 + case)
    q = torch.randn(sum(news), hq, d, generator=torch.Generator().manual_seed(case)).to(BF16).cuda()
    n = torch.tensor(lengths, dtype=torch.int32).cuda()
    call = lambda: fp8.attention_cached(q, ref.on_gpu(fp8, pool), table.cuda(), n, cu=ref.bounds(news), causal=causal)
    out, lse = call()
    check(q, out, lse, pool, table, lengths, news, causal, d ** -0.5)
    again, lse2 = call()
    assert torch.equal(again, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("batch, heads, longest", [(128, 8, 2048), (127, 8, 2048), (128, 8, 2049), (64, 32, 4096)])
def test_many_heads(fp8, batch, heads, longest):
    """Many heads' rows are each read by one workgroup up to some length of the table's rows, else shared out."""
    say("many heads", batch, heads, longest)
    past = [longest - 1] + [37 * i % 300 for i in range(batch - 1)]
    pool, table, lengths = setup([1] * batch, past, heads, 64, 64, 3)
    q = torch.randn(batch, heads, 64, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    top = torch.zeros(1, device="cuda")
    out, lse = fp8.attention_cached(q, ref.on_gpu(fp8, pool), table.cuda(), torch.tensor(lengths, dtype=torch.int32).cuda(), absmax=top)
    check(q, out, lse, pool, table, lengths, [1] * batch, True, 0.125)
    assert top.item() == out.float().abs().max().item()


@pytest.mark.parametrize("scale", [1e-30, 1e-3, 3.0])
def test_scales(fp8, scale):
    say("scale", scale)
    pool, table, lengths = setup([1, 20], [500, 40], 2, 64, 32, 1)
    for n in ("k_scale",):
        pool[n] -= 2 if scale > 1 else 0                  # scores stay below 100
    q = torch.randn(21, 4, 64, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    out, lse = fp8.attention_cached(q, ref.on_gpu(fp8, pool), table.cuda(), torch.tensor(lengths, dtype=torch.int32).cuda(),
                                    cu=ref.bounds([1, 20]), scale=scale)
    check(q, out, lse, pool, table, lengths, [1, 20], True, scale)


@pytest.mark.parametrize("news", [[20, 30, 5, 8, 3, 1], [200, 30, 5, 8, 3, 1]])
def test_places_that_are_not_there(fp8, news):
    """Queries before a sequence's first token see nothing; keys in a block without a page are zeros,
    past the table there are none; rows behind the last sequence keep what they hold."""
    heads, d, page = 2, 64, 16
    lengths = [10, 60, 33, -4, 2147483647, 48]
    say("no places", news)
    table = torch.tensor([[0, -1, 2], [9, 1, 1 << 30], [3, -5, 9], [4, 5, 6], [7, -2147483648, 8], [-1, -1, -1]], dtype=torch.int32)
    pool = ref.make_pool(9, heads, page, d, 2, stale=False)
    pool["k"][0, :, 10:], pool["v"][0, :, 10:] = 127, 255                # NaN codes behind the last token
    q = torch.randn(sum(news) + 9, 6, d, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    q[sum(news):] = float("nan")
    out, lse = torch.full((sum(news) + 9, 6, d), 7.0, dtype=BF16, device="cuda"), torch.full((6, sum(news) + 9), 7.0, device="cuda")
    fp8.attention_cached(q, ref.on_gpu(fp8, pool), table.cuda(), torch.tensor(lengths, dtype=torch.int32).cuda(),
                         cu=ref.bounds(news), scale=2.0 ** -8, out=out, lse=lse)
    check(q, out, lse, pool, table, lengths, news, True, 2.0 ** -8)
    assert (out[sum(news):] == 7).all() and (lse[:, sum(news):] == 7).all()


def test_bounds_in_no_order(fp8):
    say("wild bounds")
    pool, table, lengths = setup([1] * 5, [40, 100, 6, 60, 90], 1, 64, 16, 1)
    cu = torch.tensor([-7, 12, 5, 1000, 3, 2000], dtype=torch.int32).cuda()
    q = torch.randn(50, 4, 64, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    out, lse = fp8.attention_cached(q, ref.on_gpu(fp8, pool), table.cuda(), torch.tensor(lengths, dtype=torch.int32).cuda(), cu=cu)
    torch.cuda.synchronize()
    # the rows that one sequence alone claims are its queries: 0 .. 2 of the first, whose twelve
    # queries are the last of what it holds
    k, v = (ref.read(pool, table[:1], lengths[:1], [lengths[0]], x)[:, 0].cuda() for x in "kv")
    for i in range(3):
        n = lengths[0] - 12 + i + 1
        s = q[i].to(F64) @ k[:n].t() * 0.125
        p = torch.softmax(s, 1)
        assert ((out[i].to(F64) - p @ v[:n]).abs() <= 2 * U * (p @ v[:n].abs()) + 2 * E * (p @ v[:n].abs())).all()


@pytest.mark.parametrize("batch", [2, 400])
def test_bounds_that_overlap(fp8, batch):
    """Every second sequence claims all tokens: more rows than the call has; nothing outside is touched."""
    say("overlapping bounds", batch)
    pool, table, lengths = setup([1] * batch, [70] * batch, 1, 64, 16, 2)
    cu = torch.tensor(([0, 300] * batch)[:batch + 1], dtype=torch.int32).cuda()
    q = torch.randn(300, 4, 64, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    out = torch.full((310, 4, 64), 7.0, dtype=BF16, device="cuda")
    cache = ref.on_gpu(fp8, pool)
    fp8.attention_cached(q, cache, table.cuda(), torch.tensor(lengths, dtype=torch.int32).cuda(), cu=cu, out=out[:300])
    torch.cuda.synchronize()
    assert (out[300:] == 7).all()
    for t, n in zip(cache, ("k", "v", "k_scale", "v_scale")):
        assert torch.equal(t.cpu(), pool[n])


@pytest.mark.parametrize("slices", ["fused", "head_major"])
def test_strides(fp8, slices):
    news, past, hq, hk, d = [3, 1, 40], [50, 200, 7], 8, 2, 64
    say("strides", slices)
    pool, table, lengths = setup(news, past, hk, d, 32, 3)
    tokens, g = sum(news), torch.Generator().manual_seed(2)
    if slices == "fused":
        q = torch.randn(tokens, (hq + 2 * hk) * d, generator=g).to(BF16).cuda()[:, :hq * d].unflatten(1, (hq, d))
        out = torch.empty(tokens, 2, hq, d, dtype=BF16, device="cuda")[:, 1]
    else:
        q = torch.randn(hq, tokens, d, generator=g).to(BF16).cuda().transpose(0, 1)
        out = torch.empty(hq, tokens, d, dtype=BF16, device="cuda").transpose(0, 1)
    _, lse = fp8.attention_cached(q, ref.on_gpu(fp8, pool), table.cuda(), torch.tensor(lengths, dtype=torch.int32).cuda(),
                                  cu=ref.bounds(news), out=out)
    check(q, out, lse, pool, table, lengths, news, True, d ** -0.5)


def test_shared_pages(fp8):
    """Sequences that begin with the same pages read them alike."""
    say("shared pages")
    pool, table, _ = setup([1], [320], 2, 128, 64, 4, spare=1)
    table = torch.cat([table, table, table])
    lengths, news = [321, 128, 200], [1, 1, 1]
    q = torch.randn(3, 6, 128, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    out, lse = fp8.attention_cached(q, ref.on_gpu(fp8, pool), table.cuda(), torch.tensor(lengths, dtype=torch.int32).cuda())
    check(q, out, lse, pool, table, lengths, news, True, 128 ** -0.5)


def test_non_finite(fp8):
    """A NaN in one sequence's keys or values stays in that sequence."""
    say("non-finite")
    news, past = [1, 1, 20, 20], [100, 100, 60, 60]
    pool, table, lengths = setup(news, past, 1, 64, 32, 5)
    pool["v"][int(table[1, 1]), 0, 3, 7], pool["k"][int(table[3, 0]), 0, 3, 7] = 127, 255
    q = torch.randn(sum(news), 4, 64, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    out, lse = fp8.attention_cached(q, ref.on_gpu(fp8, pool), table.cuda(), torch.tensor(lengths, dtype=torch.int32).cuda(),
                                    cu=ref.bounds(news))
    assert torch.isfinite(out[0].float()).all() and torch.isfinite(out[2:22].float()).all()
    assert torch.isnan(out[1, :, 7]).all() and torch.isfinite(out[1, :, :7].float()).all()
    assert torch.isnan(out[22:].float()).all() and torch.isnan(lse[:, 22:]).all()


def test_generation(fp8):
    """A prompt in pieces, then tokens one at a time: each call's output is the packed
    attention of the same queries over what the cache reads back as."""
    say("generation")
    hq, hk, d, page = 10, 2, 128, 32
    batch, g = 3, torch.Generator().manual_seed(9)
    cache = fp8.kv_cache(40, hk, d, page)
    table = torch.randperm(40, generator=g).to(torch.int32)[:39].reshape(3, 13).cuda()
    lengths = torch.zeros(batch, dtype=torch.int32, device="cuda")
    for news in ([100, 33, 1], [0, 200, 64], [1, 1, 1], [5, 5, 5], [1, 1, 1], [1, 0, 1]):
        tokens, cu = sum(news), ref.bounds(news)
        qkv = torch.randn(tokens, (hq + 2 * hk) * d, generator=g).to(BF16).cuda()
        q, k, v = (t.unflatten(1, (-1, d)) for t in qkv.split([hq * d, hk * d, hk * d], 1))
        lengths += torch.tensor(news, dtype=torch.int32).cuda()
        fp8.kv_cache_write(cache, table, lengths, k, v, cu=cu)
        out, lse = fp8.attention_cached(q, cache, table, lengths, cu=cu)
        whole = lengths.tolist()
        ck, cv = fp8.kv_cache_read(cache, table, lengths, sum(whole), cu=ref.bounds(whole))
        want, lse2 = fp8.attention(q, ck, cv, cu, ref.bounds(whole), causal=True)
        # both round p and out once: twice the tolerance of one, with sums of at most 4 |v|
        assert ((out.float() - want.float()).abs() <= 2 * (U * want.float().abs() + (U + 2 * E) * 4)).all()
        assert ((lse - lse2).abs() <= 2 * E + 2.0 ** -21 * lse2.abs()).all()
        # the new tokens themselves came through one rounding (and their page's growth)
        nk, _ = fp8.kv_cache_read(cache, table, lengths, tokens, cu=cu)
        assert ((nk.float() - k.float()).abs() <= 2.0 ** -4 * k.float().abs() + 2.0 ** -10 * 8).all()


@pytest.mark.parametrize("kind", ["step", "few", "prompt"])
def test_replays(fp8, kind):
    """A write, a read and an attention captured in a graph: every replay, with other lengths and
    tokens, gives the eager calls' bytes."""
    hq, hk, d, page, batch = 8, 2, 128, 64, 6
    say("graph", kind)
    news = {"step": [1] * 6, "few": [5, 0, 3, 1, 8, 2], "prompt": [200, 1, 33, 64, 0, 130]}[kind]
    tokens, cu = sum(news), None if kind == "step" else ref.bounds(news)
    g = torch.Generator().manual_seed(3)
    table = torch.randperm(60, generator=g).to(torch.int32).reshape(6, 10).cuda()
    start = [torch.tensor([min(640, n + p) for n, p in zip(news, past)], dtype=torch.int32).cuda() for past in
             ([0, 100, 300, 63, 64, 5], [10, 0, 500, 640, 1, 65], [3, 200, 3, 100, 400, 350])]
    inputs = [torch.randn(tokens, hq + 2 * hk, d, generator=g).to(BF16).cuda() for _ in start]
    pool = ref.make_pool(60, hk, page, d, 1, stale=False)
    cache, lengths, qkv = ref.on_gpu(fp8, pool), start[0].clone(), inputs[0].clone()
    top = torch.zeros(1, device="cuda")

    def step():
        fp8.absmax_clear(top)
        fp8.kv_cache_write(cache, table, lengths, qkv[:, hq:hq + hk], qkv[:, hq + hk:], cu=cu)
        k, v = fp8.kv_cache_read(cache, table, lengths, tokens, cu=cu)
        out, lse = fp8.attention_cached(qkv[:, :hq], cache, table, lengths, cu=cu, absmax=top)
        return [*cache, k, v, out, lse, top]

    def reset(i):
        for t, n in zip(cache, ("k", "v", "k_scale", "v_scale")):
            t.copy_(pool[n])
        lengths.copy_(start[i])
        qkv.copy_(inputs[i])

    want = []
    for i in range(len(start)):
        reset(i)
        want.append([t.clone() for t in step()])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for rep in range(6):
        say("replay", rep)
        for t in got[4:]:
            t.fill_(float("nan"))
        reset(rep % len(start))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want[rep % len(start)])):
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)), (rep, i)


def test_pool_of_more_than_4_gib(fp8):
    """The last pages of a pool of 4.6 GB of keys and as many of values: the bytes that a small pool gives."""
    heads, d, page, news = 8, 128, 64, [130, 1, 40]
    say("large pool")
    g = torch.Generator().manual_seed(4)
    qkv = torch.randn(sum(news), 3 * heads, d, generator=g).to(BF16).cuda()
    q, k, v = qkv[:, :heads], qkv[:, heads:2 * heads], qkv[:, 2 * heads:]
    small, lengths = torch.tensor([[0, 1, 2], [3, 4, 5], [6, 7, 8]], dtype=torch.int32), torch.tensor([130, 1, 40], dtype=torch.int32).cuda()
    got = []
    for pages in (9, 70000):
        cache = fp8.kv_cache(pages, heads, d, page)
        table = (small + (pages - 9)).cuda()
        fp8.kv_cache_write(cache, table, lengths, k, v, cu=ref.bounds(news))
        out = fp8.attention_cached(q, cache, table, lengths, cu=ref.bounds(news))
        last = fp8.attention_cached(q[:3], cache, table, lengths)
        got.append([*fp8.kv_cache_read(cache, table, lengths, sum(news), cu=ref.bounds(news)), *out, *last])
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_two_streams(fp8):
    """Calls on two streams at once, each with its own cache and what its stream made just before."""
    news, past, hq, hk, d, page = [1] * 24, [157 * i % 900 for i in range(24)], 8, 2, 128, 64
    say("two streams")
    pools = [setup(news, past, hk, d, page, 40 + i) for i in range(2)]
    make = [torch.randn(24, hq + 2 * hk, d, generator=torch.Generator().manual_seed(i)).to(BF16).cuda() for i in range(2)]
    n = torch.tensor(pools[0][2], dtype=torch.int32).cuda()
    tables = [p[1].cuda() for p in pools]

    def chain(i, cache):
        outs = []
        for step in range(6):
            qkv = make[i] * (1 + step)                     # made on this stream
            fp8.kv_cache_write(cache, tables[i], n, qkv[:, hq:hq + hk], qkv[:, hq + hk:])
            outs += fp8.attention_cached(qkv[:, :hq], cache, tables[i], n)
        return outs

    want = [chain(i, ref.on_gpu(fp8, pools[i][0])) for i in range(2)]
    caches = [ref.on_gpu(fp8, pools[i][0]) for i in range(2)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [None, None]
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            got[i] = chain(i, caches[i])
    torch.cuda.synchronize()
    for i in range(2):
        for a, b in zip(got[i], want[i]):
            assert torch.equal(a, b)


def test_refusals(fp8):
    cache = fp8.kv_cache(4, 2, 64, 16)
    table, lengths = torch.zeros(2, 2, dtype=torch.int32).cuda(), torch.zeros(2, dtype=torch.int32).cuda()
    q = torch.zeros(2, 4, 64, dtype=BF16).cuda()
    good = dict(q=q, cache=cache, table=table, lengths=lengths)
    out, lse = fp8.attention_cached(**good)
    assert (out == 0).all() and torch.isneginf(lse).all()
    for bad in (dict(q=q.float()), dict(table=table.float()), dict(absmax=torch.zeros(1, dtype=F64, device="cuda")),
                dict(lse=lse.double()), dict(cache=cache._replace(k=cache.k.view(torch.int8)))):
        with pytest.raises(TypeError):
            fp8.attention_cached(**{**good, **bad})
    for bad in (dict(q=q[..., :32]), dict(q=q[:1]), dict(lse=lse[:2]), dict(out=out[:, :2]), dict(lengths=lengths[:1]),
                dict(cu=lengths)):
        with pytest.raises(ValueError):
            fp8.attention_cached(**{**good, **bad})
    for bad in (dict(q=q[:, :3]), dict(scale=0.0), dict(scale=float("nan")), dict(out=q)):
        with pytest.raises(fp8.Fp8Error):
            fp8.attention_cached(**{**good, **bad})
