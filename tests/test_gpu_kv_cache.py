"""Writing and reading the paged 8-bit cache against a token-by-token reference in float64:
codes and scales byte for byte (a NaN code may have either sign), every slot that is not
written as it was, values read back exactly."""
import pytest
import torch

import kv_cache_reference as ref
from gpu_util import E4M3, assert_codes_equal, say, u8

pytestmark = pytest.mark.gpu
BF16, F64 = torch.bfloat16, torch.float64


@pytest.fixture(scope="module")
def fp8():
    import fp8_precision_amd
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    return fp8_precision_amd


def draw(tokens, heads, d, seed, sigma=1.0, wide=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, heads, d, generator=g) * sigma
    if wide:                                              # magnitudes that differ from token to token
        x = x * torch.exp2(torch.rand(tokens, 1, 1, generator=g) * 2 * wide - wide)
    return x.to(BF16)


def check_write(fp8, pool, table, lengths, news, k, v, even=False, cu=None, pad=0):
    want = {n: t.clone() for n, t in pool.items()}
    ref.write(want, table, lengths, news, k, v)
    cache = ref.on_gpu(fp8, pool)
    cu = None if even else ref.bounds(news) if cu is None else cu
    kd, vd = k.cuda(), v.cuda()
    if pad:
        more = torch.full((pad, *k.shape[1:]), float("nan"), dtype=BF16, device="cuda")
        kd, vd = torch.cat([kd, more]), torch.cat([vd, more])
    fp8.kv_cache_write(cache, table.cuda(), torch.tensor(lengths, dtype=torch.int32, device="cuda"), kd, vd, cu=cu)
    torch.cuda.synchronize()
    for n, t in zip(("k", "v", "k_scale", "v_scale"), cache):
        if "scale" in n:
            assert torch.equal(t.cpu(), want[n]), n
        else:
            assert_codes_equal(u8(t), u8(want[n]), E4M3, n)
    return cache, want


CASES = [
    # new tokens, held before, heads, d, page
    ([1], [0], 1, 8, 16), ([1], [63], 2, 128, 64), ([1], [64], 2, 128, 64), ([3], [126], 1, 72, 128),
    ([5, 3, 1, 17, 40], [11, 0, 100, 15, 7], 3, 72, 16), ([0, 200, 0, 1, 33], [9, 70, 0, 64, 31], 2, 128, 32),
    ([129, 128, 127, 1], [0, 128, 1, 255], 4, 128, 128), ([1] * 70, list(range(70)), 2, 64, 16),
    ([2, 0, 1] * 50, list(range(150)), 1, 16, 32), ([700], [33], 5, 120, 64), ([4, 5, 6], [60, 59, 58], 1, 40, 64),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("wide", [0.0, 6.0])
def test_write_and_read(fp8, case, wide):
    news, past, heads, d, page = CASES[case]
    say("cache", CASES[case], wide)
    lengths = [a + b for a, b in zip(news, past)]
    table = ref.make_table(lengths, page, sum(-(-n // page) for n in lengths) + 2, case, spare=case % 2)
    pages = sum(-(-n // page) for n in lengths) + 2
    pool = ref.make_pool(pages, heads, page, d, case)
    k, v = draw(sum(news), heads, d, 2 * case, wide=wide), draw(sum(news), heads, d, 2 * case + 1, 0.03, wide)
    cache, want = check_write(fp8, pool, table, lengths, news, k, v)
    n = torch.tensor(lengths, dtype=torch.int32).cuda()
    for some in (news, lengths):                          # the call's own tokens, and whole contexts
        if sum(some) == 0:
            continue
        got = fp8.kv_cache_read(cache, table.cuda(), n, sum(some), cu=ref.bounds(some))
        for name, t in zip("kv", got):
            w = ref.read(want, table, lengths, some, name)
            assert torch.equal(torch.nan_to_num(t.cpu().to(F64), nan=1e30), torch.nan_to_num(w, nan=1e30)), name


@pytest.mark.parametrize("n,batch", [(1, 5), (1, 300), (4, 3), (5, 3), (65, 4)])
def test_as_many_each(fp8, n, batch):
    """Without bounds every sequence has as many tokens."""
    say("even", n, batch)
    past = [(7 * b) % 90 for b in range(batch)]
    lengths = [n + p for p in past]
    pages = sum(-(-x // 32) for x in lengths)
    table = ref.make_table(lengths, 32, pages, n)
    pool = ref.make_pool(pages, 2, 32, 64, n)
    k, v = draw(n * batch, 2, 64, 1, wide=3.0), draw(n * batch, 2, 64, 2, wide=3.0)
    cache, want = check_write(fp8, pool, table, lengths, [n] * batch, k, v, even=True)
    got = fp8.kv_cache_read(cache, table.cuda(), torch.tensor(lengths, dtype=torch.int32).cuda(), n * batch)
    for name, t in zip("kv", got):
        assert torch.equal(t.cpu().to(F64), ref.read(want, table, lengths, [n] * batch, name))


@pytest.mark.parametrize("one_by_one", [False, True])
def test_a_page_grows(fp8, one_by_one):
    """Tokens of rising and falling magnitude, added to pages in pieces: the page's exponent is the
    largest so far, and what it holds is what the reference's appends leave."""
    heads, d, page, total = 2, 32, 16, 50
    say("grow", one_by_one)
    g = torch.Generator().manual_seed(5)
    e = torch.randint(-12, 13, (total, 1, 1), generator=g)
    k = (torch.randn(total, heads, d, generator=g) * torch.exp2(e.float())).to(BF16)
    v = (torch.randn(total, heads, d, generator=g) * torch.exp2(torch.arange(total)[:, None, None] / 2.0 - 12)).to(BF16)
    table = ref.make_table([total], page, 6, 1)
    pool = ref.make_pool(6, heads, page, d, 3)
    done = 0
    for n in ([1] * total if one_by_one else [5, 1, 20, 3, 21]):
        cache, pool = check_write(fp8, pool, table, [done + n], [n], k[done:done + n], v[done:done + n])
        done += n
    for x, name in ((k, "k"), (v, "v")):
        e = pool[name + "_scale"].to(F64)[table[0].long()].repeat_interleave(page, 0)[:total] - 127
        back = ref.read(pool, table, [total], [total], name)
        # one rounding per value, and one more, of half the smallest code's step, for each time its page grew
        grown = 24 * 2.0 ** -10 * torch.exp2(e)[..., None]
        assert ((back - x.to(F64)).abs() <= 2.0 ** -4 * x.to(F64).abs() + grown).all()


def test_edges_of_the_scale(fp8):
    """448 2^e exactly and the next value, powers of two, zeros, the smallest and largest bf16."""
    heads, d, page = 1, 8, 16
    up = lambda x: torch.tensor([x]).to(BF16).view(torch.int16).add(1).view(BF16).item()
    tops = [448.0, up(448.0), 1.0, 1.75, up(1.75), 0.0, 2.0 ** -92, 448 * 2.0 ** -100, up(448 * 2.0 ** -100), 2.0 ** -126,
            9e-41, 3.3895e38, 448 * 2.0 ** 119, up(448 * 2.0 ** 119), 2.0 ** 127, 3.0]
    say("edges")
    k = torch.zeros(len(tops), heads, d)
    for i, t in enumerate(tops):
        k[i, 0] = torch.tensor([t, -t, t / 2, t / 3, t / 500, -t / 900, t / 20000, 0.0])
    k = k.to(BF16)
    table = torch.arange(len(tops), dtype=torch.int32)[:, None]
    pool = ref.make_pool(len(tops), heads, page, d, 1)
    cache, want = check_write(fp8, pool, table, [1] * len(tops), [1] * len(tops), k, -k, even=True)
    got, _ = fp8.kv_cache_read(cache, table.cuda(), torch.ones(len(tops), dtype=torch.int32).cuda(), len(tops))
    assert torch.equal(got.cpu().to(F64), ref.read(want, table, [1] * len(tops), [1] * len(tops), "k"))
    assert torch.isfinite(got.float()).all()


@pytest.mark.parametrize("news", [[3], [40]])
def test_non_finite_values(fp8, news):
    """A NaN gives a NaN code, an infinity saturates, and neither reaches the scale."""
    say("non-finite", news)
    k, v = draw(sum(news), 2, 64, 1), draw(sum(news), 2, 64, 2)
    k[0, 0, 3], k[1, 0, 9], k[2, 1, 0], v[1, 1, 63] = float("nan"), float("inf"), float("-inf"), float("nan")
    v[2, 0] = float("inf")
    v[:, 1, 5] = float("nan")
    table = ref.make_table([news[0] + 2], 32, 4, 1)
    check_write(fp8, ref.make_pool(4, 2, 32, 64, 1), table, [news[0] + 2], news, k, v)
    nothing = torch.full((sum(news), 2, 64), float("nan"), dtype=BF16)
    check_write(fp8, ref.make_pool(4, 2, 32, 64, 1), table, [news[0]], news, nothing, nothing)


def test_places_that_are_not_there(fp8):
    """Table entries that are no page, lengths past the table and below the new tokens, a padded
    batch: what has no place is left out and reads as zeros."""
    heads, d, page = 2, 64, 16
    news, lengths = [20, 30, 5, 8, 3], [40, 60, 3, -4, 2147483647]
    say("no places")
    table = torch.tensor([[0, -1, 2], [9, 1, 1 << 30], [3, -5, 9], [4, 5, 6], [-2147483648, 7, 8]], dtype=torch.int32)
    pool = ref.make_pool(9, heads, page, d, 2)
    k, v = draw(sum(news), heads, d, 1), draw(sum(news), heads, d, 2)
    cache, want = check_write(fp8, pool, table, lengths, news, k, v, pad=9)
    n = torch.tensor(lengths, dtype=torch.int32).cuda()
    out = torch.full((sum(news) + 9, heads, d), 7.0, dtype=BF16, device="cuda")
    got, _ = fp8.kv_cache_read(cache, table.cuda(), n, sum(news) + 9, cu=ref.bounds(news), k=out)
    w = ref.read(want, table, lengths, news, "k")
    assert torch.equal(torch.nan_to_num(got[:sum(news)].cpu().to(F64), nan=1e30), torch.nan_to_num(w, nan=1e30))
    assert (got[sum(news):] == 7.0).all()


def test_bounds_in_no_order(fp8):
    """Bounds outside the tokens or falling are held to them: nothing else is touched."""
    heads, d, page = 1, 32, 16
    say("wild bounds")
    pool = ref.make_pool(40, heads, page, d, 4)
    cache = ref.on_gpu(fp8, pool)
    table = torch.arange(40, dtype=torch.int32).reshape(5, 8).cuda()
    lengths = torch.tensor([30, 128, 7, 60, 100], dtype=torch.int32).cuda()
    cu = torch.tensor([-7, 12, 5, 1000, 3, 2000], dtype=torch.int32).cuda()
    k = draw(50, heads, d, 1).cuda()
    fp8.kv_cache_write(cache, table, lengths, k, k, cu=cu)
    out = torch.full((50, heads, d), 7.0, dtype=BF16, device="cuda")
    fp8.kv_cache_read(cache, table, lengths, 50, cu=cu, k=out)
    torch.cuda.synchronize()
    # a sequence's pages behind what it holds keep their bytes
    for b, n in enumerate(lengths.tolist()):
        for i in range(-(-n // page), 8):
            assert torch.equal(cache.k[8 * b + i].cpu(), pool["k"][8 * b + i])


@pytest.mark.parametrize("slices", ["fused", "head_major", "shared_head"])
def test_strides(fp8, slices):
    """Keys and values as slices of a projection's output, head-major, or one head for all."""
    news, past, heads, d, page = [33, 1, 20], [5, 16, 0], 4, 64, 32
    say("strides", slices)
    tokens, lengths = sum(news), [a + b for a, b in zip(news, past)]
    if slices == "fused":
        x = draw(tokens, 1, (8 + 2 * heads) * d, 3)[:, 0]
        k, v = (t.unflatten(1, (heads, d)) for t in (x[:, 8 * d:12 * d], x[:, 12 * d:]))
        kd, vd = (t.unflatten(1, (heads, d)) for t in (x.cuda()[:, 8 * d:12 * d], x.cuda()[:, 12 * d:]))
    elif slices == "head_major":
        k, v = draw(heads, tokens, d, 4).transpose(0, 1), draw(heads, tokens, d, 5).transpose(0, 1)
        kd, vd = k.transpose(0, 1).contiguous().cuda().transpose(0, 1), v.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    else:
        one = draw(tokens, 1, d, 6)
        k = v = one.expand(tokens, heads, d)
        kd = vd = one.cuda().expand(tokens, heads, d)
    table = ref.make_table(lengths, page, 9, 3)
    pool = ref.make_pool(9, heads, page, d, 3)
    want = {n: t.clone() for n, t in pool.items()}
    ref.write(want, table, lengths, news, k, v)
    cache, n = ref.on_gpu(fp8, pool), torch.tensor(lengths, dtype=torch.int32).cuda()
    fp8.kv_cache_write(cache, table.cuda(), n, kd, vd, cu=ref.bounds(news))
    assert_codes_equal(u8(cache.k), u8(want["k"]), E4M3, "k")
    assert_codes_equal(u8(cache.v), u8(want["v"]), E4M3, "v")
    # and back into interleaved slices of one tensor
    kv = torch.zeros(tokens, heads, 2, d, dtype=BF16, device="cuda")
    fp8.kv_cache_read(cache, table.cuda(), n, tokens, cu=ref.bounds(news), k=kv[:, :, 0], v=kv[:, :, 1])
    for i, name in enumerate("kv"):
        assert torch.equal(kv[:, :, i].cpu().to(F64), ref.read(want, table, lengths, news, name))


def test_refusals(fp8):
    cache = fp8.kv_cache(4, 2, 64, 16)
    table, lengths = torch.zeros(2, 2, dtype=torch.int32).cuda(), torch.ones(2, dtype=torch.int32).cuda()
    k = torch.zeros(2, 2, 64, dtype=BF16).cuda()
    fp8.kv_cache_write(cache, table, lengths * 0, k, k)       # nothing has a place
    for bad in (dict(table=table.long()), dict(lengths=lengths.long()), dict(k=k.float())):
        with pytest.raises(TypeError):
            fp8.kv_cache_write(**{**dict(cache=cache, table=table, lengths=lengths, k=k, v=k), **bad})
    for bad in (dict(table=table[0]), dict(lengths=lengths[:1]), dict(k=k[:, :1], v=k[:, :1]), dict(cu=lengths),
                dict(k=k[..., :32], v=k[..., :32]), dict(v=k[:1]), dict(k=k[:1], v=k[:1]), dict(cache=cache._replace(v=cache.v[:2])),
                dict(cache=cache._replace(k_scale=cache.k_scale[:, :1].contiguous())), dict(k=k[..., ::2], v=k[..., ::2])):
        with pytest.raises(ValueError):
            fp8.kv_cache_write(**{**dict(cache=cache, table=table, lengths=lengths, k=k, v=k), **bad})
    with pytest.raises(TypeError):
        fp8.kv_cache_write(cache, table.cpu(), lengths, k, k)
    with pytest.raises(fp8.Fp8Error):
        fp8.kv_cache_write(fp8.kv_cache(4, 2, 64, 24), table, lengths, k, k)
    with pytest.raises(fp8.Fp8Error):
        fp8.kv_cache_read(cache, table, lengths, 2, k=k, v=k)
    with pytest.raises(ValueError):
        fp8.kv_cache_read(cache, table, lengths, 3)
