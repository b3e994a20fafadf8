"""A paged cache on the CPU, token by token and in float64, and helpers of its tests."""
import torch

F64, BF16, U8, E4M3 = torch.float64, torch.bfloat16, torch.uint8, torch.float8_e4m3fn


def decode(codes):
    return codes.view(E4M3).to(F64)


def nearest(y):
    """The E4M3 code of a float64 that float32 holds or that lies below its smallest code's half."""
    return y.clamp(-448.0, 448.0).to(torch.float32).to(E4M3).view(U8)


def least_exponent(x):
    """The least e with max |x| <= 448 2^e over the finite x, held to -100 .. 119."""
    x = x[torch.isfinite(x)]
    top = x.abs().max().item() if x.numel() else 0.0
    e = -100
    while e < 119 and top > 448.0 * 2.0 ** e:
        e += 1
    return e


def held(lengths, table, page):
    """Tokens that can have a place."""
    return [min(max(int(n), 0), table.shape[1] * page) for n in lengths]


def place(pool, table, b, p):
    """(page, slot) of position p of sequence b, or None."""
    page = pool["k"].shape[2]
    if not 0 <= p < table.shape[1] * page:
        return None
    at = int(table[b, p // page])
    return (at, p % page) if 0 <= at < pool["k"].shape[0] else None


def write(pool, table, lengths, news, k, v):
    """pool: dict of CPU tensors k, v, k_scale, v_scale, changed in place; news: new tokens per sequence."""
    pages, heads, page, d = pool["k"].shape
    first = 0
    for b, (n, total) in enumerate(zip(news, lengths)):
        places = {}
        for i in range(n):
            p = max(int(total), 0) - n + i
            if place(pool, table, b, p):
                places.setdefault(p // page, []).append((i, p % page))
        for block, mine in places.items():
            at = int(table[b, block])
            rows, slots = [first + i for i, _ in mine], [s for _, s in mine]
            for name, x in (("k", k), ("v", v)):
                codes, scale = pool[name], pool[name + "_scale"]
                for h in range(heads):
                    new = x[rows, h].to(F64)
                    e = least_exponent(new)
                    if slots[0] > 0:
                        was = min(max(int(scale[at, h]) - 127, -100), 119)
                        if e <= was:
                            e = was
                        else:
                            old = codes[at, h, :slots[0]]
                            codes[at, h, :slots[0]] = nearest(decode(old) * 2.0 ** (was - e))
                    codes[at, h, slots] = nearest(new * 2.0 ** -e)
                    scale[at, h] = e + 127
        first += n


def read(pool, table, lengths, news, name):
    """float64 [tokens, heads, d] of each sequence's last tokens, zeros where there is no place."""
    pages, heads, page, d = pool[name].shape
    out = torch.zeros(sum(news), heads, d, dtype=F64)
    first = 0
    for b, (n, total) in enumerate(zip(news, lengths)):
        for i in range(n):
            where = place(pool, table, b, max(int(total), 0) - n + i)
            if where:
                e = (pool[name + "_scale"][where[0]].to(torch.int64) - 127).clamp(-100, 119)
                out[first + i] = decode(pool[name][where[0], :, where[1]]) * torch.exp2(e.to(F64))[:, None]
        first += n
    return out


def make_pool(pages, heads, page, d, seed, stale=True):
    """A pool of random codes (NaN codes among them where `stale`) and scales."""
    g = torch.Generator().manual_seed(seed)
    pool = {}
    for name in "kv":
        c = torch.randint(0, 256, (pages, heads, page, d), generator=g, dtype=torch.int16).to(U8)
        pool[name] = c if stale else torch.where((c & 127) == 127, c - 1, c)
        pool[name + "_scale"] = torch.randint(117, 122, (pages, heads), generator=g, dtype=torch.int16).to(U8)
    return pool


def make_table(lengths, page, pages, seed, spare=0):
    """Pages in no order; -1 behind a sequence's last block."""
    blocks = [-(-max(n, 0) // page) for n in lengths]
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    assert sum(blocks) <= pages
    table = torch.full((len(lengths), max(1, max(blocks)) + spare), -1, dtype=torch.int32)
    for b, n in enumerate(blocks):
        for i in range(n):
            table[b, i] = order.pop()
    return table


def on_gpu(fp8, pool):
    return fp8.KVCache(*(pool[n].cuda() for n in ("k", "v", "k_scale", "v_scale")))


def bounds(news):
    return torch.tensor([0] + news).cumsum(0).to(torch.int32).cuda()
