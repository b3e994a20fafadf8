"""The keys and values of generation held in 8 bits, as measured cases.

Writing new tokens' keys and values into a paged cache of E4M3 codes with one scale for each
page and head, reading them back, and attention that reads the cache: for single tokens, for
a few tokens at a time and for whole prompts.  Each has a plain form here (elementary torch
operations in 32 bits, rounded once at the end), a definition in 64 bits, and the call that a
user of the package makes.

The cache: sequence b's token at position p lies in page table[b, p // page] at slot p % page.
Of every page and head, the keys share one scale 2^e and the values another, e the least with
max |x| <= 448 2^e, held to -100 .. 119.  A page that is written on from its middle keeps the
larger of its scale and the new tokens', its older codes rounded to that.  A call's new tokens
are the last ones of `lengths`, and its queries are at their positions.
"""
import math

import torch

own = False

DEV = "cuda"
F32, F64, BF16, U8 = torch.float32, torch.float64, torch.bfloat16, torch.uint8
E4M3 = torch.float8_e4m3fn
E_LEAST, E_MOST, TOP = -100, 119, 448.0

# ------------------------------------------------------------------------------ cases

_PASTS = ("1000 4096 311 2047 63 64 65 3500 1291 700 2500 0 4031 15 16 1800 "
          "905 3333 1200 47 2900 128 127 129 512 1023 3075 77 640 3840 1999 256 "
          "333 444 555 3666 1777 888 2999 1 2 3 1400 1500 1600 3700 31 32 "
          "33 3900 2100 2200 2300 2400 3 9 27 81 243 729 2187 1459 17 4000")
_LONG = ("8191 1000 4096 7000 2047 64 65 3500 5291 700 6500 1 4031 15 16 1800 "
         "905 3333 7200 47 2900 128 127 129 5512 1023 7071 77 640 3840 1999 256 "
         "333 444 555 3666 1777 888 2999 8000 2 3 1400 1500 6600 3700 31 32 "
         "33 3900 2100 2200 7300 2400 3 9 27 81 243 729 2187 6561 17 4000")
_SHORT = ("500 311 640 12 700 333 421 499 530 610 288 345 402 467 503 589 "
          "620 655 671 299 318 377 436 485 512 543 601 633 668 690 305")


def listed():
    ones = lambda n: " ".join(["1"] * n)
    return [
        # a step of generation: one new token of each of 64 sequences, pages filled to any extent
        {"name": "write_step", "op": "write", "new": ones(64), "past": _PASTS, "hq": 40, "hk": 8, "d": 128, "page": 64},
        # prompts of every length on their way into the cache, some of them continued: the 14B-class batch
        {"name": "write_prompt_14b", "op": "write", "new": "4093 1 2111 0 517 1470", "past": "0 4000 100 300 0 64",
         "hq": 40, "hk": 8, "d": 128, "page": 64},
        # short continuations that begin and end inside small pages, an odd head size
        {"name": "write_odd", "op": "write", "new": "5 3 1 17 40", "past": "11 0 100 15 7", "hq": 6, "hk": 3, "d": 72,
         "page": 16},
        # contexts read back for the packed operators, 32768 tokens
        {"name": "read_prefix", "op": "read", "new": "8192 5000 1 9191 4096 2047 0 4241",
         "past": "0 0 0 0 0 0 0 0", "hq": 40, "hk": 8, "d": 128, "page": 64},
        # the ends of a few contexts, an odd head size
        {"name": "read_odd", "op": "read", "new": "100 7 33 1", "past": "29 300 0 64", "hq": 8, "hk": 4, "d": 40,
         "page": 32},
        # one query on a long context, the 7B-class layer's heads
        {"name": "attend_one", "op": "attend", "new": "1", "past": "16383", "hq": 32, "hk": 32, "d": 128, "page": 64,
         "causal": True},
        # a step of generation of 64 sequences of every length, the 14B-class layer's heads
        {"name": "attend_step_14b", "op": "attend", "new": ones(64), "past": _LONG, "hq": 40, "hk": 8, "d": 128,
         "page": 64, "causal": True},
        # one long context among short ones
        {"name": "attend_far", "op": "attend", "new": ones(32), "past": "65535 " + _SHORT, "hq": 32, "hk": 8, "d": 128,
         "page": 128, "causal": True},
        # five drafted tokens of each sequence are checked at once; small heads, small pages
        {"name": "attend_draft", "op": "attend", "new": " ".join(["5"] * 16),
         "past": "100 2000 17 1 512 3000 777 64 15 16 1234 900 4000 33 250 0", "hq": 12, "hk": 4, "d": 64, "page": 16,
         "causal": True},
        # a piece of a long prompt, its earlier pieces in the cache
        {"name": "attend_chunk_14b", "op": "attend", "new": "2048", "past": "6144", "hq": 40, "hk": 8, "d": 128,
         "page": 64, "causal": True},
        # a whole prompt of the 7B-class batch
        {"name": "attend_prompt_7b", "op": "attend", "new": "4096", "past": "0", "hq": 32, "hk": 32, "d": 128,
         "page": 64, "causal": True},
        # a prompt's piece among single tokens
        {"name": "attend_mixed", "op": "attend", "new": "1000 " + ones(31), "past": "500 2900 " + _SHORT[4:],
         "hq": 40, "hk": 8, "d": 128, "page": 32, "causal": True},
    ]


def _log_int(rng, lo, hi):
    """An integer spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _one(rng):
    op = rng.choice(["write", "read", "attend", "attend"])
    hk = rng.choice([1, 2, 3, 4, 8])
    case = {"op": op, "hq": hk * rng.choice([1, 1, 2, 4, 5, 8]), "hk": hk,
            "d": rng.choice([64, 128, 128, 8 * rng.randint(2, 16)]), "page": rng.choice([16, 32, 64, 64, 128])}
    kind = rng.choice(["step", "few", "prompt", "mixed"])
    n = _log_int(rng, 1, 64) if kind in ("step", "few") else rng.randint(1, 6)
    past = [_log_int(rng, 1, 8192) - 1 for _ in range(n)]
    if kind == "step":
        new = [1] * n
    elif kind == "few":
        most = rng.randint(2, 8)
        new = [most] * n if rng.random() < 0.5 else [rng.randint(0, most) for _ in range(n)]
    else:
        new = [_log_int(rng, 1, 4096) for _ in range(n)]
        if kind == "mixed":
            more = rng.randint(1, 24)
            new, past = new + [1] * more, past + [_log_int(rng, 1, 4096) for _ in range(more)]
    case["new"], case["past"] = " ".join(map(str, new)), " ".join(map(str, past))
    if op == "attend":
        case["causal"] = rng.random() < 0.85
    return case


def _padded(case):
    """Scores that the plain form holds, and elements of the contexts that it lays out."""
    new, past = _ints(case["new"]), _ints(case["past"])
    longest = max(n + p for n, p in zip(new, past))
    return len(new) * case["hq"] * max(new) * longest, len(new) * case["hk"] * longest * case["d"]


def draw(rng):
    """One more case; none costs more than the largest listed one of its operator."""
    tops = {}
    for c in listed():
        w, p = work(c), _padded(c)
        tops[c["op"]] = [max(a, b) for a, b in zip(tops.get(c["op"], (0, 0, 0, 0)), (w["bytes"], w["flops"], *p))]
    while True:
        case = _one(rng)
        if sum(_ints(case["new"])) == 0:
            continue
        w, p, top = work(case), _padded(case), tops[case["op"]]
        fits = case["op"] != "attend" or (p[0] <= top[2] and p[1] <= top[3])
        if fits and w["bytes"] <= top[0] and w["flops"] <= top[1]:
            return case


def _ints(text):
    return [int(n) for n in text.split()]


def _pairs(case):
    """How many (query, key) pairs are seen: query i of a sequence sees the keys up to past + i."""
    n = 0
    for new, past in zip(_ints(case["new"]), _ints(case["past"])):
        n += new * past + new * (new + 1) // 2 if case["causal"] else new * (new + past)
    return n


def work(case):
    new, past, hk, d, page = _ints(case["new"]), _ints(case["past"]), case["hk"], case["d"], case["page"]
    tokens = sum(new)
    if case["op"] in ("write", "read"):
        pages = sum((p + n - 1) // page - p // page + 1 for n, p in zip(new, past) if n)
        # two tensors: 16-bit values on one side, codes and the pages' scales on the other
        return {"bytes": 2 * (3 * tokens * hk * d + pages * hk), "flops": 2 * tokens * hk * d}
    held = [n + p for n, p in zip(new, past) if n]
    pages = sum(-(-n // page) for n in held)
    return {"bytes": 2 * hk * (sum(held) * d + pages) + tokens * case["hq"] * (4 * d + 4),
            "flops": 4 * d * case["hq"] * _pairs(case)}


# ------------------------------------------------------------------------------ inputs


def _inputs(case, seed):
    """The inputs of a case, from the seed alone: the pool, its table and lengths, and the new tokens."""
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    new, past = _ints(case["new"]), _ints(case["past"])
    hq, hk, d, page = case["hq"], case["hk"], case["d"], case["page"]
    blocks = [-(-(n + p) // page) for n, p in zip(new, past)]
    pages = sum(blocks) + 3
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    most = max(1, max(blocks))
    # the pages of the pool are dealt to the sequences in no order; a block past a sequence's end has none
    n = torch.tensor(blocks, device=DEV)
    at = torch.arange(most, device=DEV)[None, :]
    table = torch.where(at < n[:, None], order[((torch.cumsum(n, 0) - n)[:, None] + at).clamp(max=pages - 1)], -1)
    s = {"table": table.contiguous(), "lengths": torch.tensor([a + b for a, b in zip(new, past)], device=DEV).to(torch.int32),
         "tokens": sum(new), "cu": None}
    if len(set(new)) > 1:
        s["cu"] = torch.tensor([0] + new, device=DEV).cumsum(0).to(torch.int32)
    for name in "kv":
        # keys and values have channels that stand out
        gain = torch.exp(torch.randn(hk, 1, d, generator=g, device=DEV) * 0.5)
        x = torch.randn(pages, hk, page, d, generator=g, device=DEV) * gain
        # half of the pages hold tokens of less magnitude than is written next
        x = x * torch.exp2(-(torch.rand(pages, 1, 1, 1, generator=g, device=DEV) * 4 - 2).clamp(min=0))
        e = _exponent(x.abs().amax((2, 3)))
        s[name + "_codes"] = _codes(x, e[:, :, None, None])
        s[name + "_scale"] = (e + 127).to(U8)
        del x
        s[name + "_gain"] = gain[:, 0]
    # the slices of one projection's output, as in a layer
    qkv = torch.randn(s["tokens"], (hq + 2 * hk) * d, generator=g, device=DEV)
    cut = lambda a, b: qkv[:, a * d:b * d]
    cut(hq, hq + hk).mul_(s.pop("k_gain").reshape(-1))
    cut(hq + hk, hq + 2 * hk).mul_(s.pop("v_gain").reshape(-1))
    qkv = qkv.to(BF16)
    s["q"], s["k"], s["v"] = cut(0, hq).unflatten(1, (hq, d)), cut(hq, hq + hk).unflatten(1, (hk, d)), \
        cut(hq + hk, hq + 2 * hk).unflatten(1, (hk, d))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    new, past, page = _ints(case["new"]), _ints(case["past"]), case["page"]
    seq = torch.tensor([b for b, n in enumerate(new) for _ in range(n)], device=DEV, dtype=torch.int64)
    pos = torch.cat([torch.arange(p, p + n, device=DEV) for n, p in zip(new, past)])
    s["seq"], s["pos"] = seq, pos
    if case["op"] == "write":
        # every page that is written: its place in the pool, its slots held before, and which token each slot takes
        first = [0]
        for n in new:
            first.append(first[-1] + n)
        pieces = [(b, i) for b, (n, p) in enumerate(zip(new, past)) if n for i in range(p // page, (p + n - 1) // page + 1)]
        b = torch.tensor([x for x, _ in pieces], device=DEV)
        i = torch.tensor([x for _, x in pieces], device=DEV)
        start, count = torch.tensor(past, device=DEV)[b], torch.tensor(new, device=DEV)[b]
        slot = i[:, None] * page + torch.arange(page, device=DEV)[None, :] - start[:, None]
        s["page"] = s["table"][b, i].long()
        s["old"] = slot < 0
        s["fresh"] = (slot >= 0) & (slot < count[:, None])
        s["token"] = torch.where(s["fresh"], torch.tensor(first, device=DEV)[b][:, None] + slot, 0)
    if case["op"] == "attend":
        s["scale"] = case["d"] ** -0.5
        longest = max(new)
        n = torch.tensor(new, device=DEV)
        start = torch.cumsum(n, 0) - n
        inside = torch.arange(longest, device=DEV)[None, :].expand(len(new), -1)
        held = inside < n[:, None]
        s["iq"], s["uq"], s["new"] = torch.where(held, start[:, None] + inside, 0), held.nonzero(as_tuple=True), n
    return s


# ------------------------------------------------------------------------------ plain forms


def _exponent(top):
    """e of the largest magnitude: the least with top <= 448 2^e (448 = 0.875 2^9), held to its range."""
    m, x = torch.frexp(top)
    e = torch.where(m > 0.875, x - 8, x - 9)
    return torch.where(top == 0, E_LEAST, e).clamp(E_LEAST, E_MOST)


def _two_to(e):
    """2^e from its bits, -126 <= e <= 127."""
    return ((e.int() + 127) << 23).view(F32)


def _codes(x, e):
    return (x * _two_to(-e.clamp(max=126))).clamp(-TOP, TOP).to(E4M3).view(U8)


def _values(codes, scale):
    """What codes stand for, in 32 bits."""
    return codes.view(E4M3).float() * _two_to(scale.int() - 127)


def _write(s):
    page, old, fresh = s["page"], s["old"][:, None, :, None], s["fresh"][:, None, :, None]
    out = {}
    for name in "kv":
        codes, scale = s[name + "_codes"], s[name + "_scale"]
        x = torch.where(fresh, s[name].float()[s["token"]].transpose(1, 2), 0.0)
        before = torch.where(s["old"].any(1)[:, None], scale[page].int() - 127, E_LEAST)
        e = torch.maximum(_exponent(x.abs().amax((2, 3))), before)
        was = codes[page]
        again = _codes(was.view(E4M3).float(), (e - before)[:, :, None, None])
        codes[page] = torch.where(fresh, _codes(x, e[:, :, None, None]), torch.where(old, again, was))
        scale[page] = (e + 127).to(U8)
        out[name], out[name + "_scale"] = codes.view(E4M3), scale
    return out


def _read(s):
    page = s["table"][s["seq"], s["pos"] // s["case"]["page"]].long()
    slot = s["pos"] % s["case"]["page"]
    return {name: _values(s[name + "_codes"][page, :, slot], s[name + "_scale"][page][:, :, None]).to(BF16)
            for name in "kv"}


def _context(s, name):
    """[sequence, key head, position, d] of every sequence's pages, zeros past its end."""
    pages = s["table"].clamp(min=0).long()
    x = _values(s[name + "_codes"][pages], s[name + "_scale"][pages][..., None, None])
    x = x.transpose(1, 2).flatten(2, 3)
    at = torch.arange(x.shape[2], device=DEV)
    return x.masked_fill_((at[None, :] >= s["lengths"][:, None])[:, None, :, None], 0.0)


def _attend(s):
    hk, lengths, new = s["case"]["hk"], s["lengths"].long(), s["new"]
    q = s["q"].float()[s["iq"]].transpose(1, 2).unflatten(1, (hk, -1))           # [b, hk, group, i, d]
    k, v = _context(s, "k"), _context(s, "v")
    group, n = q.shape[2], q.shape[3]
    a = (q.flatten(2, 3) @ k.transpose(2, 3)).unflatten(2, (group, n)) * s["scale"]
    i = torch.arange(n, device=DEV)[None, :, None]
    j = torch.arange(k.shape[2], device=DEV)[None, None, :]
    seen = (i < new[:, None, None]) & (j < lengths[:, None, None])
    if s["case"]["causal"]:
        seen = seen & (j <= i + (lengths - new)[:, None, None])
    a = a.masked_fill_(~seen[:, None, None], -math.inf)
    top = a.amax(4, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(a - top)
    total = p.sum(4, keepdim=True)
    out = (p.flatten(2, 3) @ v).unflatten(2, (group, n)) / torch.where(total == 0, 1.0, total)
    lse = (top + torch.log(total)).squeeze(4)
    packed = lambda x: x.flatten(1, 2).transpose(1, 2)[s["uq"]]
    return {"out": packed(out).to(BF16), "lse": packed(lse).t().contiguous()}


# ------------------------------------------------------------------------------ the package's calls


def _own(s):
    import fp8_precision_amd as fp8
    cache = fp8.KVCache(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
    op = s["case"]["op"]
    if op == "write":
        fp8.kv_cache_write(cache, s["table"], s["lengths"], s["k"], s["v"], cu=s["cu"])
        return {"k": cache.k.view(E4M3), "k_scale": cache.k_scale, "v": cache.v.view(E4M3), "v_scale": cache.v_scale}
    if op == "read":
        k, v = fp8.kv_cache_read(cache, s["table"], s["lengths"], s["tokens"], cu=s["cu"])
        return {"k": k, "v": v}
    out, lse = fp8.attention_cached(s["q"], cache, s["table"], s["lengths"], cu=s["cu"], causal=s["case"]["causal"],
                                    scale=s["scale"])
    return {"out": out, "lse": lse}


def run(state):
    if own:
        return _own(state)
    return {"write": _write, "read": _read, "attend": _attend}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------ in 64 bits


def _decoded():
    """The value of every E4M3 code: a sign, four bits of exponent (bias 7), three of fraction; no infinity."""
    c = torch.arange(256, device=DEV)
    e, f = (c >> 3) & 15, (c & 7).to(F64)
    x = torch.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * _power(e - 7))
    x = torch.where((c & 128) != 0, -x, x)
    x[127] = x[255] = math.nan
    return x


def _power(e):
    """2^e in 64 bits, from its bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(F64)


def _nearest(y):
    """The E4M3 value nearest to y, ties to the even one, at most 448 in magnitude."""
    a = y.abs().clamp(max=TOP)
    step = _power(torch.frexp(a.clamp(min=2.0 ** -6))[1] - 4)      # 2^-3 of the power of two at or below a
    return torch.sign(y) * (torch.round(a / step) * step).clamp(max=TOP)


def _least(top):
    """The least e with top <= 448 2^e."""
    m, e = torch.frexp(top / TOP)
    return torch.where(top == 0, E_LEAST, torch.where(m == 0.5, e - 1, e)).clamp(E_LEAST, E_MOST)


def _exact_write(case, s):
    value, page, out = _decoded(), case["page"], {}
    for name in "kv":
        codes, scale = value[s[name + "_codes"].long()], s[name + "_scale"].int() - 127
        first = 0
        for b, (n, p) in enumerate(zip(_ints(case["new"]), _ints(case["past"]))):
            x, done = s[name][first:first + n].to(F64), 0
            first += n
            while done < n:
                at, slot = int(s["table"][b, (p + done) // page]), (p + done) % page
                take = min(page - slot, n - done)
                y = x[done:done + take].transpose(0, 1)
                e = _least(y.abs().amax((1, 2)))
                if slot:
                    e = torch.maximum(e, scale[at])
                    codes[at, :, :slot] = _nearest(codes[at, :, :slot] * _power(scale[at] - e)[:, None, None])
                codes[at, :, slot:slot + take] = _nearest(y * _power(-e)[:, None, None])
                scale[at] = e
                done += take
        out[name], out[name + "_scale"] = codes, None
    return out


def _held(case, s, name, b, value):
    """A sequence's keys or values [position, head, d]."""
    n, page = int(s["lengths"][b]), case["page"]
    at = s["table"][b, :-(-n // page)].long()
    x = value[s[name + "_codes"][at].long()] * _power(s[name + "_scale"][at].int() - 127)[:, :, None, None]
    return x.transpose(1, 2).reshape(-1, case["hk"], case["d"])[:n]


def _exact_read(case, s):
    value, new = _decoded(), _ints(case["new"])
    return {name: torch.cat([_held(case, s, name, b, value)[-n:] for b, n in enumerate(new) if n]) for name in "kv"}


def _exact_attend(case, s):
    value, group, scale = _decoded(), case["hq"] // case["hk"], case["d"] ** -0.5
    q = s["q"].to(F64)
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[1], q.shape[0], dtype=F64, device=DEV)
    first = 0
    for b, n in enumerate(_ints(case["new"])):
        if not n:
            continue
        k, v = _held(case, s, "k", b, value), _held(case, s, "v", b, value)
        rows = slice(first, first + n)
        first += n
        unseen = None
        if case["causal"]:
            unseen = torch.ones(n, len(k), dtype=torch.bool, device=DEV).triu(len(k) - n + 1)
        for h in range(case["hq"]):
            a = q[rows, h] @ k[:, h // group].t() * scale
            if unseen is not None:
                a.masked_fill_(unseen, -math.inf)
            z = torch.logsumexp(a, 1)
            out[rows, h], lse[h, rows] = torch.exp(a - z[:, None]) @ v[:, h // group], z
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = _inputs(case, seed)
    return {"write": _exact_write, "read": _exact_read, "attend": _exact_attend}[case["op"]](case, s)
