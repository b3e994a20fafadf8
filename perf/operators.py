"""The training operators around the FP8 linears, as measured cases.

Normalisation (root mean square or layer norm, with the residual sum in front and the
weight's gradient), attention over packed sequences with its backward pass, and the
cross entropy of a linear head over a large vocabulary with its gradients.  Each has a
plain form here (elementary torch operations in 32 bits, rounded once at the end), a
definition in 64 bits, and the call that a user of the package makes.
"""
import math

import torch

own = False

DEV = "cuda"
F32, F64, BF16 = torch.float32, torch.float64, torch.bfloat16
EPS = 1e-5

# ------------------------------------------------------------------------------ cases


def listed():
    return [
        # a single token's vector on its way into a block: what counts is the call itself
        {"name": "norm_one_row", "op": "norm", "dir": "forward", "rows": 1, "cols": 4096, "rms": True, "f32": False,
         "add": True},
        # the 7B-class layer's norm in front of a linear, with the residual sum in the same pass
        {"name": "norm_7b", "op": "norm", "dir": "forward", "rows": 4096, "cols": 4096, "rms": True, "f32": False,
         "add": True},
        # the 14B-class layer's norm, backward: 8192 tokens, the stream's own gradient joined
        {"name": "norm_grad_14b", "op": "norm", "dir": "backward", "rows": 8192, "cols": 5120, "rms": True,
         "f32": False, "add": True},
        # a layer norm with a bias on a 32-bit residual stream, a ragged number of tokens
        {"name": "norm_grad_layer_f32", "op": "norm", "dir": "backward", "rows": 1537, "cols": 1000, "rms": False,
         "f32": True, "add": False},
        # the 7B-class layer's attention: 4096 tokens of one sequence, as many key heads as query heads
        {"name": "attn_7b", "op": "attention", "dir": "forward", "lq": "4096", "lk": "4096", "hq": 32, "hk": 32,
         "d": 128, "causal": True},
        # the 14B-class layer's attention on 8192 packed tokens of documents of every length
        {"name": "attn_packed_14b", "op": "attention", "dir": "forward", "lq": "4093 1 2111 0 517 1470",
         "lk": "4093 1 2111 0 517 1470", "hq": 40, "hk": 8, "d": 128, "causal": True},
        # the 7B-class layer's attention, backward
        {"name": "attn_grad_7b", "op": "attention", "dir": "backward", "lq": "4096", "lk": "4096", "hq": 32,
         "hk": 32, "d": 128, "causal": True},
        # short questions against contexts of other lengths, some shorter than the question: rows that see nothing
        {"name": "attn_grad_short", "op": "attention", "dir": "backward", "lq": "37 130 1 64", "lk": "101 77 1 300",
         "hq": 12, "hk": 4, "d": 64, "causal": True},
        # the loss of a handful of tokens: the head's weight is read once
        {"name": "loss_few", "op": "loss", "dir": "forward", "tokens": 16, "d": 4096, "vocab": 32000},
        # the loss of the 14B-class batch over a large vocabulary of odd size
        {"name": "loss_large", "op": "loss", "dir": "forward", "tokens": 8192, "d": 5120, "vocab": 65521},
        # the 7B-class batch's gradients of the hidden states and of the head
        {"name": "loss_grad_7b", "op": "loss", "dir": "backward", "tokens": 4096, "d": 4096, "vocab": 32000},
        # a ragged batch and vocabulary
        {"name": "loss_grad_odd", "op": "loss", "dir": "backward", "tokens": 1001, "d": 1600, "vocab": 40007},
    ]


def _log_int(rng, lo, hi):
    """An integer spread over its logarithm; 3072 is passed over."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n + 1 if n == 3072 else n


def _log_eights(rng, lo, hi):
    n = 8 * int(round(math.exp(rng.uniform(math.log(lo / 8), math.log(hi / 8)))))
    return n + 8 if n == 3072 else n


def _one(rng):
    op, direction = rng.choice(["norm", "attention", "loss"]), rng.choice(["forward", "backward"])
    if op == "norm":
        cols = _log_eights(rng, 128, 8192) if rng.random() < 0.75 else _log_int(rng, 100, 8191)
        return {"op": op, "dir": direction, "rows": _log_int(rng, 1, 16384), "cols": cols,
                "rms": rng.random() < 0.5, "f32": rng.random() < 0.35, "add": rng.random() < 0.5}
    if op == "loss":
        return {"op": op, "dir": direction, "tokens": _log_int(rng, 1, 8192), "d": _log_eights(rng, 256, 5120),
                "vocab": _log_int(rng, 500, 65536)}
    n = rng.randint(1, 6)
    lk = [_log_int(rng, 1, 4096) for _ in range(n)]
    lq = list(lk) if rng.random() < 0.6 else [_log_int(rng, 1, 2048) for _ in range(n)]
    hk = rng.choice([1, 2, 4, 8])
    return {"op": op, "dir": direction, "lq": " ".join(map(str, lq)), "lk": " ".join(map(str, lk)),
            "hq": hk * rng.choice([1, 2, 4, 5]), "hk": hk, "d": rng.choice([64, 128, 128, 8 * rng.randint(4, 16)]),
            "causal": rng.random() < 0.7}


def draw(rng):
    """One more case; none costs more than the largest listed one of its operator."""
    top = {}
    for c in listed():
        top[c["op"]] = max(top.get(c["op"], 0), work(c)["flops"])
    while True:
        case = _one(rng)
        if 0 < work(case)["flops"] <= top[case["op"]]:
            return case


def _lens(text):
    return [int(n) for n in text.split()]


def _pairs(case):
    """How many (query, key) pairs the mask leaves: query i of a sequence sees the keys up to i + lk - lq."""
    n = 0
    for lq, lk in zip(_lens(case["lq"]), _lens(case["lk"])):
        if not case["causal"]:
            n += lq * lk
            continue
        first = max(0, lq - lk)                       # rows before it see nothing
        n += (lq - first) * (2 * (lk - lq + 1 + first) + (lq - 1 - first)) // 2
    return n


def work(case):
    back = case["dir"] == "backward"
    if case["op"] == "norm":
        n, size = case["rows"] * case["cols"], 4 if case["f32"] else 2
        stats = 4 * case["rows"] * (1 if case["rms"] else 2)
        vectors = case["cols"] * (2 if case["rms"] else 4)
        if back:                                       # dy, x (and the joined gradient) in, dx and the vectors out
            return {"bytes": n * (2 + 2 * size + (size if case["add"] else 0)) + stats + 3 * vectors, "flops": 12 * n}
        return {"bytes": n * (size + 2 + ((2 + size) if case["add"] else 0)) + stats + vectors, "flops": 8 * n}
    if case["op"] == "loss":
        t, d, v = case["tokens"], case["d"], case["vocab"]
        if back:                                       # logits again, the hidden states' and the head's gradients
            return {"bytes": 4 * (t * d + v * d) + 16 * t, "flops": 6 * t * d * v}
        return {"bytes": 2 * (t * d + v * d) + 16 * t, "flops": 2 * t * d * v}
    q = sum(_lens(case["lq"])) * case["hq"]
    kv = sum(_lens(case["lk"])) * case["hk"]
    d = case["d"]
    if back:                                           # q, k, v, out, dout in; dq, dk, dv out
        return {"bytes": 2 * d * (4 * q + 4 * kv) + 4 * q, "flops": 10 * d * case["hq"] * _pairs(case)}
    return {"bytes": 2 * d * (2 * q + 2 * kv) + 4 * q, "flops": 4 * d * case["hq"] * _pairs(case)}


# ------------------------------------------------------------------------------ inputs


def _inputs(case, seed):
    """The inputs of a case, from the seed alone."""
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    normal = lambda shape, sigma=1.0, dtype=BF16: (torch.randn(shape, generator=g, device=DEV) * sigma).to(dtype)
    if case["op"] == "norm":
        shape, wide = (case["rows"], case["cols"]), F32 if case["f32"] else BF16
        # a residual stream has channels that stand out
        gain = torch.exp(torch.randn(case["cols"], generator=g, device=DEV) * 0.5)
        s = {"x": (normal(shape, 1.0, F32) * gain + 0.1).to(wide),
             "weight": (1 + normal((case["cols"],), 0.1, F32)).to(BF16),
             "bias": None if case["rms"] else normal((case["cols"],), 0.1),
             "add": normal(shape, 0.5) if case["add"] and case["dir"] == "forward" else None}
        if case["dir"] == "backward":
            s["dy"] = normal(shape, 1e-3)
            s["dres"] = normal(shape, 1e-3, wide) if case["add"] else None
        return s
    if case["op"] == "loss":
        t, d, v = case["tokens"], case["d"], case["vocab"]
        s = {"x": normal((t, d)), "weight": normal((v, d), 0.02),
             "target": torch.randint(0, v, (t,), generator=g, device=DEV)}
        # one token in sixteen is padding or prompt, and has no target
        s["target"][torch.rand(t, generator=g, device=DEV) < 1 / 16] = -100
        if case["dir"] == "backward":
            s["dloss"] = torch.full((t,), 1.0 / t, device=DEV)
        return s
    lq, lk, hq, hk, d = _lens(case["lq"]), _lens(case["lk"]), case["hq"], case["hk"], case["d"]
    tq, tk = sum(lq), sum(lk)
    if lq == lk:                                       # slices of one projection's output, as in a layer
        qkv = normal((tq, (hq + 2 * hk) * d))
        q, kv = qkv[:, :hq * d], qkv[:, hq * d:]
    else:
        q, kv = normal((tq, hq * d)), normal((tk, 2 * hk * d))
    s = {"q": q.unflatten(1, (hq, d)), "k": kv[:, :hk * d].unflatten(1, (hk, d)),
         "v": kv[:, hk * d:].unflatten(1, (hk, d))}
    if case["dir"] == "backward":
        s["dout"] = normal((tq, hq, d), 1e-2)
    return s


def _sequences(lens, longest):
    """Where each place of a padded batch lies in the packed tokens, and where each token lies in the batch."""
    n = torch.tensor(lens, device=DEV)
    start = torch.cumsum(n, 0) - n
    inside = torch.arange(longest, device=DEV)[None, :].expand(len(lens), -1)
    held = inside < n[:, None]
    return n, torch.where(held, start[:, None] + inside, 0), held.nonzero(as_tuple=True)


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] == "norm":
        if case["dir"] == "backward":
            _, _, s["mean"], s["rstd"] = _norm(s, F32)
    elif case["op"] == "loss":
        if case["dir"] == "backward":
            s["lse"] = torch.logsumexp(s["x"].float() @ s["weight"].float().t(), 1)
    else:
        lq, lk = _lens(case["lq"]), _lens(case["lk"])
        s["scale"] = case["d"] ** -0.5
        s["nq"], s["iq"], s["uq"] = _sequences(lq, max(lq))
        s["nk"], s["ik"], s["uk"] = _sequences(lk, max(lk))
        bounds = lambda n: torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), torch.cumsum(n, 0)]).to(torch.int32)
        s["cu_q"], s["cu_k"] = bounds(s["nq"]), bounds(s["nk"])
        if case["dir"] == "backward":
            s["out"], s["lse"] = _attention(s)
    return s


# ------------------------------------------------------------------------------ plain forms


def _norm(s, f):
    """y, the summed stream, mean and reciprocal deviation, in the type f."""
    x = s["x"].to(f)
    if s["add"] is not None:
        x = x + s["add"].to(f)
    mean = None if s["case"]["rms"] else x.mean(1)
    c = x if mean is None else x - mean[:, None]
    rstd = 1 / torch.sqrt((c * c).mean(1) + EPS)
    y = c * rstd[:, None] * s["weight"].to(f)
    return (y if s["bias"] is None else y + s["bias"].to(f)), x, mean, rstd


def _norm_forward(s):
    y, x, mean, rstd = _norm(s, F32)
    out = {"y": y.to(BF16), "rstd": rstd}
    if mean is not None:
        out["mean"] = mean
    if s["add"] is not None:
        out["sum"] = x.to(s["x"].dtype)
    return out


def _norm_backward(s):
    x, dy = s["x"].float(), s["dy"].float()
    c = x if s["mean"] is None else x - s["mean"][:, None]
    h = c * s["rstd"][:, None]
    g = dy * s["weight"].float()
    dx = g - h * (g * h).mean(1, keepdim=True)
    if s["mean"] is not None:
        dx = dx - g.mean(1, keepdim=True)
    dx = dx * s["rstd"][:, None]
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    out = {"dx": dx.to(s["x"].dtype), "dweight": (dy * h).sum(0)}
    if s["bias"] is not None:
        out["dbias"] = dy.sum(0)
    return out


def _scores(s):
    """Padded queries and keys [sequence, head, place, d] and the masked scores."""
    q = s["q"].float()[s["iq"]].transpose(1, 2)
    k = s["k"].float()[s["ik"]].transpose(1, 2).repeat_interleave(s["case"]["hq"] // s["case"]["hk"], 1)
    i = torch.arange(q.shape[2], device=DEV)[None, :, None]
    j = torch.arange(k.shape[2], device=DEV)[None, None, :]
    nq, nk = s["nq"][:, None, None], s["nk"][:, None, None]
    seen = (i < nq) & (j < nk)
    if s["case"]["causal"]:
        seen = seen & (j <= i + (nk - nq))
    a = (q @ k.transpose(2, 3)) * s["scale"]
    return q, k, a.masked_fill_(~seen[:, None], -math.inf)


def _values(s):
    return s["v"].float()[s["ik"]].transpose(1, 2).repeat_interleave(s["case"]["hq"] // s["case"]["hk"], 1)


def _packed(x, at):
    """[sequence, head, place, ...] back to packed tokens [token, head, ...]."""
    return x.transpose(1, 2)[at]


def _attention(s):
    _, _, a = _scores(s)
    top = a.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(a - top)
    total = p.sum(3, keepdim=True)
    out = (p @ _values(s)) / torch.where(total == 0, 1.0, total)
    lse = (top + torch.log(total)).squeeze(3)
    return _packed(out, s["uq"]).to(BF16), _packed(lse, s["uq"]).t().contiguous()


def _attention_backward(s):
    q, k, a = _scores(s)
    v = _values(s)
    lse = torch.zeros(a.shape[:3], device=DEV).transpose(1, 2)
    lse = lse.index_put(s["uq"], s["lse"].t()).transpose(1, 2)[..., None]
    p = torch.exp(a - torch.where(lse == -math.inf, 0.0, lse))
    do = s["dout"].float()[s["iq"]].transpose(1, 2)
    dv = p.transpose(2, 3) @ do
    dp = do @ v.transpose(2, 3)
    ds = p * (dp - (p * dp).sum(3, keepdim=True)) * s["scale"]
    dq = ds @ k
    dk = ds.transpose(2, 3) @ q
    shared = lambda x: x.unflatten(1, (s["case"]["hk"], -1)).sum(2)
    return {"dq": _packed(dq, s["uq"]).to(BF16), "dk": _packed(shared(dk), s["uk"]).to(BF16),
            "dv": _packed(shared(dv), s["uk"]).to(BF16)}


def _loss_forward(s):
    z = s["x"].float() @ s["weight"].float().t()
    top = z.amax(1, keepdim=True)
    lse = top[:, 0] + torch.log(torch.exp(z - top).sum(1))
    t = s["target"]
    hit = z.gather(1, t.clamp(min=0)[:, None])[:, 0]
    return {"loss": torch.where(t < 0, 0.0, lse - hit), "lse": lse}


def _loss_backward(s):
    x, w, t = s["x"].float(), s["weight"].float(), s["target"]
    g = torch.exp(x @ w.t() - s["lse"][:, None])
    g.scatter_add_(1, t.clamp(min=0)[:, None], torch.full_like(g[:, :1], -1.0))
    g = g * torch.where(t < 0, 0.0, s["dloss"])[:, None]
    return {"dx": (g @ w).to(BF16), "dweight": (g.t() @ x).to(BF16)}


# ------------------------------------------------------------------------------ the package's calls


def _own(s):
    import fp8_precision_amd as fp8
    case = s["case"]
    if case["op"] == "norm":
        if case["dir"] == "forward":
            y, total, mean, rstd = fp8.norm(s["x"], s["weight"], s["bias"], add=s["add"], eps=EPS, rms=case["rms"])
            out = {"y": y, "rstd": rstd}
            if mean is not None:
                out["mean"] = mean
            if s["add"] is not None:
                out["sum"] = total
            return out
        dx, dw, db = fp8.norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], dres=s["dres"],
                                       want_dbias=s["bias"] is not None)
        out = {"dx": dx, "dweight": dw}
        if db is not None:
            out["dbias"] = db
        return out
    if case["op"] == "loss":
        if case["dir"] == "forward":
            loss, lse = fp8.linear_cross_entropy(s["x"], s["weight"], s["target"])
            return {"loss": loss, "lse": lse}
        dx, dw = fp8.linear_cross_entropy_backward(s["dloss"], s["x"], s["weight"], s["target"], s["lse"])
        return {"dx": dx, "dweight": dw}
    how = {"cu_q": s["cu_q"], "cu_k": s["cu_k"], "causal": case["causal"], "scale": s["scale"]}
    if case["dir"] == "forward":
        out, lse = fp8.attention(s["q"], s["k"], s["v"], **how)
        return {"out": out, "lse": lse}
    dq, dk, dv = fp8.attention_backward(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], **how)
    return {"dq": dq, "dk": dk, "dv": dv}


def run(state):
    if own:
        return _own(state)
    case = state["case"]
    if case["op"] == "norm":
        return _norm_forward(state) if case["dir"] == "forward" else _norm_backward(state)
    if case["op"] == "loss":
        return _loss_forward(state) if case["dir"] == "forward" else _loss_backward(state)
    if case["dir"] == "forward":
        out, lse = _attention(state)
        return {"out": out, "lse": lse}
    return _attention_backward(state)


# ------------------------------------------------------------------------------ in 64 bits


def _exact_norm(case, s):
    x = s["x"].to(F64) + (0 if s["add"] is None else s["add"].to(F64))
    n = x.shape[1]
    mu = torch.zeros_like(x[:, 0]) if case["rms"] else x.sum(1) / n
    h = x - mu[:, None]
    rstd = torch.rsqrt((h ** 2).sum(1) / n + EPS)
    h = h * rstd[:, None]
    w = s["weight"].to(F64)
    if case["dir"] == "forward":
        y = h * w + (0 if s["bias"] is None else s["bias"].to(F64))
        out = {"y": y, "rstd": rstd}
        if not case["rms"]:
            out["mean"] = mu
        if s["add"] is not None:
            out["sum"] = x
        return out
    dy = s["dy"].to(F64)
    dh = dy * w
    # the gradient of h = (x - mu) rstd: what lies along 1 (layer norm) and along h is taken out
    along = (dh * h).sum(1, keepdim=True) / n
    flat = 0 if case["rms"] else dh.sum(1, keepdim=True) / n
    dx = rstd[:, None] * (dh - flat - along * h) + (0 if s["dres"] is None else s["dres"].to(F64))
    out = {"dx": dx, "dweight": torch.einsum("rc,rc->c", dy, h)}
    if s["bias"] is not None:
        out["dbias"] = dy.sum(0)
    return out


def _exact_loss(case, s):
    x, w, t = s["x"].to(F64), s["weight"].to(F64), s["target"]
    z = torch.mm(x, w.t())
    lse = torch.logsumexp(z, 1)
    rows = torch.arange(len(t), device=DEV)
    has = t >= 0
    if case["dir"] == "forward":
        loss = torch.zeros_like(lse)
        loss[has] = (lse - z[rows, t.clamp(min=0)])[has]
        return {"loss": loss, "lse": lse}
    z.sub_(lse[:, None]).exp_()
    z[rows[has], t[has]] -= 1
    z *= (s["dloss"].to(F64) * has)[:, None]
    return {"dx": torch.mm(z, w), "dweight": torch.mm(z.t(), x)}


def _exact_attention(case, s):
    group, scale = case["hq"] // case["hk"], case["d"] ** -0.5
    q, k, v = (s[n].to(F64) for n in "qkv")
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[1], q.shape[0], dtype=F64, device=DEV)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    q0 = k0 = 0
    for nq, nk in zip(_lens(case["lq"]), _lens(case["lk"])):
        if nq and nk:
            for h in range(case["hq"]):
                qs, ks = slice(q0, q0 + nq), slice(k0, k0 + nk)
                qh, kh, vh = q[qs, h], k[ks, h // group], v[ks, h // group]
                a = qh @ kh.t() * scale
                if case["causal"]:
                    # ones on and below the diagonal that ends in the last row's last key
                    a = a.masked_fill(torch.ones(nq, nk, device=DEV).tril(nk - nq) == 0, -math.inf)
                z = torch.logsumexp(a, 1)
                p = torch.exp(a - z.clamp(min=-1e300)[:, None])
                out[qs, h], lse[h, qs] = p @ vh, z
                if case["dir"] == "backward":
                    do = s["dout"][qs, h].to(F64)
                    dp = do @ vh.t()
                    ds = p * (dp - (do * out[qs, h]).sum(1, keepdim=True)) * scale
                    dq[qs, h] = ds @ kh
                    dk[ks, h // group] += ds.t() @ qh
                    dv[ks, h // group] += p.t() @ do
        elif nq:
            lse[:, q0:q0 + nq] = -math.inf
        q0, k0 = q0 + nq, k0 + nk
    if case["dir"] == "forward":
        return {"out": out, "lse": lse}
    return {"dq": dq, "dk": dk, "dv": dv}


def exact(case, seed):
    s = _inputs(case, seed)
    return {"norm": _exact_norm, "loss": _exact_loss, "attention": _exact_attention}[case["op"]](case, s)
