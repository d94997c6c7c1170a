"""Cases of the paged key-value cache's operators: the plain form of each beside the library's call.

``append``  writes the new tokens' keys and values into a paged cache, with the position rotation
            of keys and queries applied on the way;
``attend``  reads the cache for one new token of each sequence (softmax attention over the
            sequence's cached tokens).

Shapes: heads query heads share kv_heads cached heads of dim elements; a cache is a pool of pages
[pages][kv_heads][page][dim], and row b of the table lists the pages of sequence b in order.
"""
import math

import torch

own = False

GOLDEN = 0.6180339887498949
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZES = {"bf16": 2, "f32": 4, "e4m3": 1}


def listed():
    return [
        # a serving step of a few conversations, one of them very long: latency of one small call
        _append("append one token of 4", batch=4, heads=32, kv_heads=8, dim=128, page=64,
                longest=131072, shortest=1),
        # the decode batch of a large server whose cache is held in 8 bits
        _append("append one token of 256", batch=256, heads=64, kv_heads=8, dim=128, page=64,
                longest=8192, shortest=1, cache="e4m3"),
        # prompts of very different lengths written in one packed call, some behind a long past
        _append("append ragged prompts", batch=8, heads=28, kv_heads=4, dim=128, page=16,
                longest=131072, shortest=0, new=4096, new_shortest=1),
        # a chunk of 4096 tokens of two sequences in full precision; adjacent pairs of the first
        # 32 elements rotate; a page size that is no power of two
        _append("append chunk f32", batch=2, heads=16, kv_heads=8, dim=64, page=48, longest=4096,
                shortest=4096, new=4096, new_shortest=4096, inputs="f32", cache="f32", rotary=32,
                style="pairs"),
        # one long document with wide heads into an 8-bit cache
        _append("append long prompt", batch=1, heads=16, kv_heads=2, dim=256, page=128,
                longest=16384, shortest=16384, new=16384, new_shortest=16384, cache="e4m3"),
        # one conversation shortly after its start: latency
        _attend("attend one short", batch=1, heads=32, kv_heads=8, dim=128, page=64, longest=512,
                shortest=512),
        # one 128K context: the whole card on one sequence
        _attend("attend one long", batch=1, heads=32, kv_heads=8, dim=128, page=64,
                longest=131072, shortest=131072),
        # a serving batch of every length up to 8192, small pages, seven queries to a cached head
        _attend("attend ragged batch", batch=64, heads=28, kv_heads=4, dim=128, page=16,
                longest=8192, shortest=1),
        # many short conversations of a small model without shared heads
        _attend("attend many short", batch=512, heads=16, kv_heads=16, dim=64, page=32,
                longest=256, shortest=1),
        # layers that see the last 1024 tokens of long sequences; older pages were given back
        _attend("attend window", batch=128, heads=32, kv_heads=8, dim=128, page=64,
                longest=131072, shortest=1, window=1024),
        # long contexts held in 8 bits
        _attend("attend e4m3", batch=32, heads=64, kv_heads=8, dim=128, page=64, longest=32768,
                shortest=2048, cache="e4m3"),
        # the same in full precision, wide heads, a page size that is no power of two
        _attend("attend f32", batch=4, heads=8, kv_heads=2, dim=256, page=48, longest=8192,
                shortest=4096, inputs="f32", cache="f32"),
    ]


def _append(name=None, new=1, new_shortest=1, inputs="bf16", cache="bf16", rotary=None,
            style="halves", **sizes):
    case = dict(op="append", inputs=inputs, cache=cache, new=new, new_shortest=new_shortest,
                rotary=sizes["dim"] if rotary is None else rotary, style=style, **sizes)
    return case if name is None else dict(case, name=name)


def _attend(name=None, inputs="bf16", cache="bf16", window=0, **sizes):
    case = dict(op="attend", inputs=inputs, cache=cache, window=window, **sizes)
    return case if name is None else dict(case, name=name)


def draw(rng):
    def log(lo, hi):
        return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))

    cap = max(work(c)["bytes"] for c in listed())
    inputs, cache = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "e4m3"),
                                ("f32", "f32")])
    heads, kv_heads = rng.choice([(32, 8), (28, 4), (16, 16), (8, 2), (64, 8), (5, 1), (12, 4),
                                  (32, 1), (40, 40), (48, 2)])
    sizes = dict(heads=heads, kv_heads=kv_heads, dim=rng.choice([64, 80, 96, 128, 128, 192, 256]),
                 page=rng.choice([8, 16, 32, 48, 64, 100, 128, 256]), batch=log(1, 512),
                 longest=log(1, 131072))
    sizes["shortest"] = rng.choice([0, 1, sizes["longest"] // 2, sizes["longest"]])
    if rng.random() < 0.4:
        new = rng.choice([1, 1, log(1, 8192)])
        sizes["longest"] = max(sizes["longest"], new)
        case = _append(inputs=inputs, cache=cache, new=new,
                       new_shortest=1 if new == 1 else rng.choice([0, 1, new]),
                       rotary=rng.choice([sizes["dim"], sizes["dim"] // 32 * 16, 16]),
                       style=rng.choice(["halves", "pairs"]), **sizes)
        if new == 1:
            case["shortest"] = max(1, case["shortest"])
    else:
        case = _attend(inputs=inputs, cache=cache, window=rng.choice([0, 0, log(1, 8192)]),
                       **sizes)
    while work(case)["bytes"] > cap:
        if case["batch"] > 1:
            case["batch"] = max(1, case["batch"] * 2 // 3)
        else:
            case["longest"] = case["longest"] * 2 // 3
            case["shortest"] = min(case["shortest"], case["longest"])
            if "new" in case:
                case["new"] = min(case["new"], case["longest"])
                case["new_shortest"] = min(case["new_shortest"], case["new"])
    return case


def _spread(most, least, batch):
    """`batch` lengths between the two ends, the first the longest, in no order."""
    return [most - int((most - least + 0.999) * (b * GOLDEN % 1.0)) for b in range(batch)]


def _lengths(case):
    """(cached tokens, new tokens among them) of every sequence."""
    total = _spread(case["longest"], case["shortest"], case["batch"])
    if case["op"] == "attend":
        return total, [0] * case["batch"]
    new = _spread(case["new"], case["new_shortest"], case["batch"])
    return [max(a, b) for a, b in zip(total, new)], new


def work(case):
    total, new = _lengths(case)
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
    size, cached = SIZES[case["inputs"]], SIZES[case["cache"]]
    if case["op"] == "append":
        rows = sum(new)
        return {"bytes": rows * dim * ((2 * heads + 2 * kv_heads) * size + 2 * kv_heads * cached),
                "flops": 3 * rows * (heads + kv_heads) * case["rotary"]}
    seen = sum(min(n, case["window"]) if case["window"] else n for n in total)
    return {"bytes": 2 * seen * kv_heads * dim * cached + case["batch"] * heads * (2 * dim * size + 4),
            "flops": 4 * seen * heads * dim}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    batch, kv_heads, page, dim = (case[k] for k in ("batch", "kv_heads", "page", "dim"))
    dtype, cached = DTYPES[case["inputs"]], DTYPES[case["cache"]]
    total, new = _lengths(case)
    # the pages in use: all of a sequence's, or those of its window or its new tokens
    first = [0] * batch
    if case["op"] == "append":
        first = [(n - m) // page for n, m in zip(total, new)]
    elif case["window"]:
        first = [max(0, n - case["window"]) // page for n in total]
    count = [-(-n // page) - f for n, f in zip(total, first)]
    pages = sum(count) + 3
    width = max(1, max(-(-n // page) for n in total))
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    at = torch.tensor([sum(count[:b]) for b in range(batch)], device="cuda")[:, None]
    column = torch.arange(width, device="cuda")[None, :]
    column = column - torch.tensor(first, device="cuda")[:, None]
    mine = (column >= 0) & (column < torch.tensor(count, device="cuda")[:, None])
    table = torch.where(mine, order[(at + column).clamp(0, pages - 1)], -1).contiguous()

    s = {"case": case, "table": table,
         "lengths": torch.tensor(total, dtype=torch.int32, device="cuda"),
         "key_scale": None, "value_scale": None}
    if case["cache"] == "e4m3":  # the scales of a calibrated cache, one to a cached head
        s["key_scale"] = 0.01 + 0.02 * torch.rand(kv_heads, generator=g, device="cuda")
        s["value_scale"] = 0.01 + 0.02 * torch.rand(kv_heads, generator=g, device="cuda")
    pool = (pages, kv_heads, page, dim)
    for name in ("key", "value"):
        x = torch.empty(pool, dtype=cached, device="cuda")
        for i in range(0, pages, 4096):
            y = normal(*x[i:i + 4096].shape)
            if s[name + "_scale"] is not None:
                y = (y / s[name + "_scale"][None, :, None, None]).clamp(-448, 448)
            x[i:i + 4096] = y.to(cached)
        s[name + "s"] = x

    if case["op"] == "append":
        rows, heads = sum(new), case["heads"]
        # the output of one projection: queries, keys and values side by side
        qkv = normal(rows, heads + 2 * kv_heads, dim).to(dtype)
        s["q"], s["k"], s["v"] = qkv.split([heads, kv_heads, kv_heads], 1)
        s["starts"] = None
        if case["new"] > 1:
            ends = [sum(new[:b]) for b in range(batch + 1)]
            s["starts"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
        half = torch.arange(case["rotary"] // 2, dtype=torch.float64, device="cuda")
        s["freqs"] = (10000.0 ** (-2 * half / case["rotary"])).float()
    else:
        # queries that favour some tokens: scores of standard deviation 2
        s["q"] = (2 * normal(batch, case["heads"], dim)).to(dtype)
    if own:
        from sparse_weight_memory_b200 import KVCache
        s["cache"] = KVCache(keys=s["keys"], values=s["values"], key_scale=s["key_scale"],
                             value_scale=s["value_scale"])
    return s


def run(s):
    case = s["case"]
    if case["op"] == "append":
        if own:
            q = s["cache"].append(s["k"], s["v"], s["table"], s["lengths"], starts=s["starts"],
                                  q=s["q"], freqs=s["freqs"], style=case["style"])
        else:
            q = append_plain(s)
        return {"q": q, "keys": s["keys"], "values": s["values"]}
    if own:
        lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
        out = s["cache"].attend(s["q"], s["table"], s["lengths"], window=case["window"], lse=lse)
        return {"out": out, "lse": lse}
    return attend_plain(s)


# -- the plain forms ------------------------------------------------------------------------------

def rotate(x, cos, sin, style):
    """x [rows, heads, dim] in 32 bits: the first 2 * cos.shape[1] elements of each head turned."""
    r = cos.shape[1]
    c, t = cos[:, None, :], sin[:, None, :]
    if style == "halves":
        a, b, rest = x[..., :r], x[..., r:2 * r], x[..., 2 * r:]
        return torch.cat([a * c - b * t, b * c + a * t, rest], -1)
    a, b, rest = x[..., 0:2 * r:2], x[..., 1:2 * r:2], x[..., 2 * r:]
    turned = torch.stack([a * c - b * t, b * c + a * t], -1).flatten(-2)
    return torch.cat([turned, rest], -1)


def stored(x, scale, dtype):
    """x [rows, kv_heads, dim] in 32 bits as the cache holds it."""
    if scale is None:
        return x.to(dtype)
    return (x / scale[None, :, None]).clamp(-448, 448).to(dtype)


def put(pool, page, slot, x):
    """Rows of x into the pool; the bytes of 8-bit elements, which torch does not index."""
    if pool.element_size() == 1:
        pool, x = pool.view(torch.uint8), x.view(torch.uint8)
    pool[page, :, slot] = x


def append_plain(s):
    case, lengths, page = s["case"], s["lengths"].long(), s["case"]["page"]
    row = torch.arange(s["k"].shape[0], device="cuda")
    if s["starts"] is None:
        seq, pos = row, lengths - 1
    else:
        seq = torch.searchsorted(s["starts"][1:].long(), row, right=True)
        pos = lengths[seq] - s["starts"][1:].long()[seq] + row
    angle = pos[:, None].double() * s["freqs"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    where = s["table"][seq, pos // page].long()
    k = rotate(s["k"].float(), cos, sin, case["style"])
    put(s["keys"], where, pos % page, stored(k, s["key_scale"], s["keys"].dtype))
    put(s["values"], where, pos % page, stored(s["v"].float(), s["value_scale"], s["values"].dtype))
    return rotate(s["q"].float(), cos, sin, case["style"]).to(s["q"].dtype)


def gathered(pool, table, scale):
    """[batch, kv_heads, tokens, dim] in 32 bits."""
    raw = pool.view(torch.uint8) if pool.element_size() == 1 else pool
    x = raw[table.long().clamp(min=0)].view(pool.dtype)  # [batch, width, kv_heads, page, dim]
    x = x.permute(0, 2, 1, 3, 4).flatten(2, 3).float()
    return x if scale is None else x.mul_(scale[None, :, None, None])


def attend_plain(s):
    case, q, table, lengths = s["case"], s["q"], s["table"], s["lengths"]
    batch, heads, dim = q.shape
    page, window = case["page"], case["window"]
    if window:  # the columns that the window of each sequence touches
        first = (lengths.long() - window).clamp(min=0) // page
        column = torch.arange((window + page - 2) // page + 1, device="cuda")[None, :]
        column = column + first[:, None]
        table = table.gather(1, column.clamp(max=table.shape[1] - 1))
        pos = (column[:, :, None] * page + torch.arange(page, device="cuda")).flatten(1)
        seen = (pos < lengths[:, None]) & (pos >= lengths[:, None] - window)
    else:
        pos = torch.arange(table.shape[1] * page, device="cuda")[None, :]
        seen = pos < lengths[:, None]
    k = gathered(s["keys"], table, s["key_scale"])
    qs = q.float().view(batch, case["kv_heads"], -1, dim)
    score = (qs @ k.transpose(2, 3)) * (1.0 / math.sqrt(dim))
    del k
    score = score.masked_fill(~seen[:, None, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    norm = weight.sum(-1, keepdim=True)
    out = (weight @ gathered(s["values"], table, s["value_scale"])) / torch.where(norm == 0, 1.0, norm)
    lse = top + torch.log(norm)
    return {"out": out.reshape(batch, heads, dim).to(q.dtype), "lse": lse.view(batch, heads)}


# -- the definition in 64 bits --------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    total, new = _lengths(case)
    page, dim = case["page"], case["dim"]
    table = s["table"].tolist()
    ks = torch.ones(case["kv_heads"], device="cuda") if s["key_scale"] is None else s["key_scale"]
    vs = torch.ones(case["kv_heads"], device="cuda") if s["value_scale"] is None else s["value_scale"]
    ks, vs = ks.double()[:, None, None], vs.double()[:, None, None]
    if case["op"] == "append":
        keys, values = s["keys"].double(), s["values"].double()
        turned = s["q"].double().clone()
        n = case["rotary"] // 2
        if case["style"] == "halves":
            one, two = slice(0, n), slice(n, 2 * n)
        else:
            one, two = slice(0, 2 * n, 2), slice(1, 2 * n, 2)
        top = math.inf if case["cache"] != "e4m3" else 448.0
        at = 0
        for b, (length, m) in enumerate(zip(total, new)):
            if not m:
                continue
            places = torch.arange(length - m, length, device="cuda")
            z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                            places.double()[:, None] * s["freqs"].double())[:, None, :]
            k = s["k"][at:at + m].double().clone()
            for x in (k, turned[at:at + m]):
                w = torch.complex(x[..., one], x[..., two]) * z
                x[..., one], x[..., two] = w.real, w.imag
            rows = torch.tensor([table[b][p] for p in range((length - m) // page, -(-length // page))],
                                device="cuda")
            p, r = rows[places // page - (length - m) // page], places % page
            keys[p, :, r] = (k / ks[:, 0]).clamp(-top, top)
            values[p, :, r] = (s["v"][at:at + m].double() / vs[:, 0]).clamp(-top, top)
            at += m
        return {"q": turned, "keys": keys, "values": values}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    share = case["heads"] // case["kv_heads"]
    for b, length in enumerate(total):
        lo = max(0, length - case["window"]) if case["window"] else 0
        if length <= lo:
            continue
        rows = torch.tensor(table[b][lo // page:-(-length // page)], device="cuda")
        cut = slice(lo % page, lo % page + length - lo)

        def tokens(pool):
            raw = pool.view(torch.uint8) if pool.element_size() == 1 else pool
            x = raw[rows].view(pool.dtype).transpose(0, 1).reshape(case["kv_heads"], -1, dim)
            return x[:, cut].double()

        k, v = tokens(s["keys"]) * ks, tokens(s["values"]) * vs
        q = s["q"][b].double().view(-1, share, dim)
        score = torch.einsum("hgd,htd->hgt", q, k) / math.sqrt(dim)
        lse[b] = torch.logsumexp(score, -1).flatten()
        weight = torch.exp(score - lse[b].view(-1, share, 1))
        out[b] = torch.einsum("hgt,htd->hgd", weight, v).reshape(-1, dim)
    return {"out": out, "lse": lse}
