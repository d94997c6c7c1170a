"""Paged key-value cache on the GPU against plain 64-bit forms.

Tolerances.  A result rounded to type T is off by half a step, u = eps(T)/2 of
it.  What the kernels add before that rounding:
  - a score is a sum of dim products held in 32 bits:
    ds <= scale * sum |q_i k_i| * (dim + 16) 2^-23, and for 8-bit caches scale * max |q| * sum |k_i| * 2^-25 more (queries in
    16-bit floats);
  - a weight 2^(s-m) is then off by ds (its exponent) and 2^-22 (exp2), twice
    (numerator and denominator); as an operand of the second product it is
    rounded to two bf16 parts (2^-16), to 11 bits (2^-11, 8-bit caches) or, in
    32 bits, not at all (2^-22 is given it);
  - the sums over n tokens run in 32 bits in n/8 steps and a join: (n/8 + 64) 2^-23.
An output is off by these shares of sum_t p_t |v_t|.  lse is off by ds, the
sums' share and the roundings of ln 2 (m + log2 l): 4 * 2^-23 (|lse| + |m|).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_weight_memory_b200 import build
    build.build()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def make_pool(g, pages, kv, page, dim, dtype, fill=None, layout="heads"):
    from sparse_weight_memory_b200 import KVCache
    scales = {}
    if dtype == E4:
        scales = {n: 0.01 + 0.02 * torch.rand(kv, generator=g, device="cuda")
                  for n in ("key_scale", "value_scale")}
    pools = []
    for n in ("key_scale", "value_scale"):
        x = torch.randn((pages, kv, page, dim), generator=g, device="cuda")
        if dtype == E4:
            x = (x / scales[n][None, :, None, None]).clamp(-448, 448)
        if fill is not None:
            x = torch.full_like(x, fill)
        pools.append(x.to(dtype))
    if layout == "tokens":  # [pages][page][kv][dim]
        pools = [p.transpose(1, 2).contiguous().transpose(1, 2) for p in pools]
    elif layout == "both":  # keys and values of a page side by side, rows padded
        both = torch.zeros((pages, 2, kv, page, dim + 16), dtype=dtype, device="cuda")
        views = [both[:, i, :, :, :dim] for i in range(2)]
        for view, p in zip(views, pools):
            view.copy_(p)
        pools = views
    return KVCache(keys=pools[0], values=pools[1], **scales)


def make_table(g, lengths, page, spare=2, first=None):
    """Every sequence's pages, in random order over the pool; -1 elsewhere."""
    count = [-(-n // page) for n in lengths]
    first = first or [0] * len(lengths)
    total = sum(c - f for c, f in zip(count, first)) + spare
    order = torch.randperm(total, generator=g, device="cuda").tolist()
    width = max(1, max(count))
    rows = []
    for c, f in zip(count, first):
        rows.append([-1] * f + [order.pop() for _ in range(c - f)] + [-1] * (width - c))
    return torch.tensor(rows, dtype=torch.int32, device="cuda"), total


def as_int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def held(cache, which):
    """A pool as the 64-bit values it stands for."""
    pool = cache.keys if which == 0 else cache.values
    x = pool.float().double()
    s = cache._scales[which]
    return x if s is None else x * s.double()[None, :, None, None]


def reference(cache, q, table, lengths, scale, window):
    """out, lse and their tolerances, from the definition in 64 bits."""
    B, H, D = q.shape
    page, kv = cache.page_size, cache.kv_heads
    K, V = held(cache, 0), held(cache, 1)
    out = torch.zeros((B, H, D), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    lse = torch.full((B, H), -math.inf, dtype=torch.float64, device="cuda")
    ltol = torch.zeros((B, H), dtype=torch.float64, device="cuda")
    u = {BF: 2.0 ** -8, F32: 2.0 ** -24}[q.dtype]
    pw = {BF: 2.0 ** -16, E4: 2.0 ** -11, F32: 2.0 ** -22}[cache.dtype]
    for b, n in enumerate(lengths):
        lo = max(0, n - window) if window else 0
        if n <= lo:
            continue
        t = torch.arange(lo, n, device="cuda")
        pg, row = table[b][t // page].long(), t % page
        ok = (pg >= 0) & (pg < cache.pages)
        pg, row = pg[ok], row[ok]
        if not len(pg):
            continue
        k, v = K[pg, :, row].transpose(0, 1), V[pg, :, row].transpose(0, 1)  # [kv, n, D]
        qb = q[b].double().view(kv, H // kv, D)
        s = scale * torch.einsum("hgd,htd->hgt", qb, k)
        ds = abs(scale) * torch.einsum("hgd,htd->hgt", qb.abs(), k.abs()).amax(-1) * (D + 16) * 2.0 ** -23
        if cache.dtype == E4:
            ds += abs(scale) * qb.abs().amax(-1) * k.abs().sum(-1).amax(-1)[:, None] * 2.0 ** -25
        p = torch.softmax(s, -1)
        sums = (len(pg) / 8 + 64) * 2.0 ** -23
        o = torch.einsum("hgt,htd->hgd", p, v)
        share = (2 * (ds + 2.0 ** -22) + pw + sums)[..., None]
        out[b] = o.reshape(H, D)
        tol[b] = (u * o.abs() + share * torch.einsum("hgt,htd->hgd", p, v.abs())).reshape(H, D)
        ls = torch.logsumexp(s, -1)
        lse[b] = ls.flatten()
        ltol[b] = (ds + 2.0 ** -22 + sums
                   + 2.0 ** -21 * (ls.abs() + s.amax(-1).abs() + 9)).flatten()
    return out, tol, lse, ltol


def check(cache, q, table, lengths, window=0, scale=None, got=None, **kw):
    lse = torch.full(q.shape[:2], float("nan"), device="cuda")
    if got is None:
        out = cache.attend(q, table, as_int32(lengths), window=window, scale=scale, lse=lse, **kw)
    else:
        out, lse = got
    want, tol, wl, ltol = reference(cache, q, table, lengths,
                                    1 / math.sqrt(cache.dim) if scale is None else scale, window)
    off = (out.double() - want).abs()
    assert out.isfinite().all()
    assert (off <= tol + 1e-37).all(), f"out off by {(off / (tol + 1e-37)).max():.3f} of its tolerance"
    empty = wl == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    off = (lse.double() - wl)[~empty].abs()
    assert (off <= ltol[~empty]).all(), f"lse off by {(off / ltol[~empty]).max():.3f} of its tolerance"
    return out, lse


LENGTHS = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 100, 1000, 0, 515]


# -- attend ---------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, E4, F32])
@pytest.mark.parametrize("heads,kv,dim,page", [
    (8, 2, 64, 16), (5, 1, 128, 100), (16, 16, 80, 32), (32, 2, 96, 8), (40, 2, 128, 1),
    (17, 1, 256, 48), (3, 3, 16, 3), (34, 2, 192, 64), (8, 8, 144, 7)])
def test_attend(dtype, heads, kv, dim, page):
    g = gen(heads * dim + page)
    table, pages = make_table(g, LENGTHS, page)
    cache = make_pool(g, pages, kv, page, dim, dtype)
    q = (2 * torch.randn((len(LENGTHS), heads, dim), generator=g, device="cuda")).to(
        F32 if dtype == F32 else BF)
    check(cache, q, table, LENGTHS)
    # a table with room for longer sequences: the work is divided another way
    wide = torch.full((len(LENGTHS), -(-9000 // page)), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    check(cache, q, wide, LENGTHS)


@pytest.mark.parametrize("dtype", [BF, E4, F32])
@pytest.mark.parametrize("dim", [32, 64, 128, 256])
@pytest.mark.parametrize("group", [1, 4, 5, 8, 9, 16, 33])
def test_attend_every_variant(dtype, dim, group):
    """Each width the kernels are built for, with few and many heads to a cached
    one, divided one tile to a warp and many."""
    g = gen(dim + group)
    for lengths in ([5, 0, 200, 31], [3000, 2900, 1, 700] * 4):
        table, pages = make_table(g, lengths, 16)
        cache = make_pool(g, pages, 2, 16, dim, dtype)
        q = torch.randn((len(lengths), 2 * group, dim), generator=g, device="cuda").to(
            F32 if dtype == F32 else BF)
        check(cache, q, table, lengths)


@pytest.mark.parametrize("dtype", [BF, E4, F32])
@pytest.mark.parametrize("window", [1, 7, 16, 100, 999, 1000, 5000])
def test_attend_window(dtype, window):
    """Pages wholly before the window are gone (-1) and not looked at."""
    g = gen(window)
    page = 24
    first = [max(0, n - window) // page if n else 0 for n in LENGTHS]
    table, pages = make_table(g, LENGTHS, page, first=first)
    cache = make_pool(g, pages, 2, page, 64, dtype)
    q = torch.randn((len(LENGTHS), 6, 64), generator=g, device="cuda").to(F32 if dtype == F32 else BF)
    errors = torch.zeros(1, dtype=torch.int32, device="cuda")
    check(cache, q, table, LENGTHS, window=window, errors=errors)
    assert errors.item() == 0


@pytest.mark.parametrize("dtype", [BF, E4, F32])
@pytest.mark.parametrize("batch,length,window", [(1, 131072, 0), (1, 4096, 0), (3, 20011, 0),
                                                 (1, 300, 0), (2, 131072, 4096)])
def test_attend_long(dtype, batch, length, window):
    """Few sequences: parts of every kind are joined, inside CTAs and across them."""
    g = gen(length + batch)
    lengths = [max(1, length - 37 * b) for b in range(batch)]
    page, dim = 64, 128
    table, pages = make_table(g, lengths, page)
    cache = make_pool(g, pages, 2, page, dim, dtype)
    q = (3 * torch.randn((batch, 8, dim), generator=g, device="cuda")).to(F32 if dtype == F32 else BF)
    check(cache, q, table, lengths, window=window)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_ragged_batches(dtype):
    """One long sequence among short ones, and more sequences than threads."""
    g = gen(3)
    for lengths in ([9000] + [3] * 40, [1] * 700 + [0] * 1200 + [40] * 300,
                    [5, 0, 0, 0, 3000, 0, 0]):
        table, pages = make_table(g, lengths, 32)
        cache = make_pool(g, pages, 2, 32, 64, dtype)
        q = torch.randn((len(lengths), 4, 64), generator=g, device="cuda").to(dtype)
        check(cache, q, table, lengths)


@pytest.mark.parametrize("dtype", [BF, E4, F32])
@pytest.mark.parametrize("layout", ["tokens", "both"])
def test_attend_layouts_and_strided_queries(dtype, layout):
    g = gen(11)
    table, pages = make_table(g, LENGTHS, 20)
    cache = make_pool(g, pages, 4, 20, 64, dtype, layout=layout)
    qkv = torch.randn((len(LENGTHS), 16, 64), generator=g, device="cuda").to(F32 if dtype == F32 else BF)
    wide = torch.full((len(LENGTHS), table.shape[1] + 5), -7, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    check(cache, qkv[:, 4:12], wide[:, :table.shape[1]], LENGTHS)


@pytest.mark.parametrize("dtype", [BF, E4, F32])
@pytest.mark.parametrize("junk", [float("nan"), float("inf"), None])
def test_attend_ignores_what_is_not_visible(dtype, junk):
    """NaN, infinity or the type's lowest value everywhere but at visible tokens."""
    if dtype == E4 and junk == float("inf"):
        junk = float("nan")  # the type has no infinity
    low = torch.finfo(dtype).min if junk is None else junk
    g = gen(5)
    page, window = 24, 50
    table, pages = make_table(g, LENGTHS, page)
    clean = make_pool(g, pages, 2, page, 96, dtype)
    dirty = make_pool(g, pages, 2, page, 96, dtype, fill=low)
    from sparse_weight_memory_b200 import KVCache
    cache = KVCache(keys=dirty.keys, values=dirty.values, key_scale=clean._scales[0],
                    value_scale=clean._scales[1])
    for b, n in enumerate(LENGTHS):
        t = torch.arange(max(0, n - window), n, device="cuda")
        pg, row = table[b][t // page].long(), t % page
        for x, y in ((cache.keys, clean.keys), (cache.values, clean.values)):
            if dtype == E4:
                x, y = x.view(torch.uint8), y.view(torch.uint8)
            x[pg, :, row] = y[pg, :, row]
    q = torch.randn((len(LENGTHS), 4, 96), generator=g, device="cuda").to(F32 if dtype == F32 else BF)
    got = (torch.empty_like(q), torch.empty(q.shape[:2], device="cuda"))
    cache.attend(q, table, as_int32(LENGTHS), window=window, out=got[0], lse=got[1])
    check(clean, q, table, LENGTHS, window=window, got=got)


@pytest.mark.parametrize("dtype", [BF, E4, F32])
def test_attend_peaked_scores(dtype):
    """One token with nearly all the weight, first, last or in the middle; scales 0 and < 0."""
    g = gen(8)
    lengths = [700, 701, 702]
    table, pages = make_table(g, lengths, 16)
    cache = make_pool(g, pages, 1, 16, 64, dtype)
    q = torch.randn((3, 2, 64), generator=g, device="cuda").to(F32 if dtype == F32 else BF)
    for b, t in enumerate([0, 350, 701]):
        at = table[b][t // 16].long(), 0, t % 16
        row = (12 * q[b, 0]).float()
        if dtype == E4:
            cache.keys.view(torch.uint8)[at] = (row / cache._scales[0][0]).clamp(-448, 448).to(E4).view(torch.uint8)
        else:
            cache.keys[at] = row.to(dtype)
    for scale in (None, 1.0, 0.0, -0.3):
        check(cache, q, table, lengths, scale=scale)


@pytest.mark.parametrize("dtype", [BF, E4, F32])
def test_attend_keeps_a_bad_score_to_its_head(dtype):
    """A NaN among the visible keys or values reaches its sequence's head (its
    element) and nothing else, bit for bit; a head whose scores are all -infinity
    has none to weigh."""
    g = gen(14)
    lengths = [5000, 1, 0, 700, 9000, 33]
    table, pages = make_table(g, lengths, 32)
    cache = make_pool(g, pages, 2, 32, 128, dtype)
    q = torch.randn((6, 8, 128), generator=g, device="cuda").to(F32 if dtype == F32 else BF)
    q[5, :, 0] = 1
    lens = as_int32(lengths)

    def attend():
        lse = torch.empty((6, 8), device="cuda")
        return cache.attend(q, table, lens, lse=lse), lse

    def put(pool, b, t, h, e, x):  # element by element: fp8 has no indexed fill
        row = pool[table[b][t // 32].item(), h, t % 32]
        row[e:e + 1].copy_(torch.tensor([x], device="cuda").to(dtype))

    want, want_lse = attend()
    put(cache.keys, 3, 111, 1, 7, math.nan)
    put(cache.values, 4, 8000, 0, 5, math.nan)
    rest = torch.ones((6, 8, 128), dtype=torch.bool, device="cuda")
    rest[3, 4:] = False
    rest[4, :4, 5] = False
    out, lse = attend()
    assert torch.equal(out[rest], want[rest]) and out[~rest].isnan().all()
    keep = torch.ones((6, 8), dtype=torch.bool, device="cuda")
    keep[3, 4:] = False
    assert torch.equal(lse[keep], want_lse[keep]) and lse[~keep].isnan().all()
    if dtype == E4:
        return  # the type has no infinity
    for t in range(33):
        put(cache.keys, 5, t, 1, 0, -math.inf)
    rest[5, 4:] = False
    out, lse = attend()
    assert torch.equal(out[rest], want[rest])
    assert (out[5, 4:] == 0).all() and (lse[5, 4:] == -math.inf).all()


def test_attend_tiny_and_huge_queries():
    """8-bit caches scale a row of queries by a power of two: rows of very
    different size, of zeros, and of one large element beside small ones."""
    g = gen(9)
    lengths = [100] * 5
    table, pages = make_table(g, lengths, 16)
    cache = make_pool(g, pages, 1, 16, 64, E4)
    q = torch.randn((5, 4, 64), generator=g, device="cuda")
    q[0] *= 1e-30
    q[1] *= 1e4
    q[2] = 0
    q[3, :, 0] = 3e4
    q[4] *= 1e-5
    check(cache, q.to(BF), table, lengths)
    check(cache, q.to(BF), table, lengths, scale=1e-4)


def test_attend_bad_pages_and_lengths():
    """Entries that are no page, and lengths beyond the table or negative: what
    is left is right, and the bits say what was met."""
    from sparse_weight_memory_b200.cache import BAD_LENGTH, BAD_PAGE
    g = gen(13)
    lengths = [100, 64, 33, 200, 16]
    table, pages = make_table(g, lengths, 16)
    cache = make_pool(g, pages, 2, 16, 64, BF)
    q = torch.randn((5, 4, 64), generator=g, device="cuda").to(BF)
    errors = torch.zeros(1, dtype=torch.int32, device="cuda")
    check(cache, q, table, lengths, errors=errors)
    assert errors.item() == 0
    table[0, 2], table[1, :], table[3, 12] = pages, -1, 2**31 - 1
    check(cache, q, table, lengths, errors=errors)
    assert errors.item() == BAD_PAGE
    errors.zero_()
    out = cache.attend(q, table[:, :5].contiguous(), as_int32([-3, 0, 33, 200, 80]), errors=errors)
    assert errors.item() == BAD_LENGTH | BAD_PAGE  # row 4's pages 1 .. 4 are -1
    want, tol, _, _ = reference(cache, q, table[:, :5], [0, 0, 33, 80, 80], 1 / 8, 0)
    assert ((out.double() - want).abs() <= tol + 1e-37).all()


def test_attend_beyond_32_bit_offsets():
    """A pool of more than 2^32 elements, with the sequence's pages at its end."""
    from sparse_weight_memory_b200 import KVCache
    kv, page, dim = 8, 64, 256
    pages = 2**32 // (kv * page * dim) + 40
    keys = torch.zeros((pages, kv, page, dim), dtype=E4, device="cuda")
    values = torch.zeros_like(keys)
    g = gen(2)
    for x in (keys, values):
        x[-32:] = torch.randn((32, kv, page, dim), generator=g, device="cuda").to(E4)
    n = 1000
    rows = [pages - 1 - i for i in range(16)]
    small = KVCache(keys=keys[-32:].clone(), values=values[-32:].clone())
    q = torch.randn((1, 16, dim), generator=g, device="cuda").to(BF)
    lse = torch.empty((1, 16), device="cuda")
    cache = KVCache(keys=keys, values=values)
    out = cache.attend(q, as_int32([rows]), as_int32([n]), lse=lse)
    check(small, q, as_int32([[r - (pages - 32) for r in rows]]), [n], got=(out, lse))
    # and a write there
    k = torch.randn((1, kv, dim), generator=g, device="cuda").to(BF)
    cache.append(k, k, as_int32([rows]), as_int32([n]))
    at = (rows[(n - 1) // page], slice(None), (n - 1) % page)
    assert torch.equal(cache.keys[at].float(), k[0].float().to(E4).float())
    assert torch.equal(cache.values[at].float(), k[0].float().to(E4).float())


def test_attend_equal_bits_and_streams():
    """The same call twice, on another stream, two at once, and replayed."""
    g = gen(21)
    lengths = [5000, 1, 0, 700, 9000, 33]
    table, pages = make_table(g, lengths, 32)
    cache = make_pool(g, pages, 2, 32, 128, BF)
    qs = [torch.randn((6, 8, 128), generator=g, device="cuda").to(BF) for _ in range(2)]
    lens = as_int32(lengths)
    want = [cache.attend(q, table, lens) for q in qs]
    check(cache, qs[0], table, lengths)
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [cache.attend(q, table, lens, stream=s) for q, s in zip(qs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    # a workspace of the caller's, whatever it holds
    size = cache.attend_workspace(6, 8)
    for fill in (0, 255):
        own = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        for _ in range(2):
            assert torch.equal(cache.attend(qs[0], table, lens, workspace=own), want[0])
    # a captured call follows new lengths, tables and queries
    graphs, outs = [], []
    q = qs[0].clone()
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(cache.attend(q, table, lens))
        graphs.append(graph)
    q.copy_(qs[1])
    lens.copy_(as_int32([4999, 0, 0, 1, 8192, 2]))
    for gr, s in zip(graphs, streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            gr.replay()
    torch.cuda.synchronize()
    for out in outs:
        assert torch.equal(out, cache.attend(q, table, lens))


def test_attend_e4m3_weights():
    """8-bit caches: weights in the products with the values are as good as their sum.
    Few tokens of opposite values leave outputs far smaller than their terms,
    whose weights' rounding then shows."""
    from sparse_weight_memory_b200 import KVCache
    g = gen(35)
    B, page, kv, heads, dim = 600, 16, 1, 8, 64
    keys = torch.zeros((B, kv, page, dim), device="cuda")
    keys[..., 0] = torch.randn((B, kv, page), generator=g, device="cuda").clamp(-2, 2)
    values = torch.randn((B, kv, page, dim), generator=g, device="cuda")
    cache = KVCache(keys=keys.to(E4), values=values.to(E4))
    q = torch.zeros((B, heads, dim), device="cuda")
    q[..., 0] = torch.rand((B, heads), generator=g, device="cuda") + 0.1
    q = q.to(BF)
    n = torch.arange(B, device="cuda", dtype=torch.int32) % 3 + 2
    table = torch.arange(B, device="cuda", dtype=torch.int32)[:, None]
    out = cache.attend(q, table, n, scale=0.5)
    s = 0.5 * q.double()[:, :, :1] * cache.keys.double()[:, 0, None, :, 0]
    s = s.masked_fill(torch.arange(page, device="cuda") >= n[:, None, None], -math.inf)
    p, v = torch.softmax(s, -1), cache.values.double()[:, 0]
    want, size = p @ v, p @ v.abs()
    # half a step of the output; a score is one product, |s| <= 1.1, and its factor off
    # by 2^-22; the exponent of up to 16 is rounded once, 2^-21; exp2 2^-22; these
    # three twice; the two parts of a weight 2^-22; the sums of up to 4 terms,
    # their join and the last factor 8 roundings
    share = 2 * (2.0 ** -22 + 2.0 ** -21 + 2.0 ** -22) + 2.0 ** -22 + 8 * 2.0 ** -23
    off = (out.double() - want).abs()
    tol = 2.0 ** -8 * want.abs() + share * size
    assert (off <= tol).all(), f"off by {(off / tol).max():.2f} of the tolerance"


@pytest.mark.parametrize("which", ["key_scale", "value_scale"])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_attend_bad_scale(which, bad):
    """A cached head whose scale is no number gives no number for its query heads, in
    sequences that are finished by a warp, joined in a CTA and joined across them,
    and leaves the other heads their bits; a sequence without tokens has nothing
    to scale."""
    from sparse_weight_memory_b200 import KVCache
    g = gen(31)
    lengths = [9000, 1, 0, 700, 40]
    table, pages = make_table(g, lengths, 32)
    cache = make_pool(g, pages, 2, 32, 64, E4)
    q = torch.randn((5, 6, 64), generator=g, device="cuda").to(BF)
    scales = {"key_scale": cache._scales[0], "value_scale": cache._scales[1]}
    scales[which] = scales[which].clone()
    scales[which][1] = bad
    broken = KVCache(keys=cache.keys, values=cache.values, **scales)
    lse, want_lse = (torch.empty((5, 6), device="cuda") for _ in range(2))
    want = cache.attend(q, table, as_int32(lengths), lse=want_lse)
    out = broken.attend(q, table, as_int32(lengths), lse=lse)
    live = [0, 1, 3, 4]
    assert torch.equal(out[:, :3], want[:, :3]) and torch.equal(lse[:, :3], want_lse[:, :3])
    assert not out[live, 3:].isfinite().any()
    assert (out[2] == 0).all() and (lse[2] == -math.inf).all()
    if which == "key_scale":
        assert out[live, 3:].isnan().all() and lse[live, 3:].isnan().all()
    else:
        assert torch.equal(lse, want_lse)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [2e-38, -2e-39, 1e-41])
def test_attend_tiny_scale(dtype, scale):
    """Scales below the smallest normal number, with products large enough to feel them."""
    from sparse_weight_memory_b200 import KVCache
    g = gen(32)
    keys = torch.zeros((4, 1, 16, 64), device="cuda")
    keys[..., 0] = 2e19 * torch.rand((4, 1, 16), generator=g, device="cuda")
    values = torch.randn((4, 1, 16, 64), generator=g, device="cuda")
    cache = KVCache(keys=keys.to(dtype), values=values.to(dtype))
    q = torch.zeros((1, 2, 64), device="cuda", dtype=dtype)
    q[:, :, 0] = 8e18
    check(cache, q, as_int32([[0, 1, 2, 3]]), [64], scale=scale)


def test_attend_rows_without_a_normal_exponent():
    """8-bit caches: rows of queries with an infinity, beside elements beyond the 16-bit
    range, and rows of denormal numbers only."""
    from sparse_weight_memory_b200 import KVCache
    g = gen(33)
    keys = torch.rand((4, 1, 16, 64), generator=g, device="cuda") + 0.5
    values = torch.randn((4, 1, 16, 64), generator=g, device="cuda")
    one = torch.full((1,), 0.5, device="cuda")
    cache = KVCache(keys=keys.to(E4), values=values.to(E4), key_scale=one, value_scale=one)
    table, lens = as_int32([[0, 1, 2, 3]] * 2), as_int32([64, 64])
    q = torch.zeros((2, 2, 64), device="cuda")
    q[:, :, 1] = 1e6
    q[:, 1] = torch.randn(64, generator=g, device="cuda")
    q[:, 0, 0] = -math.inf
    lse = torch.empty((2, 2), device="cuda")
    out = cache.attend(q.to(BF), table, lens, lse=lse)
    assert (out[:, 0] == 0).all() and (lse[:, 0] == -math.inf).all()
    check(cache, q.to(BF)[:, 1:].contiguous(), table, [64, 64])
    q = torch.randn((2, 2, 64), generator=g, device="cuda") * 2.0 ** -128
    check(cache, q.to(BF), table, [64, 64], scale=1e38)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("batch,length", [(1500, 64), (3, 2000)])
def test_attend_large_values(dtype, batch, length):
    """Values whose sum over the tokens is still within 32 bits: weights are at most 1,
    also where scores rise by less than what scales the sums anew (here by a
    factor 2^5.9)."""
    from sparse_weight_memory_b200 import KVCache
    page = 32
    pages = -(-length // page)
    keys = torch.zeros((pages, 2, page, 64), device="cuda")
    keys[1:, ..., 0] = 4.09375
    values = torch.full_like(keys, 2e38 / length)
    values[..., 1::2] *= -1
    cache = KVCache(keys=keys.to(dtype), values=values.to(dtype))
    q = torch.zeros((batch, 2, 64), device="cuda", dtype=dtype)
    q[:, :, 0] = 1
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(batch, 1)
    check(cache, q, table, [length] * batch, scale=1.0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_attend_without_weights(dtype, value):
    """A head whose visible scores are all -infinity gives 0 whatever its values are."""
    g = gen(34)
    lengths = [9000, 1, 700, 40]
    table, pages = make_table(g, lengths, 32)
    cache = make_pool(g, pages, 2, 32, 64, dtype)
    cache.keys[:, 1, :, 0] = -math.inf
    cache.values[:, 1, :, 3] = value
    q = torch.randn((4, 6, 64), generator=g, device="cuda").to(dtype)
    q[:, :, 0] = 1
    lse = torch.empty((4, 6), device="cuda")
    for width in (2, table.shape[1]):  # short contexts are divided another way
        n = [min(m, 32 * width) for m in lengths]
        out = cache.attend(q, table[:, :width].contiguous(), as_int32(n), lse=lse)
        assert (out[:, 3:] == 0).all() and (lse[:, 3:] == -math.inf).all()
        assert out[:, :3].isfinite().all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_infinite_value(dtype):
    """An infinite visible value leaves its element not finite, and the others their bits."""
    g = gen(40)
    lengths = [9000, 1, 700, 40]
    table, pages = make_table(g, lengths, 32)
    cache = make_pool(g, pages, 2, 32, 64, dtype)
    q = torch.randn((4, 6, 64), generator=g, device="cuda").to(dtype)
    lens = as_int32(lengths)
    lse, want_lse = (torch.empty((4, 6), device="cuda") for _ in range(2))
    want = cache.attend(q, table, lens, lse=want_lse)
    rest = torch.ones((4, 6, 64), dtype=torch.bool, device="cuda")
    for b, t, h, e in ((0, 8000, 0, 5), (1, 0, 1, 63), (2, 3, 1, 0), (3, 39, 0, 17)):
        cache.values[table[b, t // 32].long(), h, t % 32, e] = math.inf
        rest[b, 3 * h:3 * h + 3, e] = False
    out = cache.attend(q, table, lens, lse=lse)
    assert not out[~rest].isfinite().any()
    assert torch.equal(out[rest], want[rest]) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("dtype", [BF, E4, F32])
def test_attend_more_sequences_than_threads_joined(dtype):
    """Several sequences to a thread, and parts of long ones joined across CTAs."""
    g = gen(38)
    lengths = [1] * 700 + [0] * 1200 + [40] * 298 + [9000, 3]
    table, pages = make_table(g, lengths, 32)
    cache = make_pool(g, pages, 2, 32, 64, dtype)
    q = torch.randn((len(lengths), 4, 64), generator=g, device="cuda").to(F32 if dtype == F32 else BF)
    check(cache, q, table, lengths)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_infinite_score(dtype):
    """A +infinity among a head's scores makes that sequence's head NaN and no other,
    where a warp finishes it and where parts are joined in a CTA or across them."""
    from sparse_weight_memory_b200 import KVCache
    g = gen(39)
    lengths = [9000, 33, 700, 1, 6000]
    table, pages = make_table(g, lengths, 32)
    cache = make_pool(g, pages, 2, 32, 64, dtype)
    q = torch.randn((5, 8, 64), generator=g, device="cuda").to(dtype)
    sign = torch.tensor([1, -1, 0] * 3, device="cuda")[:8]  # of each head's element 0
    q[..., 0] = sign.to(dtype)
    places = ((0, 4321, 0), (1, 32, 1), (2, 0, 0), (2, 699, 1), (3, 0, 1))
    near = cache.keys.clone()  # with a score of no weight (-250) for the heads of sign -1
    bad = torch.zeros((5, 8), dtype=torch.bool, device="cuda")
    for b, t, h in places:
        at = (table[b, t // 32].long(), h, t % 32, 0)
        cache.keys[at], near[at] = math.inf, 2000
        bad[b, 4 * h:4 * h + 4] = sign[4 * h:4 * h + 4] >= 0  # infinity, or 0 times infinity
    lse = torch.empty((5, 8), device="cuda")
    out = cache.attend(q, table, as_int32(lengths), lse=lse)
    assert out[bad].isnan().all() and lse[bad].isnan().all()
    none = torch.zeros_like(bad)  # the only token's score is -infinity
    none[3, 4:] = sign[4:] < 0
    assert (out[none] == 0).all() and (lse[none] == -math.inf).all()
    want, tol, wl, ltol = reference(KVCache(keys=near, values=cache.values), q, table, lengths, 1 / 8, 0)
    rest = ~bad & ~none
    assert ((out.double() - want).abs() <= tol + 1e-37)[rest].all()
    assert ((lse.double() - wl).abs() <= ltol)[rest].all()


@pytest.mark.parametrize("dtype,batch,width", [(BF, 2 ** 22, 1), (F32, 2 ** 20 + 3, 1), (E4, 300001, 400)])
def test_attend_largest_batches(dtype, batch, width):
    """Up to 2^22 sequences of 0 to 3 tokens, whole segments to a CTA or divided."""
    from sparse_weight_memory_b200 import KVCache
    g = gen(43)
    page, dim = 4, 16
    keys, values = (torch.randn((batch, 1, page, dim), generator=g, device="cuda").to(dtype)
                    for _ in range(2))
    cache = KVCache(keys=keys, values=values)
    q = torch.randn((batch, 1, dim), generator=g, device="cuda").to(F32 if dtype == F32 else BF)
    lengths = torch.randint(0, 4, (batch,), generator=g, device="cuda", dtype=torch.int32)
    order = torch.randperm(batch, generator=g, device="cuda").int()
    table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
    table[:, 0] = order
    lse = torch.empty((batch, 1), device="cuda")
    out = cache.attend(q, table, lengths, lse=lse)
    raw = (lambda x: x.view(torch.uint8)) if dtype == E4 else (lambda x: x)
    k, v = (raw(x)[order.long(), 0].view(dtype).double() for x in (keys, values))
    s = (k @ q.double().transpose(1, 2))[..., 0] / 4
    size = (k.abs() @ q.double().abs().transpose(1, 2))[..., 0] / 4
    seen = torch.arange(page, device="cuda") < lengths[:, None]
    s = s.masked_fill(~seen, -math.inf)
    p = torch.softmax(s, -1).nan_to_num(0.0)
    want, terms = (p[:, None] @ v)[:, 0], (p[:, None] @ v.abs())[:, 0]
    # as in `reference`, for at most 3 tokens
    ds = size.masked_fill(~seen, 0.0).amax(-1) * (dim + 16) * 2.0 ** -23
    if dtype == E4:
        ds += q.double().abs().amax((1, 2)) * k.abs().sum(-1).amax(-1) / 4 * 2.0 ** -25
    pw = {BF: 2.0 ** -16, E4: 2.0 ** -11, F32: 2.0 ** -22}[dtype]
    share = 2 * (ds + 2.0 ** -22) + pw + 65 * 2.0 ** -23
    u = 2.0 ** -24 if dtype == F32 else 2.0 ** -8
    assert ((out[:, 0].double() - want).abs() <= u * want.abs() + share[:, None] * terms + 1e-37).all()
    some = lengths > 0
    ls = torch.logsumexp(s[some], -1)
    tol = ds[some] + 2.0 ** -22 + 65 * 2.0 ** -23 + 2.0 ** -21 * (ls.abs() + s[some].amax(-1).abs() + 9)
    assert ((lse[some, 0].double() - ls).abs() <= tol).all()
    assert (lse[~some] == -math.inf).all() and (out[~some] == 0).all()


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("dim,heads", [(64, 8), (128, 8), (128, 16), (256, 8)])
def test_attend_long_sums(dtype, dim, heads):
    """Sums over many tokens are rounded to nearest, not cut: tokens that come twice, with
    values of both signs, leave nothing, and what a cut at each step takes away
    would show.  Each sequence is about a warp's work."""
    from sparse_weight_memory_b200 import KVCache
    g = gen(44)
    batch, n, page = 1500, 25600, 64
    pages = n // page
    keys = torch.randn((pages // 2, 1, page, dim), generator=g, device="cuda") / math.sqrt(dim)
    values = torch.rand((pages // 2, 1, page, dim), generator=g, device="cuda") + 1
    cache = KVCache(keys=torch.cat([keys, keys]).to(dtype), values=torch.cat([values, -values]).to(dtype))
    q = torch.randn((batch, heads, dim), generator=g, device="cuda").to(BF)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(batch, -1)
    out = cache.attend(q, table, torch.full((batch,), n, dtype=torch.int32, device="cuda"), scale=1.0)
    k, v = (x.double().transpose(0, 1).reshape(n, dim)[:n // 2] for x in (cache.keys, cache.values))
    for b in range(0, batch, 100):
        p = torch.softmax(q[b:b + 100].double() @ k.t(), -1)  # of one half
        half = (p @ v) / 2
        # sums rise to `half` and fall again.  n/16 additions rounded to nearest, 2^-24
        # each, add up at random: six times their deviation.  Beside them, all in
        # 2^-24: 16 for the products' sums inside a tile (cut, up to four at a time),
        # 8 for the factors of two joined parts, 8 for exp2 and 2 for the weights' parts
        tol = (6 * math.sqrt(n / 16) / math.sqrt(3) + 34) * 2.0 ** -24 * half
        off = out[b:b + 100].double().abs()
        assert (off <= tol).all(), f"off by {(off / tol).max():.1f} of the tolerance"


# -- append ---------------------------------------------------------------------

def rotated(x, pos, freqs, style):
    """x [rows, heads, dim] turned in 64 bits, and the size of each element's pair."""
    x = x.double().clone()
    size = torch.zeros_like(x)
    if freqs is None:
        return x, size
    n = freqs.numel()
    one, two = ((slice(0, n), slice(n, 2 * n)) if style == "halves"
                else (slice(0, 2 * n, 2), slice(1, 2 * n, 2)))
    angle = pos.double()[:, None, None] * freqs.double()
    a, b = x[..., one].clone(), x[..., two].clone()
    size[..., one] = size[..., two] = torch.hypot(a, b)
    x[..., one] = a * angle.cos() - b * angle.sin()
    x[..., two] = b * angle.cos() + a * angle.sin()
    return x, size


def close(got, want, size, dtype, far=0):
    """Half a step of the type (of its smallest step, below the normal numbers), and
    of the pair's size 2^-21: cos, sin and their products in 32 bits.  Positions up
    to `far` add 4 roundings of the angle in 64 bits (far 2^-53 each; two or three
    in the kernel, one here)."""
    u = torch.finfo(dtype).eps / 2
    small = {E4: 2.0 ** -10, BF: 0.0, F32: 0.0}[dtype]
    off = (got.float().double() - want).abs()
    tol = torch.maximum(u * want.abs(), torch.tensor(small, dtype=torch.float64, device="cuda"))
    assert (off <= tol + (2.0 ** -21 + far * 2.0 ** -51) * size * (1 + u)).all(), (off - tol).max().item()


@pytest.mark.parametrize("inputs,dtype", [(BF, BF), (BF, E4), (BF, F32), (F32, F32), (F32, BF),
                                          (F32, E4)])
@pytest.mark.parametrize("heads,kv,dim,page,rotary,style,layout", [
    (8, 2, 128, 16, 128, "halves", "heads"), (5, 1, 64, 1, 32, "halves", "tokens"),
    (16, 16, 80, 100, 80, "pairs", "heads"), (40, 8, 96, 48, 16, "pairs", "both"),
    (0, 2, 256, 64, 256, "halves", "heads"), (3, 3, 16, 7, 0, "halves", "heads"),
    (64, 8, 192, 32, 96, "pairs", "tokens")])
def test_append(inputs, dtype, heads, kv, dim, page, rotary, style, layout):
    g = gen(heads + dim + page)
    new = [3, 0, 1, 40, 0, 17, 1, 200]
    lengths = [3, 50, 100, 4000, 0, 17, 1, 131072]
    first = [(n - m) // page for n, m in zip(lengths, new)]
    table, pages = make_table(g, lengths, page, first=first)
    cache = make_pool(g, pages, kv, page, dim, dtype, layout=layout)
    before = [cache.keys.float().clone(), cache.values.float().clone()]
    starts = as_int32([sum(new[:b]) for b in range(len(new) + 1)])
    rows = sum(new)
    padded = rows + 9  # rows behind the last sequence
    qkv = torch.randn((padded, heads + 2 * kv, dim), generator=g, device="cuda").to(inputs)
    q, k, v = qkv.split([heads, kv, kv], 1)
    freqs = (10000.0 ** (-torch.arange(rotary // 2, dtype=torch.float64, device="cuda")
                         / max(1, rotary // 2))).float() if rotary else None
    q_out = torch.full((padded, heads, dim), 7.0, dtype=inputs, device="cuda") if heads else None
    errors = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = cache.append(k, v, table, as_int32(lengths), starts=starts, q=q if heads else None,
                       freqs=freqs, style=style, q_out=q_out, errors=errors)
    assert errors.item() == 0
    seq = torch.tensor([b for b, m in enumerate(new) for _ in range(m)], device="cuda")
    pos = torch.tensor([n - m + i for n, m in zip(lengths, new) for i in range(m)], device="cuda")
    if heads:
        want, size = rotated(q[:rows], pos, freqs, style)
        close(got[:rows], want, size, inputs)
        assert (got[rows:] == 7).all()
    else:
        assert got is None
    pg, row = table[seq, pos // page].long(), pos % page
    want, size = rotated(k[:rows], pos, freqs, style)
    exact = v[:rows].float()
    if dtype == E4:
        ks, vs = (s.double()[None, :, None] for s in cache._scales)
        want, size = (want / ks).clamp(-448, 448), size / ks
        exact = (exact / cache._scales[1][None, :, None]).clamp(-448, 448)
    kf, vf = cache.keys.float().clone(), cache.values.float().clone()
    close(kf[pg, :, row].to(dtype), want, size, dtype)
    assert torch.equal(vf[pg, :, row], exact.to(dtype).float())
    for x, y in zip((kf, vf), before):  # the rest of the pool is as it was
        x[pg, :, row] = 0
        y[pg, :, row] = 0
        assert torch.equal(x, y)


@pytest.mark.parametrize("inputs,dtype", [(BF, BF), (F32, F32)])
@pytest.mark.parametrize("style", ["halves", "pairs"])
@pytest.mark.parametrize("dim,rotary", [(8, 0), (24, 16), (40, 16), (72, 64), (200, 112), (248, 48)])
def test_append_odd_widths(inputs, dtype, style, dim, rotary):
    """Heads of an odd number of 8-element groups, in part rotated, few rows and many."""
    g = gen(dim)
    heads, kv, page = 13, 2, 50
    freqs = torch.rand(rotary // 2, generator=g, device="cuda") if rotary else None
    for rows in (5, 2500):
        cache = make_pool(g, 51, kv, page, dim, dtype)
        table = torch.randperm(51, generator=g, device="cuda").int()[None]
        qkv = torch.randn((rows, heads + 2 * kv, dim), generator=g, device="cuda").to(inputs)
        q, k, v = qkv.split([heads, kv, kv], 1)
        got = cache.append(k, v, table, as_int32([rows + 40]), starts=as_int32([0, rows]), q=q,
                           freqs=freqs, style=style)
        pos = torch.arange(40, rows + 40, device="cuda")
        want, size = rotated(q, pos, freqs, style)
        close(got, want, size, inputs)
        pg, row = table[0][pos // page].long(), pos % page
        want, size = rotated(k, pos, freqs, style)
        close(cache.keys[pg, :, row], want, size, dtype)
        assert torch.equal(cache.values[pg, :, row], v.to(dtype))


@pytest.mark.parametrize("inputs,dtype", [(BF, BF), (BF, E4), (F32, F32)])
@pytest.mark.parametrize("style", ["halves", "pairs"])
def test_append_one_token_in_place(inputs, dtype, style):
    """One row a sequence, empty places in a padded batch, queries turned in place."""
    g = gen(4)
    lengths = [1, 0, 64, 65, 0, 131071, 131072]
    page, kv, heads, dim = 64, 2, 4, 64
    first = [max(0, n - 1) // page for n in lengths]
    table, pages = make_table(g, lengths, page, first=first)
    cache = make_pool(g, pages, kv, page, dim, dtype)
    before = cache.keys.float().clone()
    qkv = torch.randn((len(lengths), heads + 2 * kv, dim), generator=g, device="cuda").to(inputs)
    old = qkv.clone()
    q, k, v = qkv.split([heads, kv, kv], 1)
    freqs = torch.rand(dim // 2, generator=g, device="cuda")
    assert cache.append(k, v, table, as_int32(lengths), q=q, freqs=freqs, style=style, q_out=q) is q
    live = torch.tensor([b for b, n in enumerate(lengths) if n], device="cuda")
    dead = torch.tensor([b for b, n in enumerate(lengths) if not n], device="cuda")
    pos = torch.tensor([n - 1 for n in lengths if n], device="cuda")
    want, size = rotated(old[live, :heads], pos, freqs, style)
    close(q[live], want, size, inputs)
    assert torch.equal(qkv[dead], old[dead]) and torch.equal(qkv[:, heads:], old[:, heads:])
    pg, row = table[live, pos // page].long(), pos % page
    assert len(set(zip(pg.tolist(), row.tolist()))) == len(live)
    changed = (cache.keys.float() != before).any(-1).any(1)  # [pages, page]
    expect = torch.zeros_like(changed)
    expect[pg, row] = True
    assert torch.equal(changed, expect)


def test_append_far_positions():
    """Positions near 2^31 with a frequency of 1 radian a token: the angle needs 64 bits."""
    from sparse_weight_memory_b200 import KVCache
    top = 2**31 - 1
    page = 2**29
    cache = KVCache(keys=torch.zeros((1, 1, 1, 16), device="cuda").expand(5, 1, page, 16),
                    values=torch.zeros((1, 1, 1, 16), device="cuda").expand(5, 1, page, 16))
    q = torch.randn((3, 2, 16), generator=gen(1), device="cuda")
    kv = torch.zeros((3, 1, 16), device="cuda")
    freqs = torch.tensor([1.0, 0.7, 3e-5, 0.1, 0.9, 0.99999, 1e-9, 0.5], device="cuda")
    lengths = [top, 2**30 + 1, 12345678]
    got = cache.append(kv, kv, as_int32([[0, 1, 2, 3]] * 3), as_int32(lengths), q=q, freqs=freqs)
    want, size = rotated(q, torch.tensor(lengths, device="cuda") - 1, freqs, "halves")
    close(got, want, size, F32, far=top)


def test_append_bad_places():
    """Rows without a valid place are not stored, and the bits say why."""
    from sparse_weight_memory_b200.cache import BAD_LENGTH, BAD_PAGE
    g = gen(6)
    cache = make_pool(g, 6, 2, 8, 64, BF)
    k = torch.randn((4, 2, 64), generator=g, device="cuda").to(BF)
    table = as_int32([[0, 1], [2, 3], [4, 6], [5, -1]])

    def run(lengths, starts=None, t=table):
        before = (cache.keys.clone(), cache.values.clone())
        errors = torch.zeros(1, dtype=torch.int32, device="cuda")
        cache.append(k, k, t, as_int32(lengths), errors=errors,
                     starts=None if starts is None else as_int32(starts))
        wrote = (cache.keys != before[0]).any(-1).any(1).nonzero().tolist()
        wrote_v = (cache.values != before[1]).any(-1).any(1).nonzero().tolist()
        assert wrote == wrote_v
        cache.keys.copy_(before[0])
        cache.values.copy_(before[1])
        return errors.item(), wrote

    assert run([1, 2, 3, 4]) == (0, [[0, 0], [2, 1], [4, 2], [5, 3]])
    assert run([1, 2, 9, 9]) == (BAD_PAGE, [[0, 0], [2, 1]])       # pages 6 and -1
    assert run([17, 2, -1, 4]) == (BAD_LENGTH, [[2, 1], [5, 3]])   # beyond the table; negative
    assert run([1, 2, 3, 4], starts=[0, 1, 2, 2, 4]) == (0, [[0, 0], [2, 1], [5, 2], [5, 3]])
    assert run([1, 1, 3, 4], starts=[0, 1, 4, 4, 4]) == (BAD_LENGTH, [[0, 0]])  # 3 rows, 1 token
    assert run([1, 2, 3, 4], starts=[0, 0, 0, 0, 0]) == (0, [])


def test_append_many_sequences():
    """The search for a row's sequence: thousands of sequences, many of them empty."""
    g = gen(7)
    new = [0 if b % 3 else 1 + b % 4 for b in range(5000)]
    lengths = [m + b % 5 for b, m in enumerate(new)]
    page = 8
    table, pages = make_table(g, lengths, page)
    cache = make_pool(g, pages, 1, page, 16, F32)
    rows = sum(new)
    k = torch.randn((rows, 1, 16), generator=g, device="cuda")
    starts = [0]
    for m in new:
        starts.append(starts[-1] + m)
    cache.append(k, 2 * k, table, as_int32(lengths), starts=as_int32(starts))
    seq = torch.tensor([b for b, m in enumerate(new) for _ in range(m)], device="cuda")
    pos = torch.tensor([n - m + i for n, m in zip(lengths, new) for i in range(m)], device="cuda")
    at = table[seq, pos // page].long(), slice(None), pos % page
    assert torch.equal(cache.keys[at], k) and torch.equal(cache.values[at], 2 * k)


@pytest.mark.parametrize("style", ["halves", "pairs"])
@pytest.mark.parametrize("rows", [3, 3000])
def test_append_small_sines(style, rows):
    """cos and sin as accurate as their size, also near multiples of pi: the fraction
    of a turn is not cut to 32 bits before them."""
    from sparse_weight_memory_b200 import KVCache
    g = gen(36)
    cache = KVCache(pages=1, page_size=2 ** 16, kv_heads=1, dim=64, dtype=F32)
    lengths = as_int32([rows + 1000])
    pos = torch.arange(1000, rows + 1000, device="cuda")
    # near a multiple of half a turn, from 2^-20 to 2^-2 turns beside it, at 1001
    turns = torch.arange(1, 33, device="cuda") / 2
    turns = turns + torch.sign(torch.randn(32, generator=g, device="cuda")) * \
        2.0 ** -(2 + 18 * torch.rand(32, generator=g, device="cuda"))
    freqs = (2 * math.pi * turns.double() / 1001).float()
    q = torch.zeros((rows, 1, 64), device="cuda")  # a pair (1, 0) becomes (cos, sin)
    one, two = (slice(0, 32), slice(32, 64)) if style == "halves" else (slice(0, 64, 2), slice(1, 64, 2))
    q[..., one] = 1
    kv = torch.zeros((rows, 1, 64), device="cuda")
    got = cache.append(kv, kv, as_int32([[0]]), lengths, starts=as_int32([0, rows]), q=q,
                       freqs=freqs, style=style)[:, 0].double()
    angle = pos[:, None].double() * freqs.double()
    # the function 2^-23 and the last rounding 2^-24 of the result; the angle four
    # roundings in 64 bits; what 32 bits lose of the correction
    # of up to pi 2^-25: its second order, its factors and products 2^-45
    far = 4 * angle * 2.0 ** -53 + 2.0 ** -45
    for part, want in ((one, angle.cos()), (two, angle.sin())):
        off = (got[:, part] - want).abs()
        assert (off <= (2.0 ** -23 + 2.0 ** -24) * want.abs() + far).all(), (off / want.abs()).max().item()


# -- together -------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, E4, F32])
def test_prompt_then_tokens_beside_the_memory(dtype):
    """As a model runs them: prompts appended, then token by token append, attend
    and a step of the fast-weight memory, in one captured graph for each token;
    against causal attention over the rotated tokens in 64 bits."""
    from sparse_weight_memory_b200 import FwPKMState
    inputs = F32 if dtype == F32 else BF
    g = gen(17)
    B, heads, kv, dim, page, steps = 3, 4, 2, 64, 8, 12
    prompt = [5, 0, 21]
    total = [n + steps for n in prompt]
    table, pages = make_table(g, total, page)
    cache = make_pool(g, pages, kv, page, dim, dtype, fill=0.0)
    freqs = (100.0 ** (-torch.arange(dim // 2, device="cuda") / (dim // 2))).float()
    packed = torch.randn((sum(prompt), heads + 2 * kv, dim), generator=g, device="cuda").to(inputs)
    starts = as_int32([0, 5, 5, 26])
    lengths = as_int32(prompt)
    q, k, v = packed.split([heads, kv, kv], 1)
    cache.append(k, v, table, lengths, starts=starts, freqs=freqs)

    mem = FwPKMState(1024, 64, heads * dim, 4, 1)
    mem.set_tables(torch.randn((1, 2, 32, 32), generator=g, device="cuda"),
                   torch.randn((1024, heads * dim), generator=g, device="cuda"))
    gate = torch.full((B, 1), 0.5, device="cuda")
    qkv = torch.randn((B, heads + 2 * kv, dim), generator=g, device="cuda").to(inputs)
    qm, vm = (torch.randn((B, 1, n), generator=g, device="cuda") for n in (64, heads * dim))
    mem_out = torch.empty((B, 1, heads * dim), device="cuda")
    mem.step(qm, vm, gate, 0.0, out=mem_out)  # scratch before the capture
    torch.cuda.synchronize()

    def token():
        lengths.add_(1)
        q, k, v = qkv.split([heads, kv, kv], 1)
        q = cache.append(k, v, table, lengths, q=q, freqs=freqs)
        mem.step(qm, vm, gate, 0.0, out=mem_out)
        return q, cache.attend(q, table, lengths)

    graph = torch.cuda.CUDAGraph()
    mem.set_graphs(False)
    with torch.cuda.graph(graph):
        q_out, out = token()
    lengths.copy_(as_int32(prompt))
    seen = list(prompt)
    for _ in range(steps):
        qkv.copy_(torch.randn(qkv.shape, generator=g, device="cuda"))
        graph.replay()
        seen = [n + 1 for n in seen]
        assert lengths.tolist() == seen
        want, size = rotated(qkv[:, :heads], lengths - 1, freqs, "halves")
        close(q_out, want, size, inputs)
        want, tol, _, _ = reference(cache, q_out, table, seen, 1 / 8, 0)
        assert ((out.double() - want).abs() <= tol).all()
        assert mem_out.isfinite().all()
    # what the cache holds are the tokens: the last one's keys and values
    for b, n in enumerate(seen):
        at = table[b, (n - 1) // page].long(), slice(None), (n - 1) % page
        want, size = rotated(qkv[b:b + 1, heads:heads + kv], lengths[b:b + 1] - 1, freqs, "halves")
        got = cache.keys.float()[at][None]
        if dtype == E4:
            ks = cache._scales[0].double()[None, :, None]
            want, size = want / ks, size / ks
        close(got.to(dtype), want, size, dtype)
    mem.close()


def test_captured_behind_two_streams():
    """Calls captured where two streams meet wait for the work of both."""
    g = gen(37)
    B, heads, kv, dim, page = 5, 4, 2, 128, 16
    lengths = [3000, 1, 64, 65, 900]
    table, pages = make_table(g, lengths, page)
    cache = make_pool(g, pages, kv, page, dim, BF)
    lens = as_int32(lengths)
    freqs = torch.rand(dim // 2, generator=g, device="cuda")
    big = torch.randn((4096, 4096), generator=g, device="cuda")
    src = [torch.randn((B, heads + 2 * kv, dim), generator=g, device="cuda").to(BF) for _ in range(3)]
    fed, qkv, n = src[0].clone(), torch.empty_like(src[0]), lens.clone()
    side = torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            x = big @ big  # long enough that a call that did not wait would show
            n.copy_(lens + (x[0, 0] * 0).int())
        qkv.copy_(fed)
        main.wait_stream(side)
        q, k, v = qkv.split([heads, kv, kv], 1)
        q = cache.append(k, v, table, n, q=q, freqs=freqs)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            out = cache.attend(q, table, n)
        y = big @ big
        main.wait_stream(side)
        return q, out + (y[0, 0] * 0).to(BF)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got_q, got = step()
    for x in src[1:]:
        fed.copy_(x)
        n.fill_(1)
        qkv.zero_()
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        q, k, v = x.split([heads, kv, kv], 1)
        want_q = cache.append(k, v, table, lens, q=q, freqs=freqs)
        assert torch.equal(got_q, want_q)
        assert torch.equal(got, cache.attend(want_q, table, lens))


def test_tables_with_shared_rows():
    """Sequences that share a table row (one prefix, or the same row for all)."""
    g = gen(41)
    table, pages = make_table(g, [700], 16)
    cache = make_pool(g, pages, 2, 16, 64, BF)
    q = torch.randn((6, 4, 64), generator=g, device="cuda").to(BF)
    lens = as_int32([700, 1, 0, 512, 33, 700])
    want = cache.attend(q, table.repeat(6, 1), lens)
    assert torch.equal(cache.attend(q, table.expand(6, -1), lens), want)
    flat = table[0]
    windows = flat.unfold(0, 8, 4)[:6]  # overlapping rows
    lens = as_int32([128, 100, 3, 0, 128, 64])
    assert torch.equal(cache.attend(q, windows, lens), cache.attend(q, windows.contiguous(), lens))


def test_two_layers_and_the_memory_between_them():
    """A token through an attention layer, a memory step that reads and writes, and a second
    attention layer, each call's output the next one's input with no other kernel
    between them, captured and replayed: every bit as call by call with a
    synchronisation after each."""
    from sparse_weight_memory_b200 import FwPKMState
    g = gen(42)
    B, heads, kv, dim, page, steps = 3, 4, 2, 64, 8, 6
    start = [700, 1, 40]
    table, pages = make_table(g, [n + steps for n in start], page)
    width = heads + 2 * kv
    freqs = torch.rand(dim // 2, generator=g, device="cuda")
    subkeys = torch.randn((1, 2, 32, heads * dim // 2), generator=g, device="cuda")
    rows = torch.randn((1024, width * dim), generator=g, device="cuda")
    gate = torch.full((B, 1), 0.7, device="cuda")
    target = torch.randn((B, 1, width * dim), generator=g, device="cuda")
    fed = [torch.randn((B, width, dim), generator=g, device="cuda").to(BF) for _ in range(steps)]
    pools = [torch.randn((2, pages, kv, page, dim), generator=g, device="cuda").to(BF) for _ in range(2)]

    class Model:
        def __init__(self):
            from sparse_weight_memory_b200 import KVCache
            self.caches = [KVCache(keys=p[0].clone(), values=p[1].clone()) for p in pools]
            self.mem = FwPKMState(1024, heads * dim, width * dim, 4, 1)
            self.mem.set_graphs(False)
            self.x = torch.empty((B, width, dim), dtype=BF, device="cuda")
            self.lengths = as_int32(start)
            self.inner = torch.empty((B, 1, width * dim), device="cuda")
            self.reset()

        def reset(self):
            self.mem.set_tables(subkeys, rows)
            for c, p in zip(self.caches, pools):
                c.keys.copy_(p[0])
                c.values.copy_(p[1])
            self.lengths.copy_(as_int32(start))

        def token(self, done=lambda: None):
            self.lengths.add_(1)
            q, k, v = self.x.split([heads, kv, kv], 1)
            q = self.caches[0].append(k, v, table, self.lengths, q=q, freqs=freqs)
            done()
            out = self.caches[0].attend(q, table, self.lengths)
            done()
            self.mem.step(out.view(B, 1, heads * dim), target, gate, 0.5, out=self.inner)
            done()
            q, k, v = self.inner.view(B, width, dim).split([heads, kv, kv], 1)  # fp32 into bf16
            turned = self.caches[1].append(k, v, table, self.lengths, q=q, freqs=freqs)
            done()
            last = self.caches[1].attend(turned.to(BF), table, self.lengths)
            done()
            return out, self.inner, turned, last

    a, b = Model(), Model()
    a.x.copy_(fed[0])
    a.token()  # scratch before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = a.token()
    a.reset()
    for x in fed:
        a.x.copy_(x)
        b.x.copy_(x)
        graph.replay()
        want = b.token(torch.cuda.synchronize)
        assert all(t.isfinite().all() for t in want)
        for i, j in zip(got, want):
            assert torch.equal(i, j)
    for c, d in zip(a.caches, b.caches):
        assert torch.equal(c.keys, d.keys) and torch.equal(c.values, d.values)
    for i, j in zip(a.mem.get_tables(), b.mem.get_tables()):
        assert torch.equal(i, j)
    a.mem.close()
    b.mem.close()
