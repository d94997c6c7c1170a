"""Paged key-value cache, without a GPU: the schedule's arithmetic and the
places of new tokens (cache_schedule.cuh compiled for the host), the refusals
of both calls, and the binding's constants."""
import ctypes
import functools
import os
import re
import subprocess

import numpy as np
import pytest
import torch

from sparse_weight_memory_b200 import FwpkmError, KVCache
from sparse_weight_memory_b200 import build as fwbuild
from sparse_weight_memory_b200 import cache as binding
from sparse_weight_memory_b200.fwpkm import (FWPKM_BF16, FWPKM_EINVAL, FWPKM_ESHAPE,
                                             FWPKM_EUNSUPPORTED, FWPKM_F32, FWPKM_OK)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fwpkm_cache.h")
i32, i64 = ctypes.c_int, ctypes.c_int64

SHIM = """
#include "cache_schedule.cuh"
using namespace fwpkm;
extern "C" {
void span(int len, int window, int tile, int *o) {
  Span s = cache_span(len, window, tile);
  o[0] = s.lo; o[1] = s.len; o[2] = s.first; o[3] = s.count;
}
int extra_of(int64_t tiles, int most) { return extra_units(tiles, most); }
int warps(int64_t units, int most, int extra) { return piece_line(units, most, extra).warps; }
int64_t cut(int64_t units, int most, int extra, int w) {
  return line_cut(piece_line(units, most, extra), w);
}
int owner(int64_t units, int most, int extra, int64_t unit) {
  return line_owner(piece_line(units, most, extra), unit);
}
int64_t unit_of(int j, int extra) { return tile_unit(j, extra); }
int from(int64_t u, int extra) { return tile_from(u, extra); }
int tiles(int64_t u, int count, int extra) { return tiles_before(u, count, extra); }
int page(int d, int t) { return page_of(page_div(d), t); }
int length(int len, int width, int page, int *bad) {
  bool b; int r = cache_length(len, width, page, b); *bad = b; return r;
}
int position(int len, int before, int after, int width, int page, int *bad) {
  bool b; int r = append_position(len, before, after, width, page, b); *bad = b; return r;
}
}
"""


@pytest.fixture(scope="module")
def sched(tmp_path_factory):
    d = tmp_path_factory.mktemp("schedule")
    (d / "shim.cpp").write_text(SHIM)
    so = str(d / "shim.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover",
                    "-static-libubsan", "-shared", "-fPIC", "-I", fwbuild.CSRC,
                    str(d / "shim.cpp"), "-o", so], check=True)
    L = ctypes.CDLL(so)
    L.extra_of.argtypes, L.warps.argtypes = [i64, i32], [i64, i32, i32]
    L.cut.argtypes, L.owner.argtypes = [i64, i32, i32, i32], [i64, i32, i32, i64]
    L.unit_of.argtypes, L.from_ = [i32, i32], getattr(L, "from")
    L.from_.argtypes, L.tiles.argtypes = [i64, i32], [i64, i32, i32]
    L.cut.restype = L.unit_of.restype = i64
    return L


@pytest.fixture(scope="module")
def lib():
    fwbuild.build()
    return binding._library()


@pytest.mark.parametrize("tile", [8, 16, 32])
@pytest.mark.parametrize("window", [0, 1, 7, 16, 100, 2**31 - 1])
def test_span_covers_the_visible_tokens(sched, tile, window):
    o = (i32 * 4)()
    for n in [0, 1, tile - 1, tile, tile + 1, 99, 100, 101, 1000, 2**31 - 1]:
        sched.span(n, window, tile, o)
        lo, end, first, count = list(o)
        assert end == n and lo == (max(0, n - window) if window else 0)
        if n == 0:
            assert (first, count) == (0, 1)
        else:  # the first and the last tile hold a visible token, no tile outside does
            assert first * tile <= lo < (first + 1) * tile
            assert (first + count - 1) * tile < n <= (first + count) * tile


def test_pieces_share_the_line_out(sched):
    """Every tile of every segment belongs to one warp; pieces differ by a unit at
    most; and a segment's parts are those of its first warp to its last, none
    of them without a tile."""
    rng = np.random.default_rng(0)
    seen = set()
    for _ in range(200):
        most = int(rng.choice([1, 5, 8, 16, 592, 1184, 2368]))
        big = int(np.exp(rng.uniform(0, np.log(3000))))
        counts = [int(c) for c in rng.integers(1, big + 1, int(rng.integers(1, 60)))]
        extra = sched.extra_of(sum(counts), most)
        seen.add(extra)
        assert extra == (0 if sum(counts) <= most else 2)
        at = np.cumsum([0] + [c + extra for c in counts])
        line = (int(at[-1]), most, extra)
        n = sched.warps(*line)
        cuts = [sched.cut(*line, w) for w in range(n + 1)]
        sizes = np.diff(cuts)
        assert 1 <= n <= most and cuts[0] == 0 and cuts[-1] == at[-1]
        assert sizes.max() - sizes.min() <= 1 and (n == 1 or sizes.min() > extra)
        for c, first in zip(counts, at[:-1]):
            unit = [int(first) + sched.unit_of(j, extra) for j in range(c)]
            assert unit[-1] < first + c + extra
            owner = np.searchsorted(cuts, unit, side="right") - 1
            for j in {0, c - 1, c // 2}:
                assert sched.owner(*line, unit[j]) == owner[j]
            assert set(owner) == set(range(owner[0], owner[-1] + 1))
            for w in range(owner[0], owner[-1] + 1):  # where the warp enters the segment
                j = sched.from_(max(0, cuts[w] - int(first)), extra)
                assert j == int(np.searchsorted(owner, w))
                end = sched.tiles(cuts[w + 1] - int(first), c, extra)
                assert end == int(np.searchsorted(owner, w, side="right"))
    assert seen == {0, 2}


def test_largest_line_stays_within_64_bits(sched):
    total = (1 << 22) * ((1 << 28) + 2)  # B * heads segments of 2^31 tokens
    line = (total, 2368, 2)
    assert sched.cut(*line, 2368) == total
    assert sched.owner(*line, total - 1) == 2367
    assert sched.owner(*line, 0) == 0


def test_page_of_a_token_is_the_quotient(sched):
    top = 2**31 - 1
    rng = np.random.default_rng(1)
    sizes = [*range(1, 40), 48, 63, 64, 65, 100, 127, 1000, 2**16 + 1, 2**30, 2**30 + 1, top - 1,
             top, *(int(x) for x in rng.integers(1, top, 50))]
    for d in sizes:
        tokens = {0, 1, d - 1, d, top, top - 1, top // d * d, max(0, top // d * d - 1),
                  *(int(x) for x in rng.integers(0, top, 30)),
                  *(int(x) * d % (top + 1) for x in rng.integers(0, top, 10))}
        for t in tokens:
            if t <= top:
                assert sched.page(d, t) == t // d


def test_lengths_stay_within_the_table(sched):
    bad = i32()
    for n, width, page, want in [(0, 3, 16, 0), (48, 3, 16, 48), (49, 3, 16, 48), (-1, 3, 16, 0),
                                 (2**31 - 1, 2**31 - 1, 2**31 - 1, 2**31 - 1),
                                 (-2**31, 1, 1, 0)]:
        assert sched.length(n, width, page, ctypes.byref(bad)) == want
        assert bool(bad.value) == (n != want)


def test_places_of_new_tokens(sched):
    """A row is stored only where its page is an entry of the table, whatever
    lengths and starts the call was given."""
    bad = i32()
    top = 2**31 - 1
    for n in [-top - 1, -1, 0, 1, 16, 47, 48, 49, top]:
        for before in [-top - 1, -1, 0, 1, 15, top]:
            for after in [-top - 1, 0, 1, 2, 48, top]:
                pos = sched.position(n, before, after, 3, 16, ctypes.byref(bad))
                if n < 0 or after < 1 or n < after:
                    assert pos == -1 and bad.value
                    continue
                assert pos == n - after
                ok = before >= 0 and before + after <= n and pos // 16 < 3
                assert bool(bad.value) == (not ok)


# -- refusals -----------------------------------------------------------------

FAKE = 1 << 20  # an aligned address that nothing reads: every call here is refused first


def pool(**kw):
    c = binding._Cache(FAKE, FAKE, 8 * 16 * 64, 16 * 64, 64, 4, 16, 8, 64, FWPKM_BF16, None, None)
    for name, v in kw.items():
        setattr(c, name, v)
    return c


def batch(**kw):
    b = binding._Batch(2, 3, 3, FAKE, FAKE)
    for name, v in kw.items():
        setattr(b, name, v)
    return b


APPEND = dict(rows=2, in_dtype=FWPKM_BF16, k=FAKE, k_stride=512, v=FAKE, v_stride=512, q=FAKE,
              q_stride=1024, q_out=2 * FAKE, q_out_stride=1024, heads=16, starts=None, rotary=64,
              style=0, freqs=FAKE, errors=None, stream=None)
ATTEND = dict(heads=16, q_dtype=FWPKM_BF16, q=FAKE, q_stride=1024, scale=0.125, window=0, out=2 * FAKE,
              lse=None, workspace=FAKE, workspace_bytes=1 << 40, errors=None, stream=None)


def call(lib, fn, args, c, b, **kw):
    args = dict(args, **kw)
    return fn(None if c is None else ctypes.byref(c), None if b is None else ctypes.byref(b),
              *args.values())


POOL_REFUSALS = [
    (dict(keys=None), FWPKM_EINVAL), (dict(values=None), FWPKM_EINVAL),
    (dict(keys=FAKE + 8), FWPKM_EINVAL), (dict(dtype=3), FWPKM_EINVAL),
    (dict(dtype=-1), FWPKM_EINVAL), (dict(dim=0), FWPKM_ESHAPE), (dict(dim=60), FWPKM_ESHAPE),
    (dict(dim=264), FWPKM_ESHAPE), (dict(dtype=2, dim=72), FWPKM_ESHAPE),
    (dict(pages=0), FWPKM_ESHAPE), (dict(pages=2**31), FWPKM_ESHAPE),
    (dict(page_size=0), FWPKM_ESHAPE), (dict(kv_heads=0), FWPKM_ESHAPE),
    (dict(row_stride=68), FWPKM_ESHAPE), (dict(head_stride=-8), FWPKM_ESHAPE),
    (dict(page_stride=2**41), FWPKM_ESHAPE), (dict(pages=2**30, page_stride=2**40), FWPKM_ESHAPE),
    (dict(key_scale=FAKE), FWPKM_EINVAL),
]
BATCH_REFUSALS = [
    (dict(B=0), FWPKM_ESHAPE), (dict(B=2**22 + 1), FWPKM_ESHAPE),
    (dict(table_width=0), FWPKM_ESHAPE), (dict(table_stride=-1), FWPKM_ESHAPE),
    (dict(table=None), FWPKM_EINVAL), (dict(lengths=None), FWPKM_EINVAL),
    (dict(lengths=FAKE + 2), FWPKM_EINVAL),
]


@pytest.mark.parametrize("kw,status", POOL_REFUSALS)
def test_pool_refusals(lib, kw, status):
    assert call(lib, lib.fwpkm_cache_append, APPEND, pool(**kw), batch()) == status
    assert call(lib, lib.fwpkm_cache_attend, ATTEND, pool(**kw), batch()) == status
    assert lib.fwpkm_last_error().decode()


@pytest.mark.parametrize("kw,status", BATCH_REFUSALS)
def test_batch_refusals(lib, kw, status):
    assert call(lib, lib.fwpkm_cache_append, APPEND, pool(), batch(**kw)) == status
    assert call(lib, lib.fwpkm_cache_attend, ATTEND, pool(), batch(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(in_dtype=2), FWPKM_EINVAL), (dict(rows=-1), FWPKM_ESHAPE), (dict(rows=3), FWPKM_ESHAPE),
    (dict(rotary=8), FWPKM_ESHAPE), (dict(rotary=80), FWPKM_ESHAPE),
    (dict(rotary=-16), FWPKM_ESHAPE), (dict(style=2), FWPKM_EINVAL), (dict(freqs=None), FWPKM_EINVAL),
    (dict(q=None), FWPKM_EINVAL), (dict(q_out=None), FWPKM_EINVAL), (dict(heads=0), FWPKM_ESHAPE),
    (dict(k=None), FWPKM_EINVAL), (dict(v=None), FWPKM_EINVAL), (dict(k=FAKE + 2), FWPKM_EINVAL),
    (dict(k_stride=511), FWPKM_ESHAPE), (dict(v_stride=504), FWPKM_ESHAPE),
    (dict(q_stride=1020), FWPKM_ESHAPE), (dict(q_out=FAKE, q_out_stride=2048), FWPKM_EINVAL),
])
def test_append_refusals(lib, kw, status):
    assert call(lib, lib.fwpkm_cache_append, APPEND, pool(), batch(), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(heads=12), FWPKM_ESHAPE), (dict(heads=0), FWPKM_ESHAPE), (dict(heads=8192), FWPKM_ESHAPE),
    (dict(q_dtype=2), FWPKM_EINVAL), (dict(q_dtype=FWPKM_F32), FWPKM_EUNSUPPORTED),
    (dict(q=None), FWPKM_EINVAL), (dict(q_stride=1016), FWPKM_ESHAPE), (dict(out=None), FWPKM_EINVAL),
    (dict(out=FAKE + 4), FWPKM_EINVAL), (dict(out=FAKE, q=FAKE), FWPKM_EINVAL), (dict(scale=float("nan")), FWPKM_EINVAL),
    (dict(scale=float("inf")), FWPKM_EINVAL), (dict(scale=3e38), FWPKM_EINVAL),
    (dict(window=-1), FWPKM_EINVAL),
    (dict(workspace=None), FWPKM_EINVAL), (dict(workspace=FAKE + 16), FWPKM_EINVAL),
    (dict(workspace_bytes=1000), FWPKM_EINVAL),
])
def test_attend_refusals(lib, kw, status):
    assert call(lib, lib.fwpkm_cache_attend, ATTEND, pool(), batch(), **kw) == status


@pytest.mark.parametrize("fn,args,c,kw", [
    ("append", APPEND, dict(), dict(starts=FAKE + 2)), ("append", APPEND, dict(), dict(freqs=FAKE + 1)),
    ("append", APPEND, dict(), dict(errors=FAKE + 2)),
    ("append", APPEND, dict(dtype=2, key_scale=FAKE + 2), dict()),
    ("attend", ATTEND, dict(dtype=2, value_scale=FAKE + 1), dict()),
    ("attend", ATTEND, dict(), dict(lse=FAKE + 2)), ("attend", ATTEND, dict(), dict(errors=FAKE + 3)),
])
def test_words_that_are_not_aligned(lib, fn, args, c, kw):
    """The kernels read and write them as 32-bit words."""
    call_ = getattr(lib, "fwpkm_cache_" + fn)
    assert call(lib, call_, args, pool(**c), batch(), **kw) == FWPKM_EINVAL
    assert "4-byte aligned" in lib.fwpkm_last_error().decode()


def test_null_descriptors_and_large_batches(lib):
    assert call(lib, lib.fwpkm_cache_append, APPEND, None, batch()) == FWPKM_EINVAL
    assert call(lib, lib.fwpkm_cache_append, APPEND, pool(), None) == FWPKM_EINVAL
    assert call(lib, lib.fwpkm_cache_attend, ATTEND, None, batch()) == FWPKM_EINVAL
    assert call(lib, lib.fwpkm_cache_attend, ATTEND, pool(), None) == FWPKM_EINVAL
    assert call(lib, lib.fwpkm_cache_attend, ATTEND, pool(), batch(B=2**19)) == FWPKM_ESHAPE
    assert lib.fwpkm_cache_attend_workspace(None, 1, 8) == FWPKM_EINVAL
    assert lib.fwpkm_cache_attend_workspace(ctypes.byref(pool()), 0, 8) == FWPKM_ESHAPE
    assert lib.fwpkm_cache_attend_workspace(ctypes.byref(pool()), 1, 9) == FWPKM_ESHAPE
    assert lib.fwpkm_cache_attend_workspace(ctypes.byref(pool()), 1, 8) > 0


def test_no_rows_are_no_work(lib):
    """rows = 0 (an empty packed batch) launches nothing, so it needs no device."""
    assert call(lib, lib.fwpkm_cache_append, APPEND, pool(), batch(), rows=0, starts=FAKE,
                k=None, v=None) == FWPKM_OK


# -- the binding ------------------------------------------------------------------

def test_binding_constants_and_exports(lib):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    values = {n: int(v) for n, v in re.findall(r"\b(FWPKM_[A-Z0-9_]+)\s*=?\s+(\d+)u?\b", src)}
    assert values["FWPKM_E4M3"] == binding.E4M3
    assert values["FWPKM_ROTATE_HALVES"] == binding.ROTATE["halves"]
    assert values["FWPKM_ROTATE_PAIRS"] == binding.ROTATE["pairs"]
    assert values["FWPKM_CACHE_BAD_PAGE"] == binding.BAD_PAGE
    assert values["FWPKM_CACHE_BAD_LENGTH"] == binding.BAD_LENGTH
    names = set(re.findall(r"\b(fwpkm_cache_[a-z_]+)\s*\(", src))
    assert names == {"fwpkm_cache_append", "fwpkm_cache_attend", "fwpkm_cache_attend_workspace"}
    for n in names:
        assert hasattr(lib, n)


def cpu_cache(**kw):
    return KVCache(**dict(dict(pages=4, page_size=16, kv_heads=2, dim=64, device="cpu"), **kw))


def cpu_args(**kw):
    bf = torch.bfloat16
    a = dict(k=torch.zeros(2, 2, 64, dtype=bf), v=torch.zeros(2, 2, 64, dtype=bf),
             table=torch.zeros(2, 3, dtype=torch.int32), lengths=torch.ones(2, dtype=torch.int32),
             q=torch.zeros(2, 4, 64, dtype=bf))
    return dict(a, **kw)


@pytest.mark.parametrize("kw,error", [
    (dict(k=torch.zeros(2, 3, 64, dtype=torch.bfloat16)), FwpkmError),
    (dict(k=torch.zeros(3, 2, 64, dtype=torch.bfloat16)), FwpkmError),
    (dict(k=torch.zeros(2, 2, 64, dtype=torch.float16)), TypeError),
    (dict(v=torch.zeros(2, 2, 64)), TypeError),
    (dict(v=torch.zeros(2, 64, 2, dtype=torch.bfloat16).transpose(1, 2)), FwpkmError),
    (dict(table=torch.zeros(3, 3, dtype=torch.int32)), FwpkmError),
    (dict(table=torch.zeros(2, 3)), TypeError),
    (dict(table=torch.zeros(3, 2, dtype=torch.int32).t()), FwpkmError),
    (dict(lengths=torch.ones(2, dtype=torch.int64)), TypeError),
    (dict(lengths=torch.ones(4, dtype=torch.int32)[::2]), FwpkmError),
    (dict(q=torch.zeros(1, 4, 64, dtype=torch.bfloat16)), FwpkmError),
    (dict(q=None, q_out=torch.zeros(2, 4, 64, dtype=torch.bfloat16)), FwpkmError),
    (dict(q_out=torch.zeros(2, 5, 64, dtype=torch.bfloat16)), FwpkmError),
    (dict(starts=torch.zeros(2, dtype=torch.int32)), FwpkmError),
    (dict(freqs=torch.zeros(8, dtype=torch.float64)), TypeError),
    (dict(style="thirds"), FwpkmError), (dict(errors=torch.zeros(1)), TypeError),
    (dict(), FwpkmError),  # a cache that is not on a CUDA device
])
def test_binding_refuses_append(lib, kw, error):
    with pytest.raises(error):
        cpu_cache().append(**cpu_args(**kw))


@pytest.mark.parametrize("kw,error", [
    (dict(q=torch.zeros(3, 4, 64, dtype=torch.bfloat16)), FwpkmError),
    (dict(q=torch.zeros(2, 4, 32, dtype=torch.bfloat16)), FwpkmError),
    (dict(q=torch.zeros(2, 3, 64, dtype=torch.bfloat16)), FwpkmError),
    (dict(q=torch.zeros(2, 4, 64, dtype=torch.float16)), TypeError),
    (dict(out=torch.zeros(2, 4, 64)), TypeError),
    (dict(out=torch.zeros(2, 2, 64, dtype=torch.bfloat16)), FwpkmError),
    (dict(lse=torch.zeros(2, 5)), FwpkmError), (dict(lse=torch.zeros(2, 4, dtype=torch.int32)), TypeError),
    (dict(workspace=torch.zeros(4)), TypeError), (dict(), FwpkmError),
])
def test_binding_refuses_attend(lib, kw, error):
    a = cpu_args(**kw)
    a.pop("k"), a.pop("v")
    with pytest.raises(error):
        cpu_cache().attend(**a)


@pytest.mark.parametrize("kw,error", [
    (dict(dim=60), FwpkmError), (dict(dim=512), FwpkmError), (dict(pages=0), FwpkmError),
    (dict(kv_heads=None), FwpkmError), (dict(dtype=torch.float16), TypeError),
    (dict(dim=72, dtype=torch.float8_e4m3fn), FwpkmError), (dict(keys=torch.zeros(1)), FwpkmError),
    (dict(key_scale=torch.ones(3)), FwpkmError),
    (dict(keys=torch.zeros(4, 16, 2, 64), values=torch.zeros(4, 2, 16, 64)), FwpkmError),
])
def test_binding_refuses_caches(lib, kw, error):
    with pytest.raises(error):
        cpu_cache(**kw)


def test_binding_refuses_sizes_beyond_an_int(lib):
    """Sizes and windows that would wrap around on their way into the library (tensors
    without storage stand in for the large ones)."""
    bf, far = torch.bfloat16, 2**32 + 2
    empty = functools.partial(torch.empty, device="meta")
    long = dict(k=empty(far, 2, 64, dtype=bf), v=empty(far, 2, 64, dtype=bf), q=None)
    many = dict(table=empty(far, 3, dtype=torch.int32), lengths=empty(far, dtype=torch.int32))
    for kw in (long, many, dict(table=empty(2, far, dtype=torch.int32)),
               dict(q=empty(2, far, 64, dtype=bf))):
        with pytest.raises(FwpkmError, match="2\\^31"):
            cpu_cache().append(**cpu_args(**kw))
    for window in (-1, 2**31, far, -far):
        a = cpu_args(window=window)
        a.pop("k"), a.pop("v")
        with pytest.raises(FwpkmError, match="window"):
            cpu_cache().attend(**a)
    pool = empty(4, 2, far, 64, dtype=bf)
    with pytest.raises(FwpkmError, match="2\\^31"):
        KVCache(keys=pool, values=pool)


def test_pool_layouts(lib):
    """Pools [pages][page_size][kv_heads][dim] and pools interleaved in one tensor."""
    both = torch.zeros(4, 2, 16, 2, 64, dtype=torch.bfloat16)
    c = KVCache(keys=both[:, 0].transpose(1, 2), values=both[:, 1].transpose(1, 2))
    assert (c.pages, c.kv_heads, c.page_size, c.dim) == (4, 2, 16, 64)
    assert (c._c.page_stride, c._c.head_stride, c._c.row_stride) == (2 * 16 * 128, 64, 128)


def test_tables_may_overlap(lib):
    """Rows that overlap, and one row for all, as the library takes them: such tables pass
    the binding's checks (and are refused for the cache's device)."""
    row = torch.zeros(8, dtype=torch.int32)
    for table in (row.expand(2, -1), row.unfold(0, 6, 2)):
        with pytest.raises(FwpkmError, match="not on a CUDA device"):
            cpu_cache().append(**cpu_args(table=table))
    assert cpu_cache()._batch(row.expand(2, -1), torch.ones(2, dtype=torch.int32)).table_stride == 0


@pytest.mark.parametrize("name", ["k", "v", "q", "freqs"])
def test_binding_refuses_to_drop_gradients(lib, name):
    """No gradients pass: an input that requires them is refused while they are recorded."""
    a = cpu_args(freqs=torch.ones(32))
    a[name] = a[name].clone().requires_grad_()
    calls = [lambda: cpu_cache().append(**a)]
    if name == "q":
        calls.append(lambda: cpu_cache().attend(a["q"], a["table"], a["lengths"]))
    for call_ in calls:
        with pytest.raises(FwpkmError, match="no gradients") as e:
            call_()
        assert e.value.status == FWPKM_EUNSUPPORTED
        with torch.no_grad(), pytest.raises(FwpkmError, match="not on a CUDA device"):
            call_()
