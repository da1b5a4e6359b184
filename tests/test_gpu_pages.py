"""Page operations on the GPU against the oracle: every entry of the tables and
every byte of the cache equal."""
import numpy as np
import pytest
import torch

from gpu_util import say
from paged_util import random_table

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def up(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def same(got, want):
    np.testing.assert_array_equal(got.cpu().numpy(), want)


def state(seed, rows, longest, slots, planes, elems, slack, dtype=np.int16, dead=0):
    """A cache, page table, lengths and counts; `dead` rows hold nothing."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, longest + 1, rows).astype(np.int32)
    lens[rng.permutation(rows)[:dead]] = 0
    width = -(-longest // slots) + 1
    used = int(sum(-(-int(n) // slots) for n in lens))
    pages = used + slack
    table = random_table(rng, lens, slots, pages, width)
    refs = np.zeros(pages, np.int32)
    refs[table[table >= 0]] = 1
    info = np.iinfo(dtype)
    cache = rng.integers(info.min, info.max, (planes, pages, elems)).astype(dtype)
    return rng, cache, table, lens, refs


# page sizes of 1 element and of odd bytes, one that ends inside a 16-byte
# vector, one past a workgroup's 16 KiB part, several planes
SIZES = [(1, 1, np.uint8), (2, 7, np.uint8), (3, 33, np.int16), (2, 4096, np.int32), (1, 8195, np.int16), (5, 8192, np.int16)]
AS_TORCH = {np.uint8: torch.uint8, np.int16: torch.bfloat16, np.int32: torch.int32}


def up_cache(c):
    t = up(c)
    return t.view(torch.bfloat16) if c.dtype == np.int16 else t


def down_cache(t):
    return (t.view(torch.int16) if t.dtype == torch.bfloat16 else t).cpu().numpy()


@pytest.mark.parametrize("planes,elems,dtype", SIZES)
def test_copy(stg, orc, planes, elems, dtype):
    rng, cache, *_ = state(1, 4, 30, 4, planes, elems, 20, dtype)
    n = cache.shape[1]
    order = rng.permutation(n)
    src, dst = order[: n // 2].astype(np.int32), order[n // 2: 2 * (n // 2)].astype(np.int32)
    src[0], dst[1] = -1, n  # skipped
    say("pages_copy", planes, n, elems, np.dtype(dtype).name)
    t = up_cache(cache)
    stg.pages_copy(t, up(src), up(dst))
    orc.pages_copy(cache, src, dst)
    np.testing.assert_array_equal(down_cache(t), cache)


def test_copy_strided_planes(stg):
    """A view of some planes and pages of a larger pool: nothing outside it changes."""
    pool = torch.arange(4 * 10 * 24, dtype=torch.int32, device=DEV).view(4, 10, 24)
    want = pool.clone()
    view = pool[1:3, 2:9, :20]
    say("pages_copy on a view")
    stg.pages_copy(view, up(np.array([0, 6], np.int32)), up(np.array([3, 1], np.int32)))
    want[1:3, 5, :20] = want[1:3, 2, :20].clone()
    want[1:3, 3, :20] = want[1:3, 8, :20].clone()
    assert torch.equal(pool, want)


@pytest.mark.parametrize("n", [0, 1])
def test_copy_of_none(stg, n):
    cache = torch.ones((2, 3, 4), device=DEV)
    idx = torch.zeros(n, dtype=torch.int32, device=DEV)
    say("pages_copy of", n)
    stg.pages_copy(cache[:, :3 * n], idx, idx + 2)
    assert bool((cache == 1).all())


@pytest.mark.parametrize("planes,elems,dtype", SIZES)
@pytest.mark.parametrize("slots", [1, 5, 16])
def test_free_then_fork(stg, orc, planes, elems, dtype, slots):
    rng, cache, table, lens, refs = state(2, 24, 70, slots, planes, elems, 30, dtype, dead=3)
    rows = rng.permutation(24)
    children, stay = rows[:9].astype(np.int32), rows[9:]
    parents = rng.choice(stay, 9).astype(np.int32)
    listed = np.concatenate([children, [children[0], -1, 24]]).astype(np.int32)  # one twice, two out of range
    c, t, n, r = up_cache(cache), up(table), up(lens), up(refs)
    short = torch.full((1,), -9, dtype=torch.int32, device=DEV)
    say("pages_free, pages_fork", planes, elems, slots)
    stg.pages_free(t, n, r, up(listed))
    orc.pages_free(table, lens, refs, listed)
    for got, want in ((t, table), (n, lens), (r, refs)):
        same(got, want)
    p, k = parents.copy(), children.copy()
    p[3], k[5] = 99, -2  # skipped
    stg.pages_fork(c, t, n, r, slots, up(p), up(k), shortfall=short)
    assert int(short) == orc.pages_fork(cache, table, lens, refs, slots, p, k)
    for got, want in ((t, table), (n, lens), (r, refs)):
        same(got, want)
    np.testing.assert_array_equal(down_cache(c), cache)


def test_fork_without_enough_pages(stg, orc):
    """Children past the last free page are cut to their full pages."""
    _, cache, table, lens, refs = state(3, 12, 40, 8, 2, 40, 3, dead=6)
    parents = np.repeat(np.flatnonzero(lens % 8 != 0)[:1], 6).astype(np.int32)
    children = np.flatnonzero(lens == 0)[:6].astype(np.int32)
    c, t, n, r = up_cache(cache), up(table), up(lens), up(refs)
    short = torch.zeros(1, dtype=torch.int32, device=DEV)
    say("pages_fork, three free pages for six children")
    stg.pages_fork(c, t, n, r, 8, up(parents), up(children), shortfall=short)
    want = orc.pages_fork(cache, table, lens, refs, 8, parents, children)
    assert int(short) == want == 3
    for got, w in ((t, table), (n, lens), (r, refs)):
        same(got, w)
    np.testing.assert_array_equal(down_cache(c), cache)


def test_fork_of_rows_with_holes(stg, orc):
    """Entries of the parent that name no page are -1 in the child, and a last
    page that is not there takes no page."""
    _, cache, table, lens, refs = state(4, 8, 40, 8, 1, 16, 9)
    lens[6:], table[6:] = 0, -1
    lens[0], table[0] = 21, -1
    table[0, :3] = [-5, 1 << 30, -1]
    refs[:] = 0
    refs[table[(table >= 0) & (table < refs.size)]] = 1
    lens[1] = 1 << 30  # longer than its row
    child = np.array([6, 7], np.int32)
    c, t, n, r = up_cache(cache), up(table), up(lens), up(refs)
    say("pages_fork of holes")
    stg.pages_fork(c, t, n, r, 8, up(np.array([0, 1], np.int32)), up(child))
    orc.pages_fork(cache, table, lens, refs, 8, np.array([0, 1], np.int32), child)
    for got, w in ((t, table), (n, lens), (r, refs)):
        same(got, w)
    np.testing.assert_array_equal(down_cache(c), cache)


@pytest.mark.parametrize("planes,elems,dtype", SIZES)
def test_compact(stg, orc, planes, elems, dtype):
    rng, cache, table, lens, refs = state(5, 30, 60, 4, planes, elems, 60, dtype)
    refs[table[3, :2]] += 1  # shared pages
    table[20, -1], table[21, -1] = -7, 1 << 29  # no pages
    table[22, -1] = np.flatnonzero(refs == 0)[0]  # names a free page
    c, t, r = up_cache(cache), up(table), up(refs)
    say("pages_compact", planes, elems)
    remap = stg.pages_compact(c, t, r)
    want = orc.pages_compact(cache, table, refs)
    same(remap, want)
    same(t, table)
    same(r, refs)
    np.testing.assert_array_equal(down_cache(c), cache)
    again = stg.pages_compact(c, t, r)  # nothing is left to move
    live = int((refs > 0).sum())
    same(again, np.where(refs > 0, np.arange(refs.size), -1))
    assert (refs[:live] > 0).all()
    same(t, table)
    np.testing.assert_array_equal(down_cache(c), cache)


@pytest.mark.parametrize("pages,live", [(1, 0), (1, 1), (4096, 0), (4096, 4096), (4097, 1), (8192, 4096), (20000, 12345),
                                        (12288, 8192)])
def test_compact_pools(stg, orc, pages, live):
    """Pools of one scan workgroup and of several, with the border at, before and past a workgroup's end."""
    rng = np.random.default_rng(pages + live)
    refs = np.zeros(pages, np.int32)
    refs[rng.permutation(pages)[:live]] = rng.integers(1, 4, live)
    ids = np.flatnonzero(refs)
    table = np.full((3, max(1, -(-live // 3))), -1, np.int32)
    table.reshape(-1)[:live] = rng.permutation(ids)
    cache = rng.integers(0, 1 << 30, (2, pages, 5)).astype(np.int32)
    c, t, r = up(cache), up(table), up(refs)
    say("pages_compact", pages, live)
    remap = stg.pages_compact(c, t, r)
    same(remap, orc.pages_compact(cache, table, refs))
    same(t, table)
    same(r, refs)
    same(c, cache)


@pytest.mark.parametrize("pages", [40, 4096, 9000])
@pytest.mark.parametrize("slots", [1, 7, 16])
def test_reserve(stg, orc, pages, slots):
    rng = np.random.default_rng(pages + slots)
    rows, width = 37, 80
    lens = rng.integers(0, 3 * slots, rows).astype(np.int32)
    lens[5], lens[6] = -3, width * slots + 9  # clamped
    n_new = rng.integers(0, 2 * slots + 2, rows).astype(np.int32)
    n_new[1], n_new[7], n_new[8] = 70 * slots, 0, -4
    refs = (rng.random(pages) < 0.6).astype(np.int32)
    live = np.flatnonzero(refs)
    table = np.full((rows, width), -1, np.int32)
    for b in range(rows):
        c = min(width, -(-max(0, int(lens[b])) // slots))
        table[b, :c] = rng.choice(live, c)
    table[9, :4] = -1  # entries before the length stay as they are
    t, n, r = up(table), up(lens), up(refs)
    short = torch.zeros(1, dtype=torch.int32, device=DEV)
    say("pages_reserve", pages, slots)
    stg.pages_reserve(t, n, up(n_new), r, slots, shortfall=short)
    assert int(short) == orc.pages_reserve(table, lens, n_new, refs, slots)
    same(t, table)
    same(r, refs)
    same(n, lens)


def test_graph_replays(stg, orc):
    """A decode loop's page operations under capture, replayed between eager work."""
    _, cache, table, lens, refs = state(6, 16, 60, 8, 2, 64, 20, dead=5)
    children = np.flatnonzero(lens == 0)[:3].astype(np.int32)
    parents = np.flatnonzero(lens > 0)[:3].astype(np.int32)
    first = [up_cache(cache), up(table), up(lens), up(refs)]
    c, t, n, r = (x.clone() for x in first)
    p, k, new = up(parents), up(children), torch.ones(16, dtype=torch.int32, device=DEV)
    ws = torch.empty(stg.pages_workspace(cache.shape[1], 16), dtype=torch.uint8, device=DEV)
    remap = torch.empty(cache.shape[1], dtype=torch.int32, device=DEV)

    def step():
        stg.pages_fork(c, t, n, r, 8, p, k, workspace=ws)
        stg.pages_reserve(t, n, new, r, 8, workspace=ws)
        stg.pages_free(t, n, r, p)
        stg.pages_compact(c, t, r, remap=remap, workspace=ws)

    def reset():
        for x, y in zip((c, t, n, r), first):
            x.copy_(y)
        remap.fill_(-5)

    say("page operations: eager, then captured")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    want = [x.clone() for x in (c, t, n, r, remap)]
    orc.pages_fork(cache, table, lens, refs, 8, parents, children)
    orc.pages_reserve(table, lens, np.ones(16, np.int32), refs, 8)
    orc.pages_free(table, lens, refs, parents)
    orc.pages_compact(cache, table, refs)
    same(t, table)
    same(r, refs)
    np.testing.assert_array_equal(down_cache(c), cache)
    reset()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(3):
        say("replay", i)
        reset()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for got, w in zip((c, t, n, r, remap), want):
            assert torch.equal(got.view(torch.uint8), w.view(torch.uint8))
