"""Forking and ending requests, compacting the cache and copying pages, against plain loops (whole numbers: equal)."""
import random

import pytest
import torch

import kda_linear_attention_bounded_gb300 as kda
from cache_refs import D, compact_reference, fork_reference, free_reference, i32, page_case

pytestmark = pytest.mark.gpu


def strided(table, more):
    """The table in rows `more` wider, which are kept."""
    B, width = len(table), len(table[0]) if table else 3
    wide = torch.full((max(B, 1), width + more), -9, dtype=torch.int32, device="cuda")
    if B:
        wide[:B, :width] = i32(table)
    return wide[:B, :width], wide


# ---------------------------------------------------------------- forking
def fork(table, lens, parents, children, free, page, more=0):
    t, wide = strided(table, more)
    n = i32(lens)
    src, dst = (torch.full((len(parents),), -5, dtype=torch.int32, device="cuda") for _ in range(2))
    used, ws = i32([-5]), kda.make_workspace()
    kda.fork_requests(t, n, i32(parents), i32(children), i32(free), page, copy_src=src, copy_dst=dst, pages_used=used, workspace=ws)
    assert (wide[:, t.shape[1]:] == -9).all()
    return t.tolist(), n.tolist(), src.tolist(), dst.tolist(), int(used), kda.read_device_status(ws)


def fork_case(prompts, copies, longest, page, seed, padding=0):
    table, lens, total = page_case(prompts, longest, page, seed)
    width = len(table[0])
    table += [[-3] * width for _ in range(prompts * copies)]
    lens += [0] * (prompts * copies)
    parents = [p for p in range(prompts) for _ in range(copies)]
    children = list(range(prompts, prompts * (1 + copies)))
    random.Random(seed).shuffle(children)
    return table, lens, parents + [-1] * padding, children + [-1] * padding, list(range(total, total + prompts * copies + 1))


@pytest.mark.parametrize("prompts,copies,longest,page", [
    (1, 1, 1, 1), (1, 4, 33, 16), (3, 7, 500, 16), (48, 5, 300, 64), (255, 1, 40, 5), (300, 3, 90, 24), (1, 700, 9000, 16)])
def test_fork(prompts, copies, longest, page):
    x = fork_case(prompts, copies, longest, page, seed=prompts + copies, padding=copies % 3)
    want = fork_reference(*x, page)
    assert fork(*x, page, more=3) == (*want[:5], 0)


def test_fork_with_padding_between():
    table, lens, parents, children, free = fork_case(6, 2, 100, 16, seed=1)
    parents[3] = children[7] = -1
    want = fork_reference(table, lens, parents, children, free, 16)
    assert fork(table, lens, parents, children, free, 16) == (*want[:5], 0)


@pytest.mark.parametrize("keep", [0, 1, 5])
def test_fork_free_list_used_up(keep):
    x = list(fork_case(40, 2, 100, 16, seed=2))
    x[4] = x[4][:keep]
    *want, refused = fork_reference(*x, 16)
    assert refused > 0
    assert fork(*x, 16) == (*want, kda.KDA_DEVICE_NO_PAGES)


def test_fork_skips_what_is_none():
    table, lens, parents, children, free = fork_case(5, 1, 60, 16, seed=3)
    lens[0], lens[1], lens[2] = 17, -4, 16 * len(table[0]) + 1
    table[0][:2] = [1, 2]
    lens[3] = lens[4] = 20
    parents[3] = len(lens)
    children[4] = parents[4]
    got = fork(table, lens, parents, children, free, 16)
    want = fork_reference(table, lens, parents[:1], children[:1], free, 16)
    assert got[0] == want[0] and got[1] == want[1] and got[4] == 1
    assert got[2] == want[2] + [-1] * 4 and got[3] == want[3] + [-1] * 4
    assert got[5] == kda.KDA_DEVICE_BAD_COUNT | kda.KDA_DEVICE_BAD_INDEX


def test_no_forks():
    assert fork([[1, 2]], [20], [], [], [4], 16)[4] == 0


# ---------------------------------------------------------------- ending
def release(table, lens, rows, page, total, more=0):
    t, _ = strided(table, more)
    n, free, count = i32(lens), torch.full((total,), -5, dtype=torch.int32, device="cuda"), i32([-5])
    ws = kda.make_workspace()
    kda.release_requests(t, n, i32(rows), page, free_pages=free, num_free=count, workspace=ws)
    return n.tolist(), free.tolist(), int(count), kda.read_device_status(ws)


@pytest.mark.parametrize("B,longest,page,shared", [
    (1, 1, 1, 1), (5, 100, 16, 1), (64, 3000, 16, 1), (64, 3000, 16, 8), (700, 90, 5, 4), (3, 40000, 2, 3), (40, 20000, 64, 4)])
def test_release(B, longest, page, shared):
    table, lens, total = page_case(B, longest, page, seed=B + page, shared=shared)
    rows = random.Random(B).sample(range(B), B // 3) + [-1]
    rows += rows[:1]   # one of them twice
    after = [0 if b in rows else n for b, n in enumerate(lens)]
    assert release(table, lens, rows, page, total, more=2) == (after, *free_reference(table, after, page, total), 0)


def test_release_of_all_and_none():
    table, lens, total = page_case(20, 300, 16, seed=4)
    assert release(table, lens, list(range(20)), 16, total) == ([0] * 20, list(range(total)), total, 0)
    assert release(table, lens, [], 16, total) == (lens, *free_reference(table, lens, 16, total), 0)
    assert release([], [], [], 16, 40) == ([], list(range(40)), 40, 0)
    assert release(table, [0] * 20, [], 16, 0) == ([0] * 20, [], 0, 0)


def test_release_of_many_pages():
    # more ids than one window of bits
    total = 3_500_000
    table = [[0, 31, 32, 1_572_863, 1_572_864, total - 1, 1_600_000], [3_200_000, 64, 3_145_728, 3_145_727, -9, -9, -9]]
    lens = [7, 4]
    t, n = i32(table), i32(lens)
    free, count = torch.empty(total, dtype=torch.int32, device="cuda"), i32([0])
    kda.release_requests(t, n, i32([]), 1, free_pages=free, num_free=count)
    used = torch.zeros(total, dtype=torch.bool, device="cuda")
    used[t[0].long()] = True
    used[t[1, :4].long()] = True
    want = torch.nonzero(~used)[:, 0].to(torch.int32)
    assert int(count) == want.numel() and torch.equal(free[:want.numel()], want) and (free[want.numel():] == -1).all()


def test_release_of_what_is_none():
    table, lens, total = page_case(12, 200, 16, seed=5)
    lens[1], lens[2], lens[4] = -3, 16 * len(table[0]) + 1, 40
    table[4][1] = total
    got = release(table, lens, [0, 99], 16, total)
    lens[0] = 0
    seen = list(lens)
    seen[1] = seen[2] = 0
    table[4][1] = table[4][0]
    assert got == (lens, *free_reference(table, seen, 16, total),
                   kda.KDA_DEVICE_BAD_COUNT | kda.KDA_DEVICE_BAD_INDEX | kda.KDA_DEVICE_BAD_PAGE)


# ---------------------------------------------------------------- compacting
def compact(table, lens, page, total, room, in_place=False, more=0):
    t, _ = strided(table, more)
    new = t if in_place else torch.full_like(t, -6)
    lists = [torch.full((n,), -5, dtype=torch.int32, device="cuda") for n in (room, room, total, 1)]
    ws = kda.make_workspace()
    kda.compact_pages(t, i32(lens), page, new_table=new, copy_src=lists[0], copy_dst=lists[1], free_pages=lists[2],
                      num_free=lists[3], workspace=ws)
    return (new.tolist(), *(x.tolist() for x in lists[:3]), int(lists[3])), kda.read_device_status(ws)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,longest,page,shared,extra", [
    (1, 1, 1, 1, 2.0), (5, 100, 16, 1, 1.5), (64, 3000, 16, 8, 1.2), (300, 90, 5, 4, 3.0), (3, 30000, 2, 3, 1.9), (9, 500, 64, 1, 1.0)])
def test_compact(B, longest, page, shared, extra, in_place):
    table, lens, total = page_case(B, longest, page, seed=B + page, shared=shared, extra=extra)
    room = total // 2 + B % 2
    keep = table if in_place else [[-6] * len(table[0])] * B
    got, status = compact(table, lens, page, total, room, in_place, more=1)
    assert status == 0
    assert got == compact_reference(table, lens, page, total, room, keep)


def test_compact_nothing_and_what_is_compact():
    table, lens, total = page_case(4, 100, 16, seed=6)
    got, _ = compact(table, [0] * 4, 16, total, total)
    assert got == ([[-6] * len(table[0])] * 4, [-1] * total, [-1] * total, list(range(total)), total)
    new, *_ = compact(table, lens, 16, total, total, True)[0]
    again, *rest = compact(new, lens, 16, total, total, True)[0]
    assert again == new and set(rest[0]) == {-1}


def test_compact_many_pages():
    total = 3_500_000
    table = [[0, 31, 3_499_999, 1_572_863, 1_572_864, 2, 1_600_000], [3_200_000, 4, 3_145_728, 3_145_727, -9, -9, -9]]
    t = i32(table)
    src, dst = (torch.empty(total // 2, dtype=torch.int32, device="cuda") for _ in range(2))
    free, count = torch.empty(total, dtype=torch.int32, device="cuda"), i32([0])
    kda.compact_pages(t, i32([7, 4]), 1, new_table=t, copy_src=src, copy_dst=dst, free_pages=free, num_free=count)
    moves = sorted(x for r in table for x in r if x > 10)
    assert src[:9].tolist() == moves + [-1] and dst[:9].tolist() == [1, 3, 5, 6, 7, 8, 9, 10, -1]
    assert (src[8:] == -1).all() and (dst[8:] == -1).all()
    to = dict(zip(moves, [1, 3, 5, 6, 7, 8, 9, 10]))
    assert t.tolist() == [[to.get(x, x) for x in r] for r in table]
    assert int(count) == total - 11 and torch.equal(free[:total - 11], torch.arange(11, total, device="cuda").int())


def test_compact_of_what_is_none():
    table, lens, total = page_case(12, 200, 16, seed=7)
    lens[1], lens[2], lens[4] = -3, 16 * len(table[0]) + 1, 40
    table[4][1], table[4][2] = total, -1
    got, status = compact(table, lens, 16, total, total)
    seen = list(lens)
    seen[1] = seen[2] = 0
    assert status == kda.KDA_DEVICE_BAD_COUNT | kda.KDA_DEVICE_BAD_PAGE
    assert got == compact_reference(table, seen, 16, total, total, [[-6] * len(table[0])] * 12)


# ---------------------------------------------------------------- tables that the whole GPU marks
WIDE = [(700, 400, 1, 1, None), (700, 1600, 4, 8, None), (4, 5, 1, 1, 70000), (33, 90, 16, 1, 4000), (2, 100000, 1, 1, None)]


@pytest.mark.parametrize("B,longest,page,shared,width", WIDE)
def test_release_in_wide_tables(B, longest, page, shared, width):
    table, lens, total = page_case(B, longest, page, seed=B + page, shared=shared, width=width)
    rows = random.Random(B).sample(range(B), B // 3) + [-1]
    after = [0 if b in rows else n for b, n in enumerate(lens)]
    assert release(table, lens, rows, page, total, more=1) == (after, *free_reference(table, after, page, total), 0)


@pytest.mark.parametrize("B,longest,page,shared,width", WIDE)
def test_compact_in_wide_tables(B, longest, page, shared, width):
    table, lens, total = page_case(B, longest, page, seed=B + page, shared=shared, width=width, extra=1.7)
    room = total // 2 + 1
    got, status = compact(table, lens, page, total, room, in_place=True, more=1)
    assert status == 0 and got == compact_reference(table, lens, page, total, room, table)


@pytest.mark.parametrize("total,lens", [(5000, [3, 2]), (5000, [0, 0]), (70001, [900, 1300]), (70001, [900, 1500]), (150, [3, 140])])
def test_wide_tables_of_a_nearly_free_cache(total, lens):
    # more free pages than the list's memory has room for before the marks
    ids = random.Random(total).sample(range(total), sum(lens))
    table = [ids[:lens[0]] + [-4] * (70000 - lens[0]), ids[lens[0]:] + [-4] * (70000 - lens[1])]
    want = free_reference(table, lens, 1, total)
    assert release(table, lens, [-1], 1, total) == (lens, *want, 0)
    got, status = compact(table, lens, 1, total, total, in_place=True)
    assert status == 0 and got == compact_reference(table, lens, 1, total, total, table)


@pytest.mark.parametrize("off", [1, 2, 3])
def test_wide_tables_with_lists_anywhere(off):
    # the free list at any 4 bytes, ids and lengths that are none, again from a graph
    table, lens, total = page_case(300, 700, 1, seed=off, width=800)
    lens[5], lens[6], lens[7] = -1, 801, 30
    table[7][3], table[7][29], table[7][30] = -2, total, total + 1
    rows = [0, 300, 44]
    buffer = torch.full((total + 8,), -5, dtype=torch.int32, device="cuda")
    t, start, count, ws = i32(table), i32(lens), i32([0]), kda.make_workspace()
    n, free = start.clone(), buffer[off:off + total]
    call = lambda: kda.release_requests(t, n, i32_rows, 1, free_pages=free, num_free=count, workspace=ws)
    i32_rows = i32(rows)
    seen = [0 if b in (0, 44) or x < 0 or x > 800 else x for b, x in enumerate(lens)]
    read = [list(r) for r in table]
    read[7][3] = read[7][29] = read[7][0]
    want = free_reference(read, seen, 1, total)
    lens[0] = lens[44] = 0
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):
        assert (free.tolist(), int(count)) == want and n.tolist() == lens
        assert buffer[:off].tolist() == [-5] * off and buffer[off + total:].tolist() == [-5] * (8 - off)
        assert kda.read_device_status(ws) == kda.KDA_DEVICE_BAD_COUNT | kda.KDA_DEVICE_BAD_INDEX | kda.KDA_DEVICE_BAD_PAGE
        free.fill_(-5)
        n.copy_(start)
        graph.replay()
        torch.cuda.synchronize()


# ---------------------------------------------------------------- copying
def buffers_of(total, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    both = n(total, 2, 16, 2, D).bfloat16()
    wide = n(total, 40)
    return [n(total, 16, 2, D).bfloat16(), both[:, 0], both[:, 1], n(total, 4, D, D), n(total, 3, 1032).half(),
            wide[:, :8], (n(total, 16) * 50).to(torch.uint8), (n(total, 5000) * 50).to(torch.int64)], both, wide


@pytest.mark.parametrize("pairs", [0, 1, 7, 40, 5000])
def test_copy(pairs):
    total = max(2 * pairs + 5, 9) if pairs < 100 else pairs * 2 + 5
    r = random.Random(pairs)
    if pairs < 100:
        buffers, _, wide = buffers_of(total, pairs)
    else:   # more pairs than are listed at once
        buffers = [torch.randn((total, 40, 4), device="cuda"), torch.randn((total, 1, 12), device="cuda")]
        wide = buffers[0]
    ids = r.sample(range(total), 2 * pairs)
    src, dst = ids[:pairs], ids[pairs:]
    for at in r.sample(range(pairs), pairs // 3):   # entries without a copy
        if at % 2:
            src[at] = -1
        else:
            dst[at] = -1
    want = [b.clone() for b in buffers]
    live = [(a, b) for a, b in zip(src, dst) if a >= 0 and b >= 0]
    if live:
        a, b = (torch.tensor(x, device="cuda") for x in zip(*live))
        for w in want:
            w[b] = w[a]
    outside = wide[:, 8:].clone()
    ws = kda.make_workspace()
    kda.copy_pages(buffers, i32(src), i32(dst), workspace=ws)
    assert kda.read_device_status(ws) == 0
    for w, b in zip(want, buffers):
        assert torch.equal(w, b)
    if pairs < 100:
        assert torch.equal(outside, wide[:, 8:])


def test_copy_leaves_out_what_is_none():
    x = torch.randn((10, 64), device="cuda")
    want = x.clone()
    want[5] = want[4]
    ws = kda.make_workspace()
    kda.copy_pages([x], i32([1, 10, 4, 3, -2]), i32([10, 2, 5, 3, 8]), workspace=ws)
    assert kda.read_device_status(ws) == kda.KDA_DEVICE_BAD_PAGE
    assert torch.equal(x, want)


def test_copy_of_many_buffers():
    # more than one launch takes
    buffers = [torch.randn((6, 4 * (1 + i % 3)), device="cuda") for i in range(300)]
    want = [b.clone() for b in buffers]
    for w in want:
        w[5], w[0] = w[1], w[2]
    kda.copy_pages(tuple(buffers), i32([1, 2]), i32([5, 0]))
    for w, b in zip(want, buffers):
        assert torch.equal(w, b)


def test_copy_beyond_32_bits():
    x = torch.zeros((70000, 40000), dtype=torch.uint8, device="cuda")
    assert x.numel() > 2 ** 31
    x[69999] = torch.arange(40000, device="cuda") % 251
    kda.copy_pages([x], i32([69999, 69999]), i32([3, 69001]))
    assert torch.equal(x[3], x[69999]) and torch.equal(x[69001], x[69999]) and not x[69000].any() and not x[69002].any()


def test_page_calls_in_a_graph():
    """Fork, copy, release and compact captured once and replayed with other lengths."""
    page, B, width = 16, 12, 9
    case = lambda seed: page_case(B, 16 * width, page, seed, extra=2.0, width=width)  # noqa: E731
    t0, l0, _ = case(8)
    total = 2 * B * width + 2
    table, lens, new = i32(t0), i32(l0), torch.zeros((B, width), dtype=torch.int32, device="cuda")
    cache = torch.randn((total, page, 1, D), device="cuda").bfloat16()
    parents, children = i32([0, 1, -1]), i32([10, 11, -1])
    src, dst, used = i32([0] * 3), i32([0] * 3), i32([0])
    csrc, cdst = (torch.zeros(total // 2, dtype=torch.int32, device="cuda") for _ in range(2))
    free, count, free2, count2 = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (total, 1, total, 1))
    ws = kda.make_workspace()

    def calls():
        kda.release_requests(table, lens, children, page, free_pages=free, num_free=count, workspace=ws)
        kda.fork_requests(table, lens, parents, children, free, page, copy_src=src, copy_dst=dst, pages_used=used, workspace=ws)
        kda.copy_pages([cache], src, dst, workspace=ws)
        kda.compact_pages(table, lens, page, new_table=new, copy_src=csrc, copy_dst=cdst, free_pages=free2, num_free=count2,
                          workspace=ws)
        kda.copy_pages([cache], csrc, cdst, workspace=ws)

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for seed in (9, 10):
        t, n, _ = case(seed)
        table.copy_(i32(t))
        lens.copy_(i32(n))
        old = cache.clone()
        graph.replay()
        torch.cuda.synchronize()
        n[10] = n[11] = 0
        free_want, num = free_reference(t, n, page, total)
        assert free.tolist() == free_want and int(count) == num
        ft, fl, fs, fd, fu, _ = fork_reference(t, n, [0, 1], [10, 11], free_want, page)
        assert (table.tolist(), lens.tolist(), src.tolist(), dst.tolist(), int(used)) == (ft, fl, fs + [-1], fd + [-1], fu)
        for b in range(B):   # every request's tokens are where the new table says
            for c in range(-(-fl[b] // page)):
                was = fs[fd.index(ft[b][c])] if ft[b][c] in fd and ft[b][c] >= 0 else ft[b][c]
                assert torch.equal(cache[new[b, c]], old[was]), (b, c)
    assert kda.read_device_status(ws) == 0
