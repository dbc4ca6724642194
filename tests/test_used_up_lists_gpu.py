"""Free lists as release_requests and compact_pages leave them, of the cache's whole length with -1 behind the free ids, handed on
as they are: they end at the first -1, whatever their length."""
import random

import pytest
import torch

import kda_linear_attention_bounded_gb300 as kda
from cache_refs import D, fork_reference, free_reference, i32
from test_pages_gpu import fork, fork_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("keep", [0, 1, 5, 200])
def test_fork_ends_at_the_lists_first_negative_id(keep):
    # (2 x 200 forks: more than are counted at once)
    x = list(fork_case(200, 2, 100, 16, seed=2))
    ids = x[4]
    x[4] = ids[:keep]
    *want, refused = fork_reference(*x, 16)
    assert refused > 0
    for behind in ([-1], [-1] * 500, [-7] + ids[keep:]):
        x[4] = ids[:keep] + behind
        assert fork(*x, 16) == (*want, kda.KDA_DEVICE_NO_PAGES)


def test_fork_of_whole_pages_needs_no_list():
    table, lens, parents, children, free = fork_case(6, 2, 100, 16, seed=3)
    lens[:6] = [16, 0, 32, 16, 16, 32]
    want = fork_reference(table, lens, parents, children, [], 16)
    assert fork(table, lens, parents, children, [-1] * 4, 16) == (*want[:5], 0)


def test_fork_takes_all_that_the_list_has():
    x = list(fork_case(30, 2, 100, 16, seed=4))
    need = sum(x[1][p] % 16 != 0 for p in x[2])
    x[4] = x[4][:need]
    *want, refused = fork_reference(*x, 16)
    assert refused == 0
    x[4] = x[4] + [-1] * 3
    assert fork(*x, 16) == (*want, 0)


def nearly_full(seed, total, page, keep):
    """(table, lens): ten prompts, a row that holds all pages left but `keep`, one that ends, ten children to be."""
    r = random.Random(seed)
    lens = [r.randint(0, 9) * page + r.randint(1, page - 1) for _ in range(10)]
    ids = r.sample(range(total), total)
    rows = []
    for n in lens:
        rows.append([ids.pop() for _ in range(-(-n // page))])
    ended = [ids.pop() for _ in range(keep)]
    lens += [page * len(ids), page * keep]
    rows += [ids, ended]
    table = [x + [-3] * (total - len(x)) for x in rows] + [[-3] * total for _ in range(10)]
    return table, lens + [0] * 10


def test_release_then_fork_in_a_nearly_full_cache():
    """The whole list from call to call, its length read by no host: eager, and replayed."""
    page, total = 16, 150
    parents, children = list(range(10)), list(range(12, 22))
    t, n = nearly_full(1, total, page, 3)
    table, lens, ws = i32(t), i32(n), kda.make_workspace()
    cache = torch.randn((total, page, 1, D), device="cuda").bfloat16()
    src, dst, used, count = i32([0] * 10), i32([0] * 10), i32([0]), i32([0])
    free, ends, d_parents, d_children = i32([0] * total), i32([11]), i32(parents), i32(children)

    def calls():
        kda.release_requests(table, lens, ends, page, free_pages=free, num_free=count, workspace=ws)
        kda.fork_requests(table, lens, d_parents, d_children, free, page, copy_src=src, copy_dst=dst, pages_used=used, workspace=ws)
        kda.copy_pages([cache], src, dst, workspace=ws)

    def check(t, n, keep):
        n = n[:11] + [0] + n[12:]
        want, num = free_reference(t, n, page, total)
        assert num == keep
        ft, fl, fs, fd, fu, refused = fork_reference(t, n, parents, children, want[:num], page)
        assert refused == 10 - keep
        assert (table.tolist(), lens.tolist(), src.tolist(), dst.tolist(), int(used)) == (ft, fl, fs, fd, fu)
        assert kda.read_device_status(ws) == (kda.KDA_DEVICE_NO_PAGES if refused else 0)

    calls()
    check(t, n, 3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for seed, keep in ((2, 7), (3, 0), (4, 1)):
        t, n = nearly_full(seed, total, page, keep)
        table.copy_(i32(t))
        lens.copy_(i32(n))
        graph.replay()
        torch.cuda.synchronize()
        check(t, n, keep)
