"""Step tables from free lists as release_requests leaves them: as long as the cache has pages, -1 behind the free ids."""
import pytest
import torch

import kda_linear_attention_bounded_gb300 as kda
from cache_refs import free_reference, i32
from test_step_tables_gpu import case, reference, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,most_old,most_new,page", [(300, 90, 40, 16), (7, 100, 30, 16), (1100, 60, 20, 4), (3, 10, 4000, 256)])
def test_list_ends_at_the_ids_behind_which_are_none(B, most_old, most_new, page):
    table, old, new, free = case(B, most_old, most_new, page, seed=B)
    for keep in (0, 1, 7, 40, len(free) - 4):
        keep = min(max(keep, 0), len(free))
        want = reference(table, old, new, free[:keep], page, sum(new) + 3)
        for behind in (1, 60, len(free)):
            assert run(table, old, new, free[:keep] + [-1] * behind, page, sum(new) + 3) == want, (keep, behind)


def test_release_then_step_in_a_nearly_full_cache():
    """Every step's list is release's whole one, its length read by no host: eager, and replayed."""
    page, total, B, width = 16, 20, 6, 12
    table, lens, ws = i32([[-3] * width] * B), i32([0] * B), kda.make_workspace()
    free, count, none = i32([0] * total), i32([0]), i32([-1])
    new = i32([0] * B)
    outs = dict(cu_seqlens=i32([0] * (B + 1)), kv_lens=i32([0] * B), positions=i32([0] * 400),
                slot_map=torch.zeros(400, dtype=torch.int64, device="cuda"), pages_used=i32([0]))

    def calls():
        kda.release_requests(table, lens, none, page, free_pages=free, num_free=count, workspace=ws)
        kda.step_tables(table, lens, new, free, page, workspace=ws, **outs)

    t, n, refused = [[-3] * width for _ in range(B)], [0] * B, 0
    graph = None
    for step in ([40, 3, 0, 17, 16, 90], [100, 0, 1, 0, 0, 70], [1, 15, 1, 17, 1, 1], [1] * 6, [17] * 6, [60, 60, 0, 0, 0, 1]):
        new.copy_(i32(step))
        if graph is None:
            calls()
            torch.cuda.synchronize()
        else:
            graph.replay()
            torch.cuda.synchronize()
        ids, num = free_reference(t, n, page, total)
        want = reference(t, n, step, ids[:num], page, 400)
        got = (table.tolist(), outs["cu_seqlens"].tolist(), outs["kv_lens"].tolist(), outs["positions"].tolist(),
               outs["slot_map"].tolist(), int(outs["pages_used"]))
        assert got == want[:6]
        assert int(count) == num
        refused |= want[6]
        t, n = want[0], want[2]
        lens.copy_(outs["kv_lens"])
        if graph is None:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                calls()
    assert refused == kda.KDA_DEVICE_NO_PAGES == kda.read_device_status(ws)
