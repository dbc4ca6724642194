"""Step tables with the lengths brought forward in place (kv_lens is seq_lens), and what may not overlap."""
import pytest
import torch

import kda_linear_attention_bounded_gb300 as kda
from test_step_tables_gpu import case, reference

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _outs(B, rows):
    return dict(cu_seqlens=torch.empty(B + 1, dtype=torch.int32, device="cuda"),
                positions=torch.empty(rows, dtype=torch.int32, device="cuda"),
                slot_map=torch.empty(rows, dtype=torch.int64, device="cuda"),
                pages_used=torch.empty(1, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("B,most_old,most_new,page", [(1, 40, 50, 16), (64, 3000, 1, 16), (512, 900, 2000, 16),
                                                      (1025, 70, 12, 16), (5, 500, 6000, 1)])
def test_lengths_in_place(B, most_old, most_new, page):
    table, old, new, free = case(B, most_old, most_new, page, seed=B)
    rows = sum(new) + 5
    want = reference(table, old, new, free, page, rows)
    d_table, lens, o, ws = _i32(table), _i32(old), _outs(B, rows), kda.make_workspace()
    kda.step_tables(d_table, lens, _i32(new), _i32(free), page, kv_lens=lens, workspace=ws, **o)
    got = (d_table.tolist(), o["cu_seqlens"].tolist(), lens.tolist(), o["positions"].tolist(), o["slot_map"].tolist(),
           int(o["pages_used"]), kda.read_device_status(ws))
    assert got == want


def test_steps_replayed_in_place():
    # a captured step, replayed: the lengths move on by themselves (every request's pages are there already)
    B, page, width = 70, 16, 12
    table = torch.arange(B * width, dtype=torch.int32, device="cuda").view(B, width)
    first = [r % 100 + 16 * (r % 3) for r in range(B)]
    lens, ones, o, ws = _i32(first), torch.ones(B, dtype=torch.int32, device="cuda"), _outs(B, B), kda.make_workspace()
    free = torch.arange(B * width, B * width + B, dtype=torch.int32, device="cuda")

    def step():
        kda.step_tables(table, lens, ones, free, page, kv_lens=lens, workspace=ws, **o)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    for i in range(1, 5):
        graph.replay()
        torch.cuda.synchronize()
        assert lens.tolist() == [n + 1 + i for n in first] and o["positions"].tolist() == [n + i for n in first]
    assert kda.read_device_status(ws) == 0


def test_overlapping_buffers_are_refused():
    o = _outs(3, 9)
    lens, new, free, table = _i32([5, 0, 7]), _i32([1, 2, 0]), _i32([0, 1, 2, 3]), _i32([[4, 5]] * 3)
    kv = torch.empty(3, dtype=torch.int32, device="cuda")
    wide = torch.zeros(8, dtype=torch.int32, device="cuda")
    for args in (dict(kv_lens=new), dict(kv_lens=wide[:3], cu_seqlens=wide[2:6]), dict(kv_lens=kv, pages_used=free[2:3]),
                 dict(kv_lens=table.view(-1)[:3])):
        with pytest.raises(kda.KdaError):
            kda.step_tables(table, lens, new, free, 16, **{**o, **args})


def test_what_lies_between_the_tables_rows():
    # the lengths, their sums and the count in the gaps of a table with wide rows
    table, old, new, free = case(6, 90, 40, 16, seed=7)
    width, rows = len(table[0]), sum(new) + 3
    want = reference(table, old, new, free, 16, rows)
    room = torch.full((6, width + 8), -9, dtype=torch.int32, device="cuda")
    room[:, :width] = _i32(table)
    gap = lambda r, n: room[r, width:width + n]  # noqa: E731
    lens, kv, cu, used, fresh = gap(0, 6), gap(1, 6), gap(2, 7), gap(5, 1), gap(3, 6)
    lens.copy_(_i32(old))
    fresh.copy_(_i32(new))
    o, ws = _outs(6, rows), kda.make_workspace()
    o.update(cu_seqlens=cu, pages_used=used)
    kda.step_tables(room[:, :width], lens, fresh, _i32(free), 16, kv_lens=kv, workspace=ws, **o)
    got = (room[:, :width].tolist(), cu.tolist(), kv.tolist(), o["positions"].tolist(), o["slot_map"].tolist(), int(used),
           kda.read_device_status(ws))
    assert got == want
