"""Step tables on the GPU against a plain loop over requests and tokens (whole numbers: equal)."""
import random

import pytest
import torch

import kda_linear_attention_bounded_gb300 as kda

pytestmark = pytest.mark.gpu


def reference(table, old, new, free, page, rows):
    """What the call leaves behind, request by request: the status bits too."""
    table = [list(r) for r in table]
    width = len(table[0]) if table else 0
    cu, kv, pos, slot, status, needed, used = [0], [], [0] * rows, [-1] * rows, 0, 0, 0
    t = 0
    for r, (o, n) in enumerate(zip(old, new)):
        if o < 0 or n < 0:
            status |= kda.KDA_DEVICE_BAD_COUNT
            o, n = max(o, 0), 0
        had, has = -(-o // page), -(-(o + n) // page)
        refused = has > width
        if not refused and has > had:
            if needed + has - had > len(free):
                refused = True
            else:
                for j in range(has - had):
                    table[r][had + j] = free[needed + j]
                used = needed + has - had
            needed += has - had
        if refused:
            status |= kda.KDA_DEVICE_NO_PAGES
        kv.append(o if refused else o + n)
        for i in range(n):
            if t < rows:
                p = o + i
                pos[t] = p
                if not refused:
                    if table[r][p // page] < 0:
                        status |= kda.KDA_DEVICE_BAD_SLOT
                    else:
                        slot[t] = table[r][p // page] * page + p % page
            else:
                status |= kda.KDA_DEVICE_BAD_COUNT
            t += 1
        cu.append(t)
    return table, cu, kv, pos, slot, used, status


def run(table, old, new, free, page, rows, stride=None):
    i32 = lambda v, n=None: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    B, width = len(old), len(table[0]) if table else 4
    wide = torch.full((max(B, 1), stride or max(width, 1)), -9, dtype=torch.int32, device="cuda")
    d_table = wide[:B, :width]
    if B and width:
        d_table.copy_(i32(table))
    outs = {"cu_seqlens": torch.full((B + 1,), -7, dtype=torch.int32, device="cuda"),
            "kv_lens": torch.full((B,), -7, dtype=torch.int32, device="cuda"),
            "positions": torch.full((rows,), -7, dtype=torch.int32, device="cuda"),
            "slot_map": torch.full((rows,), -7, dtype=torch.int64, device="cuda"),
            "pages_used": torch.full((1,), -7, dtype=torch.int32, device="cuda")}
    ws = kda.make_workspace()
    kda.step_tables(d_table, i32(old), i32(new), i32(free), page, workspace=ws, **outs)
    status = kda.read_device_status(ws)
    assert stride is None or (wide[:, width:] == -9).all()
    return (d_table.tolist(), outs["cu_seqlens"].tolist(), outs["kv_lens"].tolist(), outs["positions"].tolist(),
            outs["slot_map"].tolist(), int(outs["pages_used"]), status)


def case(B, most_old, most_new, page, seed, spare=3, width=None):
    r = random.Random(seed)
    old = [r.randint(0, most_old) for _ in range(B)]
    new = [r.choice([0, 1, 1, r.randint(0, most_new)]) for _ in range(B)]
    width = width or max([-(-(o + n) // page) for o, n in zip(old, new)] + [1])
    had = [-(-o // page) for o in old]
    ids = list(range(sum(had) + sum(-(-(o + n) // page) for o, n in zip(old, new)) + spare))
    r.shuffle(ids)
    table, at = [], 0
    for h in had:
        h = min(h, width)
        table.append(ids[at:at + h] + [-1] * (width - h))
        at += h
    return table, old, new, ids[at:]


@pytest.mark.parametrize("B,most_old,most_new,page", [
    (1, 0, 1, 1), (1, 40, 50, 16), (7, 100, 30, 16), (64, 3000, 1, 16), (255, 50, 9, 5), (256, 64, 64, 64),
    (257, 200, 40, 48), (1025, 70, 12, 16), (2500, 30, 3, 4), (5, 500, 6000, 1), (3, 10, 4000, 256)])
def test_tables(B, most_old, most_new, page):
    table, old, new, free = case(B, most_old, most_new, page, seed=B)
    rows = sum(new) + 5
    assert run(table, old, new, free, page, rows) == reference(table, old, new, free, page, rows)


def test_strided_rows_are_kept():
    table, old, new, free = case(9, 90, 40, 16, seed=1)
    assert run(table, old, new, free, 16, sum(new), stride=len(table[0]) + 3) == \
        reference(table, old, new, free, 16, sum(new))


def test_nothing_new_and_no_requests():
    table, old, _, free = case(6, 90, 40, 16, seed=2)
    assert run(table, old, [0] * 6, free, 16, 4) == reference(table, old, [0] * 6, free, 16, 4)
    assert run([], [], [], [1], 16, 3)[1:] == ([0], [], [0] * 3, [-1] * 3, 0, 0)


def test_too_few_rows():
    table, old, new, free = case(9, 90, 40, 16, seed=3)
    got = run(table, old, new, free, 16, sum(new) - 11)
    assert got == reference(table, old, new, free, 16, sum(new) - 11)
    assert got[-1] == kda.KDA_DEVICE_BAD_COUNT


def test_free_list_used_up():
    table, old, new, free = case(300, 90, 40, 16, seed=4)
    for keep in (0, 1, 7, 40):
        got = run(table, old, new, free[:keep], 16, sum(new))
        assert got == reference(table, old, new, free[:keep], 16, sum(new))
        assert got[-1] == kda.KDA_DEVICE_NO_PAGES


def test_table_row_used_up():
    table, old, new, free = case(40, 90, 60, 16, seed=5, width=7)
    got = run(table, old, new, free, 16, sum(new))
    assert got == reference(table, old, new, free, 16, sum(new))
    assert got[-1] == kda.KDA_DEVICE_NO_PAGES


def test_bad_lengths_and_bad_pages():
    table, old, new, free = case(20, 90, 40, 16, seed=6)
    old[3], new[5] = -4, -1
    old[8], new[8] = 33, 2
    table[8][2] = -1   # the page that token 33 is in
    got = run(table, old, new, free, 16, sum(max(n, 0) for n in new))
    want = reference(table, old, new, free, 16, sum(max(n, 0) for n in new))
    assert got == want
    assert got[-1] == kda.KDA_DEVICE_BAD_COUNT | kda.KDA_DEVICE_BAD_SLOT


def test_lengths_beyond_int32():
    got = run([[0, -1], [1, -1]], [2 ** 31 - 1, 1], [1, 1], [5], 16, 4)
    assert got == ([[0, -1], [1, -1]], [0, 0, 1], [2 ** 31 - 1, 2], [1, 0, 0, 0], [17, -1, -1, -1], 0,
                   kda.KDA_DEVICE_BAD_COUNT | kda.KDA_DEVICE_NO_PAGES)


def test_same_inputs_again_in_a_graph():
    table, old, new, free = case(33, 200, 70, 16, seed=7)
    B, rows = 33, sum(new) + 2
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    d = [i32(table), i32(old), i32(new), i32(free)]
    outs = dict(cu_seqlens=i32([0] * (B + 1)), kv_lens=i32([0] * B), positions=i32([0] * rows),
                slot_map=torch.zeros(rows, dtype=torch.int64, device="cuda"), pages_used=i32([0]))
    ws = kda.make_workspace()
    kda.step_tables(*d, 16, workspace=ws, **outs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.step_tables(*d, 16, workspace=ws, **outs)
    table2, old2, new2, free2 = case(33, 150, 50, 16, seed=8, width=len(table[0]))
    new2 = [min(n, 2) for n in new2]
    for t, v in zip(d, (table2, old2, new2, free2)):
        t[tuple(slice(0, n) for n in torch.tensor(v).shape)] = i32(v)[:t.shape[0]] if t.dim() == 1 else i32(v)
    graph.replay()
    torch.cuda.synchronize()
    want = reference(table2, old2, new2, d[3].tolist(), 16, rows)
    got = (d[0].tolist(), outs["cu_seqlens"].tolist(), outs["kv_lens"].tolist(), outs["positions"].tolist(),
           outs["slot_map"].tolist(), int(outs["pages_used"]), kda.read_device_status(ws))
    assert got == want
