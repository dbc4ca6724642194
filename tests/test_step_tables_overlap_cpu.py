"""Step tables refuse buffers that overlap (fake, aligned device addresses; never dereferenced)."""
import ctypes

import pytest

from kda_linear_attention_bounded_gb300 import build as kbuild

P = ctypes.c_void_p
B, WIDTH, STRIDE, FREE, ROWS = 4, 8, 10, 5, 7
SIZE = {"table": 4 * ((B - 1) * STRIDE + WIDTH), "old": 4 * B, "new": 4 * B, "free": 4 * FREE, "cu": 4 * (B + 1), "kv": 4 * B,
        "pos": 4 * ROWS, "slot": 8 * ROWS, "used": 4}
APART = {name: 0x10000000 + 0x1000 * i for i, name in enumerate(SIZE)}
WRITTEN = ("table", "cu", "kv", "pos", "slot", "used")


def call(*, stride=STRIDE, width=WIDTH, b=B, num_free=FREE, page=16, rows=ROWS, **at):
    from kda_linear_attention_bounded_gb300 import _binding
    kbuild.build()
    x = {**APART, **at}
    return _binding.load().kda_step_tables(P(x["table"]), stride, width, P(x["old"]), P(x["new"]), b, P(x["free"]), num_free, page,
                                           rows, P(x["cu"]), P(x["kv"]), P(x["pos"]), P(x["slot"]), P(x["used"]), P(0x20000000),
                                           1024, None)


def test_other_refusals_with_buffers_apart():
    for bad in (dict(table=None), dict(stride=7), dict(old=None), dict(new=None), dict(b=-1), dict(free=None), dict(num_free=-1),
                dict(page=0), dict(page=-16), dict(rows=-1), dict(rows=2 ** 31), dict(cu=None), dict(kv=None), dict(pos=None),
                dict(slot=None), dict(used=None), dict(width=-1), dict(table=APART["table"] + 2), dict(slot=APART["slot"] + 4),
                dict(cu=APART["cu"] + 1)):
        assert call(**bad) == 1, bad


@pytest.mark.parametrize("a", WRITTEN)
@pytest.mark.parametrize("b", SIZE)
def test_overlaps_are_refused(a, b):
    if a == b:
        return
    step = 8 if "slot" in (a, b) else 4
    last = (SIZE[b] - 1) // step * step   # the last place of b where a may begin
    first = (SIZE[a] - 1) // step * step  # and the other way round
    for at in ({a: APART[b]}, {a: APART[b] + last}, {b: APART[a] + first}):
        if (a, b) == ("kv", "old") and at[a if a in at else b] == APART[b if a in at else a]:
            continue                      # in place
        assert call(**at) == 1, at
    if (a, b) == ("kv", "old"):
        assert call(kv=APART["old"] + 4) == 1 and call(kv=APART["old"] - 4) == 1


def test_every_row_of_the_table_counts():
    # (what lies between the rows is tested where the call may run)
    for r in range(B):
        row = APART["table"] + 4 * STRIDE * r
        for at in (row, row + 4 * (WIDTH - 1), row - SIZE["cu"] + 4):
            assert call(cu=at) == 1, (r, at - row)
        assert call(new=row + 4) == 1 and call(used=row + 8) == 1
    assert call(slot=APART["table"] - SIZE["slot"] + 8) == 1
