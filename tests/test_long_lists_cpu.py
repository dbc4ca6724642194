"""Lists so long that 32-bit places in them would wrap are refused on the host."""
import pytest

import test_step_tables_overlap_cpu as tables
from test_cache_cpu import FAKE, _copy, _fork, _prefix, lib  # noqa: F401

SPACE = 1 << 40   # (between any two of the fake addresses)


def places(*names):
    return {n: SPACE * (i + 1) for i, n in enumerate(names)}


@pytest.mark.parametrize("n", [2 ** 31 - 65536, 2 ** 31 - 4096, 2 ** 31 - 1])
def test_long_lists(lib, n):  # noqa: F811
    assert _fork(lib, forks=n, **places("table", "lens", "parents", "children", "free_pages", "src", "dst", "used")) == 1
    assert _release_rows(lib, n) == 1
    assert _copy(lib, count=n, src=SPACE, dst=2 * SPACE) == 1
    assert _prefix(lib, groups=n, ws_bytes=1 << 45) == 1
    assert tables.call(b=n, **places(*tables.SIZE)) == 1


def _release_rows(lib, n):  # noqa: F811
    import ctypes
    P = ctypes.c_void_p
    at = places("table", "lens", "rows", "free", "num")
    return lib.kda_release_requests(P(at["table"]), 8, 8, P(at["lens"]), 4, P(at["rows"]), n, 16, P(at["free"]), 9, P(at["num"]),
                                    P(FAKE), 1024, None)
