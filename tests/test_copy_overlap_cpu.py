"""Buffers of copy_pages that meet are refused on the host; buffers that lie between one another's pages are taken.  (Fake, aligned
addresses; without entries to copy an accepted call launches nothing.)"""
import itertools
import random
import time

import pytest

from test_cache_cpu import _copy, lib  # noqa: F401


def refused(lib, buffers, pages):
    far = 1 << 44   # (the lists and the workspace, behind all buffers)
    rc = _copy(lib, buffers=buffers, pages=pages, count=0, src=far, dst=far + 4096, ws=far + 8192)
    assert rc in (0, 1)
    return rc == 1


def meet(buffers, pages):
    """By going through all pages."""
    spans = sorted((at + i * stride, at + i * stride + n) for at, stride, n in buffers if n for i in range(pages))
    return any(b[0] < a[1] for a, b in itertools.pairwise(spans))


def layers(count, each, pages, order):
    """count buffers of one tensor [pages, count, each bytes]."""
    x = [(i * each, count * each, each) for i in range(count)]
    return [x[i] for i in order]


@pytest.mark.parametrize("count,pages", [(2, 1), (2, 6), (7, 3), (300, 5)])
def test_buffers_apart(lib, count, pages):  # noqa: F811
    r = random.Random(count)
    behind = [(i * 512 * pages, 512, 512) for i in range(count)]
    among = layers(count, 512, pages, range(count))
    for x in (behind, among):
        for order in (x, x[::-1], r.sample(x, count), x + [(0, 0, 0), (512, 512, 0)]):
            assert not refused(lib, order, pages)
        for bad in (x + [x[-1]], [x[1]] + x, x[::-1] + [(x[0][0] + 16, x[0][1], 512)]):
            assert meet(bad, pages) and refused(lib, bad, pages)
    # both kinds, and pages of other strides among them
    mixed = among + [(512 * count * pages + at, s, n) for at, s, n in behind]
    assert not refused(lib, r.sample(mixed, 2 * count), pages)
    assert refused(lib, mixed + [(512 * count * pages - 16, 32, 32)], pages)


def test_other_strides(lib):  # noqa: F811
    for x, pages, want in (([(0, 64, 16), (16, 128, 16)], 9, False), ([(0, 64, 16), (16, 112, 16)], 3, True), ([(0, 64, 16), (16, 112, 16)], 2, False),
                           ([(0, 4096, 512), (512, 512, 512)], 7, False), ([(0, 4096, 512), (512, 512, 512)], 8, True),
                           ([(4096, 64, 64), (0, 1024, 32), (512, 1024, 32)], 4, False)):
        assert meet(x, pages) == want and refused(lib, x, pages) == want and refused(lib, x[::-1], pages) == want


def test_random(lib):  # noqa: F811
    r = random.Random(2)
    found = [0, 0]
    for _ in range(4000):
        pages, base = r.randint(1, 6), 16 * r.randint(1, 12)
        x = []
        for _ in range(r.randint(2, 5)):
            n = 16 * r.randint(0, 3)
            x.append((16 * r.randint(0, 60), base if r.random() < 0.7 and base >= n else max(n, 16 * r.randint(1, 12)), n))
        want = meet(x, pages)
        found[want] += 1
        assert refused(lib, x, pages) == want, (x, pages)
    assert min(found) > 500


def test_many_pages(lib):  # noqa: F811
    pages = 1 << 22
    t = time.time()
    assert not refused(lib, layers(256, 4096, pages, range(256)), pages)
    assert refused(lib, layers(256, 4096, pages, range(256)) + [(4096 * 255, 4096 * 256, 16)], pages)
    assert not refused(lib, [(0, 2 ** 14, 2 ** 13), (2 ** 13, 2 ** 15, 2 ** 13)], pages)
    assert time.time() - t < 20   # (not page by page for each pair)
