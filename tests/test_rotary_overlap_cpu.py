"""Key and value rows of rotary_to_pages that meet, of one tensor or of both: what the host's search finds against going through all
rows, and what the call refuses (fake, aligned addresses; a refused call launches and reads nothing)."""
import itertools
import random
import subprocess

import pytest

from kda_linear_attention_bounded_gb300 import build as kbuild
from test_cache_cpu import _rotary, addresses, lib  # noqa: F401

PROGRAM = """
#include <cstdio>
#include "kda_layout.h"
int main() {
  long long x[10];
  while (true) {
    for (int i = 0; i < 10; ++i)
      if (std::scanf("%lld", x + i) != 1) return 0;
    const int P = (int)x[7], T = (int)x[8], H = (int)x[9];
    const uint16_t *at = (const uint16_t *)(1ll << 46);
    const kda::Pages k = {at, x[1], x[2], x[3]}, v = {(const uint16_t *)((1ll << 46) + 2 * x[0]), x[4], x[5], x[6]};
    std::printf("%d", kda::rows_apart(k, P, T, H) && kda::rows_apart(v, P, T, H) && !kda::pages_meet(k, v, P, T, H));
  }
}
"""


@pytest.fixture(scope="module")
def apart(tmp_path_factory):
    """apart([(offset of the values behind the keys, key strides, value strides, sizes), ..]): what the search says of each."""
    at = tmp_path_factory.mktemp("layout")
    (at / "main.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", f"-I{kbuild.CSRC}", str(at / "main.cpp"), "-o", str(at / "main")], check=True)

    def ask(cases):
        text = "\n".join(" ".join(map(str, (off, *kp, *vp, *sizes))) for off, kp, vp, sizes in cases)
        done = subprocess.run([str(at / "main")], input=text, capture_output=True, text=True, check=True, timeout=60)
        assert len(done.stdout) == len(cases)
        return [c == "1" for c in done.stdout]

    return ask


def meets(off, kp, vp, sizes):
    """By going through all rows."""
    every = [at + sum(s * i for s, i in zip(strides, x)) for at, strides in ((0, kp), (off, vp))
             for x in itertools.product(*map(range, sizes))]
    every.sort()
    return any(b - a < 128 for a, b in zip(every, every[1:]))


# keys and values in one buffer, apart: (offset, key strides, value strides), for 6 pages of 8 tokens and 2 heads
P, T, H = 6, 8, 2
LAYOUTS = {
    "one behind the other": (P * T * H * 128, (T * H * 128, H * 128, 128), (T * H * 128, H * 128, 128)),
    "by page": (T * H * 128, (2 * T * H * 128, H * 128, 128), (2 * T * H * 128, H * 128, 128)),
    "by token": (H * 128, (2 * T * H * 128, 2 * H * 128, 128), (2 * T * H * 128, 2 * H * 128, 128)),
    "by head": (128, (2 * T * H * 128, 2 * H * 128, 256), (2 * T * H * 128, 2 * H * 128, 256)),
    "values heads first": (T * H * 128, (2 * T * H * 128, H * 128, 128), (2 * T * H * 128, 128, T * 128)),
    "layers by page, values before": (-3 * T * H * 128, (8 * T * H * 128, H * 128, 128), (8 * T * H * 128, H * 128, 128)),
    "rows with room between": (136, (T * H * 280, H * 280, 280), (T * H * 280, H * 280, 280)),
    "heads outermost": (P * T * 128, (T * 128, 128, 2 * P * T * 128), (T * 128, 128, 2 * P * T * 128)),
    "strides that do not nest": (7 * 128, (14 * T * 128, 14 * 128, 3 * 128), (14 * T * 128, 14 * 128, 3 * 128)),
}


@pytest.mark.parametrize("name", LAYOUTS)
def test_layouts(lib, apart, name):  # noqa: F811
    off, kp, vp = LAYOUTS[name]
    assert not meets(off, kp, vp, (P, T, H)) and apart([(off, kp, vp, (P, T, H))]) == [True]
    # values moved onto keys, by heads, tokens, pages or a part of a row: refused by the call, too
    a = addresses(10)
    for to in (0, kp[2], -kp[2], kp[1], -kp[1], kp[0], (P - 1) * kp[0], kp[0] + kp[1] - kp[2], 120, -8):
        assert meets(to, kp, vp, (P, T, H)) and apart([(to, kp, vp, (P, T, H))]) == [False]
        assert _rotary(lib, kp=kp, vp=vp, pages=P, page=T, v_pages=a[6] + 2 * to) == 1, to


def test_rows_of_one_tensor(lib, apart):  # noqa: F811
    far, good = 1 << 22, (2048, 256, 128)
    for strides in ((128, 128, 128), (2048, 256, 256), (2048, 128, 128), (1024, 256, 128), (256, 2048, 1024), (2040, 256, 128), (2048, 256, 136)):
        for kp, vp in ((strides, good), (good, strides)):
            assert meets(far, kp, vp, (P, T, H)) and apart([(far, kp, vp, (P, T, H))]) == [False]
            assert _rotary(lib, kp=kp, vp=vp, pages=P, page=T) == 1, (kp, vp)
    for strides in (good, (2048, 128, 1024), (128, 6 * 256, 6 * 128), (2112, 264, 136), (1 << 18, 384, 256 * 3 * 8)):
        assert not meets(far, strides, strides, (P, T, H)) and apart([(far, strides, good, (P, T, H))]) == [True], strides
    # one page, token or head alone may have any stride
    assert apart([(far, (0, 256, 128), (8, 256, 128), (1, T, H)), (far, (T * 128, 128, 0), (T * 128, 128, 8), (P, T, 1)),
                  (far, (128, 0, 0), (128, 8, 8), (P, 1, 1))]) == [True] * 3
    # a place behind all memory
    assert _rotary(lib, kp=(1 << 62, 256, 128)) == 1


def test_random_layouts(apart):
    r = random.Random(1)
    cases = []
    for _ in range(6000):
        sizes = (r.randint(1, 4), r.randint(1, 5), r.randint(1, 3))
        unit = lambda: 128 * r.randint(1, 14) + r.choice([0, 0, 0, 8, 64])  # noqa: E731
        kp, vp = (unit() * r.choice([1, 4]), unit(), unit()), (unit() * r.choice([1, 4]), unit(), unit())
        if r.random() < 0.7:
            vp = kp
        cases.append((r.choice([1, -1]) * r.choice([0, 128, 136, 256, 1000, r.randint(0, 900) * 8]), kp, vp, sizes))
    want = [not meets(*c) for c in cases]
    assert apart(cases) == want
    assert 600 < sum(want) < 5400


def test_large_caches(apart):
    """A search that goes through pages, tokens or heads one by one would not come back."""
    n, many = 1 << 24, 2 ** 31 - 1
    assert apart([(256, (2 ** 12, 512, 128), (2 ** 12, 512, 128), (n, 8, 2)),
                  (n * 2 ** 11, (2 ** 11, 256, 128), (2 ** 11, 256, 128), (n, 8, 2)),
                  (2 ** 10, (2 ** 11, 128, 2 ** 35), (2 ** 11, 128, 2 ** 35), (n, 8, 4))]) == [True] * 3
    assert apart([(n // 2 * 2 ** 11, (2 ** 11, 256, 128), (2 ** 11, 256, 128), (n, 8, 2)),
                  (120, (2 ** 12, 512, 128), (2 ** 12, 512, 128), (n, 8, 2)),
                  (8, (128, 128, 128), (128, 128, 128), (many, many, 4096)),
                  (0, (136, 128, 144), (136, 152, 160), (many, 1 << 20, 4096))]) == [False] * 4


def test_no_pages(apart):
    assert apart([(0, (2048, 256, 128), (2048, 256, 128), (0, 8, 2)), (0, (2048, 256, 128), (2048, 256, 128), (1, 8, 2))]) == [True, False]
