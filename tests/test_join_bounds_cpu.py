"""Rows that say where the parts of a cut item lie: whatever they say, as after a kernel that gave up, no part lies outside the
workspace; and what a kernel can say is taken."""
import os
import subprocess

from kda_linear_attention_bounded_gb300 import build as kbuild

PROGRAM = """
#include <climits>
#include <cstdio>
#include "kda_hybrid.h"
#include "kda.h"
using namespace kda;
int main() {
  long long bad = 0, taken = 0;
  const auto look = [&](int parts, int cut) {
    if (!paged_parts_there(parts, cut)) return;
    ++taken;
    for (int n = 0; n < parts; ++n) bad += paged_part_slot(cut, n) < 0 || paged_part_slot(cut, n) >= 2 * kPagedMaxCtas;
  };
  for (int parts = -600; parts <= 600; ++parts)
    for (int cut = -600; cut <= 600; ++cut) look(parts, cut);
  const unsigned edges[] = {0u, 1u, 2u, 0x7fffffffu, 0x80000000u, 0xffffffffu, 0x7f800000u, 0xff800000u, 0x3f800000u, 0x40000000u,
                            0x7ffffffeu, 0x80000001u, 0x7fffff00u, 0x80000100u};
  for (unsigned a : edges)
    for (unsigned b : edges) look(static_cast<int>(a), static_cast<int>(b));
  for (int s = 1; s < kPagedMaxCtas; ++s)            // an item cut at the beginning of stretch s, over n stretches from there on
    for (int n = 1; s + n <= kPagedMaxCtas; ++n) bad += !paged_parts_there(n + 1, s);
  std::printf("%lld %lld\\n", bad, taken);
}
"""


def test_parts_lie_in_the_workspace(tmp_path):
    (tmp_path / "main.cpp").write_text(PROGRAM)
    cuda = os.path.dirname(os.path.dirname(kbuild._nvcc())) or "/usr/local/cuda"
    subprocess.run(["g++", "-std=c++17", "-O1", f"-I{kbuild.CSRC}", f"-I{kbuild.INCLUDE}", f"-I{cuda}/include", str(tmp_path / "main.cpp"),
                    "-o", str(tmp_path / "main")], check=True)
    bad, taken = map(int, subprocess.run([str(tmp_path / "main")], capture_output=True, text=True, check=True).stdout.split())
    assert bad == 0 and taken >= 303 * 304 // 2
    with open(f"{kbuild.CSRC}/kda_prefix_attention.cu") as f:   # the join asks before it follows a row's words
        text = f.read()
    assert "paged_parts_there(__float_as_int(end.z), cut) ?" in text
