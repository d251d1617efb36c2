"""The tree forward's ring of tiles, its header compiled for the host: every entry is
loaded once, each loader's in order, and wherever a loader stops, the copies that
it waits for are all that can be on their way."""
import os
import shutil
import subprocess

import pytest

from packed_varlen_non_gb300 import build

PROGRAM = r"""
#include <cstdio>
#include "tree_ring.h"
using namespace h3::ring;
template <bool kTwo> void list(int me, int first, int copies, int steps) {
  std::printf("%d %d %d %d", kTwo ? 1 : 0, me, first, steps);
  for (int c = 0; c < copies; ++c) std::printf(" %u", copy_entry<kTwo>(c, me, first, steps));
  std::printf("\n");
}
int main() {
  std::printf("%d", kSlots);
  for (int n = 0; n < 100; ++n) std::printf(" %d", first_on_its_way(n));
  std::printf("\n");
  for (int steps = 1; steps < 40; ++steps) {
    for (int me = 0; me < 2; ++me) list<false>(me, me, steps, steps);
    for (int lead = 0; lead < 2; ++lead)  // the stream that begins has the odd tile
      for (int me = 0; me < 2; ++me) {
        const int first = me ^ lead;
        list<true>(me, first, 2 * ((steps + 1 - first) / 2), steps);
      }
  }
}
"""


@pytest.fixture(scope="module")
def lines(tmp_path_factory):
    d = tmp_path_factory.mktemp("ring")
    (d / "ring.cpp").write_text(PROGRAM)
    exe = str(d / "ring")
    subprocess.run([shutil.which("g++") or "g++", "-std=c++17", "-Wall", "-Werror", "-I" + build.CSRC, str(d / "ring.cpp"), "-o", exe],
                   check=True)
    out = subprocess.run([exe], check=True, capture_output=True, text=True).stdout
    return [[int(x) for x in line.split()] for line in out.splitlines()]


def test_every_entry_is_loaded_once_and_in_order(lines):
    loads = {}
    for two, me, first, steps, *entries in lines[1:]:
        assert entries == sorted(set(entries))
        key = (two, steps, me ^ first if two else 0)
        loads.setdefault(key, []).extend(entries)
    assert len(loads) == 39 * 3
    for (two, steps, _), entries in loads.items():
        assert sorted(entries) == list(range(2 * steps))


def test_a_loader_that_stops_waits_for_all_that_is_on_its_way(lines):
    slots, *first = lines[0]
    for two, me, start, steps, *entries in lines[1:]:
        for issued in range(1, len(entries) + 1):
            # its last copy went out when the entry `slots` before it had been used, and those before that one
            late = [c for c in range(issued) if entries[c] > entries[issued - 1] - slots]
            assert late[0] >= first[issued] and late[-1] == issued - 1
            assert issued - first[issued] <= 3
    assert first[0] == 0


def test_the_header_is_part_of_the_build():
    assert "tree_ring.h" in build.HEADERS and os.path.exists(os.path.join(build.CSRC, "tree_ring.h"))
