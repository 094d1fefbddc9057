"""The shared memory of the linear attention's tensor-core pass, form by form, from its header on
the host: every barrier and word lies within what the launch asks for."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "chunk_wise_weight_gate_b200", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "linattn_smem.h"
using namespace ipttt::la;
template <int A, int C, bool S> void show() {
  using M = Smem<A, C, S>;
  std::printf("%d %d %d %d %d %d %d %d %d %d %d %d %d\n", A, C, (int)S, M::NS, M::at_ring, M::at_lo, M::at_f, M::at_tabs,
              M::at_bars, M::bars(M::NS), M::at_words, M::WORDS, M::BYTES);
}
int main() {
  show<64, 64, false>(); show<64, 64, true>(); show<64, 128, false>(); show<64, 128, true>();
  show<128, 64, false>(); show<128, 64, true>(); show<128, 128, false>(); show<128, 128, true>();
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no C++ compiler")
def test_every_form_stays_within_its_shared_memory(tmp_path):
    src, exe = tmp_path / "smem.cpp", tmp_path / "smem"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    rows = [list(map(int, r.split())) for r in subprocess.run([str(exe)], capture_output=True, text=True).stdout.splitlines()]
    assert len(rows) == 8
    for A, C, state, ns, ring, lo, f, tabs, bars, nbars, words, nwords, size in rows:
        tile = 2 * 128 * max(A, C)
        assert ring == (0 if state else 2 * tile)
        assert ns >= 3 and lo >= ring + ns * tile                            # the ring's tiles
        assert f >= lo + 2 * 128 * A * (2 if state else 1)                   # the scaled keys' lower halves
        assert tabs >= f + (0 if state else 2 * A * C)                       # the state's bf16 copy
        assert bars >= tabs + 2 * 4 * (128 + 129 + 32) and bars % 8 == 0     # two heads' tables of powers
        # two barriers a tile of the ring, and 19 that the roles share; then four words or more
        assert nbars >= 2 * ns + 19 and words >= bars + 8 * nbars and nwords >= 4
        assert size >= words + 4 * nwords
        assert size <= 227 * 1024
        # tiles and halves start where the 128-byte swizzle repeats
        assert all(x % 1024 == 0 for x in (ring, lo, f, tabs))
