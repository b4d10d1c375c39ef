"""The hand-offs between the warp roles of the block-attention cache kernel, run on the host (CPU only).

csrc/role_waits.h is plain C++; a small program gives it copies, barriers and a clock of its own, some
of which never complete, and the tests read what it did.
"""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "calibration_free_kv_gb300", "csrc")


def _run(tmp_path, body):
    """Lines printed by a program with this main."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no C++ compiler")
    src = tmp_path / "roles.cc"
    src.write_text('#include <stdio.h>\n#include <algorithm>\n#include <vector>\n#include "role_waits.h"\n'
                   "using namespace kvarn::blk;\n" + body)
    exe = tmp_path / "roles"
    r = subprocess.run([gxx, "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I", CSRC, str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, (r.returncode, r.stdout, r.stderr)
    return r.stdout.split("\n")[:-1]


def test_drain_waits_for_the_issued_copies(tmp_path):
    # a ring of 3 slots; the copies of the pages from `stop` on are not issued (the call was given up):
    # the drain waits for the last copies issued into each slot, at the phase that each completes
    lines = _run(tmp_path, r"""
int main() {
  for (int stop = 0; stop <= 8; ++stop) {
    CopyRing ring(3);
    std::vector<std::pair<int, unsigned>> issued;
    for (int page = 0; page < 8; ++page) {
      if (page >= stop) continue;
      issued.push_back({ring.slot, ring.phase});
      ring.next();
    }
    printf("%d:", stop);
    ring.drain([&](int slot, unsigned parity) {
      printf(" %d/%u", slot, parity);
      return true;
    });
    printf(" |");
    for (size_t i = issued.size() > 3 ? issued.size() - 3 : 0; i < issued.size(); ++i)
      printf(" %d/%u", issued[i].first, issued[i].second);
    printf("\n");
  }
}
""")
    assert len(lines) == 9
    for stop, line in enumerate(lines):
        got, want = line.split(":")[1].split("|")
        assert got.split() == want.split() and len(got.split()) == min(stop, 3)
    assert lines[5] == "5: 2/0 0/1 1/1 | 2/0 0/1 1/1"


def test_drain_reports_a_copy_that_did_not_land(tmp_path):
    # every copy is waited for all the same
    lines = _run(tmp_path, r"""
int main() {
  for (int lost = -1; lost < 4; ++lost) {
    CopyRing ring(4);
    for (int i = 0; i < 6; ++i) ring.next();
    int waits = 0;
    const bool all = ring.drain([&](int slot, unsigned) {
      ++waits;
      return slot != lost;
    });
    printf("%d %d\n", (int)all, waits);
  }
}
""")
    assert lines == ["1 4"] + ["0 4"] * 4
