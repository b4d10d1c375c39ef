"""The hand-offs between the warp roles of the block-attention cache kernel, run on the host (CPU only).

csrc/role_waits.h is plain C++; a small program gives it copies, barriers and a clock of its own, some
of which never complete, and the tests read what it did.
"""

import os
import re
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


def test_roles_end_after_the_same_segments(tmp_path):
    # a publisher and four roles in any order of steps; at each step a role whose segment is not there
    # may give up.  No role takes a segment that was not published, and all end at the same one.
    lines = _run(tmp_path, r"""
#include <random>
int main() {
  std::mt19937 rng(1);
  int early = 0, whole = 0;
  for (int trial = 0; trial < 20000; ++trial) {
    uint32_t gate = 1;              // segment 0 is published from the start
    const int segments = 1 + rng() % 6;
    const int impatience = 2 + rng() % 60;
    int next = 1, at[4] = {}, ended[4] = {};
    bool closed_seen = false;
    auto cas = [&](uint32_t was, uint32_t is) {
      const uint32_t old = gate;
      if (old == was) gate = is;
      return old;
    };
    std::vector<char> left(64, 0);  // whether the segment has pages: what a publisher writes first
    left[0] = 1;
    int published = 1;
    for (int step = 0; step < 4000; ++step) {
      const int who = rng() % 5;
      if (who == 4) {  // publishes the segments, then the end; a closed gate ends it too
        if (next <= segments && !closed_seen) {
          left[next] = next < segments;
          if (gate_publish(cas, next)) published = next + 1;
          else closed_seen = true;
          ++next;
        }
        continue;
      }
      if (ended[who]) continue;
      const int k = at[who];
      const bool complete = published > k;
      if (!complete && rng() % impatience != 0) continue;
      if (!complete) gate |= kGateClosed;
      if (gate_open(gate, k) && !complete) return 1;  // would take what is not there
      if (gate_open(gate, k) && left[k]) at[who] = k + 1;
      else ended[who] = 1;
    }
    for (int r = 0; r < 4; ++r)
      if (!ended[r] || at[r] != at[0]) return 2;
    at[0] < segments ? ++early : ++whole;
  }
  printf("%d %d\n", early > 1000, whole > 1000);
}
""")
    assert lines == ["1 1"]


def test_a_wait_for_a_long_segment_lasts_while_pages_are_issued(tmp_path):
    # made-up time, 1 ms a look at the clock: pages issued every 3 s keep a wait of 60 s alive, none
    # for 4 s ends it
    lines = _run(tmp_path, r"""
int main() {
  for (int every : {3, 5}) {
    uint64_t t = 0;
    long polls = 0;
    const bool done = wait_progress([&] { ++polls; return t >= 60000000000ull; },
                                    [&] { return (int)(t / (every * 1000000000ull)); },
                                    [&] { return t += 1000000; });
    printf("%d %llu\n", (int)done, (unsigned long long)(t / 1000000000ull));
  }
  int looks = 0;
  printf("%d\n", (int)wait_progress([] { return true; }, [&] { return ++looks; }, [&] { return (uint64_t)++looks; }));
  printf("%d\n", looks);
}
""")
    assert lines == ["1 60", "0 4", "1", "0"]


def test_a_phase_left_behind_does_not_pass_for_a_page(tmp_path):
    # one stage's barrier of two arrivals a page (the MMAs' completion and the issuing thread's).  The
    # completion of the stage's first page never comes; the pages are then issued one by one after the
    # abort, and a wait for a page may not end before that page is issued, though the barrier's parity
    # reads as complete a page early.
    lines = _run(tmp_path, r"""
int main() {
  int arrivals = 0, issued = 0, misread = 0;
  auto phase = [&] { return arrivals / 2; };
  for (int page = 0; page < 6; ++page) {
    // the wait of a role that is a page ahead of the MMA warp: the page is issued after 1000 looks
    int looks = 0, ended_at = -1;
    auto issue = [&] {
      arrivals += page == 0 ? 1 : 2;  // the first completion is lost
      ++issued;
    };
    wait_page(
        [&] {
          if (++looks == 1000) issue();
          const bool complete = (phase() & 1) != (page & 1);
          if (complete && issued <= page) ++misread;
          return complete;
        },
        [&] { return issued > page; }, [] { return true; }, [] {}, [] { return (uint64_t)1; });
    ended_at = looks;
    printf("%d %d\n", issued, (int)(ended_at >= 1000));
  }
  printf("%d\n", (int)(misread > 0));
}
""")
    # the model does meet a barrier that reads as complete too early
    assert lines == ["%d 1" % (i + 1) for i in range(6)] + ["1"]


def test_a_wait_for_a_page_runs_out_after_two_seconds(tmp_path):
    # by the clock, however quick or slow a poll is: made-up time that a poll moves by 1 ns or 1 ms
    lines = _run(tmp_path, r"""
int main() {
  for (uint64_t step : {40ull, 1000000ull}) {
    for (int mode = 0; mode < 4; ++mode) {  // MMAs not issued; issued; a copy; issued by another's abort
      uint64_t t = 1, aborted_at = 0;
      bool aborted = mode == 3;
      wait_page([&] { t += step; return false; }, [&] { return mode != 0; }, [&] { return aborted; },
                [&] { if (!aborted) aborted_at = t; aborted = true; }, [&] { return t; });
      printf("%.1f %.1f\n", aborted_at / 1e9, t / 1e9);
    }
  }
  // a page that completes is not reported, and the clock is not read for a quick one
  int looks = 0, clocks = 0;
  bool aborted = false;
  wait_page([&] { return ++looks == 200; }, [] { return true; }, [&] { return aborted; }, [&] { aborted = true; },
            [&] { return (uint64_t)++clocks; });
  printf("%d %d %d\n", looks, clocks, (int)aborted);
}
""")
    # the first look at the clock is after 256 polls (0.26 s of the slow ones)
    assert lines[:4] == ["2.0 10.0", "2.0 2.0", "2.0 2.0", "0.0 0.0"]
    assert lines[4:8] == ["2.3 10.5", "2.3 2.3", "2.3 2.3", "0.0 0.3"]
    assert lines[8] == "200 0 0"


def test_named_barriers_take_converged_warps():
    # the aligned barriers are reached through three wrappers only; a warp's threads meet after every
    # poll and every elected section, and none leaves an elected section for a barrier of its own
    with open(os.path.join(CSRC, "block_attention.cu")) as fh:
        text = re.sub(r"//.*", "", fh.read())
    assert len(re.findall(r'"[^"]*\bbar(?:rier)?\.[^"]*"', text)) == 3
    assert not re.search(r"elect_one\(\)\s*\)\s*(continue|return|break)", text)
    kernel = text[text.index("block_cache_kernel(BlockParams"):text.index("block_raw_kernel(BlockParams")]
    loader = kernel[kernel.index("if (warp == kLoadWarp)"):kernel.index("} else if (warp >= kQueryWarp)")]
    roles = kernel[kernel.index("auto segment ="):].replace(loader, "")  # the loader is one thread
    lines = [line.strip() for line in roles.split("\n") if line.strip()]
    polls = [i for i, line in enumerate(lines) if re.search(r"\b(wait|wait_qk|wait_pv|wait_segment|mbar_wait)\(", line)]
    assert len(polls) >= 8
    for i in polls:
        rest = lines[i + 1:]
        while re.search(r"\b(wait|wait_qk|wait_pv)\(", rest[0]):  # polls of other warps of the role
            rest = rest[1:]
        assert rest[0] == "__syncwarp();", (lines[i], rest[0])
    assert loader.rstrip().endswith("__syncwarp();")
    for m in re.finditer(r"if \(elect_one\(\)\)", roles):
        after = roles[m.start():]
        depth, at = 0, after.index(")") + 2
        while True:  # the end of the elected statement
            depth += {"{": 1, "}": -1}.get(after[at], 0)
            if (after[at] == "}" or after[at] == ";") and depth == 0:
                break
            at += 1
        assert after[at + 1:].strip().startswith("__syncwarp();")
