"""The end of a ring's producer on the CPU (csrc/ring_landing.h, which the layers' kernels
include): with fake barriers, for every point at which a role may give up, all loads
that the unit's CTAs issued are waited for before its CTAs can leave."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dlrm_embedding_bag_b200", "csrc")

MODEL = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "ring_landing.h"

static int checks = 0;
#define CHECK(c) \
  do { \
    ++checks; \
    if (!(c)) { std::printf("line %d: %s\n", __LINE__, #c); std::exit(1); } \
  } while (0)

// The barriers of a unit's ring: phase i / STAGES of stage i % STAGES belongs to step i.
template <int STAGES>
struct Ring {
  std::vector<int> armed, landed_by_wait;  // by step
  int phase[STAGES] = {};                  // armed so far
  explicit Ring(int n) : armed(n + 2 * STAGES), landed_by_wait(n + 2 * STAGES) {}
  void arm(int s) { armed[phase[s]++ * STAGES + s] = 1; }
  void wait(int s, int parity) {
    // the wait is for the last armed phase, whose parity it has to be given: with the
    // other one it would return at once
    CHECK(phase[s] > 0);
    const int step = (phase[s] - 1) * STAGES + s;
    CHECK(parity == ((phase[s] - 1) & 1));
    landed_by_wait[step] = 1;
  }
};

// One CTA: `issued` steps; the products read `read` of them before something gave up.
template <int STAGES>
void one_cta(int issued, int read, bool gave_up) {
  Ring<STAGES> r(issued);
  for (int i = 0; i < issued; ++i) r.arm(i % STAGES);
  dlrm::land_loads<STAGES, false>(
      true, gave_up, issued, [&](int s, int p) { r.wait(s, p); }, [&](int) { CHECK(false); },
      [&](int) { CHECK(false); }, [&]() -> int { CHECK(false); return 0; });
  for (int i = read; i < issued; ++i) CHECK(r.landed_by_wait[i]);
}

// A pair: the leader armed and issued `a` steps, the other issued `b`, the products read
// `read`. When the other's number comes too late (late), at least the leader's own land.
template <int STAGES>
void pair(int a, int b, int read, bool gave_up, bool late) {
  Ring<STAGES> r(a > b ? a : b);
  for (int i = 0; i < a; ++i) r.arm(i % STAGES);
  int told = -1;
  dlrm::land_loads<STAGES, true>(
      false, false, b, [&](int, int) { CHECK(false); }, [&](int) { CHECK(false); },
      [&](int n) { told = n; }, [&]() -> int { CHECK(false); return 0; });
  CHECK(told == b);
  dlrm::land_loads<STAGES, true>(
      true, gave_up, a, [&](int s, int p) { r.wait(s, p); }, [&](int s) { r.arm(s); },
      [&](int) { CHECK(false); }, [&]() -> int { CHECK(gave_up); return late ? -1 : told; });
  const int end = (a > b || late) ? a : b;
  for (int i = read; i < end; ++i) CHECK(r.landed_by_wait[i]);
  // and nothing was armed that no load was issued for
  for (int i = end; i < static_cast<int>(r.armed.size()); ++i) CHECK(!r.armed[i]);
}

template <int STAGES>
void all() {
  for (int issued = 0; issued <= 4 * STAGES; ++issued)
    for (int read = issued > STAGES ? issued - STAGES : 0; read <= issued; ++read)
      for (int gave_up = 0; gave_up < 2; ++gave_up) one_cta<STAGES>(issued, read, gave_up);
  for (int a = 0; a <= 4 * STAGES; ++a)
    for (int read = a > STAGES ? a - STAGES : 0; read <= a; ++read) {
      for (int b = read; b <= a; ++b) pair<STAGES>(a, b, read, true, false);
      pair<STAGES>(a, a, read, false, false);
      // the other went on while stages came free: its step i needs step i - STAGES read
      for (int b = a + 1; b <= read + STAGES; ++b) {
        pair<STAGES>(a, b, read, true, false);
        pair<STAGES>(a, b, read, true, true);
      }
    }
}

int main() {
  all<1>(); all<2>(); all<3>(); all<6>(); all<8>();
  std::printf("%d\n", checks);
}
"""


def test_all_loads_land_wherever_a_role_gives_up(tmp_path):
    src = tmp_path / "model.cpp"
    src.write_text(MODEL)
    exe = tmp_path / "model"
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, str(src), "-o",
                    str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    assert int(r.stdout) > 10000


@pytest.mark.parametrize("kernel,leader", [("tokens/linear_int8.cu", "!PAIR || rank == 0"),
                                           ("linear.cu", "rank == 0")])
def test_the_layers_producer_ends_so(kernel, leader):
    """Every producer calls it, whatever happened: not under a condition on a give-up."""
    src = open(os.path.join(CSRC, kernel)).read()
    body = src[src.index("if (warp == 0) {"):src.index("} else if (warp == 1) {")]
    call = body.index("land_loads<")
    # directly in the producer thread's block: two levels deep, behind the loop over tiles
    depth = body[:call].count("{") - body[:call].count("}")
    assert depth == 2
    assert re.search(r"\(\s*" + re.escape(leader) + r", timed_out, g,", body[call:])
    # ranks other than 0 without a pair: only where a cluster splits a tile along K
    assert ("SPLIT" in src) == ("!PAIR" in leader)
