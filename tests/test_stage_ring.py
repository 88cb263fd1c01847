"""csrc/stage_ring.h on the host: a producer that leaves early waits for
exactly the fills that may be in flight.  Every state of a ring that the
protocol reaches (fills read by the consumer, fills armed), and every
subset of the unread fills still in flight, against a model of the stages'
barriers (a wait for a parity passes iff the barrier's current phase has
the other one)."""

import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_128_gb300", "csrc")

MODEL = r"""
#include <cstdio>
#include <vector>
#include "stage_ring.h"

int main() {
  long states = 0;
  for (int n = 1; n <= 8; ++n)
    for (int read = 0; read <= 3 * n; ++read)
      for (int armed = read; armed <= read + n; ++armed)
        for (int mask = 0; mask < 1 << (armed - read); ++mask) {
          // fill i of the ring has landed iff i < read or its bit is set
          std::vector<int> phases(n, 0);  // completed phases of each stage's barrier
          std::vector<bool> flying(armed, false);
          for (int i = 0; i < armed; ++i) {
            flying[i] = i >= read && !(mask >> (i - read) & 1);
            if (!flying[i]) ++phases[i % n];
          }
          int waits = 0;
          bool good = true;
          pagedkv::fills_in_flight(armed, n, [&](int stage, int parity) {
            ++waits;
            if ((phases[stage] & 1) != parity) return;  // passes at once
            // blocks until the stage's fill in flight lands; there has to be one, and that has to be enough
            bool landed = false;
            for (int i = stage; i < armed; i += n)
              if (flying[i] && !landed) {
                flying[i] = false;
                landed = true;
                ++phases[stage];
              }
            good = good && landed && (phases[stage] & 1) != parity;
          });
          for (bool f : flying) good = good && !f;
          good = good && waits == (armed < n ? armed : n);
          if (!good) {
            std::printf("n %d read %d armed %d mask %x\n", n, read, armed, mask);
            return 1;
          }
          ++states;
        }
  std::printf("%ld\n", states);
  return 0;
}
"""


def test_fills_in_flight(tmp_path):
    cxx = os.environ.get("CXX", "g++")
    if not shutil.which(cxx):
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "ring.cpp", tmp_path / "ring"
    src.write_text(MODEL)
    subprocess.run([cxx, "-std=c++17", "-O2", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    done = subprocess.run([str(exe)], capture_output=True, text=True)
    assert done.returncode == 0, done.stdout
    assert int(done.stdout) > 1000
