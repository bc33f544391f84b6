"""The end of a GEMM pipeline that gave up (csrc/pipeline_end.h), compiled for the host and run on a model of the
full barriers: no stage counts as landed while a copy into it is in flight, and every one does afterwards."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "invariant_expert_routing_gb300", "csrc")

MODEL = r"""
#include <cstdio>
#include <cstdlib>
#include <random>
#include <utility>
#include <vector>
#include "pipeline_end.h"

struct Barrier {                       // one arrival a phase, and bytes
  int phase = 0, pending = 1;
  long bytes = 0;
  void next() { if (pending == 0 && bytes == 0) { ++phase; pending = 1; } }
  void arm(long b) { bytes += b; if (--pending < 0) { std::puts("armed twice"); std::exit(1); } next(); }
  void complete(long b) { bytes -= b; next(); }
  bool done(unsigned parity) const { return (unsigned)(phase & 1) != parity; }
};
#define CHECK(c) do { if (!(c)) { std::printf("%s: %d loads, %d by the other, %d consumed, %d stages\n", #c, even, odd, used, S); return 1; } } while (0)

// pair: the even CTA arms a stage for both CTAs' bytes; alone: for its own.
int run(std::mt19937& g, bool pair) {
  auto rnd = [&](int n) { return (int)(g() % (unsigned)n); };
  const int S = 1 + rnd(9), n = rnd(6 * S);
  std::vector<long> tx(n + 1);
  for (auto& b : tx) b = rnd(2) ? 3 : 7;
  std::vector<Barrier> bars(S);
  std::vector<std::pair<int, long>> flying;
  int even = 0, odd = 0, used = 0;
  auto land = [&] {
    const int i = rnd((int)flying.size());
    bars[flying[i].first % S].complete(flying[i].second);
    flying.erase(flying.begin() + i);
  };
  for (int step = rnd(8 * n + 2); step > 0; --step) {   // cut off anywhere
    switch (rnd(5)) {
      case 0:
        if (even < n && even < used + S) { bars[even % S].arm((pair ? 2 : 1) * tx[even]); flying.push_back({even, tx[even]}); ++even; }
        break;
      case 1:
        if (pair && odd < n && odd < used + S) { flying.push_back({odd, tx[odd]}); ++odd; }
        break;
      case 2:
        if (!flying.empty()) land();
        break;
      default:
        if (used < even && (!pair || used < odd) && bars[used % S].done((unsigned)(used / S) & 1u)) ++used;
    }
  }
  if (pair) {
    auto never = [](int) { std::puts("the wrong side"); std::exit(1); };
    moe::settle_pair_loads(true, even, odd, [&](int i) { bars[i % S].complete(tx[i]); }, never);
    moe::settle_pair_loads(false, odd, even, never, [&](int i) { bars[i % S].arm(tx[i]); });
  }
  std::vector<std::pair<int, unsigned>> waits;
  moe::wait_last_loads(even > odd ? even : odd, S, [&](int s, unsigned parity) { waits.push_back({s, parity}); });
  while (!flying.empty()) {
    for (auto& f : flying) {
      bool waited = false;
      for (auto& w : waits) waited |= w.first == f.first % S && !bars[w.first].done(w.second);
      CHECK(waited);
    }
    land();
  }
  for (auto& w : waits) CHECK(bars[w.first].done(w.second));
  return 0;
}

int main() {
  std::mt19937 g(7);
  for (int i = 0; i < 200000; ++i)
    if (run(g, i & 1)) return 1;
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_no_copy_outlives_the_wait(tmp_path):
    src, exe = tmp_path / "model.cpp", tmp_path / "model"
    src.write_text(MODEL)
    subprocess.check_call(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)])
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
