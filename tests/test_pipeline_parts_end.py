"""The end of a pair's pipeline whose loads several warps request in turn (csrc/pipeline_end.h), on the model of the
full barriers of test_pipeline_end.py: no copy into a stage outlives the wait, and every wait ends."""
import shutil
import subprocess

import pytest

from tests.test_pipeline_end import CSRC, MODEL

RUN = r"""
// Warp w of each CTA issues loads w, w + parts, ... in order, none before the stage was consumed.
int run(std::mt19937& g) {
  auto rnd = [&](int n) { return (int)(g() % (unsigned)n); };
  const int S = 1 + rnd(8), parts = 1 + rnd(5), n = rnd(6 * S);
  std::vector<long> tx(n + 1);
  for (auto& b : tx) b = 1 + rnd(9);
  std::vector<Barrier> bars(S);
  std::vector<std::pair<int, long>> flying;
  std::vector<int> count[2] = {std::vector<int>(parts), std::vector<int>(parts)};
  int used = 0;
  auto land = [&] {
    const int i = rnd((int)flying.size());
    bars[flying[i].first % S].complete(flying[i].second);
    flying.erase(flying.begin() + i);
  };
  for (int step = rnd(20 * n + 2); step > 0; --step) {   // cut off anywhere
    const int odd = rnd(2), w = rnd(parts), i = count[odd][w] * parts + w;
    switch (rnd(4)) {
      case 0: case 1:
        if (i < n && i < used + S) {
          if (!odd) bars[i % S].arm(2 * tx[i]);
          flying.push_back({i, tx[i]});
          ++count[odd][w];
        }
        break;
      case 2:
        if (!flying.empty()) land();
        break;
      default:
        if (used < n && moe::load_issued(count[0].data(), parts, used) && moe::load_issued(count[1].data(), parts, used) &&
            bars[used % S].done((unsigned)(used / S) & 1u)) ++used;
    }
  }
  const int *even = count[0].data(), *odd = count[1].data();
  auto never = [](int) { std::puts("the wrong side"); std::exit(1); };
  moe::settle_pair_parts(true, even, odd, parts, S, [&](int i) { bars[i % S].complete(tx[i]); }, never);
  moe::settle_pair_parts(false, odd, even, parts, S, never, [&](int i) { bars[i % S].arm(tx[i]); });
  std::vector<std::pair<int, unsigned>> waits;
  moe::wait_pair_parts(even, odd, parts, S, [&](int s, unsigned parity) { waits.push_back({s, parity}); });
  while (!flying.empty()) {
    for (auto& f : flying) {
      bool waited = false;
      for (auto& w : waits) waited |= w.first == f.first % S && !bars[w.first].done(w.second);
      if (!waited) { std::printf("load %d not waited for (%d consumed, %d stages, %d warps)\n", f.first, used, S, parts); return 1; }
    }
    land();
  }
  for (auto& w : waits) if (!bars[w.first].done(w.second)) { std::printf("stage %d never ends\n", w.first); return 1; }
  return 0;
}

int main() {
  std::mt19937 g(11);
  for (int i = 0; i < 200000; ++i)
    if (run(g)) return 1;
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_no_copy_outlives_the_wait(tmp_path):
    src, exe = tmp_path / "model.cpp", tmp_path / "model"
    head = MODEL[:MODEL.index("#define CHECK")]
    src.write_text(head + RUN)
    subprocess.check_call(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)])
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout


PARITY = r"""
#include <cstdio>
#include <random>
#include <vector>
// Warps w, w + parts, ... of one CTA wait for a stage by the parity of its empty barrier alone.  Returns the loads that
// went into a stage whose load before had not been consumed.
long early(std::mt19937& g, int S, int parts, int n) {
  auto rnd = [&](int k) { return (int)(g() % (unsigned)k); };
  std::vector<int> freed(S), count(parts);   // phases completed of each empty barrier
  std::vector<bool> full(n);
  int used = 0;
  long bad = 0;
  for (int idle = 0; used < n && idle < 100000; ++idle) {
    const int w = rnd(parts), i = count[w] * parts + w;
    if (rnd(3) && i < n) {
      const int s = i % S;
      const unsigned parity = ((unsigned)(i / S) & 1u) ^ 1u;
      if (((unsigned)(freed[s] - 1) & 1u) == parity) {   // the last completed phase has this parity
        bad += i >= used + S;
        full[i] = true;
        ++count[w];
      }
    } else if (full[used]) {
      ++freed[used % S];
      ++used;
    }
  }
  return bad;
}
int main() {
  std::mt19937 g(3);
  long good = 0, over = 0;
  for (int i = 0; i < 20000; ++i) {
    const int S = 2 + (int)(g() % 7);
    good += early(g, S, 1 + (int)(g() % (unsigned)S), 60);
    over += early(g, S, S + 1 + (int)(g() % 3), 60);
  }
  std::printf("%ld %ld\n", good, over);
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_as_many_requesting_warps_as_stages_at_most(tmp_path):
    """What the kernels assert: up to that many a stage's parity is never mistaken; more of them do overwrite stages."""
    src, exe = tmp_path / "parity.cpp", tmp_path / "parity"
    src.write_text(PARITY)
    subprocess.check_call(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", str(src), "-o", str(exe)])
    good, over = map(int, subprocess.run([str(exe)], capture_output=True, text=True, timeout=120, check=True).stdout.split())
    assert good == 0 and over > 0
