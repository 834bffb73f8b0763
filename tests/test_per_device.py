"""State that the rotary and cross-entropy launchers make once a device (function
attributes, resident clusters): a small host program over the header they use, and the
launchers' use of it."""

import os
import re
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "adamw_optimizer_step_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "per_device.h"

struct State { int err = 0; int resident = 0; };

int main() {
  static gbo::PerDevice<State> per;
  int made[3] = {0, 0, 0};
  auto of = [&](int dev, int sms) {
    return per.of(dev, [&](State &s) { ++made[dev]; s.resident = sms; s.err = dev == 1 ? 98 : 0; });
  };
  // a second device gets its own state, whatever the first one got; each is made once
  const State *a = of(0, 152), *b = of(1, 148), *c = of(0, 7);
  if (!a || !b || a != c || a == b) return 1;
  if (a->resident != 152 || a->err != 0 || b->resident != 148 || b->err != 98) return 2;
  if (made[0] != 1 || made[1] != 1) return 3;
  // from several threads: made once, and seen whole
  std::vector<std::thread> threads;
  int bad[8] = {};
  for (int k = 0; k < 8; ++k) threads.emplace_back([&, k] { bad[k] = of(2, 33)->resident != 33; });
  for (auto &t : threads) t.join();
  for (int k = 0; k < 8; ++k) if (bad[k]) return 4;
  if (made[2] != 1) return 5;
  // out of range: told, not touched
  auto never = [](State &) { std::printf("made"); };
  return per.of(-1, never) || per.of(gbo::kMaxDevices, never) ? 6 : 0;
}
"""


def test_state_of_each_device(tmp_path):
    src, exe = tmp_path / "p.cpp", tmp_path / "p"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe), "-lpthread"], check=True)
    assert subprocess.run([str(exe)], capture_output=True, timeout=60).returncode == 0


def test_the_launchers_keep_nothing_for_the_process():
    for name in ("rotary.cu", "xent_tc.cu"):
        text = open(os.path.join(CSRC, name)).read()
        assert not re.search(r"once_flag|call_once", text), name
        # every raised limit belongs to a device's state
        assert text.count("cudaFuncSetAttribute") == text.count("static PerDevice<"), name
