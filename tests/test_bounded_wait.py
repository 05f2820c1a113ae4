"""The end of the chained recurrence's bounded wait (csrc/wait.hpp), on the
host: whichever look is the last, a state is written before the wait ends, and
it is a number only where the state was found."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "rl_experience_collection_amd", "csrc")

PROGRAM = r"""
#include "wait.hpp"
#include <cmath>
#include <cstdio>
int main() {
  for (uint32_t budget = 0; budget < 5; ++budget)
    for (uint32_t found = 0; found < 8; ++found) {  // the look that finds it
      uint32_t left = budget, looks = 0;
      float state = 7.0f;  // another tile's, left in the same place
      bool walking = true;
      while (walking) {
        const bool done = looks++ == found;
        if (rl::wait_over(done, left)) {
          state = done ? 1.0f : NAN;
          walking = false;
        }
        if (looks > 100) return 1;
      }
      const bool in_time = found <= budget;
      if (in_time ? state != 1.0f : !std::isnan(state)) return 2;
      if (looks != (in_time ? found : budget) + 1) return 3;
    }
  std::puts("ok");
}
"""


def test_a_wait_that_ends_has_written_its_state(tmp_path):
    src, exe = tmp_path / "wait.cpp", tmp_path / "wait"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", (r.returncode, r.stderr)


def test_the_kernel_ends_its_waits_there_only():
    """No place of the scan tests or counts down the looks by itself."""
    text = open(os.path.join(CSRC, "recur.hip")).read()
    assert text.count("wait_over(") == 2
    assert "left == 0" not in text and "--left" not in text
