"""How a grid of more threads than a launch takes is cut into launches (launch_parts.h), on the CPU."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include "launch_parts.h"
static void fail(const char *what, long long g, long long t) { std::printf("%s: %lld x %lld\n", what, g, t); std::exit(1); }
int main() {
  const long long limit = 1LL << 32, most = (1LL << 31) - 1;
  for (long long t = 64; t <= 1024; t += 64)
    for (long long g : {0LL, 1LL, 7LL, limit / t - 8, limit / t - 1, limit / t, limit / t + 1, 2 * (limit / t), 1LL << 24, (1LL << 25) + 5, most}) {
      if (g > most) continue;
      long long at = 0;
      int calls = 0;
      const int st = wt::launch_parts(g, t, 0, [&](uint32_t first, uint32_t count) {
        if (first != at) fail("a gap", g, t);
        if (first % 8) fail("out of step", g, t);
        if (count == 0 || (long long)count * t >= limit) fail("too large a part", g, t);
        at += count, ++calls;
        return 0;
      });
      if (st != 0 || at != g) fail("not all of it", g, t);
      if (g > 0 && g * t < limit - 8 * t && calls != 1) fail("more than one launch", g, t);
      calls = 0;
      const int refused = wt::launch_parts(g, t, 0, [&](uint32_t, uint32_t) { return ++calls, 5; });
      if (refused != (g ? 5 : 0) || calls != (g ? 1 : 0)) fail("went on after a failure", g, t);
    }
  std::printf("parts ok\n");
}
"""


def test_parts_cover_the_grid_and_fit_a_launch(tmp_path):
    src, exe = tmp_path / "parts.cpp", tmp_path / "parts"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", os.path.join(ROOT, "bf16_fp8_weight_amd", "csrc"), str(src), "-o",
                    str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "parts ok" in r.stdout, r.stdout + r.stderr


def test_launches_that_may_exceed_one_grid_go_through_it():
    """Every launch of a kernel whose grid grows with rows, columns and experts without a limit of its own."""
    csrc = os.path.join(ROOT, "bf16_fp8_weight_amd", "csrc")
    for name, launches in (("expert_run.h", 1), ("mxfp4.hip", 2), ("act_quant.hip", 1)):
        text = open(os.path.join(csrc, name)).read()
        assert text.count("hipLaunchKernelGGL(") == launches == text.count("dim3(count)"), name
