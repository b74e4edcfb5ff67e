"""Which phase of a stage's barrier a fill of a ring completes, and which fills
may still be on their way: csrc/ring.cuh, compiled for the host, against
barriers that are counted along.  No GPU needed."""

import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_layer_side_gb300",
                    "csrc")

PROGRAM = r"""
#include "ring.cuh"
#include <cstdio>
// As an mbarrier answers: whether the phase with this parity is over.
struct Barrier {
  int phase = 0;
  bool over(unsigned parity) const { return ((unsigned)phase & 1u) != parity; }
};
int main() {
  long checked = 0;
  for (int stages = 1; stages <= 10; ++stages)
    for (int issued = 0; issued <= 45; ++issued) {
      // all fills but the last of each stage have landed; of those any may have
      const int n = issued < stages ? issued : stages;
      for (int landed = 0; landed < (1 << n); ++landed) {
        Barrier full[10];
        int fill_of[10];
        for (int f = 0; f < issued; ++f) {
          if (f >= stages) ++full[f % stages].phase;  // the fill before
          fill_of[f % stages] = f;
        }
        for (int s = 0; s < n; ++s)
          if (landed >> s & 1) ++full[s].phase;
        int waits = 0;
        for (int f = mok::last_fills_from(issued, stages); f < issued; ++f, ++waits) {
          const int s = f % stages;
          if (fill_of[s] != f) return printf("stages %d, issued %d: fill %d is not its stage's last\n", stages, issued, f), 1;
          if (full[s].over(mok::fill_parity(f, stages)) != (bool)(landed >> s & 1))
            return printf("stages %d, issued %d, landed %x: fill %d\n", stages, issued, landed, f), 1;
          ++checked;
        }
        if (waits != n) return printf("stages %d, issued %d: %d waits\n", stages, issued, waits), 1;
      }
    }
  printf("%ld checked\n", checked);
  return 0;
}
"""


def test_last_fills_are_told_from_landed_ones(tmp_path):
    compiler = shutil.which("g++") or shutil.which("c++")
    if compiler is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "ring.cpp", tmp_path / "ring"
    src.write_text(PROGRAM)
    subprocess.run([compiler, "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    done = subprocess.run([str(exe)], capture_output=True, text=True)
    assert done.returncode == 0 and "checked" in done.stdout, done.stdout


def test_the_feed_forward_kernel_waits_for_them():
    """Past the loop of the copies, whatever became of it, and on the barriers that count them."""
    text = open(os.path.join(CSRC, "ffn.cu")).read()
    few = text[text.index("ffn_few_kernel("):]
    copies = few[few.index("ffn_loads<MODE>("):few.index("} else if (warp == 1 && rank == 0) {")]
    assert "if (!ok) {" not in copies
    assert "last_fills_from(i, stages)" in copies and copies.count("fill_parity(f, stages)") == 2
    assert copies.index("if (rank == 0) {") < copies.index("last_fills_from")
    # the matrix instructions' end is waited for past an abort too
    sums = few[few.index("const bool summed"):few.index("cluster_sync();\n  const int row0")]
    assert "mbar_drain(&ctl->done, 0, kWaitLimitNs)" in sums
