"""How attention lays out its work, on the host: the lengths of items stay inside the 32 bits in which the kernels hold them, up
to the longest sequences that a call may have."""
import os
import shutil
import subprocess

import pytest

import hybrid_draft_tree_gb300 as g
from hybrid_draft_tree_gb300 import _build

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>

#include "kv_internal.cuh"

int main() {
  const int most = 0x7FFFFFFF - 256;  // keys of a row
  long long plans = 0, widest = 0;
  for (int batch : {1, 2, 64, 1024})
    for (int slots : {1, 3, 16, 61, 64})
      for (int group : {1, 4, 8, 130})
        for (int heads : {1, 8})
          for (int dim : {64, 128})
            for (int prefix : {0, 1, 900, 1 << 30, most - 4096})
              for (int own : {1, 117, 4000, 1 << 29, 1 << 30, 2000000000, most})
                for (int window : {0, 500})
                  for (int eight = 0; eight < 2; ++eight)
                    for (int capped = 0; capped < 2; ++capped) {
                      const long long left = (long long)most - slots - prefix;
                      const int ctx = (int)(own < left ? own : left);
                      const auto p = graft::plan_kv_attend(batch, slots, group, heads, dim, prefix, ctx, window, eight, capped, 152);
                      const long long np = (prefix + 127LL) / 128, no = ((long long)ctx + slots + 127) / 128;
                      const long long joined = (p.packed ? 0 : np) + no;
                      // an item's place and a block more, as the kernels add them up
                      const long long a = p.packed ? p.fixed_a + (np + 1) * p.step_a : 0, b = p.fixed_b + (joined + 1) * p.step_b;
                      if (a > widest) widest = a;
                      if (b > widest) widest = b;
                      if (a > 0xFFFFFFFFLL || b > 0xFFFFFFFFLL || p.step_b < 1 || p.fixed_b < 1 || (p.packed && p.step_a < 1)) {
                        std::printf("batch %d slots %d group %d heads %d dim %d prefix %d ctx %d window %d eight %d capped %d: %lld %lld\n",
                                    batch, slots, group, heads, dim, prefix, ctx, window, eight, capped, a, b);
                        return 1;
                      }
                      // the CTAs ahead of the split take all of the packed line, in pieces of a block and more
                      if (p.split && (p.chunk_a < p.step_a || p.chunk_a * p.split < p.items_a * (p.fixed_a + np * p.step_a))) {
                        std::printf("split %d chunk %lld\n", p.split, (long long)p.chunk_a);
                        return 1;
                      }
                      ++plans;
                    }
  std::printf("%lld %lld\n", plans, widest);
  return 0;
}
"""


def test_items_of_the_longest_sequences_stay_inside_32_bits(tmp_path):
    if shutil.which("nvcc") is None:
        pytest.skip("no nvcc")
    src, exe = tmp_path / "plan.cu", tmp_path / "plan"
    src.write_text(PROGRAM)
    g.load()                                   # builds the library where it is missing
    subprocess.check_call(["nvcc", "-O1", "-std=c++17", "-I" + _build.CSRC, "-I" + _build.INCLUDE, str(src), "-o", str(exe),
                           _build.LIB, "-Xlinker", "-rpath=" + os.path.dirname(_build.LIB)])
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout
    plans, widest = map(int, run.stdout.split())
    assert plans == 4 * 5 * 4 * 2 * 2 * 5 * 7 * 2 * 2 * 2 and widest > 2 ** 31     # the limit was in reach
