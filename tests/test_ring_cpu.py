"""The last waits of a thread that fills a ring of stages, on the host: the
header that the kernels use, compiled with a model of the barriers."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "weight_only_quantized_wql_gb300", "csrc")

MODEL = r"""
#include <cstdio>
#include <cstdlib>
#include "ring.cuh"

// Two producers share a ring; producer p stops after fills[p] of them.  A fill
// in flight lands only when its own producer waits for it: landed[p][slot] is the
// number of that producer's fills of the slot known to have landed.
int main() {
  for (int ring = 1; ring <= 12; ++ring)
    for (int f0 = 0; f0 <= 40; ++f0)
      for (int ahead = 0; ahead <= ring; ++ahead) {
        const int fills[2] = {f0, f0 + ahead};      // one gave up, the other got further
        for (int p = 0; p < 2; ++p) {
          int waits = 0;
          bool seen[12] = {};
          wql::drain_ring(fills[p], ring, [&](int slot, uint32_t parity) {
            int last = -1;                           // its last fill of the slot
            for (int i = slot; i < fills[p]; i += ring) last = i;
            if (last < 0 || seen[slot] || parity != (uint32_t)((last / ring) & 1)) {
              printf("ring %d fills %d: slot %d parity %u\n", ring, fills[p], slot, parity);
              exit(1);
            }
            seen[slot] = true;
            ++waits;
            return slot != 1;
          });
          for (int s = 0; s < ring; ++s)
            if (seen[s] != (s < fills[p])) { printf("slot %d of %d left\n", s, ring); exit(1); }
          if (waits != (fills[p] < ring ? fills[p] : ring)) exit(1);
        }
      }
  // a wait that fails is reported, and the others are waited for all the same
  int waits = 0;
  const bool ok = wql::drain_ring(9, 4, [&](int s, uint32_t) { ++waits; return s != 2; });
  return ok || waits != 4 || !wql::drain_ring(0, 4, [](int, uint32_t) { return false; });
}
"""


def test_every_fill_of_either_producer_is_waited_for(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    src, exe = tmp_path / "ring.cpp", tmp_path / "ring"
    src.write_text(MODEL)
    subprocess.run([cxx, "-std=c++17", "-x", "c++", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


def test_both_producers_of_the_product_wait_for_their_fills():
    """The weight's and the tokens' thread can stop at different fills."""
    with open(os.path.join(CSRC, "mx_logits.cu")) as f:
        code = f.read()
    weight = code[code.index("TMA: the weight and its scales"):code.index("TMA: the tokens")]
    tokens = code[code.index("TMA: the tokens"):code.index("tensor cores ----")]
    assert "drain_fills(fills)" in weight and "drain_fills(fills)" in tokens
