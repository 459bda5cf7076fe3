"""The ring of the cache attention (csrc/cache_ring.cuh) as a host program: which slots are waited for, filled and
drained, with waits that give up at every place; and what the kernel does with a wait that gave up."""

import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "lsh_attention_hash_b200", "csrc")

MODEL = r"""
#include <stdio.h>
#include <stdlib.h>
#include "cache_ring.cuh"
#define CHECK(x) do { if (!(x)) { printf("line %d: %s (stages %d fail %d)\n", __LINE__, #x, kS, fail); exit(1); } } while (0)

template <int kS, int kW>
void runs() {
  const int sizes[] = {0, 1, 2, 3, 4, 5, 7, 8, 9, 12, 13, 16, 33};
  for (int warp = 0; warp < kW; ++warp)
    for (int fail = -1; fail < 40; ++fail)     // the wait that gives up, -1: none
      for (int late = 0; late <= kS; ++late) { // copies that never land either (drained in vain)
        int slot = 0, waits = 0;
        uint32_t phase = 0;
        int filled[kS] = {}, stage[kS];
        bool flying[kS] = {};
        bool gone = false;
        for (int n : sizes) {  // stretches one after the other, as a block's pieces are
          int next = warp;
          auto issue = [&](int st, int s) {
            CHECK(!gone && st < n && !flying[s]);
            flying[s] = true;
            stage[s] = st;
            ++filled[s];
          };
          for (int i = 0, s = slot; i < kS; ++i) {
            if (warp + i * kW < n) issue(warp + i * kW, s);
            s = s + 1 == kS ? 0 : s + 1;
          }
          int drained = 0;
          const bool ok = lsh::cache::run_stages<kS, kW>(
              warp, n, slot, phase,
              [&](int s, uint32_t parity) {
                CHECK(!gone && flying[s] && stage[s] == next && parity == (uint32_t)((filled[s] - 1) & 1));
                return waits++ != fail;
              },
              [&](int s, uint32_t parity) {
                CHECK(flying[s] && parity == (uint32_t)((filled[s] - 1) & 1));
                flying[s] = false;
                ++drained;
              },
              [&](int st, int s) {
                CHECK(!gone && stage[s] == st && st == next && st < n);
                flying[s] = false;  // landed, and free after this call
                next += kW;
              },
              issue);
          CHECK(ok == (waits <= fail || fail < 0));
          for (int s = 0; s < kS; ++s) CHECK(!flying[s]);  // nothing is on its way any more
          if (!ok) {
            CHECK(drained >= 1);
            gone = true;
            break;  // the kernel returns
          }
          CHECK(drained == 0 && next >= n);
        }
      }
}
int main() {
  runs<1, 4>(); runs<2, 4>(); runs<3, 4>(); runs<2, 1>();
  printf("ok\n");
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_ring_order_and_drains(tmp_path):
    src, exe = tmp_path / "model.cpp", tmp_path / "model"
    src.write_text(MODEL)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout


def test_a_wait_that_gave_up_ends_the_block():
    """Lanes decide about a wait together, and every block barrier behind the stages takes all warps out."""
    with open(os.path.join(CSRC, "cache_attend.cuh")) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    kernel = code[code.index("cache_attend_kernel(const"):code.index("cache_join_kernel(const")]
    assert "mbar_wait(" not in kernel  # each lane for itself: some could go on to a warp's shuffles alone
    assert "mbar_try_wait" not in kernel and "stage_wait(" in kernel
    wait = code[code.index("bool stage_wait("):]
    wait = wait[:wait.index("\n}\n")]
    assert wait.count("return true") == wait.count("if (__all_sync(0xffffffffu, tc::mbar_try_wait(bar, parity))) return true;") == 2
    assert wait.count("return false") == wait.count("if (__shfl_sync(0xffffffffu, bail, 0)) return false;") == 1
    after = kernel[kernel.index("run_stages<"):]
    barriers = re.findall(r"__syncthreads\w*\([^;]*;", after)
    # one for more pages (then one behind the look-up), one before the ring's memory is used again
    assert after.count("if (__syncthreads_or(!ok)) return;") == 2
    assert after.index("__syncthreads_or") < after.index("look_up()")
    assert after.rindex("__syncthreads_or") < after.index("om[")
    assert len(barriers) == 4
