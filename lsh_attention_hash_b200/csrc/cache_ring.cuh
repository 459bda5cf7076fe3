// How a warp takes its stages of a stretch of keys through its ring of shared-memory slots (plain C++, so that the
// order of waits, copies and drains is tested without a GPU).
//
// Warp w of W has stages w, w + W, ...; the copies of the first kStages of them are on their way into the
// slots from `slot` on.  A slot's copies end phases 0, 1, 0, ... of its barrier, and `phase` is the one that the slots
// from `slot` on are in (those before it: the next).
//
// When a wait gives up, the copies that are on their way are waited for (drain, with a limit of its own) and
// nothing more is copied or consumed: the caller leaves, as the shared memory may not be reused before.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define LSH_RING_FN __device__ __forceinline__
#else
#define LSH_RING_FN inline
#endif

namespace lsh {
namespace cache {

template <int kStages, int kWarps, typename Wait, typename Drain, typename Consume, typename Issue>
LSH_RING_FN bool run_stages(int warp, int n_stage, int& slot, uint32_t& phase, Wait wait, Drain drain, Consume consume,
                            Issue issue) {
  for (int st = warp; st < n_stage; st += kWarps) {
    if (!wait(slot, phase)) {
      for (int i = 0, s = slot; i < kStages; ++i) {
        if (st + i * kWarps < n_stage) drain(s, s < slot ? phase ^ 1u : phase);
        s = s + 1 == kStages ? 0 : s + 1;
      }
      return false;
    }
    consume(st, slot);
    if (st + kStages * kWarps < n_stage) issue(st + kStages * kWarps, slot);
    if (++slot == kStages) {
      slot = 0;
      phase ^= 1;
    }
  }
  return true;
}

}  // namespace cache
}  // namespace lsh
