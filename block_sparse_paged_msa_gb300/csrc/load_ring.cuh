// The loader's side of a ring of shared-memory stages.  Plain C++ as well: its
// protocol is tested on the host.  Not part of the ABI.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define MSA_RING_FN __device__ __forceinline__
#else
#define MSA_RING_FN inline
#endif

namespace msa {

// Copies go to the stages in turn, each once its stage is free.  A stage's barrier
// counts one armed copy a phase: armed again while bytes are outstanding its arrival
// count underflows, and the phases that follow (and what drain() asks for) are no
// longer the copies'.  So after a wait that gave up nothing more is copied.
template <int N>
struct LoadRing {
  int stage = 0;               // of the next copy
  int copies = 0;              // armed so far
  uint32_t phase = 0;          // parity of the stage's use
  bool going = true;           // no wait gave up

  // wait(stage, parity of `empty`): false = it gave up
  template <typename Wait>
  MSA_RING_FN bool free(Wait wait) {
    if (going) going = wait(stage, phase ^ 1u);
    return going;
  }
  // the copy to `stage` is armed
  MSA_RING_FN void armed() {
    ++copies;
    if (++stage == N) {
      stage = 0;
      phase ^= 1u;
    }
  }
  // wait(stage, parity of `full`) for the last copy of every stage
  template <typename Wait>
  MSA_RING_FN void drain(Wait wait) const {
    for (int i = 0; i < N && i < copies; ++i) wait(i, (uint32_t)(((copies - 1 - i) / N) & 1));
  }
};

}  // namespace msa
