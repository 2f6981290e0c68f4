// Places in a ring of stages in shared memory, each with a barrier that says it is full and one that says
// it is empty (head.cu).  Host code too, so that it can be tested without a GPU.
#pragma once

#ifdef __CUDACC__
#define PROFK_RING __host__ __device__ __forceinline__
#else
#define PROFK_RING inline
#endif

namespace profk {

// Where a copy goes, or a product's operands are: a stage, and how often the ring has been gone round (by its parity).
struct RingPlace {
  int stage = 0;
  unsigned turn = 0;
  PROFK_RING void next(int stages) {
    if (++stage == stages) {
      stage = 0;
      turn ^= 1;
    }
  }
  PROFK_RING void back(int stages) {
    if (stage == 0) {
      stage = stages;
      turn ^= 1;
    }
    --stage;
  }
  // The parities to wait for: that the copy of this turn is there, and that what the turn before
  // brought has been used (in the first turn the barrier's phase before its first: the ring begins empty).
  PROFK_RING unsigned full() const { return turn; }
  PROFK_RING unsigned empty() const { return turn ^ 1; }
};

// The end of the copying, `at` being the place that the next copy would have gone to and `issued` the number of
// stages that have been copied to: waits until all of them have been used (wait_empty(place), false where that
// gives up, and of the stages without a copy at once true).  Where it gives up, nobody may
// be waiting for them any more, but copies may still be writing: the last one to each stage is waited for
// (wait_full(place)), from the last of all backwards.
template <typename WaitEmpty, typename WaitFull>
PROFK_RING void leave_ring(RingPlace at, int issued, int stages, WaitEmpty wait_empty, WaitFull wait_full) {
  bool used = true;
  RingPlace place = at;
  for (int i = 0; i < stages && used; ++i) {
    used = wait_empty(place);
    place.next(stages);
  }
  if (used) return;
  for (int i = 0; i < issued; ++i) {
    at.back(stages);
    wait_full(at);
  }
}

}  // namespace profk
