// What a producer of a shared-memory ring does at its end, so that no load of its
// unit (a CTA, or a CTA pair) is in flight when a CTA leaves, whichever role of the
// kernel gave up on a bounded wait. Written over the barriers' operations alone, so
// that the rule can be checked on the CPU.
#pragma once

#if defined(__CUDACC__)
#define DLRM_RING_FN __device__ __forceinline__
#else
#define DLRM_RING_FN inline
#endif

namespace dlrm {

// Step i loads into stage i % STAGES, and its bytes complete phase i / STAGES of that
// stage's barrier. This producer issued the steps [0, steps).
//
// One CTA (LEADER, not PAIR): it waits for its last STAGES steps; those before have
// been read by the products. Nothing has to have failed: the products' thread may be
// the one that gave up, and where all went well they have landed already.
//
// A pair: both CTAs' bytes are counted on the leader's barriers, which the leader
// arms. The other one says how many steps it issued (tell). A leader that gave up
// waits for that number (told; negative: not said in time) and arms the steps that the
// other went beyond it, at most STAGES, for that one's bytes (arm), before it waits.
//
// wait(stage, parity), arm(stage) and told() are bounded.
template <int STAGES, bool PAIR, class Wait, class Arm, class Tell, class Told>
DLRM_RING_FN void land_loads(bool leader, bool gave_up, int steps, Wait wait, Arm arm, Tell tell,
                             Told told) {
  if (PAIR && !leader) {
    tell(steps);
    return;
  }
  int end = steps;
  if (PAIR && gave_up) {
    const int other = told();
    for (; end < other; ++end) arm(end % STAGES);
  }
  for (int i = end > STAGES ? end - STAGES : 0; i < end; ++i) wait(i % STAGES, (i / STAGES) & 1);
}

}  // namespace dlrm
