// drain.cuh - which loads a pair of CTAs still has in flight when it gives up
// (plain C++, so that the CPU tests compile it as it stands).
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define MOE_HD __host__ __device__ __forceinline__
#else
#define MOE_HD inline
#endif

namespace moe {

// A ring of `stages`; load j goes to stage j % stages, and ends that stage's
// barrier's phase j / stages.  A pair's loads all count on its first CTA's
// barriers: the first CTA's load of a stage arrives there, expecting both
// CTAs' bytes.  first, second: how many loads each has issued when both have
// stopped; a stage is loaded again once both loads of it were used, so the
// counts of a stage differ by one at most.  (One CTA alone: second = first.)
struct StageDrain {
  bool wait;         // something may be in flight: wait for the phase
  uint32_t parity;   // of that phase
  bool arrive;       // the second CTA alone loaded: arrive, expecting its bytes
  bool make_up;      // the first CTA alone loaded: count the second's bytes,
                     // which never come
};

MOE_HD StageDrain stage_drain(uint32_t first, uint32_t second, uint32_t stages, uint32_t stage) {
  const uint32_t a = first > stage ? (first - stage - 1) / stages + 1 : 0;    // loads of this stage
  const uint32_t b = second > stage ? (second - stage - 1) / stages + 1 : 0;
  const uint32_t n = a > b ? a : b;
  return StageDrain{n != 0, (n - 1) & 1u, b > a, a > b};
}

}  // namespace moe
