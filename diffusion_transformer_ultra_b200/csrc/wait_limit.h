// When a bounded wait on the device ends.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define UG_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define UG_HOST_DEVICE inline
#endif

namespace ug {

// A wait takes at least kWaitLooks looks, of up to 20 us each, and kMostLooks at most.
constexpr uint32_t kWaitLooks = 2048, kMostLooks = 1u << 26;

// Whether a wait that began at timer value t0 has run out at `now`, after `looks` looks.  The timer is the
// machine's clock in nanoseconds, which may be stepped: the difference is taken as signed, so that a step
// back is not a time of 2^64 ns, and a step forward is outlasted by the looks.  One that was stepped far back
// would hold a wait until it has caught up: the looks end that.
UG_HOST_DEVICE bool wait_over(uint64_t now, uint64_t t0, uint64_t limit_ns, uint32_t looks) {
  return (static_cast<int64_t>(now - t0) > static_cast<int64_t>(limit_ns) && looks >= kWaitLooks) || looks >= kMostLooks;
}

}  // namespace ug
