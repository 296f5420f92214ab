// The loop of every bounded wait: ``ready`` until it holds or ``now`` has moved by more than ``most``.
//
// A thread may be held up between a try that failed and its look at the clock (preemption, a long queue of other warps'
// instructions).  So the last word is a try, not the clock: what is ready when the limit has passed is not a timeout, and
// threads that wait for the same event rarely disagree.
//
// The event and the clock are template parameters so that the loop can be checked on a host (a header of its own, with no
// CUDA include).
#pragma once

#ifndef KDN_HOST_DEVICE
#ifdef __CUDACC__
#define KDN_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define KDN_HOST_DEVICE inline
#endif
#endif

namespace kdn {

template <class Ready, class Now>
KDN_HOST_DEVICE bool wait_bounded(Ready ready, Now now, long long most) {
  if (ready()) return true;
  const long long t0 = now();
  while (!ready())
    if (now() - t0 > most) return ready();
  return true;
}

}  // namespace kdn
