// How many pages a reservation needs, and whether a pool can have them.  A call may list 2^18 rows of up to 2^30 pages
// each, so the sum takes 64 bits; what exceeds the pool is refused before anything is handed out.
//
// A header of its own, with no CUDA include, so that the sums can be checked on a host.
#pragma once

#ifndef KDN_HOST_DEVICE
#ifdef __CUDACC__
#define KDN_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define KDN_HOST_DEVICE inline
#endif
#endif

namespace kdn {

KDN_HOST_DEVICE int pages_of(int len, int page_size) { return (len + page_size - 1) / page_size; }

using PageSum = unsigned long long;

// Pages that a row of len tokens needs for count more; len + count is within the table (at most 2^30).
KDN_HOST_DEVICE PageSum more_pages(int len, int count, int page_size) {
  return (PageSum)(pages_of(len + count, page_size) - pages_of(len, page_size));
}
KDN_HOST_DEVICE bool pool_too_small(PageSum need, int num_pages) { return need > (PageSum)num_pages; }

}  // namespace kdn
