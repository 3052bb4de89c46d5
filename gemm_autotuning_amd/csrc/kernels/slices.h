// slices.h -- joining the partial sums of a k-split inside one launch: each
// workgroup stores its slice's partials, and the last one to finish adds
// them in slice order.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gtk {

// Sum of the S slice partials w[q * stride], q ascending.  The device-scope
// loads are issued BIG (then 8, 4 and 2) at a time before any is added, so
// the reduction costs about S/BIG + 3 memory round trips rather than S (BIG =
// 8 where registers are scarce: 16-wave workgroups have 128 per lane).
template <int BATCH>
__device__ __forceinline__ void sum_batches(const float* w, int64_t stride, int S, int& q, float& v) {
  for (; q + BATCH <= S; q += BATCH) {
    float t[BATCH];
#pragma unroll
    for (int j = 0; j < BATCH; ++j)
      t[j] = __hip_atomic_load(w + (int64_t)(q + j) * stride, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
    for (int j = 0; j < BATCH; ++j) v += t[j];
  }
}
template <int BIG = 32>
__device__ __forceinline__ float sum_slices(const float* w, int64_t stride, int S) {
  float v = 0.f;
  int q = 0;
  if constexpr (BIG > 8) sum_batches<BIG>(w, stride, S, q, v);
  sum_batches<8>(w, stride, S, q, v);
  sum_batches<4>(w, stride, S, q, v);
  sum_batches<2>(w, stride, S, q, v);
  for (; q < S; ++q) v += __hip_atomic_load(w + (int64_t)q * stride, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return v;
}

// Counts this workgroup's K slice as finished for its column block; is_last
// (workgroup-shared) is set in every thread when it was the S-th.  Partial
// sums stored before the call are visible to the last workgroup's loads
// after it.  The workgroup barrier orders every thread's partial stores
// before thread 0's counter increment, a device-scope release, which is
// cumulative and so publishes them all.  The increments form one release
// sequence on the counter; the last workgroup's thread 0 read-modifies the
// value the others left, then issues a device-scope acquire fence, so every
// earlier workgroup's release synchronizes with that fence, and the second
// barrier orders the fence before every thread's later loads.  One
// device-scope release per workgroup (it writes back the XCD's L2) and one
// acquire (it invalidates it) in the last workgroup of each column block.
__device__ __forceinline__ void last_slice_handshake(unsigned* counter, int S, int tid, int& is_last) {
  __syncthreads();
  if (tid == 0) {
    const unsigned prev = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_AGENT);
    is_last = (prev == (unsigned)(S - 1));
    if (is_last) __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  }
  __syncthreads();
}

}  // namespace gtk
