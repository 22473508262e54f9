// What a thread block still waits for after a bounded wait has run out: its own
// asynchronous copies into a ring in shared memory, which must land before the
// ring's memory serves another purpose or another block.  Host and device code,
// shared by the kernels and a host-side check.
#pragma once
#include <cstdint>

#if defined(__CUDACC__)
#define MLA_RHD __host__ __device__ __forceinline__
#else
#define MLA_RHD inline
#endif

namespace mla {

// A ring of `slots` slots is filled in order, fill f into slot f % slots, and
// completes phase f / slots of the slot's full barrier; fill f is issued only
// when fill f - slots has been used, so what may be in flight lies in the last
// `slots` fills before `end`.  Calls wait(slot, parity) for those that
// issued(f) says were issued.
template <typename Issued, typename Wait>
MLA_RHD void drain_ring(int end, int slots, Issued issued, Wait wait) {
  for (int f = end > slots ? end - slots : 0; f < end; ++f)
    if (issued(f)) wait(f % slots, (uint32_t)(f / slots) & 1u);
}

}  // namespace mla
