// Rules of the rings of shared-memory slots that the integer 4-bit projection
// kernels fill by asynchronous copies.  A slot has a `full` barrier, armed by
// the loader for each copy, and an `empty` one, on which its readers release
// it; the n-th use of a ring of S slots is phase n / S of slot n % S.  Plain
// C++, so that the rules can be run on the host too.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define BSR_RING_FN __host__ __device__ __forceinline__
#else
#define BSR_RING_FN inline
#endif

namespace bsr {

// Waits for every copy that may be in flight after `issued` uses of a ring of
// `slots`: the last use of each slot.  wait(slot, parity) is bounded and says
// whether that phase of the slot's `full` barrier has completed.
//
// The CTA must not exit, nor use the slots for anything else, under a copy.  So
// the loader calls this at its end, or once the readers are done if any wait of
// the CTA ran out: its own waits do not tell, for the reader may be the one that
// gave up, after the loader's last issue.
//
// A reader whose wait ran out releases no slot any more: the copy may still be
// on its way, and the loader would arm the `full` barrier again in the same
// phase.  The loader then gives up too.
template <class Wait>
BSR_RING_FN void drain_ring(uint32_t issued, uint32_t slots, Wait wait) {
  for (uint32_t j = issued > slots ? issued - slots : 0u; j < issued; ++j)
    if (!wait(j % slots, (j / slots) & 1u)) return;
}

}  // namespace bsr
