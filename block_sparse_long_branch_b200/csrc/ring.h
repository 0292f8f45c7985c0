// ring.h -- the last uses of a ring of barriers, to wait on before its memory goes.
//
// Use n of `bars` barriers taken in turn is on barrier n % bars, in its phase n / bars.  A
// barrier's uses complete in order, so who has waited for the last use of every barrier
// has waited for all.  Copies on different barriers may land in any order: the last copy
// alone says nothing of the others.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define MSA_DEVICE __device__ __forceinline__
#else
#define MSA_DEVICE inline
#endif

namespace msa {

// The i-th from the end of `uses`, i < bars, counted a round later so that it is no less than
// 0 (later = uses + bars - 1 - i): below `bars` there were not so many uses; else it is on
// barrier later % bars, and this is the parity to wait for.
MSA_DEVICE uint32_t ring_parity(uint32_t later, uint32_t bars) { return (later / bars + 1) & 1; }

// The parity of the last use of barrier i, when the next use is of barrier `slot` in a phase
// of parity `phase`.  For a barrier not yet used it is 1: the phase "before the first", for
// which a wait passes at once.
MSA_DEVICE uint32_t ring_last_parity(uint32_t i, uint32_t slot, uint32_t phase) {
  return i < slot ? phase : phase ^ 1;
}

}  // namespace msa
