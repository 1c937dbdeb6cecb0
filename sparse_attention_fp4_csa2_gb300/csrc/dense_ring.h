// Which barrier and phase say that a slot of the dense readout's ring is free
// again.  (Plain C++: the host test of the protocol includes it too.)
//
// Round r fills every slot once: a K round's slots are filled by all
// dequantising warps, a V round's slot s by warp s alone.  Before its part of
// round r a K round's warp waits until round r - 1 has been read from every
// slot, a V round's until it has from its own.  A parity wait cannot tell a
// phase from the second one before it, and after a V round a warp knows of its
// own slot only, so round r's release goes to barrier (r mod 4, s) in phase
// r / 4.  A wait for round r - 1 could then be taken in only while round r - 5
// has not been released, and that is behind every warp: there are never three
// V rounds in a row, so one of the rounds r - 4 .. r - 1 was a K round r', the
// warp waited there for round r' - 1 >= r - 5 on every slot, and that round's
// fill of a slot had itself waited for the slot's round before, and so on down
// to r - 5.  (With one barrier per slot the releases of different slots would
// have to arrive in the order of their products, which nothing promises.)
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define CSA2_RING_FN __host__ __device__ __forceinline__
#else
#define CSA2_RING_FN inline
#endif

namespace csa2 {

constexpr int kRingSets = 4;   // barriers per slot

CSA2_RING_FN uint32_t ring_set(uint32_t round) { return round % kRingSets; }
CSA2_RING_FN uint32_t ring_parity(uint32_t round) { return (round / kRingSets) & 1u; }

}  // namespace csa2
