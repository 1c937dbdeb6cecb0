// What a row warp of the gathered readout waits for before it converts the queries
// of its CTA's n-th token, n >= 1 (the first token's are the softmax warps').  (Plain
// C++: the host test of the protocol includes it too.)
//
// Token n's copy completes phase n of q_raw, its conversion phase n of q_ready, and
// the copy of token n + 1 is issued only after the products that read token n's
// converted queries.  A parity wait cannot tell a phase from the second one before
// it: a wait for phase 1 of q_raw ends at once while phase 0 is still open, and a
// row warp gets there that early when the first token has a single step (the first
// two slots are free from the start).  So q_ready's phase n - 1 comes first.  That
// wait is exact, since phase n needs this warp's own arrival; behind it phase n - 1
// of q_raw is complete, and phase n + 1 cannot be before this warp has converted.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define CSA2_Q_FN __host__ __device__ __forceinline__
#else
#define CSA2_Q_FN inline
#endif

namespace csa2 {

struct QWait {
  bool ready;       // of q_ready, else of q_raw
  uint32_t phase;
};
constexpr int kQWaits = 2;
CSA2_Q_FN QWait q_wait(uint32_t n, int i) { return i == 0 ? QWait{true, n - 1} : QWait{false, n}; }

}  // namespace csa2
