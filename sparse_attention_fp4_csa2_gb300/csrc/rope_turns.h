// RoPE phases in fixed point.  (Plain C++: the host test of the bound includes
// it too.)
//
// A frequency is kept as a fraction of a turn per position, in units of 2^-64
// turns, step_j = floor(2^64 inv_j / (2 pi)), inv_j = fl32(theta^(-2j/64)).  Its
// product with a position wraps modulo whole turns by itself.  The step is
// less than 1 + 2^-20 units short, so for positions below 2^22 the phase is
// less than 2^-41.9 turns, 2^-39.3 rad, behind: an absolute bound, which many
// ulp of a cos or sin next to zero can lie within, but far below the smallest
// step of the row's E4M3 codes (2^-17.8 of its largest value).
#pragma once
#include <cmath>
#include <cstdint>

#ifdef __CUDACC__
#define CSA2_ROPE_FN __host__ __device__ __forceinline__
#else
#define CSA2_ROPE_FN inline
#endif

namespace csa2 {

constexpr int kRopePairs = 32;

struct RopeTurns {
  uint64_t step[kRopePairs];
};

inline RopeTurns rope_turns(float theta) {
  // 1 / (2 pi) = 0x0.28BE60DB9391054A7F09D5F47D4D3770... (binary expansion)
  constexpr uint64_t kHi = 0x28BE60DB9391054Aull, kLo = 0x7F09D5F47D4D3770ull;
  RopeTurns t;
  for (int j = 0; j < kRopePairs; ++j) {
    const float inv = (float)std::pow((double)theta, -(2.0 * j) / (2.0 * kRopePairs));
    int ex;
    const uint64_t m = (uint64_t)std::ldexp(std::frexp(inv, &ex), 24);   // inv = m * 2^(ex - 24), ex <= 1
    const unsigned __int128 lo = (unsigned __int128)m * kLo;
    const unsigned __int128 prod = (unsigned __int128)m * kHi + (uint64_t)(lo >> 64);   // 2^64 m / (2 pi)
    const int sh = 24 - ex;
    t.step[j] = sh >= 128 ? 0 : (uint64_t)(prod >> sh);
  }
  return t;
}

// Position p's phase as quarter turns (0 .. 3) and what is left, at most an
// eighth of a turn, as half turns rounded once to fp32.
CSA2_ROPE_FN float rope_phase(uint64_t step, int64_t p, uint32_t &quarter) {
  const uint64_t phase = step * (uint64_t)p;
  const uint64_t q = (phase + (1ull << 61)) >> 62;
  quarter = (uint32_t)(q & 3);
  return (float)(int64_t)(phase - (q << 62)) * 0x1p-63f;
}

}  // namespace csa2
