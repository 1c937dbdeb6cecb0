// Which rows a step's query token sees (window_attn and tree_attn).
#pragma once
#include "kernels.cuh"

namespace csa2 {

// 8-bit rows of a smaller scale count as zeros (2^-64).
constexpr float kTinyScale = 5.421010862427522e-20f;

// Of token gp: its sequence, the positions that its window may hold, end - left ..
// end - 1 (those below 0 hold no key), and its extra rows, a bit each.  False for
// a packed token behind the last sequence.  Called by whole warps.  Nothing read
// from the device makes an address: whatever ctx_len, cu and the masks hold, seq <
// batch and places in a ring come from a remainder.
struct StepToken {
  int64_t seq, end;
  int left;
  uint64_t extra;
};

__device__ __forceinline__ uint64_t low_bits(int n) { return n >= 64 ? ~0ull : (1ull << n) - 1; }

__device__ __forceinline__ bool step_token(const StepRows &s, int64_t gp, StepToken &t) {
  if (s.cu) {   // packed tokens: a causal window and the first tokens as sinks
    int b;
    if (!find_sequence(s.cu, s.batch, gp, b)) return false;
    const int32_t len = s.ctx_len[b];
    const int64_t at = s.cu[b], ctx = max(len, 0);
    t.seq = b;
    t.end = max(ctx + (gp - at) + 1, (int64_t)0);
    t.left = s.win;
    const int64_t before = t.end - s.win;   // positions that the window has left behind
    t.extra = low_bits((int)(before < s.extras ? (before > 0 ? before : 0) : s.extras));
    if (len < 0 || (s.win > 0 && min(ctx, (int64_t)s.win - 1) + (s.cu[b + 1] - at) > s.ring)) set_error(CSA2_DEV_ERR_INDEX);
  } else {      // a tree's tokens: the rows their mask names, and the window's rest
    t.seq = (int64_t)((uint32_t)gp / (uint32_t)s.extras);
    const int32_t len = s.ctx_len[t.seq];
    if (len < 0) set_error(CSA2_DEV_ERR_INDEX);
    t.extra = s.mask[gp] & low_bits(s.extras);
    t.end = max(len, 0);
    t.left = max(s.win - __popcll(t.extra), 0);
  }
  return true;
}

// A lane holds x and y of two rows at its own column; neighbouring lanes exchange,
// so that the even one has two columns of the first row (bf16) and the odd one two
// of the second.
__device__ __forceinline__ uint32_t lane_pair(bool odd, float x, float y) {
  const float other = __shfl_xor_sync(0xffffffffu, odd ? x : y, 1);
  const __nv_bfloat162 v = odd ? __floats2bfloat162_rn(other, y) : __floats2bfloat162_rn(x, other);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// Channel d (a lane's; a warp's 32 are consecutive) of rows `row` and row + 1.
__device__ __forceinline__ void put_pair(__nv_bfloat16 *out, int64_t row, int d, float x, float y) {
  const bool odd = d & 1;
  *reinterpret_cast<uint32_t *>(out + (row + odd) * D + (d & ~1)) = lane_pair(odd, x, y);
}

}  // namespace csa2
