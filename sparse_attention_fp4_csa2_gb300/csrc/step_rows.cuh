// Which rows a step's query token sees (window_attn and tree_attn).
#pragma once
#include "kernels.cuh"

namespace csa2 {

// 8-bit rows of a smaller scale count as zeros (2^-64).
constexpr float kTinyScale = 5.421010862427522e-20f;

// Where the weights go to the tensor cores as fp16 (all but window_attn.cu), a key
// is held as fp16 values over a scale f of its own size: the weight is 2^(logit - m)
// f with m the largest logit + log2 f, at most 1 (2^8 between raises), so that what
// it loses below fp16's normal range is 2^-25 of about the largest contribution of
// any key, whatever the keys' sizes are.  Both divisions are by powers of two and
// exact in fp16:
//   an entry's f is the power of two of its largest block scale, x 4 (its codes reach
//   6, so f is 2^-7 .. 2^10 and the values are below 3);
//   an 8-bit row's f is its scale x 2^8 (its codes reach 448 = 1.75 x 2^8);
// so that keys of one size have nearly the same f.  (An entry's size is that of its
// scales: a block of zero codes under a large one counts too.  The writers leave none.)
// What it costs: 32 x 64 drafted tokens 310 us, with f = 1 for entries and a row's scale
// 303; but entries of zeros beside rows of 1e-6 then came out as nothing.
//   a key of nothing but zero codes has f = 2^-56: it never sets m beside others, and up to
//   row scales of 2^50 beside it 2^(logit - m) f is an fp32 number that gives back
//   its weight in the row sum.
constexpr float kZeroScale = 1.3877787807814457e-17f;   // 2^-56
constexpr uint32_t kRowNorm = 0x1C001C00u;              // fp16 2^-8, twice

// fp16 magnitudes of four E4M3 scales (two a word, NaNs beside others left out)
// joined with those of `m`.
__device__ __forceinline__ __half2 scales_size(uint32_t sc, __half2 m) {
  const uint32_t x = e4m3x2_to_half2((uint16_t)sc), y = e4m3x2_to_half2((uint16_t)(sc >> 16));
  return __hmax2(m, __hmax2(__habs2(*reinterpret_cast<const __half2 *>(&x)), __habs2(*reinterpret_cast<const __half2 *>(&y))));
}

// The larger half's fp16 bits.
__device__ __forceinline__ uint32_t larger_half(__half2 m) {
  const uint32_t u = *reinterpret_cast<const uint32_t *>(&m);
  return max(u & 0xFFFFu, u >> 16);
}

// A key's f, and what its values are multiplied by on their way (two fp16 numbers).
// Of an entry: size, its largest block scale's fp16 bits; of a row: its scale, and 0
// for the codes of a tiny one.  zero: all its codes are zeros.
__device__ __forceinline__ float key_scale(bool entry, uint32_t size, float scale, bool zero, uint32_t &norm) {
  const uint32_t e = min(size >> 10, 23u);   // exponent field, 6 .. 23 (a NaN stays one in the values)
  const bool tiny = !entry && scale < kTinyScale;
  norm = entry ? (28u - e) * 0x04000400u : tiny ? 0u : kRowNorm;
  return zero || tiny ? kZeroScale : entry ? __uint_as_float((e + 114u) << 23) : scale * 256.0f;
}

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
