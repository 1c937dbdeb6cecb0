// Work split of the dense readout (csa2_cross_attn, csa2_prefix_attn).
//
// A unit is a pair of query tokens of one sequence (128 query rows) against
// one step of kDenseStep entries.  The units of all pairs, sequence by
// sequence and pair by pair, form one line that the workers (clusters of two
// CTAs) cut into equal contiguous ranges, whatever the sequences' lengths: a
// worker's range is the end of one pair, whole pairs, and the start of
// another.  A pair inside one range is finished there; the others leave one
// partial per range, merged by dense_combine_kernel.  So a worker has at most
// two partials: slot 2w for the pair that holds the range's first unit, slot
// 2w + 1 for a pair that starts inside the range.
#pragma once
#include "kernels.cuh"

namespace csa2 {

constexpr int kDenseStep = 256;      // entries per unit
constexpr int kDenseWorkers = 76;    // most workers (one CTA pair per two SMs)

// A pair that several workers share, for the combine: its first token, how many
// tokens it has, its first partial's slot (the following ones are the even
// slots of the following workers) and how many partials (0: no such pair).
struct __align__(16) DenseShared {
  int32_t token, tokens, slot, n;
};

struct DenseArgs {
  const __nv_bfloat16 *q;      // [seqs][n_q][64][512]
  const uint8_t *kv;           // [seqs][cap][288]
  const int32_t *n_vis;        // [seqs], or NULL: n_max entries each
  int64_t cap;
  int32_t n_max;
  int32_t seqs, n_q;
  int32_t workers;
  int32_t split;               // combine: warps per head (1, 2, 4 or 8)
  __nv_bfloat16 *out;          // [seqs][n_q][64][512]
  float *lse;                  // [seqs][n_q][64] or NULL
  const float *own_out;        // another part of each token's softmax to merge in
  const float *own_lse;        // (fp32 rows and natural log-sum-exps), or NULL
  __half *part;                // [2 workers][2 tokens][64][512] normalised partials
  float *part_lse;             // [2 workers][2 tokens][64] their natural log-sum-exps
  DenseShared *shared;         // [workers], by pair if there are fewer pairs than workers, else by first worker
};

__device__ __forceinline__ int dense_len(const DenseArgs &a, int b) {
  if (!a.n_vis) return a.n_max;
  const int n = __ldg(a.n_vis + b);
  if (n < 0 || n > a.n_max) set_error(CSA2_DEV_ERR_NVIS);
  return n < 0 ? 0 : n > a.n_max ? a.n_max : n;
}

__device__ __forceinline__ int dense_steps(int n) { return n / kDenseStep + (n % kDenseStep ? 1 : 0); }

// The units of all sequences, and how many workers have a range (a.workers,
// but no more than there are units: no range is empty); a whole warp calls it.
__device__ __forceinline__ void dense_units(const DenseArgs &a, int lane, int64_t &total, int &workers) {
  int64_t steps = 0;
  if (!a.n_vis) {
    steps = (int64_t)a.seqs * dense_steps(a.n_max);
  } else {
    for (int i = lane; i < a.seqs; i += 32) steps += dense_steps(dense_len(a, i));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) steps += __shfl_xor_sync(0xffffffffu, steps, o);
  }
  total = steps * ((a.n_q + 1) / 2);
  workers = (int)(total < a.workers ? total : a.workers);
}

// a / b for a >= 0, b > 0: in 32 bits where they fit (a 64-bit division takes
// some hundred instructions, several of them in a row before the first load).
__device__ __forceinline__ int64_t dense_div(int64_t a, int64_t b) {
  return (a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// Worker w's range starts at unit floor(w total / workers).
__device__ __forceinline__ int64_t dense_range(int64_t total, int workers, int w) {
  return dense_div(total * w, workers);
}

// The worker whose range holds unit u (the last one for any u past the line).
__device__ __forceinline__ int dense_worker(int64_t total, int workers, int64_t u) {
  return u < total ? (int)dense_div((u + 1) * workers - 1, total) : workers - 1;
}

// The sequence that holds unit u and its first unit; a whole warp calls it (32
// lengths at a time: with a length per step, the last worker of 4,096 short
// sequences would set out 80 us late).  b = a.seqs if the lengths have shrunk
// since they were counted: this walk and dense_next end then, whatever n_vis
// holds while the call runs.
__device__ __forceinline__ void dense_find(const DenseArgs &a, int64_t u, int lane, int &b, int64_t &seq0) {
  const int64_t pairs = (a.n_q + 1) / 2;
  if (!a.n_vis) {
    const int64_t s = pairs * dense_steps(a.n_max);
    b = (int)dense_div(u, s);
    seq0 = b * s;
    return;
  }
  int64_t base = 0;
  for (int c = 0; c < a.seqs; c += 32) {
    int64_t x = c + lane < a.seqs ? pairs * dense_steps(dense_len(a, c + lane)) : 0;
    const int64_t own = x;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, u < base + x);
    if (past) {
      const int from = __ffs(past) - 1;
      b = c + from;
      seq0 = base + __shfl_sync(0xffffffffu, x - own, from);
      return;
    }
    base += __shfl_sync(0xffffffffu, x, 31);
  }
  b = a.seqs;
  seq0 = base;
}

// A worker's walk over its range, one segment (a pair and its steps inside
// the range) at a time.
struct DenseWalk {
  int64_t at, end;        // the unit that comes next, the range's end
  int64_t start;          // the range's first unit
  int64_t seq0;           // first unit of sequence b
  int b, len, steps;      // the sequence, its entries and steps
};

struct DenseSegment {
  int b, pair;
  int len;                // entries of the sequence
  int s0, s1;             // steps [s0, s1) of the pair
  bool whole;             // every step of the pair
  int slot;               // partial slot otherwise
};

// The walk of worker w, the units of all pairs and the workers that have a
// range; a whole warp calls it.
__device__ __forceinline__ DenseWalk dense_walk(const DenseArgs &a, int w, int lane, int64_t &total, int &workers) {
  DenseWalk k;
  k.seq0 = 0;
  k.b = k.len = 0;
  if (a.n_vis && a.seqs <= 32) {   // one length per lane, one scan
    const int len = lane < a.seqs ? dense_len(a, lane) : 0;
    const int64_t own = (int64_t)((a.n_q + 1) / 2) * dense_steps(len);
    int64_t x = own;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    total = __shfl_sync(0xffffffffu, x, 31);
    workers = (int)(total < a.workers ? total : a.workers);
    k.start = k.at = w < workers ? dense_range(total, workers, w) : 0;
    k.end = w < workers ? dense_range(total, workers, w + 1) : 0;
    const uint32_t past = __ballot_sync(0xffffffffu, k.at < x);
    if (past) {
      k.b = __ffs(past) - 1;
      k.seq0 = __shfl_sync(0xffffffffu, x - own, k.b);
      k.len = __shfl_sync(0xffffffffu, len, k.b);
    }
  } else {
    dense_units(a, lane, total, workers);
    k.start = k.at = w < workers ? dense_range(total, workers, w) : 0;
    k.end = w < workers ? dense_range(total, workers, w + 1) : 0;
    if (k.at < k.end) {
      dense_find(a, k.at, lane, k.b, k.seq0);
      if (k.b < a.seqs)
        k.len = dense_len(a, k.b);
      else
        k.end = k.at;
    }
  }
  k.steps = dense_steps(k.len);
  return k;
}

// The next segment; false at the range's end.  Any thread, no warp operation.
__device__ __forceinline__ bool dense_next(const DenseArgs &a, int w, DenseWalk &k, DenseSegment &g) {
  if (k.at >= k.end) return false;
  const int64_t pairs = (a.n_q + 1) / 2;
  while (k.at >= k.seq0 + pairs * k.steps) {   // at < end <= total: some sequence holds it
    if (k.b + 1 >= a.seqs) return false;
    k.seq0 += pairs * k.steps;
    ++k.b;
    k.len = dense_len(a, k.b);
    k.steps = dense_steps(k.len);
  }
  const int64_t rel = k.at - k.seq0;
  g.b = k.b;
  g.pair = (int)dense_div(rel, k.steps);
  g.len = k.len;
  g.s0 = (int)(rel - (int64_t)g.pair * k.steps);
  const int64_t left = k.end - k.at;
  g.s1 = left < k.steps - g.s0 ? g.s0 + (int)left : k.steps;
  g.whole = g.s0 == 0 && g.s1 == k.steps;
  g.slot = 2 * w + (k.at == k.start ? 0 : 1);
  k.at += g.s1 - g.s0;
  return true;
}

}  // namespace csa2
