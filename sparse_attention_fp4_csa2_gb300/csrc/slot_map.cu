// From the lengths of a step's requests, the positions and cache rows that the
// writers take (csa2_slot_map).
//
// Token r of sequence b sits at position p = ctx[b] + r and has row p mod ring
// of the sequence's ring; the entries that the step completes are ctx[b] / m ..
// (ctx[b] + new[b]) / m - 1, entry e at position m e + m - 1 and row e of the
// sequence's main cache.  Token i of the packed step belongs to the last
// sequence whose exclusive prefix sum of the lengths is at most i.
//
// What it has to move: 8 bytes a sequence in, 16 out, 20 bytes a token and 16 an
// entry out; small calls are the launch and the scan's latency.  One launch, no
// pass between CTAs: each CTA scans all the lengths itself (8,192 at most, which
// stay in L2), keeps both prefix sums and the lengths before the step in shared
// memory and takes every gridDim-th stretch of the tokens and entries, finding a
// token's sequence by binary search there.  Measured in graphs: 32 sequences of one
// token 2.8 us, 999 of five 4.9, 196,000 tokens and 98,000 entries of 64 sequences
// 4.8 (1.1 TB/s); a call from Python takes 6.6.
#include "kernels.cuh"

namespace csa2 {

namespace {

constexpr int kMapThreads = 512;

struct SlotArgs {
  const int32_t *ctx_len, *new_len;
  csa2_slot_maps out;
  int64_t cap, ring, n_tokens, n_entries;
  int32_t batch, m;
};

// Exclusive prefix sums of two counts per thread over the CTA (threads from 32 *
// warps on have none); the totals in every thread.
__device__ __forceinline__ void scan_pair(int64_t &a, int64_t &b, int64_t (*part)[2], int warps, int64_t &ta, int64_t &tb) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t a0 = a, b0 = b;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int64_t x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) {
      a += x;
      b += y;
    }
  }
  if (lane == 31) {
    part[warp][0] = a;
    part[warp][1] = b;
  }
  __syncthreads();
  ta = tb = 0;
  int64_t ba = 0, bb = 0;
  for (int w = 0; w < warps; ++w) {
    if (w == warp) {
      ba = ta;
      bb = tb;
    }
    ta += part[w][0];
    tb += part[w][1];
  }
  a += ba - a0;
  b += bb - b0;
}

__global__ void __launch_bounds__(kMapThreads) slot_map_kernel(const SlotArgs a) {
  extern __shared__ int32_t sums[];   // [batch + 1] tokens, [batch + 1] entries, [batch] tokens before the step
  __shared__ int64_t part[kMapThreads / 32][2];
  int32_t *tok = sums, *ent = sums + a.batch + 1, *ctx = ent + a.batch + 1;
  pdl_wait();
  const int per = (a.batch + blockDim.x - 1) / blockDim.x;
  const int b0 = min((int)threadIdx.x * per, a.batch), b1 = min(b0 + per, a.batch);
  int64_t t = 0, e = 0;
  for (int b = b0; b < b1; ++b) {
    const int64_t c = max(a.ctx_len[b], 0), n = max(a.new_len[b], 0);
    t += n;
    e += (c + n) / a.m - c / a.m;
  }
  int64_t tokens, entries;
  scan_pair(t, e, part, ((a.batch + per - 1) / per + 31) / 32, tokens, entries);
  const bool first = blockIdx.x == 0;
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    const int32_t c0 = a.ctx_len[b], n0 = a.new_len[b];
    const int64_t c = max(c0, 0), n = max(n0, 0);
    // sums past 32 bits name no token of the outputs: they stay at the largest
    tok[b] = (int32_t)min(t, (int64_t)INT32_MAX);
    ent[b] = (int32_t)min(e, (int64_t)INT32_MAX);
    ctx[b] = (int32_t)c;
    t += n;
    e += (c + n) / a.m - c / a.m;
    if (first) {
      a.out.cu[b] = tok[b];
      a.out.entry_cu[b] = ent[b];
      a.out.n_vis[b] = (int32_t)min(min((c + n) / a.m, a.cap), (int64_t)INT32_MAX);
      a.out.swa_len[b] = (int32_t)min(min(c + n, a.ring), (int64_t)INT32_MAX);
      bad |= c0 < 0 || n0 < 0 || (c + n) / a.m > a.cap;
    }
  }
  if (threadIdx.x == 0) {
    tok[a.batch] = (int32_t)min(tokens, (int64_t)INT32_MAX);
    ent[a.batch] = (int32_t)min(entries, (int64_t)INT32_MAX);
    if (first) {
      a.out.cu[a.batch] = tok[a.batch];
      a.out.entry_cu[a.batch] = ent[a.batch];
      bad |= tokens > a.n_tokens || entries > a.n_entries;
    }
  }
  if (bad) set_error(CSA2_DEV_ERR_NVIS);
  __syncthreads();
  pdl_release();
  // tokens, then entries, on one line
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < a.n_tokens + a.n_entries; i += stride) {
    const bool entry = i >= a.n_tokens;
    const int64_t at = entry ? i - a.n_tokens : i;
    const int32_t *cu = entry ? ent : tok;
    int32_t seq = -1;
    int64_t pos = -1, slot = -1;
    if (at < cu[a.batch]) {
      seq = last_not_above(cu, 0, a.batch, (int32_t)at);
      const int32_t r = (int32_t)at - cu[seq];
      if (entry) {
        const int64_t e1 = (int64_t)(ctx[seq] >> (a.m - 1)) + r;
        pos = e1 * a.m + a.m - 1;
        if (e1 < a.cap) slot = seq * a.cap + e1;
      } else {
        pos = (int64_t)ctx[seq] + r;
        // (a row that a later token of the step takes again is written once, by that one)
        if (tok[seq + 1] - tok[seq] - r <= a.ring)
          slot = (int64_t)seq * a.ring +
                 (((uint64_t)pos | (uint64_t)a.ring) >> 32 ? pos % a.ring : (uint32_t)pos % (uint32_t)a.ring);
      }
    }
    if (!entry) a.out.tok_seq[at] = seq;
    (entry ? a.out.entry_pos : a.out.pos)[at] = pos;
    (entry ? a.out.slot : a.out.swa_slot)[at] = slot;
  }
}

}  // namespace

cudaError_t launch_slot_map(const int32_t *ctx_len, const int32_t *new_len, int32_t batch, int32_t m, int64_t cap,
                            int64_t ring, int64_t n_tokens, int64_t n_entries, const csa2_slot_maps &out, int num_sms,
                            cudaStream_t stream) {
  SlotArgs a;
  a.ctx_len = ctx_len;
  a.new_len = new_len;
  a.out = out;
  a.cap = cap;
  a.ring = ring;
  a.n_tokens = n_tokens;
  a.n_entries = n_entries;
  a.batch = batch;
  a.m = m;
  int64_t ctas = (n_tokens + n_entries + kMapThreads - 1) / kMapThreads;
  // (a CTA per SM: every one scans all the lengths; with four per SM 196,000 tokens
  // and 98,000 entries of 64 sequences took 9.3 us against 4.7)
  ctas = ctas < 1 ? 1 : ctas < num_sms ? ctas : num_sms;
  const size_t smem = ((size_t)3 * batch + 2) * sizeof(int32_t);
  if (smem > 48 * 1024) {   // (less needs no attribute)
    // the largest batch's, so that a call of another thread's never lowers it
    const cudaError_t e = cudaFuncSetAttribute(slot_map_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)((3 * kMaxMapBatch + 2) * sizeof(int32_t)));
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(slot_map_kernel, dim3((unsigned)ctas), dim3(kMapThreads), smem, stream, 0u, a);
}

}  // namespace csa2
