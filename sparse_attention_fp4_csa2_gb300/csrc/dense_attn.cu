// Dense readout: every entry of a sequence's main-KV cache, for query tokens
// that all see the same entries (csa2_cross_attn), and the shared prefix of
// csa2_prefix_attn.  For a token and head h over entries n < N:
//   o_h = sum_n softmax_n(q_h . k_n / sqrt(512)) k_n,
// key = value = the dequantised 512-d entry.
//
// This is the plain form of the kernel: fp32 on the CUDA cores, one CTA per
// token of a unit's pair, entries dequantised 32 at a time into shared memory.
#include "dense_plan.cuh"

namespace csa2 {

namespace {

constexpr float kScale = 0.04419417382415922f;   // 1 / sqrt(512)
constexpr int kTile = 32;
constexpr int kPitch = D + 1;
constexpr size_t kSmem = (size_t)(H * D + kTile * kPitch) * 4;

__device__ __forceinline__ float e2m1(uint32_t c) {
  const float mag = (c & 6) ? __uint_as_float((((c >> 1) & 3) + 126u) << 23 | (c & 1) << 22) : 0.5f * (c & 1);
  return (c & 8) ? -mag : mag;
}

__global__ void __launch_bounds__(256) dense_attn_kernel(const DenseArgs a) {
  extern __shared__ float smem[];
  float *qs = smem, *ks = smem + H * D;
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int w = blockIdx.x >> 1, r = blockIdx.x & 1;
  DenseWalk walk = dense_walk(a, w, lane);
  DenseSegment g;
  while (dense_next(a, w, walk, g)) {
    const int t = 2 * g.pair + r;
    if (t >= a.n_q) continue;
    const int64_t token = (int64_t)g.b * a.n_q + t;
    __syncthreads();
    for (int i = tid; i < H * D; i += blockDim.x) qs[i] = __bfloat162float(a.q[token * H * D + i]) * kScale;
    float m[8], l[8], acc[8][16];
#pragma unroll
    for (int h = 0; h < 8; ++h) {
      m[h] = -INFINITY;
      l[h] = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[h][i] = 0.0f;
    }
    const int64_t n1 = g.s1 * kDenseStep < g.len ? g.s1 * kDenseStep : g.len;
    for (int64_t n0 = g.s0 * kDenseStep; n0 < n1; n0 += kTile) {
      __syncthreads();
      for (int i = tid; i < kTile * 256; i += blockDim.x) {
        const int key = i >> 8, c = i & 255;
        float lo = 0.0f, hi = 0.0f;
        if (n0 + key < n1) {
          const uint8_t *e = a.kv + ((int64_t)g.b * a.cap + n0 + key) * ENTRY_BYTES;
          const float s = e4m3_to_f32(e[256 + (c >> 3)]);
          lo = e2m1(e[c] & 15) * s;
          hi = e2m1(e[c] >> 4) * s;
        }
        ks[key * kPitch + 2 * c] = lo;
        ks[key * kPitch + 2 * c + 1] = hi;
      }
      __syncthreads();
      float x[8];
#pragma unroll
      for (int h = 0; h < 8; ++h) x[h] = 0.0f;
      for (int d = 0; d < D; ++d) {
        const float k = ks[lane * kPitch + d];
#pragma unroll
        for (int h = 0; h < 8; ++h) x[h] = fmaf(qs[(warp * 8 + h) * D + d], k, x[h]);
      }
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        if (n0 + lane >= n1) x[h] = -INFINITY;
        float mx = x[h];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float mn = fmaxf(m[h], mx), f = expf(m[h] - mn);
        x[h] = expf(x[h] - mn);
        float s = x[h];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        l[h] = l[h] * f + s;
        m[h] = mn;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[h][i] *= f;
      }
      for (int k = 0; k < kTile; ++k) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = ks[k * kPitch + lane + 32 * i];
#pragma unroll
        for (int h = 0; h < 8; ++h) {
          const float p = __shfl_sync(0xffffffffu, x[h], k);
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[h][i] = fmaf(p, v[i], acc[h][i]);
        }
      }
    }
    // a whole pair is finished here (with the other part of the softmax, if
    // any); the rest leave a normalised partial
#pragma unroll
    for (int h = 0; h < 8; ++h) {
      const int head = warp * 8 + h;
      const float lse = m[h] + logf(l[h]), inv = 1.0f / l[h];
      if (g.whole) {
        const int64_t row = token * H + head;
        float wd = 1.0f, wo = 0.0f, tot = lse;
        if (a.own_lse) {
          const float lo = a.own_lse[row], mx = fmaxf(lse, lo);
          const float ed = expf(lse - mx), eo = expf(lo - mx);
          wd = ed / (ed + eo);
          wo = eo / (ed + eo);
          tot = mx + logf(ed + eo);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int d = lane + 32 * i;
          float o = acc[h][i] * inv * wd;
          if (a.own_lse) o += wo * a.own_out[row * D + d];
          a.out[row * D + d] = __float2bfloat16_rn(o);
        }
        if (lane == 0 && a.lse) a.lse[row] = tot;
      } else {
        const int64_t row = ((int64_t)g.slot * 2 + r) * H + head;
#pragma unroll
        for (int i = 0; i < 16; ++i) a.part[row * D + lane + 32 * i] = __float2half_rn(acc[h][i] * inv);
        if (lane == 0) a.part_lse[row] = lse;
      }
    }
  }
}

// One CTA per token: the token's partials (and the other part of its
// softmax) with the weights exp(lse_i - lse), lse the log-sum-exp over all of
// them.  Warp w merges heads 8w .. 8w + 7; lane l owns channels 16 l .. + 15.
// Partials are fp16 rows, normalised, so within the entries' range of +-2688:
// their rounding (2^-12 of a row) is below the bf16 output's (2^-9).
__global__ void __launch_bounds__(256) dense_combine_kernel(const DenseArgs a) {
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t token = blockIdx.x;
  const int b = (int)(token / a.n_q), t = (int)(token % a.n_q), r = t & 1;
  int64_t before, total;
  int workers;
  dense_units(a, b, lane, before, total, workers);
  const int64_t steps = dense_steps(dense_len(a, b));
  const int64_t u0 = before + (int64_t)(t >> 1) * steps;
  int w0 = 0, w1 = -1;   // no segment
  if (steps > 0) {
    w0 = dense_worker(total, workers, u0);
    w1 = dense_worker(total, workers, u0 + steps - 1);
    if (w0 == w1) return;   // finished by its worker
  }
#pragma unroll 1
  for (int h = 0; h < 8; ++h) {
    const int head = warp * 8 + h;
    const int64_t row = token * H + head;
    auto part_row = [&](int w) {
      const int slot = 2 * w + (dense_range(total, workers, w) >= u0 ? 0 : 1);
      return ((int64_t)slot * 2 + r) * H + head;
    };
    float mx = a.own_lse ? a.own_lse[row] : -INFINITY;
    for (int w = w0; w <= w1; ++w) mx = fmaxf(mx, a.part_lse[part_row(w)]);
    float acc[16], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
    if (mx > -INFINITY) {
      if (a.own_lse) {
        const float e = expf(a.own_lse[row] - mx);
        sum = e;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = e * a.own_out[row * D + lane * 16 + i];
      }
      for (int w = w0; w <= w1; ++w) {
        const int64_t pr = part_row(w);
        const float e = expf(a.part_lse[pr] - mx);
        sum += e;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = fmaf(e, __half2float(a.part[pr * D + lane * 16 + i]), acc[i]);
      }
    }
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) a.out[row * D + lane * 16 + i] = __float2bfloat16_rn(acc[i] * inv);
    if (lane == 0 && a.lse) a.lse[row] = sum > 0.0f ? mx + logf(sum) : -INFINITY;
  }
}

}  // namespace

size_t dense_scratch_bytes() {
  return (size_t)2 * kDenseWorkers * 2 * H * (D * sizeof(__half) + sizeof(float));
}

cudaError_t launch_dense_attn(const void *q, const uint8_t *kv, const int32_t *n_vis, int64_t n_max, int64_t cap,
                              int32_t seqs, int32_t n_q, void *out, float *lse, const float *own_out,
                              const float *own_lse, void *scratch, int num_sms, cudaStream_t stream, int *launches) {
  DenseArgs a;
  a.q = static_cast<const __nv_bfloat16 *>(q);
  a.kv = kv;
  a.n_vis = n_vis;
  a.n_max = n_max;
  a.cap = cap;
  a.seqs = seqs;
  a.n_q = n_q;
  const int64_t most = (int64_t)seqs * ((n_q + 1) / 2) * ((n_max + kDenseStep - 1) / kDenseStep);
  const int64_t workers = most < num_sms / 2 ? most : num_sms / 2;
  a.workers = (int32_t)(workers < 1 ? 1 : workers > kDenseWorkers ? kDenseWorkers : workers);
  a.out = static_cast<__nv_bfloat16 *>(out);
  a.lse = lse;
  a.own_out = own_out;
  a.own_lse = own_lse;
  a.part = static_cast<__half *>(scratch);
  a.part_lse = reinterpret_cast<float *>(a.part + (size_t)2 * kDenseWorkers * 2 * H * D);
  cudaError_t e = cudaSuccess;
  if (most > 0) {
    e = cudaFuncSetAttribute(dense_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(dense_attn_kernel, dim3((unsigned)(2 * a.workers)), dim3(256), kSmem, stream, 0u, a);
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  e = launch_pdl(dense_combine_kernel, dim3((unsigned)((int64_t)seqs * n_q)), dim3(256), 0, stream, 0u, a);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace csa2
