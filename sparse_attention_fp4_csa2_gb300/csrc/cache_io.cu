// csa2_swa_quant_write and the cache read-backs (csa2_kv_read, csa2_swa_read,
// csa2_indexer_k_read).
//
// Both directions are streams with a few operations per byte, so they are
// bound by HBM for many rows and by launch latency for a decode step's few.
// One warp handles a row (half a warp an indexer key) and every load and
// store of a warp covers contiguous 16-, 8- or 4-byte pieces.
#include "kernels.cuh"
#include "rope_turns.h"

namespace csa2 {

static_assert(kRopePairs == ROPE_DIM / 2, "one frequency per rotated pair");

namespace {

// Positions of kv_quant_write: [0, 2^22).
constexpr int64_t kMaxRopePos = int64_t(1) << 22;

// cos and sin of position p's rotation for one frequency: the phase in fixed
// point (rope_turns.h, so no double-precision reduction is needed: GB300 has
// few FP64 units, and 32,768 rows of double sincos alone would take over 100 us
// against 7.5 us of memory traffic), the quarter turns taken out exactly and
// the rest through sincospif: within 2 ulp of fp32 plus 2^-39.
__device__ __forceinline__ void rope_cos_sin(uint64_t step, int64_t p, float &c, float &s) {
  uint32_t quarter;
  const float half_turns = rope_phase(step, p, quarter);
  float sr, cr;
  sincospif(half_turns, &sr, &cr);
  const bool odd = quarter & 1;
  const float a = odd ? sr : cr, b = odd ? cr : sr;
  c = ((quarter + 1) & 2) ? -a : a;
  s = (quarter & 2) ? -b : b;
}

__device__ __forceinline__ uint32_t cvt_e4m3x2(float hi, float lo) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// x / s by the reciprocal r = fl(1 / s) and one correction with the exact
// remainder (P. Markstein, "Computation of elementary functions on the IBM
// RISC System/6000 processor", 1990): the correctly rounded quotient, unless
// it lies within 2^-46 of the middle of two floats.  s, r normal and positive;
// a zero keeps its sign.
__device__ __forceinline__ float quotient(float x, float s, float r) {
  const float q = x * r;
  return copysignf(fmaf(fmaf(-q, s, x), r, q), x);
}

// A warp writes R rows, one after the other, all loads first.  Lane l owns
// channels 16 l .. + 15: it loads 32 bytes and stores 16 bytes of codes.  The
// RoPE pairs, which lanes 28 to 31 hold, pass through shared memory so that
// lane j rotates pair j (products and sums rounded separately).  Latency bounds
// it (the pass through shared memory, then the loads, at 41 % of the warps; the
// schedulers are 53 % busy, DRAM 25 %), not HBM: 32,768 rows (50 MB, 7.5 us at
// the copy rate) took 22.5 us with a rounded division per channel and shuffled
// rotations, 13.2 us in this form.  One row per warp is slower for many rows
// (14.6 us).
template <int R>
__global__ void __launch_bounds__(256) swa_quant_write_kernel(const __nv_bfloat16 *__restrict__ latent, int64_t n,
                                                              const int64_t *__restrict__ pos,
                                                              const int64_t *__restrict__ slot,
                                                              uint8_t *__restrict__ swa, float *__restrict__ swa_scale,
                                                              int64_t rows, const RopeTurns turns) {
  pdl_wait();   // the inputs' producer is complete past here (programmatic launch)
  __shared__ __align__(16) float tails[8][ROPE_DIM];
  const int lane = threadIdx.x & 31;
  const int64_t e0 = ((int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * R;
  uint4 u[R][2];
  int64_t row[R], p[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    row[r] = -1;
    p[r] = 0;
    if (e0 + r < n) {
      const uint4 *src = reinterpret_cast<const uint4 *>(latent + (e0 + r) * D + lane * 16);
      u[r][0] = ld_nc_v4(src);
      u[r][1] = ld_nc_v4(src + 1);
      row[r] = __ldg(slot + e0 + r);
      if (pos) p[r] = __ldg(pos + e0 + r);
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (e0 + r >= n) return;
    if (row[r] == -1) continue;   // a place without a token
    if (row[r] < 0 || row[r] >= rows || p[r] < 0 || p[r] >= kMaxRopePos) {
      if (lane == 0) set_error(CSA2_DEV_ERR_INDEX);
      continue;
    }
    const uint32_t w[8] = {u[r][0].x, u[r][0].y, u[r][0].z, u[r][0].w, u[r][1].x, u[r][1].y, u[r][1].z, u[r][1].w};
    float x[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    if (pos) {
      float cj, sj;
      rope_cos_sin(turns.step[lane], p[r], cj, sj);
      // lanes 28 .. 31 hold the 32 pairs: each lane takes its own through shared memory
      float *tail = tails[threadIdx.x >> 5];
      if (lane >= (D - ROPE_DIM) / 16) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float4 *>(tail + (lane - (D - ROPE_DIM) / 16) * 16 + 4 * i) =
              make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
      }
      __syncwarp();
      const float2 v = *reinterpret_cast<const float2 *>(tail + 2 * lane);
      *reinterpret_cast<float2 *>(tail + 2 * lane) =
          make_float2(__fsub_rn(__fmul_rn(v.x, cj), __fmul_rn(v.y, sj)), __fadd_rn(__fmul_rn(v.x, sj), __fmul_rn(v.y, cj)));
      __syncwarp();
      if (lane >= (D - ROPE_DIM) / 16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 o = *reinterpret_cast<const float4 *>(tail + (lane - (D - ROPE_DIM) / 16) * 16 + 4 * i);
          x[4 * i] = o.x;
          x[4 * i + 1] = o.y;
          x[4 * i + 2] = o.z;
          x[4 * i + 3] = o.w;
        }
      }
      __syncwarp();
    }
    float amax = 0.0f;   // NaNs do not count
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
    const float scale = __fdiv_rn(amax, 448.0f);
    uint32_t q[4] = {0, 0, 0, 0};
    if (scale >= 0x1p-100f && scale <= 0x1p+100f) {
      const float inv = __frcp_rn(scale);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        q[i >> 1] |= cvt_e4m3x2(quotient(x[2 * i + 1], scale, inv), quotient(x[2 * i], scale, inv)) << (16 * (i & 1));
    } else if (scale > 0.0f) {
#pragma unroll 1
      for (int i = 0; i < 8; ++i) {
        float lo = 0.0f, hi = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j == i) {
            lo = x[2 * j];
            hi = x[2 * j + 1];
          }
        const uint32_t c = cvt_e4m3x2(__fdiv_rn(hi, scale), __fdiv_rn(lo, scale)) << (16 * (i & 1));
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j == i >> 1) q[j] |= c;
      }
    } else {   // zeros, but a NaN beside nothing else stays one
#pragma unroll
      for (int i = 0; i < 16; ++i) q[i >> 2] |= (x[i] != x[i] ? 0x7Fu : 0u) << (8 * (i & 3));
    }
    *reinterpret_cast<uint4 *>(swa + row[r] * D + lane * 16) = make_uint4(q[0], q[1], q[2], q[3]);
    if (lane == 0) swa_scale[row[r]] = scale;
  }
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// x s rounded to odd: of the two floats around the product, which differ by
// one in the last place unless it is exact, the one whose last bit is set (S.
// Boldo, G. Melquiond, "Emulation of FMA and correctly rounded sums: proved
// algorithms using rounding to odd", 2008).  A second rounding to fewer bits
// is then the product's own.
__device__ __forceinline__ float mul_odd(float x, float s) {
  const float down = __fmul_rd(x, s), up = __fmul_ru(x, s);
  return __float_as_uint(down) & 1 ? down : up;
}

// half2 (a pair of decoded codes) times a scale, rounded once to bf16.
// EXACT: the products have at most 24 bits (E2M1 codes).
template <bool EXACT>
__device__ __forceinline__ uint32_t scaled_bf16x2(uint32_t h2, float scale) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h2));
  return EXACT ? bf16x2(f.x * scale, f.y * scale) : bf16x2(mul_odd(f.x, scale), mul_odd(f.y, scale));
}

// UE8M0 byte -> 2^(b - 127) (255 is NaN).
__device__ __forceinline__ float ue8m0_to_f32(uint32_t b) {
  return b == 0 ? __uint_as_float(0x00400000u) : b == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(b << 23);
}

enum { kFmtKv = 0, kFmtSwa = 1, kFmtIk = 2 };

struct ReadArgs {
  const uint8_t *codes;    // kv entries, SWA rows or MXFP4 code plane
  const void *scales;      // SWA: fp32 [rows]; MXFP4: bytes [rows][4]
  const int32_t *idx;      // [batch][k] or NULL
  __nv_bfloat16 *out;      // [batch][k][512 or 128]
  int64_t cap, total;      // rows per sequence, batch * k
  int64_t k;
};

// (sequence, place) of output row i.
__device__ __forceinline__ void locate(const ReadArgs &a, int64_t i, int64_t &b, int64_t &j) {
  if (a.total >> 32)
    b = i / a.k;
  else
    b = (uint32_t)i / (uint32_t)a.k;   // a 64-bit division is four times the instructions
  j = i - b * a.k;
}

// One output piece of 8 channels: its codes and its scale.
struct Piece {
  uint2 c;
  float scale;
};

template <int FMT>
__device__ __forceinline__ Piece load_piece(const ReadArgs &a, int64_t row, int piece) {
  Piece r;
  if (FMT == kFmtKv) {
    const uint8_t *src = a.codes + row * ENTRY_BYTES;
    r.c = make_uint2(ld_nc_u32(src + 4 * piece), 0u);
    r.scale = e4m3_to_f32(__ldg(src + 256 + (piece >> 1)));
  } else if (FMT == kFmtSwa) {
    r.c = __ldg(reinterpret_cast<const uint2 *>(a.codes + row * D + 8 * piece));
    r.scale = __ldg(static_cast<const float *>(a.scales) + row);
  } else {
    r.c = make_uint2(ld_nc_u32(a.codes + row * (DI / 2) + 4 * piece), 0u);
    r.scale = ue8m0_to_f32(__ldg(static_cast<const uint8_t *>(a.scales) + row * 4 + (piece >> 2)));
  }
  return r;
}

template <int FMT>
__device__ __forceinline__ uint4 decode_piece(const Piece &p) {
  uint32_t h[4];
  if (FMT == kFmtSwa) {
    h[0] = e4m3x2_to_half2((uint16_t)(p.c.x & 0xFFFF));
    h[1] = e4m3x2_to_half2((uint16_t)(p.c.x >> 16));
    h[2] = e4m3x2_to_half2((uint16_t)(p.c.y & 0xFFFF));
    h[3] = e4m3x2_to_half2((uint16_t)(p.c.y >> 16));
  } else {
    e2m1x8_to_half2x4(p.c.x, h);
  }
  constexpr bool kExact = FMT != kFmtSwa;
  return make_uint4(scaled_bf16x2<kExact>(h[0], p.scale), scaled_bf16x2<kExact>(h[1], p.scale),
                    scaled_bf16x2<kExact>(h[2], p.scale), scaled_bf16x2<kExact>(h[3], p.scale));
}

// Output rows in pieces of 8 channels (16 bytes), 64 per entry and window
// row (lane l stores pieces l and 32 + l) and 16 per indexer key (half a warp
// each, so a warp step covers two keys).  A warp takes R consecutive steps
// and issues all their loads before the first store.  HBM bounds it for many
// rows: 262,144 main-KV entries in order (344 MB) in 54.4 us, 6.32 TB/s, 0.93 of
// the copy rate; few rows are a launch (1.3 us in a graph for 128 window rows).
template <int FMT, int R>
__global__ void __launch_bounds__(256) cache_read_kernel(const ReadArgs a) {
  pdl_wait();
  constexpr int kHalves = FMT == kFmtIk ? 1 : 2;   // pieces per lane and row
  constexpr int kRows = FMT == kFmtIk ? 2 : 1;     // rows per warp step
  constexpr int kWidth = FMT == kFmtIk ? DI : D;
  const int lane = threadIdx.x & 31;
  const int sub = FMT == kFmtIk ? lane >> 4 : 0;
  const int piece = FMT == kFmtIk ? lane & 15 : lane;
  const int64_t first = ((int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * (R * kRows) + sub;
  if (first - sub >= a.total) return;
  int64_t row[R], b, j;
  Piece p[R][kHalves];
  locate(a, first, b, j);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t i = first + r * kRows;
    row[r] = -1;
    if (i < a.total) {
      const int64_t id = a.idx ? (int64_t)__ldg(a.idx + i) : j;
      if (id >= a.cap) {
        if (piece == 0) set_error(CSA2_DEV_ERR_INDEX);
      } else if (id >= 0) {
        row[r] = b * a.cap + id;
      }
    }
    for (j += kRows; j >= a.k; j -= a.k) ++b;
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
      if (row[r] >= 0) p[r][h] = load_piece<FMT>(a, row[r], piece + 32 * h);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t i = first + r * kRows;
    if (i >= a.total) continue;
    uint4 *dst = reinterpret_cast<uint4 *>(a.out + i * kWidth);
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
      dst[piece + 32 * h] = row[r] >= 0 ? decode_piece<FMT>(p[r][h]) : make_uint4(0, 0, 0, 0);
  }
}

template <int FMT>
cudaError_t launch_read(const ReadArgs &a, cudaStream_t stream) {
  constexpr int kRows = FMT == kFmtIk ? 2 : 1;
  const int64_t steps = (a.total + kRows - 1) / kRows;
  // few rows: one step per warp and one warp per block, over all SMs (in a graph,
  // entries: 512 rows 1.6 us against 2.8 with 8 warps of 4 steps, 2,048 rows 2.4
  // against 2.8, 4,096 rows 3.5 against 2.8, 32,768 rows 17.8 against 6.8)
  if (steps <= 2048)
    return launch_pdl(cache_read_kernel<FMT, 1>, dim3((unsigned)steps), dim3(32), 0, stream, 0u, a);
  const int64_t blocks = (steps + 31) / 32;   // 8 warps x 4 steps
  return launch_pdl(cache_read_kernel<FMT, 4>, dim3((unsigned)blocks), dim3(256), 0, stream, 0u, a);
}

}  // namespace

cudaError_t launch_swa_quant_write(const void *latent, int64_t n, const int64_t *pos, const int64_t *slot, uint8_t *swa,
                                   float *swa_scale, int64_t rows, float rope_theta, cudaStream_t stream) {
  // the frequencies of the last theta of this host thread (32 powers: 4 us)
  thread_local RopeTurns turns = {};
  thread_local float theta = 0.0f;
  if (pos && theta != rope_theta) {
    turns = rope_turns(rope_theta);
    theta = rope_theta;
  }
  const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(latent);
  // a decode step's few rows: one warp per block, so that they spread over the
  // SMs (in a graph, 128 rows 2.0 us against 3.0 with 8 warps of 2 rows, 1,024
  // rows 2.4 against 3.1, 2,048 rows 3.0 against 3.1, 8,192 rows 6.1 against 5.0)
  if (n <= 1024)
    return launch_pdl(swa_quant_write_kernel<1>, dim3((unsigned)n), dim3(32), 0, stream, 0u, src, n, pos, slot, swa,
                      swa_scale, rows, turns);
  return launch_pdl(swa_quant_write_kernel<2>, dim3((unsigned)((n + 15) / 16)), dim3(256), 0, stream, 0u, src, n, pos,
                    slot, swa, swa_scale, rows, turns);
}

cudaError_t launch_kv_read(const uint8_t *kv, int64_t batch, int64_t cap, const int32_t *idx, int64_t k, void *out,
                           cudaStream_t stream) {
  const ReadArgs a{kv, nullptr, idx, static_cast<__nv_bfloat16 *>(out), cap, batch * k, k};
  return launch_read<kFmtKv>(a, stream);
}

cudaError_t launch_swa_read(const uint8_t *swa, const float *swa_scale, int64_t batch, int64_t rows, const int32_t *idx,
                            int64_t k, void *out, cudaStream_t stream) {
  const ReadArgs a{swa, swa_scale, idx, static_cast<__nv_bfloat16 *>(out), rows, batch * k, k};
  return launch_read<kFmtSwa>(a, stream);
}

cudaError_t launch_indexer_k_read(const uint8_t *k_fp4, int64_t batch, int64_t cap, const int32_t *idx, int64_t k,
                                  void *out, cudaStream_t stream) {
  const ReadArgs a{k_fp4, k_fp4 + batch * cap * (DI / 2), idx, static_cast<__nv_bfloat16 *>(out), cap, batch * k, k};
  return launch_read<kFmtIk>(a, stream);
}

}  // namespace csa2
