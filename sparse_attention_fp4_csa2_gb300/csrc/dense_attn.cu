// Dense readout: every entry of a sequence's main-KV cache, for query tokens
// that all see the same entries (csa2_cross_attn), and the shared prefix of
// csa2_prefix_attn.  For a token and head h over entries n < N:
//   o_h = sum_n softmax_n(q_h . k_n / sqrt(512)) k_n,
// key = value = the dequantised 512-d entry (E2M1 x E4M3, exact in fp16).
//
// Per (token, entry) this is 4 * 64 * 512 flop on 288 bytes, so it is bound by
// the tensor cores.  A pair of tokens, one per CTA of a two-CTA cluster, runs
// on tcgen05 cta_group::2 with M = 128 (64 heads of each token) and N = 256,
// the only single-token-per-SM shape that reaches the full rate (64 clocks per
// K = 16 step measured; N = 128 takes 58 of its ideal 32, and a one-CTA M = 64
// N = 256 takes 155): S = Q K^T for a step of 256 entries in 32 such steps,
// O += P V in 2 x 16.  Each CTA then needs the keys of its half of the step
// over all 512 channels (B of the first product), and its half of the channels
// over all 256 keys (B of the second).  The 512-channel fp32 accumulator takes
// half of the tensor memory and two S tiles the rest, so nothing larger fits,
// and Q takes 64 KB of shared memory and P 32 KB, so a dequantised step cannot
// stay until its second use: entries are dequantised twice, streamed through
// one ring of 16 KB slots in the order in which the products consume them.
//
// Warps of a CTA: 0-3 softmax (one thread per tensor-memory lane: a head and
// half of the step's keys), 4-11 dequantisation (entries loaded into registers
// a step ahead), 12 the products (in the even CTA).  The products' order is
//   S(0), S(1), O(0), S(2), O(1), ...
// so that the softmax of one step runs beside the next step's first product.
//
// Every wait is bounded; after one runs out every role falls through its
// waits, the CTAs meet at the end and the output is undefined
// (CSA2_DEV_ERR_TIMEOUT).
#include "dense_plan.cuh"

namespace csa2 {

namespace {

constexpr int kSoftWarps = 4, kDeqWarps = 8;
constexpr int kMmaWarpD = kSoftWarps + kDeqWarps;
constexpr int kThreadsD = (kMmaWarpD + 1) * 32;
constexpr int kSlots = 8;
constexpr int kSlotBytes = 16384;             // 128 keys x 64 channels, or 32 keys x 256 channels
constexpr int kQBytesD = H * D * 2;
constexpr int kPBytes = H * kDenseStep * 2;
constexpr int kAtomD = H * 128;               // 64 rows x 128 bytes (Q, P)
constexpr uint32_t kColOut = 256;             // tensor memory: S tiles at 0 and 128, O at 256
constexpr float kLogitD = 0.06375871295460785f;   // log2(e) / sqrt(512)
constexpr float kLn2D = 0.69314718055994531f;
// P = 2^(x - m + kBias) with a reference m that is raised only when a step
// exceeds it by 2^kLazyD: at most 2^15 (fp16), and a key 2^-31 below the
// reference still counts, so 64K such keys lose less than 2^-15 of the sum.
constexpr float kLazyD = 8.0f, kBias = 7.0f;
constexpr uint32_t kIdescS = idesc_f16(0, 0, 0, 256, 128);
constexpr uint32_t kIdescO = idesc_f16(0, 0, /*B MN-major*/ 1, 256, 128);

struct __align__(16) CtlD {
  uint64_t full[kSlots], free[kSlots];        // full: both CTAs' warps arrive at the even CTA
  uint64_t q_full, q_free, s_full[2], p_full, p_free, done;
  uint32_t tmem_base;
  volatile uint32_t abort;
  float red[2][128];
};

constexpr size_t kSmemD = 1024 + (size_t)kQBytesD + kPBytes + kSlots * kSlotBytes + sizeof(CtlD);
static_assert(kSmemD <= 232448, "dense readout exceeds the shared-memory limit");

__device__ __forceinline__ void wait_d(CtlD &S, uint64_t *bar, uint32_t parity) {
  if (S.abort) return;
  if (!mbar_wait_cluster(bar, parity)) S.abort = 1;
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// 32 channels of one entry (16 bytes of codes, their two scales in the low
// half of sc) as fp16 into chunks c0 .. c0 + 3 of a 128-byte row whose 16-byte
// chunks are XOR-swizzled by sw.
__device__ __forceinline__ void put32(uint8_t *row, int c0, int sw, const uint4 &v, uint32_t sc) {
  const uint32_t s = e4m3x2_to_half2((uint16_t)sc);
  const uint32_t s0 = __byte_perm(s, 0, 0x1010), s1 = __byte_perm(s, 0, 0x3232);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h[4];
    e2m1x8_to_half2x4(w[i], h);
    const uint32_t si = i < 2 ? s0 : s1;
    *reinterpret_cast<uint4 *>(row + (((c0 + i) ^ sw) << 4)) =
        make_uint4(hmul2_u32(h[0], si), hmul2_u32(h[1], si), hmul2_u32(h[2], si), hmul2_u32(h[3], si));
  }
}

// ---------------------------------------------------------- dequantisation
// Slot order: per segment K(0), then K(i + 1) and V(i) for each step i.
//   K(i), 8 slots: this CTA's 128 keys of the step, 64 channels per slot,
//     [128 keys][128 B];
//   V(i), 8 slots: 32 keys of the step per slot, this CTA's 256 channels,
//     [4 x 64 channels][32 keys][128 B].
// Thread (key, half) of a K slot and (64 channels, key, half) of a V slot
// handles 32 channels, 16 bytes of codes: two neighbours read a full sector
// and eight write eight different bank groups.  Keys past the sequence's
// length become zeros.
struct DeqRegs {
  uint4 v[8];
  uint32_t sc[8];
};

__device__ void dense_dequant(const DenseArgs &a, CtlD &S, uint8_t *qs, uint8_t *ring, int w, uint32_t rank, int pt,
                              int lane) {
  const int hf = pt & 1, key = pt >> 1;
  const int vkey = key & 31, vatom = key >> 5;
  uint32_t full_at[kSlots];
#pragma unroll
  for (int s = 0; s < kSlots; ++s) full_at[s] = dsmem_addr(&S.full[s], 0);
  const uint32_t q_full_at = dsmem_addr(&S.q_full, 0);
  DenseWalk walk = dense_walk(a, w, lane);
  DenseSegment g;
  uint32_t round = 0;   // 8-slot rounds so far
  uint32_t item = 0;
  DeqRegs kr, vr;
  while (dense_next(a, w, walk, g)) {
    const uint8_t *base = a.kv + (int64_t)g.b * a.cap * ENTRY_BYTES;
    auto load_k = [&](int64_t step) {
      const int64_t n = step * kDenseStep + (int)rank * 128 + key;
      if (n < g.len) {
        const uint8_t *e = base + n * ENTRY_BYTES;
#pragma unroll
        for (int p = 0; p < 8; ++p) kr.v[p] = ld_nc_v4(e + 32 * p + 16 * hf);
        const uint4 s0 = ld_nc_v4(e + 256), s1 = ld_nc_v4(e + 272);
        const uint32_t sw[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
        for (int p = 0; p < 8; ++p) kr.sc[p] = sw[p];
      } else {
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          kr.v[p] = make_uint4(0, 0, 0, 0);
          kr.sc[p] = 0;
        }
      }
    };
    auto load_v = [&](int64_t step) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t n = step * kDenseStep + 32 * j + vkey;
        if (n < g.len) {
          const uint8_t *e = base + n * ENTRY_BYTES + (int)rank * 128 + vatom * 32;
          vr.v[j] = ld_nc_v4(e + 16 * hf);
          vr.sc[j] = ld_nc_u32(base + n * ENTRY_BYTES + 256 + (int)rank * 16 + vatom * 4);
        } else {
          vr.v[j] = make_uint4(0, 0, 0, 0);
          vr.sc[j] = 0;
        }
      }
    };
    auto emit = [&](const DeqRegs &r, uint8_t *row0, int sw) {
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        if (round) wait_d(S, &S.free[s], (round - 1) & 1u);
        put32(row0 + s * kSlotBytes, 4 * hf, sw, r.v[s], hf ? r.sc[s] >> 16 : r.sc[s]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(full_at[s]);
      }
      ++round;
    };
    auto emit_k = [&]() { emit(kr, ring + key * 128, key & 7); };
    auto emit_v = [&]() { emit(vr, ring + vatom * 4096 + vkey * 128, vkey & 7); };

    load_k(g.s0);
    load_v(g.s0);
    // Q of this CTA's token, bf16 -> fp16 (zeros for the missing token of an odd count)
    const int t = 2 * g.pair + (int)rank;
    const uint4 *src = reinterpret_cast<const uint4 *>(a.q + ((int64_t)g.b * a.n_q + t) * (H * D));
    if (item) wait_d(S, &S.q_free, (item - 1) & 1u);
#pragma unroll 1
    for (int i0 = 0; i0 < H * D / 8; i0 += 256 * 8) {
      uint4 u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = t < a.n_q ? ld_nc_v4(src + i0 + i * 256 + pt) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = i0 + i * 256 + pt, r = at >> 6, c = at & 63;
        const uint32_t x[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
        uint32_t h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = half2_bits(__uint_as_float(x[j] << 16), __uint_as_float(x[j] & 0xFFFF0000u));
        *reinterpret_cast<uint4 *>(qs + (c >> 3) * kAtomD + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
            make_uint4(h[0], h[1], h[2], h[3]);
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive_cluster(q_full_at);
    ++item;

    emit_k();
    if (g.s0 + 1 < g.s1) load_k(g.s0 + 1);
#pragma unroll 1
    for (int64_t i = g.s0; i < g.s1; ++i) {
      if (i + 1 < g.s1) {
        emit_k();
        if (i + 2 < g.s1) load_k(i + 2);
      }
      emit_v();
      if (i + 1 < g.s1) load_v(i + 1);
    }
  }
  // every slot this CTA filled has been read, and no commit is still to
  // arrive here, before the CTA ends
  if (round)
#pragma unroll 1
    for (int s = 0; s < kSlots; ++s) wait_d(S, &S.free[s], (round - 1) & 1u);
  if (item) wait_d(S, &S.q_free, (item - 1) & 1u);
}

// ---------------------------------------------------------------- products
__device__ void dense_products(const DenseArgs &a, CtlD &S, uint8_t *qs, uint8_t *ps, uint8_t *ring, uint32_t tmem,
                               int w, DenseWalk walk) {
  const uint64_t qd = smem_desc(smem_u32(qs), 16, 1024);
  const uint64_t pd = smem_desc(smem_u32(ps), 16, 1024);
  const uint64_t kd = smem_desc(smem_u32(ring), 16, 1024);
  const uint64_t vd = smem_desc(smem_u32(ring), 4096, 1024);
  DenseSegment g;
  uint32_t round = 0, item = 0, n = 0;
  while (dense_next(a, w, walk, g)) {
    const int64_t steps = g.s1 - g.s0;
    auto scores = [&](uint32_t tile) {
#pragma unroll 1
      for (int s = 0; s < kSlots; ++s) {
        wait_d(S, &S.full[s], round & 1u);
        tc_fence_after();
        const uint64_t qa = qd + (uint64_t)(s * kAtomD >> 4), kb = kd + (uint64_t)(s * kSlotBytes >> 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) mma_f16_pair(tmem + tile * 128, qa + 2 * i, kb + 2 * i, kIdescS, (s | i) ? 1u : 0u);
        mma_commit_pair(&S.free[s]);
      }
      ++round;
      mma_commit_pair(&S.s_full[tile]);
    };
    wait_d(S, &S.q_full, item & 1u);
    ++item;
    scores(n & 1u);
    if (steps == 1) mma_commit_pair(&S.q_free);
#pragma unroll 1
    for (int64_t i = 0; i < steps; ++i, ++n) {
      if (i + 1 < steps) {
        scores((n + 1) & 1u);
        if (i + 2 == steps) mma_commit_pair(&S.q_free);
      }
      wait_d(S, &S.p_full, n & 1u);
      tc_fence_after();
#pragma unroll 1
      for (int s = 0; s < kSlots; ++s) {
        wait_d(S, &S.full[s], round & 1u);
        tc_fence_after();
        const uint64_t pa = pd + (uint64_t)((s >> 1) * kAtomD >> 4) + 4 * (s & 1);
        const uint64_t vb = vd + (uint64_t)(s * kSlotBytes >> 4);
        const uint32_t acc = (i || s) ? 1u : 0u;
        mma_f16_pair(tmem + kColOut, pa, vb, kIdescO, acc);
        mma_f16_pair(tmem + kColOut + 128, pa, vb + 512, kIdescO, acc);
        mma_f16_pair(tmem + kColOut, pa + 2, vb + 128, kIdescO, 1u);
        mma_f16_pair(tmem + kColOut + 128, pa + 2, vb + 512 + 128, kIdescO, 1u);
        mma_commit_pair(&S.free[s]);
      }
      ++round;
      mma_commit_pair(&S.p_free);
    }
  }
  // every product has completed before the teardown, also after a wait ran out
  mma_commit_pair(&S.done);
  mbar_wait_cluster(&S.done, 0);
}

// ----------------------------------------------------------------- softmax
// Thread tid holds head tid % 64: of S the keys 128 (tid / 64) .. + 127 of a
// step, of O the channels 256 (tid / 64) .. + 255.
__device__ void dense_softmax(const DenseArgs &a, CtlD &S, uint8_t *ps, uint32_t tmem, int w, uint32_t rank, int tid,
                              int lane, int warp) {
  const uint32_t p_full_at = dsmem_addr(&S.p_full, 0);
  const uint32_t row = tmem + ((uint32_t)(32 * warp) << 16);
  const int h = tid & 63, kh = tid >> 6;
  uint8_t *prow = ps + 2 * kh * kAtomD + h * 128;
  DenseWalk walk = dense_walk(a, w, lane);
  DenseSegment g;
  uint32_t n = 0;
  while (dense_next(a, w, walk, g)) {
    float m = 0.0f, l = 0.0f;
#pragma unroll 1
    for (int64_t i = g.s0; i < g.s1; ++i, ++n) {
      const uint32_t st = row + (n & 1u) * 128;
      const int64_t left = g.len - i * kDenseStep;
      const int valid = (left < kDenseStep ? (int)left : kDenseStep) - 128 * kh;   // of this thread's 128 keys
      wait_d(S, &S.s_full[n & 1u], (n >> 1) & 1u);
      tc_fence_after();
      float mx = -INFINITY;
#pragma unroll 1
      for (int c = 0; c < 128; c += 32) {
        uint32_t u[32];
        tmem_ld32(st + c, u);
        tmem_ld_wait();
        if (c + 32 <= valid) {
#pragma unroll
          for (int j = 0; j < 32; ++j) mx = fmaxf(mx, __uint_as_float(u[j]));
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (c + j < valid) mx = fmaxf(mx, __uint_as_float(u[j]));
        }
      }
      S.red[n & 1u][tid] = mx;
      bar_named(1, 128);
      mx = fmaxf(mx, S.red[n & 1u][tid ^ 64]) * kLogitD;
      // O(n - 1) is complete: P is free, O may be rescaled
      if (n) wait_d(S, &S.p_free, (n - 1) & 1u);
      tc_fence_after();
      if (i == g.s0) {
        m = mx;
      } else {
        const bool raise = mx > m + kLazyD;
        if (__any_sync(0xffffffffu, raise)) {
          const float f = raise ? ex2_approx(m - mx) : 1.0f;
          if (raise) m = mx;
          l *= f;
#pragma unroll 1
          for (int c = 0; c < 256; c += 32) {
            uint32_t u[32];
            tmem_ld32(row + kColOut + c, u);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) u[j] = __float_as_uint(__uint_as_float(u[j]) * f);
            tmem_st32(row + kColOut + c, u);
          }
          tmem_st_wait();
        }
      }
      const float off = kBias - m;
#pragma unroll 1
      for (int c = 0; c < 128; c += 32) {
        uint32_t u[32];
        tmem_ld32(st + c, u);
        tmem_ld_wait();
        uint32_t pk[16];
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          float x0 = fmaf(__uint_as_float(u[j]), kLogitD, off), x1 = fmaf(__uint_as_float(u[j + 1]), kLogitD, off);
          if (c + 32 > valid) {
            if (c + j >= valid) x0 = -INFINITY;
            if (c + j + 1 >= valid) x1 = -INFINITY;
          }
          const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
          l += p0 + p1;
          pk[j >> 1] = half2_bits(p0, p1);
        }
        uint8_t *dst = prow + (c >> 6) * kAtomD;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint4 *>(dst + (((((c & 63) >> 3) + j) ^ (h & 7)) << 4)) =
              make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(p_full_at);
    }
    // ------------------------------------------------------------ segment end
    S.red[n & 1u][tid] = l;
    bar_named(1, 128);
    l += S.red[n & 1u][tid ^ 64];
    bar_named(1, 128);   // red is written again by the next step
    const float lse = (m - kBias + log2f(l)) * kLn2D;
    wait_d(S, &S.p_free, (n - 1) & 1u);
    tc_fence_after();
    const int t = 2 * g.pair + (int)rank;
    if (t >= a.n_q) continue;
    // the weights of this part and of the other part of the softmax
    const int64_t tok_row = ((int64_t)g.b * a.n_q + t) * H;
    float wd = S.abort ? 0.0f : 1.0f / l, wo = 0.0f, total = lse;
    if (g.whole && a.own_lse) {
      const float lo = a.own_lse[tok_row + h], mm = fmaxf(lse, lo);
      const float ed = expf(lse - mm), eo = expf(lo - mm);
      wd *= ed / (ed + eo);
      wo = eo / (ed + eo);
      total = mm + logf(ed + eo);
    }
    if (kh == 0) {
      if (!g.whole)
        a.part_lse[((int64_t)g.slot * 2 + rank) * H + h] = lse;
      else if (a.lse)
        a.lse[tok_row + h] = total;
    }
    // O through the warp's 8 KB of the P buffer, 64 channels at a time, so
    // that each row leaves in 128-byte pieces
    uint8_t *stage = ps + warp * 8192;
    const int h0 = 32 * (warp & 1);
#pragma unroll 1
    for (int c = 0; c < 256; c += 64) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t u[32];
        tmem_ld32(row + kColOut + c + 32 * e, u);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<float4 *>(stage + lane * 256 + (((8 * e + j) ^ (lane & 7)) << 4)) =
              make_float4(__uint_as_float(u[4 * j]) * wd, __uint_as_float(u[4 * j + 1]) * wd,
                          __uint_as_float(u[4 * j + 2]) * wd, __uint_as_float(u[4 * j + 3]) * wd);
      }
      __syncwarp();
      const int pc = lane & 15;
#pragma unroll 4
      for (int rr = 0; rr < 32; rr += 2) {
        const int r = rr + (lane >> 4);
        float4 o = *reinterpret_cast<const float4 *>(stage + r * 256 + ((pc ^ (r & 7)) << 4));
        const int d = 256 * kh + c + 4 * pc;
        if (g.whole) {
          const int64_t at = (tok_row + h0 + r) * D + d;
          if (a.own_lse) {
            const float x = __shfl_sync(0xffffffffu, wo, r);
            const float4 y = *reinterpret_cast<const float4 *>(a.own_out + at);
            o = make_float4(fmaf(x, y.x, o.x), fmaf(x, y.y, o.y), fmaf(x, y.z, o.z), fmaf(x, y.w, o.w));
          }
          const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x, o.y), hi = __floats2bfloat162_rn(o.z, o.w);
          *reinterpret_cast<uint2 *>(a.out + at) =
              make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
        } else {
          const int64_t at = (((int64_t)g.slot * 2 + rank) * H + h0 + r) * D + d;
          *reinterpret_cast<uint2 *>(a.part + at) = make_uint2(half2_bits(o.x, o.y), half2_bits(o.z, o.w));
        }
      }
      __syncwarp();
    }
    tc_fence_before();   // O is read before the next segment's products (ordered by p_full)
  }
}

__global__ void __launch_bounds__(kThreadsD, 1) dense_attn_kernel(const DenseArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *qs = base, *ps = qs + kQBytesD, *ring = ps + kPBytes;
  CtlD &S = *reinterpret_cast<CtlD *>(ring + kSlots * kSlotBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const int w = blockIdx.x >> 1;
  if (tid == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&S.full[s], 2 * kDeqWarps);
      mbar_init(&S.free[s], 1);
    }
    mbar_init(&S.q_full, 2 * kDeqWarps);
    mbar_init(&S.q_free, 1);
    mbar_init(&S.s_full[0], 1);
    mbar_init(&S.s_full[1], 1);
    mbar_init(&S.p_full, 2 * kSoftWarps);
    mbar_init(&S.p_free, 1);
    mbar_init(&S.done, 1);
    S.abort = 0;
    fence_barrier_init();
  }
  pdl_wait();   // past here the kernel before this one is complete (programmatic launch)
  __syncthreads();
  if (warp == kMmaWarpD) {
    tmem_alloc_pair(&S.tmem_base, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' barriers and tensor memory are set up
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;

  if (warp < kSoftWarps) {
    dense_softmax(a, S, ps, tmem, w, rank, tid, lane, warp);
  } else if (warp < kMmaWarpD) {
    dense_dequant(a, S, qs, ring, w, rank, tid - kSoftWarps * 32, lane);
  } else if (rank == 0) {
    const DenseWalk walk = dense_walk(a, w, lane);
    if (lane == 0) dense_products(a, S, qs, ps, ring, tmem, w, walk);
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // neither CTA reads or signals the other past here
  pdl_release();
  if (warp == kMmaWarpD) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
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
    e = cudaFuncSetAttribute(dense_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemD);
    if (e != cudaSuccess) return e;
    e = launch_pdl(dense_attn_kernel, dim3((unsigned)(2 * a.workers)), dim3(kThreadsD), kSmemD, stream, 2u, a);
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  e = launch_pdl(dense_combine_kernel, dim3((unsigned)((int64_t)seqs * n_q)), dim3(256), 0, stream, 0u, a);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace csa2
