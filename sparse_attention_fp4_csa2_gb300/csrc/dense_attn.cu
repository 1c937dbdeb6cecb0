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
constexpr int kThreadsD = (kMmaWarpD + 1) * 32;   // 128 registers a thread, no role spills
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
  uint64_t full[kSlots], free[kSlots];        // full, q_full, p_full: both CTAs arrive at the even CTA
  uint64_t q_full, q_free, s_full[2], p_full, p_free, done;
  uint32_t tmem_base;
  volatile uint32_t abort;
  float red[2][128];
};

constexpr size_t kSmemD = 1024 + (size_t)kQBytesD + kPBytes + kSlots * kSlotBytes + sizeof(CtlD);
static_assert(kSmemD <= 232448, "dense readout exceeds the shared-memory limit");

// A wait for arrivals of this CTA or of the tensor cores, and one that is also
// ordered after the other CTA's arrivals.
__device__ __forceinline__ void wait_d(CtlD &S, uint64_t *bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity) || S.abort) return;
  if (!mbar_wait(bar, parity)) S.abort = 1;
}
__device__ __forceinline__ void wait_pair(CtlD &S, uint64_t *bar, uint32_t parity) {
  if (mbar_try_wait_cluster(bar, parity) || S.abort) return;
  if (!mbar_wait_cluster(bar, parity)) S.abort = 1;
}

__device__ __forceinline__ void st_shared_v4(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ float2 half2_floats(uint32_t u) {
  return __half22float2(*reinterpret_cast<const __half2 *>(&u));
}

// ---------------------------------------------------------- dequantisation
// Slot order: per segment K(0), then K(i + 1) and V(i) for each step i.
//   K(i), 8 slots: this CTA's 128 keys of the step, 64 channels per slot,
//     [128 keys][128 B];
//   V(i), 8 slots: 32 keys of the step per slot, this CTA's 256 channels,
//     [4 x 64 channels][32 keys][128 B].
// A lane takes 32 channels (16 bytes of codes, two scales) of a key and eight
// lanes read 128 contiguous bytes of an entry, so that a load touches few
// lines: the L1 / shared-memory data pipe is what the kernel runs against
// (two lanes per key and 16 lines a load took it 16 passes).  Of K a warp holds
// 16 keys over all channels, four slots at a time; of V it fills slot `warp`
// alone.  The eight lanes of a key write four slots (or channel blocks) at
// the same offset, so each starts at another 16-byte chunk: chunk i ^ (lane %
// 8 / 2) of its four at step i, eight bank groups for eight lanes.  Keys past
// the sequence's length become zeros.
struct DeqRegs {
  uint4 v[8];
  uint32_t sc[8];
};

// 32 channels into a 128-byte swizzled row: `at` is the place of the lane's
// first chunk, chunk i of its order at ^ 16 i; o = lane % 8 / 2.
__device__ __forceinline__ void put32(uint32_t at, const uint4 &v, uint32_t sc, bool o1, bool o2) {
  const uint32_t e = e4m3x2_to_half2((uint16_t)sc);
  const uint32_t s0 = __byte_perm(e, 0, o2 ? 0x3232 : 0x1010), s1 = __byte_perm(e, 0, o2 ? 0x1010 : 0x3232);
  const uint32_t x = o1 ? v.y : v.x, y = o1 ? v.x : v.y, z = o1 ? v.w : v.z, u = o1 ? v.z : v.w;
  const uint32_t w[4] = {o2 ? z : x, o2 ? u : y, o2 ? x : z, o2 ? y : u};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h[4];
    e2m1x8_to_half2x4(w[i], h);
    const uint32_t si = i < 2 ? s0 : s1;
    st_shared_v4(at ^ (uint32_t)(i << 4), hmul2_u32(h[0], si), hmul2_u32(h[1], si), hmul2_u32(h[2], si),
                 hmul2_u32(h[3], si));
  }
}

// Q of a token, bf16 -> fp16 (zeros for the missing token of an odd count).
template <int T>
__device__ __forceinline__ void convert_q(const DenseArgs &a, const DenseSegment &g, uint32_t rank, uint8_t *qs, int i0) {
  const int t = 2 * g.pair + (int)rank;
  const uint4 *src = reinterpret_cast<const uint4 *>(a.q + ((int64_t)g.b * a.n_q + t) * (H * D));
#pragma unroll 1
  for (; i0 < H * D / 8; i0 += T * 8) {
    uint4 u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = t < a.n_q ? ld_nc_v4(src + i0 + i * T) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = i0 + i * T, r = at >> 6, c = at & 63;
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
}

__device__ void dense_dequant(const DenseArgs &a, CtlD &S, uint8_t *qs, uint8_t *ring, int w, DenseWalk walk,
                              uint32_t rank, int pt, int lane) {
  const int warp = pt >> 5, key4 = lane >> 3, c8 = lane & 7;
  const int o = c8 >> 1;
  const bool o1 = o & 1, o2 = o & 2;
  const uint32_t z = (uint32_t)((4 * (c8 & 1)) ^ key4 ^ o) << 4;
  const uint32_t k_at = smem_u32(ring) + (uint32_t)(o * kSlotBytes + (16 * warp + key4) * 128) + z;
  const uint32_t v_at = smem_u32(ring) + (uint32_t)(warp * kSlotBytes + o * 4096 + key4 * 128) + z;
  const uint32_t full_at = dsmem_addr(&S.full[0], 0), q_full_at = dsmem_addr(&S.q_full, 0);
  DenseSegment g;
  uint32_t round = 0;   // 8-slot rounds so far
  uint32_t item = 0;
  DeqRegs kr, vr;
  while (dense_next(a, w, walk, g)) {
    const uint8_t *base = a.kv + (int64_t)g.b * a.cap * ENTRY_BYTES;
    auto load_piece = [&](DeqRegs &r, int i, int n, int half) {   // channels 256 half + 32 c8 .. of entry n
      r.v[i] = make_uint4(0, 0, 0, 0);
      r.sc[i] = 0;
      if (n < g.len) {
        const uint8_t *e = base + (int64_t)n * ENTRY_BYTES;
        r.v[i] = ld_nc_v4(e + 128 * half + 16 * c8);
        r.sc[i] = ld_nc_u16(e + 256 + 16 * half + 2 * c8);
      }
    };
    auto load_k = [&](int step) {   // [channel half][4 keys]
#pragma unroll
      for (int i = 0; i < 8; ++i)
        load_piece(kr, i, step * kDenseStep + (int)rank * 128 + 16 * warp + 4 * (i & 3) + key4, i >> 2);
    };
    auto load_v = [&](int step) {   // [4 keys]
#pragma unroll
      for (int i = 0; i < 8; ++i) load_piece(vr, i, step * kDenseStep + 32 * warp + 4 * i + key4, (int)rank);
    };
    auto emit_k = [&]() {
#pragma unroll
      for (int hc = 0; hc < 2; ++hc) {
        if (round)
#pragma unroll
          for (int s = 0; s < 4; ++s) wait_d(S, &S.free[4 * hc + s], (round - 1) & 1u);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          put32((k_at + (uint32_t)(4 * hc * kSlotBytes + i * 512)) ^ (uint32_t)((i & 1) << 6), kr.v[4 * hc + i],
                kr.sc[4 * hc + i], o1, o2);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane < 4) mbar_arrive_pair(full_at + 8 * (4 * hc + lane), 1);
      }
      ++round;
    };
    auto emit_v = [&]() {
      if (round) wait_d(S, &S.free[warp], (round - 1) & 1u);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        put32((v_at + (uint32_t)(i * 512)) ^ (uint32_t)((i & 1) << 6), vr.v[i], vr.sc[i], o1, o2);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_pair(full_at + 8 * warp, kDeqWarps);
      ++round;
    };

    load_k(g.s0);
    load_v(g.s0);
    if (item) {   // the first segment's Q is the softmax warps' (they have nothing else to do then)
      wait_d(S, &S.q_free, (item - 1) & 1u);
      convert_q<kDeqWarps * 32>(a, g, rank, qs, pt);
      if (lane == 0) mbar_arrive_pair(q_full_at, 1);
    }
    ++item;

    emit_k();
    if (g.s0 + 1 < g.s1) load_k(g.s0 + 1);
#pragma unroll 1
    for (int i = g.s0; i < g.s1; ++i) {
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
    const int steps = g.s1 - g.s0;
    auto scores = [&](uint32_t tile) {
#pragma unroll 1
      for (int s = 0; s < kSlots; ++s) {
        wait_pair(S, &S.full[s], round & 1u);
        tc_fence_after();
        const uint64_t qa = qd + (uint64_t)(s * kAtomD >> 4), kb = kd + (uint64_t)(s * kSlotBytes >> 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) mma_f16_pair(tmem + tile * 128, qa + 2 * i, kb + 2 * i, kIdescS, (s | i) ? 1u : 0u);
        mma_commit_pair(&S.free[s]);
      }
      ++round;
      mma_commit_pair(&S.s_full[tile]);
    };
    wait_pair(S, &S.q_full, item & 1u);
    ++item;
    scores(n & 1u);
    if (steps == 1) mma_commit_pair(&S.q_free);
#pragma unroll 1
    for (int i = 0; i < steps; ++i, ++n) {
      if (i + 1 < steps) {
        scores((n + 1) & 1u);
        if (i + 2 == steps) mma_commit_pair(&S.q_free);
      }
      wait_pair(S, &S.p_full, n & 1u);
      tc_fence_after();
#pragma unroll 1
      for (int s = 0; s < kSlots; ++s) {
        wait_pair(S, &S.full[s], round & 1u);
        tc_fence_after();
        const uint64_t pa = pd + (uint64_t)((s >> 1) * kAtomD >> 4) + 4 * (s & 1);
        const uint64_t vb = vd + (uint64_t)(s * kSlotBytes >> 4);
        const uint32_t acc = (i || s) ? 1u : 0u;
        mma_f16_pair_a_fill(tmem + kColOut, pa, vb, kIdescO, acc);
        mma_f16_pair_a_last(tmem + kColOut + 128, pa, vb + 512, kIdescO, acc);
        mma_f16_pair_a_fill(tmem + kColOut, pa + 2, vb + 128, kIdescO, 1u);
        mma_f16_pair_a_last(tmem + kColOut + 128, pa + 2, vb + 512 + 128, kIdescO, 1u);
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
__device__ void dense_softmax(const DenseArgs &a, CtlD &S, uint8_t *qs, uint8_t *ps, uint32_t tmem, int w, DenseWalk walk,
                              uint32_t rank, int tid, int lane, int warp) {
  const uint32_t p_full_at = dsmem_addr(&S.p_full, 0);
  const uint32_t row = tmem + ((uint32_t)(32 * warp) << 16);
  const int h = tid & 63, kh = tid >> 6;
  uint8_t *prow = ps + 2 * kh * kAtomD + h * 128;
  DenseSegment g;
  {
    DenseWalk peek = walk;
    if (dense_next(a, w, peek, g)) {
      convert_q<kSoftWarps * 32>(a, g, rank, qs, tid);
      if (lane == 0) mbar_arrive_pair(dsmem_addr(&S.q_full, 0), kDeqWarps / kSoftWarps);
    }
  }
  uint32_t n = 0;
  while (dense_next(a, w, walk, g)) {
    float m = 0.0f, l = 0.0f;
#pragma unroll 1
    for (int i = g.s0; i < g.s1; ++i, ++n) {
      const uint32_t st = row + (n & 1u) * 128;
      const int left = g.len - i * kDenseStep;
      const int valid = (left < kDenseStep ? left : kDenseStep) - 128 * kh;   // of this thread's 128 keys
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
    pdl_wait();   // own_out, own_lse
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
    // O as 16-bit rows through the warp's 8 KB of the P buffer, 128 channels at
    // a time, so that every row leaves in 256-byte pieces: bf16 if it is the
    // output, else (a partial, or this part of the softmax next to the other)
    // fp16, whose rounding (2^-11 of a value) is below the output's (2^-8)
    uint8_t *stage = ps + warp * 8192;
    const int h0 = 32 * (warp & 1);
    const bool final_rows = g.whole && !a.own_lse;
    uint16_t *dst = g.whole ? reinterpret_cast<uint16_t *>(a.out) + (tok_row + h0) * D
                            : reinterpret_cast<uint16_t *>(a.part) + (((int64_t)g.slot * 2 + rank) * H + h0) * D;
    const int pc = lane & 15;
#pragma unroll 1
    for (int c = 0; c < 256; c += 128) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t u[32];
        tmem_ld32(row + kColOut + c + 32 * e, u);
        tmem_ld_wait();
        uint32_t k[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float x = __uint_as_float(u[2 * j]) * wd, y = __uint_as_float(u[2 * j + 1]) * wd;
          k[j] = final_rows ? bf16x2_bits(x, y) : half2_bits(x, y);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint4 *>(stage + lane * 256 + (((4 * e + j) ^ (lane & 7)) << 4)) =
              make_uint4(k[4 * j], k[4 * j + 1], k[4 * j + 2], k[4 * j + 3]);
      }
      __syncwarp();
#pragma unroll 8
      for (int rr = 0; rr < 32; rr += 2) {
        const int r = rr + (lane >> 4);
        uint4 v = *reinterpret_cast<const uint4 *>(stage + r * 256 + ((pc ^ (r & 7)) << 4));
        const int64_t at = (int64_t)r * D + 256 * kh + c + 8 * pc;
        if (g.whole && a.own_lse) {
          const float x = __shfl_sync(0xffffffffu, wo, r);
          const float4 *own = reinterpret_cast<const float4 *>(a.own_out + (tok_row + h0) * D + at);
          const float4 y = own[0], z = own[1];
          const float2 f0 = half2_floats(v.x), f1 = half2_floats(v.y), f2 = half2_floats(v.z), f3 = half2_floats(v.w);
          v = make_uint4(bf16x2_bits(fmaf(x, y.x, f0.x), fmaf(x, y.y, f0.y)),
                         bf16x2_bits(fmaf(x, y.z, f1.x), fmaf(x, y.w, f1.y)),
                         bf16x2_bits(fmaf(x, z.x, f2.x), fmaf(x, z.y, f2.y)),
                         bf16x2_bits(fmaf(x, z.z, f3.x), fmaf(x, z.w, f3.y)));
        }
        *reinterpret_cast<uint4 *>(dst + at) = v;
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
  // Past pdl_wait the kernel before this one is complete (programmatic launch).
  // Behind the sparse readout of the same call (own_lse) nothing but its
  // results needs that wait, and it has itself waited for everything before
  // it when it lets this kernel start: the two run side by side, and only the
  // segments' ends wait.  (Their CTAs cannot share an SM, whose shared memory
  // each of them fills, so neither can they share its tensor memory.)
  if (!a.own_lse) pdl_wait();
  const DenseWalk walk = dense_walk(a, w, lane);
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
    dense_softmax(a, S, qs, ps, tmem, w, walk, rank, tid, lane, warp);
  } else if (warp < kMmaWarpD) {
    dense_dequant(a, S, qs, ring, w, walk, rank, tid - kSoftWarps * 32, lane);
  } else {
    if (rank == 0 && elect_one()) dense_products(a, S, qs, ps, ring, tmem, w, walk);
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

// Merges the pairs that several workers share, with the weights exp(lse_i -
// lse), lse the log-sum-exp over all their partials (and the other part of the
// softmax).  kByPair (fewer pairs than workers): kCtas CTAs for each pair.
// Otherwise at most one pair lies across each range's start: kCtas CTAs for
// each worker take the pair across its start, if that is the pair's first.  A
// CTA takes kHeads heads of one token, kWarps warps per head, each every
// kWarps-th partial: eight warps where a pair has many partials, one where it
// has two or three.  The CTAs past those write the sequences without entries.
template <bool kByPair>
struct Combine {
  static constexpr int kHeads = kByPair ? 1 : 8, kWarps = kByPair ? 8 : 1;
  static constexpr int kCtas = 2 * (H / kHeads);
};
constexpr int kEmptyCtas = 64;

__device__ __forceinline__ void put_row16(const DenseArgs &a, int64_t row, int lane, const float (&o)[16]) {
  uint32_t u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = bf16x2_bits(o[2 * i], o[2 * i + 1]);
  uint4 *dst = reinterpret_cast<uint4 *>(a.out + row * D + lane * 16);
  dst[0] = make_uint4(u[0], u[1], u[2], u[3]);
  dst[1] = make_uint4(u[4], u[5], u[6], u[7]);
}

// Tokens with no entry at all: the other part of the softmax alone, or zeros.
__device__ __forceinline__ void rest_rows(const DenseArgs &a, int64_t row0, int64_t rows, int warp, int warps, int lane) {
  for (int64_t row = row0 + warp; row < row0 + rows; row += warps) {
    float o[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = a.own_out ? a.own_out[row * D + lane * 16 + i] : 0.0f;
    put_row16(a, row, lane, o);
    if (lane == 0 && a.lse) a.lse[row] = a.own_lse ? a.own_lse[row] : -INFINITY;
  }
}

template <bool kByPair>
__global__ void __launch_bounds__(256) dense_combine_kernel(const DenseArgs a) {
  using C = Combine<kByPair>;
  __shared__ float red[kByPair ? C::kWarps : 1][D];
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t pairs = (a.n_q + 1) / 2;
  const int groups = kByPair ? (int)(a.seqs * pairs) : a.workers;
  const int group = blockIdx.x / C::kCtas, cta = blockIdx.x - group * C::kCtas;
  if (group >= groups) {
    const int ctas = gridDim.x - groups * C::kCtas, me = (blockIdx.x - groups * C::kCtas) * 8 + warp;
    for (int b = 0; b < a.seqs; ++b)
      if (dense_len(a, b) == 0) rest_rows(a, (int64_t)b * a.n_q * H, (int64_t)a.n_q * H, me, ctas * 8, lane);
    return;
  }
  // the pair, its first unit and its steps
  int b = kByPair ? (int)(group / pairs) : 0;
  int64_t before, total, pair, u0;
  int workers, steps;
  dense_units(a, b, lane, before, total, workers);
  if (kByPair) {
    pair = group - b * pairs;
    steps = dense_steps(dense_len(a, b));
    if (steps == 0) return;
    u0 = before + pair * steps;
  } else {
    if (group == 0 || group >= workers) return;
    const int64_t at = dense_range(total, workers, group);
    steps = dense_steps(dense_len(a, 0));
    while (at >= before + pairs * steps) {
      before += pairs * steps;
      steps = dense_steps(dense_len(a, ++b));
    }
    pair = (at - before) / steps;
    u0 = before + pair * steps;
    if (at == u0) return;   // no pair lies across this start
  }
  const int w0 = dense_worker(total, workers, u0);
  const int n = dense_worker(total, workers, u0 + steps - 1) - w0 + 1;   // partials
  if (n == 1 || (!kByPair && w0 != group - 1)) return;   // finished by its worker; an earlier start's
  const int r = cta & 1, hw = warp / C::kWarps, part = warp % C::kWarps;
  const int head = (cta >> 1) * C::kHeads + hw;
  const int64_t t = 2 * pair + r;
  if (t >= a.n_q) return;
  const int64_t row = ((int64_t)b * a.n_q + t) * H + head;
  // partial i's row: slot 2 (w0 + i), but the first one's is odd where the
  // pair starts inside the range
  const int64_t row0 = ((int64_t)4 * w0 + r) * H + head;
  const int64_t odd = dense_range(total, workers, w0) < u0 ? 2 * H : 0;
  auto part_row = [&](int i) { return row0 + (int64_t)i * (4 * H) + (i == 0 ? odd : 0); };
  constexpr int kPer = (kDenseWorkers + 31) / 32;
  float e[kPer], own = a.own_lse ? a.own_lse[row] : -INFINITY, mx = own;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    e[i] = 32 * i + lane < n ? a.part_lse[part_row(32 * i + lane)] : -INFINITY;
    mx = fmaxf(mx, e[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    e[i] = expf(e[i] - mx);
    sum += e[i];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  own = expf(own - mx);
  sum += own;
  float acc[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
  if (part == 0 && a.own_out) {
    const float4 *src = reinterpret_cast<const float4 *>(a.own_out + row * D + lane * 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = src[i];
      acc[4 * i] = own * v.x;
      acc[4 * i + 1] = own * v.y;
      acc[4 * i + 2] = own * v.z;
      acc[4 * i + 3] = own * v.w;
    }
  }
#pragma unroll 1
  for (int i0 = part; i0 < n; i0 += 4 * C::kWarps) {   // four partials in flight
    uint4 v[4][2];
    float f[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = i0 + k * C::kWarps;
      v[k][0] = v[k][1] = make_uint4(0, 0, 0, 0);
      if (i < n) {
        const uint4 *src = reinterpret_cast<const uint4 *>(a.part + part_row(i) * D + lane * 16);
        v[k][0] = src[0];
        v[k][1] = src[1];
      }
      f[k] = 0.0f;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const float x = __shfl_sync(0xffffffffu, e[j], i & 31);
        if (i >> 5 == j) f[k] = x;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t u[8] = {v[k][0].x, v[k][0].y, v[k][0].z, v[k][0].w, v[k][1].x, v[k][1].y, v[k][1].z, v[k][1].w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 x = half2_floats(u[j]);
        acc[2 * j] = fmaf(f[k], x.x, acc[2 * j]);
        acc[2 * j + 1] = fmaf(f[k], x.y, acc[2 * j + 1]);
      }
    }
  }
  const float inv = 1.0f / sum;
  if constexpr (kByPair) {
    // thread (part, lane) adds up channels 2 tid, 2 tid + 1 over the warps
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4 *>(&red[part][lane * 16 + 4 * i]) =
          make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
    __syncthreads();
    float x = 0.0f, y = 0.0f;
#pragma unroll
    for (int p = 0; p < C::kWarps; ++p) {
      const float2 v = *reinterpret_cast<const float2 *>(&red[p][2 * tid]);
      x += v.x;
      y += v.y;
    }
    reinterpret_cast<uint32_t *>(a.out + row * D)[tid] = bf16x2_bits(x * inv, y * inv);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] *= inv;
    put_row16(a, row, lane, acc);
  }
  if (part == 0 && lane == 0 && a.lse) a.lse[row] = mx + logf(sum);
}

// Every token when the prefix has no entry.
__global__ void __launch_bounds__(256) dense_rest_kernel(const DenseArgs a) {
  pdl_wait();
  const int warps = blockDim.x >> 5;
  rest_rows(a, 0, (int64_t)a.seqs * a.n_q * H, blockIdx.x * warps + (threadIdx.x >> 5), gridDim.x * warps,
            threadIdx.x & 31);
}

}  // namespace

namespace {

// The most workers that can have a range, for up to `tokens` query tokens.
int64_t dense_workers(int64_t tokens, int64_t n_max) {
  const int64_t steps = (n_max + kDenseStep - 1) / kDenseStep;
  return steps == 0 ? 1 : tokens >= kDenseWorkers || steps >= kDenseWorkers || tokens * steps >= kDenseWorkers ? kDenseWorkers : tokens * steps;
}

}  // namespace

size_t dense_scratch_bytes(int64_t tokens, int64_t n_max) {
  return (size_t)dense_workers(tokens, n_max) * 2 * 2 * H * (D * sizeof(__half) + sizeof(float));
}

cudaError_t launch_dense_attn(const void *q, const uint8_t *kv, const int32_t *n_vis, int64_t n_max, int64_t cap,
                              int32_t seqs, int32_t n_q, void *out, float *lse, const float *own_out,
                              const float *own_lse, void *scratch, int num_sms, cudaStream_t stream, int *launches) {
  DenseArgs a;
  a.q = static_cast<const __nv_bfloat16 *>(q);
  a.kv = kv;
  a.n_vis = n_vis;
  a.n_max = (int32_t)n_max;
  a.cap = cap;
  a.seqs = seqs;
  a.n_q = n_q;
  const int64_t most = (int64_t)seqs * ((n_q + 1) / 2) * ((n_max + kDenseStep - 1) / kDenseStep);
  int64_t workers = dense_workers((int64_t)seqs * n_q, n_max);
  workers = workers < most ? workers : most;
  workers = workers < num_sms / 2 ? workers : num_sms / 2;
  a.workers = (int32_t)(workers < 1 ? 1 : workers);
  a.out = static_cast<__nv_bfloat16 *>(out);
  a.lse = lse;
  a.own_out = own_out;
  a.own_lse = own_lse;
  a.part = static_cast<__half *>(scratch);
  a.part_lse = reinterpret_cast<float *>(a.part + (size_t)2 * a.workers * 2 * H * D);
  if (most == 0) {
    const int64_t rows = (int64_t)seqs * n_q * H;
    const cudaError_t e = launch_pdl(dense_rest_kernel, dim3((unsigned)(rows < 4096 ? (rows + 7) / 8 : 512)), dim3(256), 0,
                                     stream, 0u, a);
    if (e == cudaSuccess) ++*launches;
    return e;
  }
  cudaError_t e = cudaFuncSetAttribute(dense_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemD);
  if (e != cudaSuccess) return e;
  e = launch_pdl(dense_attn_kernel, dim3((unsigned)(2 * a.workers)), dim3(kThreadsD), kSmemD, stream, 2u, a);
  if (e != cudaSuccess) return e;
  ++*launches;
  const int64_t pairs = (int64_t)seqs * ((n_q + 1) / 2);
  const unsigned empty = n_vis ? kEmptyCtas : 0;
  e = pairs < a.workers ? launch_pdl(dense_combine_kernel<true>, dim3((unsigned)pairs * Combine<true>::kCtas + empty),
                                     dim3(256), 0, stream, 0u, a)
                        : launch_pdl(dense_combine_kernel<false>, dim3((unsigned)a.workers * Combine<false>::kCtas + empty),
                                     dim3(256), 0, stream, 0u, a);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace csa2
