// Dense readout: every entry of a sequence's main-KV cache, for query tokens
// that all see the same entries (csa2_cross_attn), and the shared prefix of
// csa2_prefix_attn.  For a token and head h over entries n < N:
//   o_h = sum_n softmax_n(q_h . k_n / sqrt(512)) k_n,
// key = value = the dequantised 512-d entry (E2M1 x E4M3, exact in fp16).
//
// Per (token, entry) this is 4 * 64 * 512 flop on 288 bytes, so two tokens or
// more are bound by the tensor cores.  A pair of tokens, one per CTA of a
// two-CTA cluster, runs on tcgen05 cta_group::2 with M = 128 (64 heads of each
// token) and N = 256: S = Q K^T for a step of 256 entries in 32 instructions,
// O += P V in 32, 64 clocks each.  Each CTA then needs the keys of its half of
// the step over all 512 channels (B of the first product) and its half of the
// channels over all 256 keys (B of the second).  The 512-channel fp32
// accumulator takes half of the tensor memory and two S tiles the rest, so no
// larger tile fits; Q takes 64 KB of shared memory and P 32 KB, so a
// dequantised step cannot stay until its second use: entries are dequantised
// twice, streamed through one ring of 16 KB slots in the order in which the
// products consume them.
//
// Warps of a CTA: 0-3 softmax (one thread per tensor-memory lane: a head and
// half of the step's keys), 4-11 dequantisation (entries loaded into registers
// a step ahead), 12 the products (in the even CTA) and the copies of Q, which
// start as soon as the last product with the Q before is done.  The first
// loads are sent before the CTA pair's set-up is awaited.  The products' order
// is
//   S(0), S(1), O(0), S(2), O(1), ...
// so that the softmax of one step runs beside the next step's first product.
//
// What bounds it: the L1 / shared-memory data pipe of the SM, which is full.  A
// step passes 2,816 wavefronts of tensor-core operands (P is read once for two
// products), 2,730 of fp16 stores (K, V, P) and 2,220 of arriving entry sectors
// (32 bytes each) in 7,950 clocks, against 4,096 of the products alone.
// Measured: 2 x 512 tokens over 16,384 entries 1.66 ms (1,321 TFLOP/s, 0.69 of a
// bf16 library product's burst rate); 32 tokens over 65,536 entries 225 us
// (1,224); one token over 65,536 31 us, of which four steps take 16 and the
// first entries' arrival, the last rows' way out and the combine the rest.
// Between two pairs the products rest about 3 us: the accumulator has to be read
// out before the next pair's first product into it.
//
// Every wait is bounded; after one runs out every role falls through its
// waits, the CTAs meet at the end and the output is undefined
// (CSA2_DEV_ERR_TIMEOUT).
#include "dense_plan.cuh"
#include "dense_ring.h"

namespace csa2 {

namespace {

constexpr int kSoftWarps = 4, kDeqWarps = 8;
constexpr int kMmaWarpD = kSoftWarps + kDeqWarps;
constexpr int kThreadsD = (kMmaWarpD + 1) * 32;   // 128 registers a thread
constexpr int kSlots = 8;
constexpr int kSlotBytes = 16384;             // 128 keys x 64 channels, or 32 keys x 256 channels
constexpr int kQBytesD = H * D * 2;
constexpr int kPBytes = H * kDenseStep * 2;
constexpr int kAtomD = H * 128;               // 64 rows x 128 bytes (Q, P)
constexpr uint32_t kColOut = 256;             // tensor memory: S tiles at 0 and 128, O at 256
constexpr float kLogitD = 0.06375871295460785f;   // log2(e) / sqrt(512)
constexpr float kLn2D = 0.69314718055994531f;
// P = 2^((s - m) kLogitD + kBias), s = q . k, with a reference m that is raised
// only when a step exceeds it by 2^kLazyD: at most 2^15 (fp16), and a key 2^-31
// below the reference still counts, so 64K such keys lose less than 2^-15 of
// the sum.  The difference comes before the scale: of scaled products of 2^24
// and more, one rounding against the reference is whole powers of two.
constexpr float kLazyD = 8.0f, kBias = 7.0f;
constexpr uint32_t kIdescS = idesc_f16(0, 0, 0, 256, 128);
constexpr uint32_t kIdescO = idesc_f16(0, 0, /*B MN-major*/ 1, 256, 128);

struct __align__(16) CtlD {
  uint64_t full[kSlots];                      // full, q_full, p_full: both CTAs arrive at the even CTA
  uint64_t free[kRingSets][kSlots];
  uint64_t q_raw, q_full, q_free, s_full[2], p_full, p_free, done;
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

// Waits until both CTAs of the pair have set up their barriers and tensor
// memory (each thread once).
__device__ __forceinline__ uint32_t pair_ready(const CtlD &S) {
  tc_fence_before();
  bar_named(2, kThreadsD);
  cluster_sync();
  tc_fence_after();
  return S.tmem_base;
}

// Q of this CTA's token of a segment: eight boxes of [64 heads][64 channels],
// bf16, each a 128B-swizzled column of the Q region; completes q_raw.
__device__ __forceinline__ void load_q(const DenseArgs &a, CtlD &S, const CUtensorMap &tm_q, uint8_t *qs,
                                       const DenseSegment &g, uint32_t rank) {
  const int t = 2 * g.pair + (int)rank;
  if (t >= a.n_q) {   // the missing token of an odd count: zeros, written by convert_q
    mbar_arrive(&S.q_raw);
    return;
  }
  mbar_arrive_expect_tx(&S.q_raw, (uint32_t)kQBytesD);
  const int32_t y = (int32_t)(((int64_t)g.b * a.n_q + t) * H);
#pragma unroll 1
  for (int c = 0; c < 8; ++c) tma_load_2d(qs + c * kAtomD, &tm_q, 64 * c, y, &S.q_raw);
}

// Q in place from bf16 to fp16 (two-byte slots of the same layout), by
// kThreads threads.
template <int kThreads>
__device__ __forceinline__ void convert_q(const DenseArgs &a, const DenseSegment &g, uint32_t rank, uint8_t *qs, int t) {
  const bool zero = 2 * g.pair + (int)rank >= a.n_q;
  uint4 *q = reinterpret_cast<uint4 *>(qs);
#pragma unroll 4
  for (int i = t; i < kQBytesD / 16; i += kThreads) {
    const uint4 v = q[i];
    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      h[j] = zero ? 0u : half2_bits(__uint_as_float(x[j] << 16), __uint_as_float(x[j] & 0xFFFF0000u));
    q[i] = make_uint4(h[0], h[1], h[2], h[3]);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

__device__ void dense_dequant(const DenseArgs &a, CtlD &S, uint8_t *qs, uint8_t *ring, int w, DenseWalk walk, uint32_t rank,
                              int pt, int lane) {
  const int warp = pt >> 5, key4 = lane >> 3, c8 = lane & 7;
  const int o = c8 >> 1;
  const bool o1 = o & 1, o2 = o & 2;
  const uint32_t z = (uint32_t)((4 * (c8 & 1)) ^ key4 ^ o) << 4;
  const uint32_t k_at = smem_u32(ring) + (uint32_t)(o * kSlotBytes + (16 * warp + key4) * 128) + z;
  const uint32_t v_at = smem_u32(ring) + (uint32_t)(warp * kSlotBytes + o * 4096 + key4 * 128) + z;
  const uint32_t full_at = dsmem_addr(&S.full[0], 0);
  uint32_t round = 0;   // 8-slot rounds so far
  uint32_t item = 0;
  DeqRegs kr, vr;
  auto load_piece = [&](DeqRegs &r, int i, const uint8_t *base, int len, int n, int half) {
    r.v[i] = make_uint4(0, 0, 0, 0);
    r.sc[i] = 0;
    if (n < len) {
      const uint8_t *e = base + (int64_t)n * ENTRY_BYTES;
      r.v[i] = ld_nc_v4(e + 128 * half + 16 * c8);
      r.sc[i] = ld_nc_u16(e + 256 + 16 * half + 2 * c8);
    }
  };
  auto load_k = [&](int b, int len, int step) {   // [channel half][4 keys]
    const uint8_t *base = a.kv + (int64_t)b * a.cap * ENTRY_BYTES;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      load_piece(kr, i, base, len, step * kDenseStep + (int)rank * 128 + 16 * warp + 4 * (i & 3) + key4, i >> 2);
  };
  auto load_v = [&](int b, int len, int step) {   // [4 keys]
    const uint8_t *base = a.kv + (int64_t)b * a.cap * ENTRY_BYTES;
#pragma unroll
    for (int i = 0; i < 8; ++i) load_piece(vr, i, base, len, step * kDenseStep + 32 * warp + 4 * i + key4, (int)rank);
  };
  // A slot is free again when the products of its round before are done (in
  // every wait of dense_ring.h's protocol the round before is the one meant).
  auto wait_free = [&](int s) { wait_d(S, &S.free[ring_set(round - 1)][s], ring_parity(round - 1)); };
  auto emit_k = [&]() {
#pragma unroll
    for (int hc = 0; hc < 2; ++hc) {
      if (round)
#pragma unroll
        for (int s = 0; s < 4; ++s) wait_free(4 * hc + s);
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
    if (round) wait_free(warp);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      put32((v_at + (uint32_t)(i * 512)) ^ (uint32_t)((i & 1) << 6), vr.v[i], vr.sc[i], o1, o2);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive_pair(full_at + 8 * warp, kDeqWarps);
    ++round;
  };

  DenseSegment g, next;
  bool more = dense_next(a, w, walk, g);
  if (more) {
    load_k(g.b, g.len, g.s0);
    load_v(g.b, g.len, g.s0);
  }
  pair_ready(S);
  while (more) {
    more = dense_next(a, w, walk, next);
    if (item) {   // the first segment's Q is the softmax warps' (they have nothing else to do then)
      wait_d(S, &S.q_raw, item & 1u);
      convert_q<kDeqWarps * 32>(a, g, rank, qs, pt);
      if (lane == 0) mbar_arrive_pair(dsmem_addr(&S.q_full, 0), 1);
    }
    ++item;
    emit_k();
    if (g.s0 + 1 < g.s1)
      load_k(g.b, g.len, g.s0 + 1);
#pragma unroll 1
    for (int i = g.s0; i < g.s1; ++i) {
      if (i + 1 < g.s1) {
        emit_k();
        if (i + 2 < g.s1)
          load_k(g.b, g.len, i + 2);
      }
      emit_v();
      if (i + 1 < g.s1)
        load_v(g.b, g.len, i + 1);
    }
    g = next;
    if (more) {
      load_k(g.b, g.len, g.s0);
      load_v(g.b, g.len, g.s0);
    }
  }
  // every slot this CTA filled has been read, and no commit is still to
  // arrive here, before the CTA ends
  if (round)
#pragma unroll 1
    for (int s = 0; s < kSlots; ++s) wait_free(s);
}

// ---------------------------------------------------------------- products
// A Q copy still in flight when the roles have fallen through after a wait that
// ran out must land before the CTA's memory goes.  Copy i completes phase i of
// q_raw and is sent for after i - 1 has landed, so the last one's parity is
// enough.  Bounded, and not cut short by S.abort.
__device__ __forceinline__ void drain_q(CtlD &S, uint32_t copies) {
  if (copies) mbar_wait(&S.q_raw, (copies - 1) & 1u);
}

// One thread of the even CTA.  `g`: the first segment, whose Q is on its way;
// the next one's is sent for when the last S of a segment is done.
__device__ void dense_products(const DenseArgs &a, CtlD &S, const CUtensorMap &tm_q, uint8_t *qs, uint8_t *ps,
                               uint8_t *ring, uint32_t tmem, int w, DenseWalk walk, DenseSegment g, bool more) {
  const uint64_t qd = smem_desc(smem_u32(qs), 16, 1024);
  const uint64_t pd = smem_desc(smem_u32(ps), 16, 1024);
  const uint64_t kd = smem_desc(smem_u32(ring), 16, 1024);
  const uint64_t vd = smem_desc(smem_u32(ring), 4096, 1024);
  uint32_t round = 0, item = 0, n = 0, copies = more ? 1u : 0u;
  while (more) {
    const int steps = g.s1 - g.s0;
    auto scores = [&](uint32_t tile) {
#pragma unroll 1
      for (int s = 0; s < kSlots; ++s) {
        wait_pair(S, &S.full[s], round & 1u);
        tc_fence_after();
        const uint64_t qa = qd + (uint64_t)(s * kAtomD >> 4), kb = kd + (uint64_t)(s * kSlotBytes >> 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) mma_f16_pair(tmem + tile * 128, qa + 2 * i, kb + 2 * i, kIdescS, (s | i) ? 1u : 0u);
        mma_commit_pair(&S.free[ring_set(round)][s]);
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
      if (i + 1 == steps) {
        more = dense_next(a, w, walk, g);
        wait_pair(S, &S.q_free, (item - 1) & 1u);
        if (more && !S.abort) {
          load_q(a, S, tm_q, qs, g, 0);
          ++copies;
        }
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
        mma_commit_pair(&S.free[ring_set(round)][s]);
      }
      ++round;
      mma_commit_pair(&S.p_free);
    }
  }
  // every product has completed before the teardown, also after a wait ran out
  mma_commit_pair(&S.done);
  mbar_wait_cluster(&S.done, 0);
  drain_q(S, copies);
}

// One thread of the odd CTA: its own token's Q, and what the combine has to
// know of a pair that starts in this worker's range and ends in another's (the
// range's last pair at most).
__device__ void dense_odd(const DenseArgs &a, CtlD &S, const CUtensorMap &tm_q, uint8_t *qs, int w, DenseWalk walk,
                          DenseSegment g, bool more, int64_t total, int workers) {
  const int pairs = (a.n_q + 1) / 2;
  const bool by_pair = (int64_t)a.seqs * pairs < a.workers;
  if (!by_pair) a.shared[w].n = 0;
  uint32_t item = 0, copies = more ? 1u : 0u;
  while (more) {
    if (g.s0 == 0 && (by_pair || !g.whole)) {
      // (a segment that reaches its pair's end is whole here)
      const int steps = dense_steps(g.len);
      const int64_t u0 = g.whole ? 0 : walk.end - g.s1;
      DenseShared d;
      d.token = g.b * a.n_q + 2 * g.pair;
      d.tokens = 2 * g.pair + 1 < a.n_q ? 2 : 1;
      d.slot = g.slot;
      d.n = g.whole ? 0 : dense_worker(total, workers, u0 + steps - 1) - w + 1;
      a.shared[by_pair ? g.b * pairs + g.pair : w] = d;
    }
    wait_d(S, &S.q_free, item & 1u);
    ++item;
    more = dense_next(a, w, walk, g);
    if (more && !S.abort) {
      load_q(a, S, tm_q, qs, g, 1);
      ++copies;
    }
  }
  // no product reads this CTA's memory past here, also after a wait ran out
  mbar_wait_cluster(&S.done, 0);
  drain_q(S, copies);
}

// ----------------------------------------------------------------- softmax
// Thread tid holds head tid % 64: of S the keys 128 (tid / 64) .. + 127 of a
// step, of O the channels 256 (tid / 64) .. + 255.
__device__ void dense_softmax(const DenseArgs &a, CtlD &S, const CUtensorMap &tm_out, const CUtensorMap &tm_part,
                              uint8_t *qs, uint8_t *ps, int w, DenseWalk walk, uint32_t rank, int tid, int lane,
                              int warp) {
  pair_ready(S);
  {
    DenseWalk peek = walk;
    DenseSegment first;
    if (dense_next(a, w, peek, first)) {
      wait_d(S, &S.q_raw, 0);
      convert_q<kSoftWarps * 32>(a, first, rank, qs, tid);
      if (lane == 0) mbar_arrive_pair(dsmem_addr(&S.q_full, 0), kDeqWarps / kSoftWarps);
    }
  }
  const uint32_t tmem = S.tmem_base;
  const uint32_t p_full_at = dsmem_addr(&S.p_full, 0);
  const uint32_t row = tmem + ((uint32_t)(32 * warp) << 16);
  const int h = tid & 63, kh = tid >> 6;
  uint8_t *prow = ps + 2 * kh * kAtomD + h * 128;
  DenseSegment g;
  uint32_t n = 0;
  DenseSegment next;
  bool more = dense_next(a, w, walk, g);
  for (; more; g = next) {
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
      for (int c = 0; c < 128; c += 64) {
        uint32_t u[2][32];
        tmem_ld32(st + c, u[0]);
        tmem_ld32(st + c + 32, u[1]);
        tmem_ld_wait();
        float m2[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (c + 64 <= valid) {
#pragma unroll
          for (int j = 0; j < 64; ++j) m2[j & 3] = fmaxf(m2[j & 3], __uint_as_float(u[j >> 5][j & 31]));
        } else {
#pragma unroll
          for (int j = 0; j < 64; ++j)
            if (c + j < valid) m2[j & 3] = fmaxf(m2[j & 3], __uint_as_float(u[j >> 5][j & 31]));
        }
        mx = fmaxf(mx, fmaxf(fmaxf(m2[0], m2[1]), fmaxf(m2[2], m2[3])));
      }
      S.red[n & 1u][tid] = mx;
      bar_named(1, 128);
      mx = fmaxf(mx, S.red[n & 1u][tid ^ 64]);
      // O(n - 1) is complete: P is free, O may be rescaled
      if (n) wait_d(S, &S.p_free, (n - 1) & 1u);
      tc_fence_after();
      if (i == g.s0) {
        m = mx;
      } else {
        const bool raise = mx > m + kLazyD / kLogitD;
        if (__any_sync(0xffffffffu, raise)) {
          const float f = raise ? ex2_approx((m - mx) * kLogitD) : 1.0f;
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
#pragma unroll 1
      for (int c = 0; c < 128; c += 64) {
        uint32_t u[2][32];
        tmem_ld32(st + c, u[0]);
        tmem_ld32(st + c + 32, u[1]);
        tmem_ld_wait();
        uint8_t *dst = prow + (c >> 6) * kAtomD;
        float l0 = 0.0f, l1 = 0.0f;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          uint32_t pk[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int e = 8 * q + 2 * j;
            float x0, x1;
            f32x2_unpack(f32x2_fma(f32x2_add(f32x2_pack(__uint_as_float(u[e >> 5][e & 31]),
                                                        __uint_as_float(u[e >> 5][(e & 31) + 1])), f32x2_pack(-m, -m)),
                                   f32x2_pack(kLogitD, kLogitD), f32x2_pack(kBias, kBias)), x0, x1);
            if (c + 64 > valid) {
              if (c + e >= valid) x0 = -INFINITY;
              if (c + e + 1 >= valid) x1 = -INFINITY;
            }
            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
            l0 += p0;
            l1 += p1;
            pk[j] = half2_bits(p0, p1);
          }
          *reinterpret_cast<uint4 *>(dst + ((q ^ (h & 7)) << 4)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
        l += l0 + l1;
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_pair(p_full_at, 1);
    }
    // ------------------------------------------------------------ segment end
    S.red[n & 1u][tid] = l;
    bar_named(1, 128);
    l += S.red[n & 1u][tid ^ 64];
    bar_named(1, 128);   // red is written again by the next step
    const float lse = (m * kLogitD + (log2f(l) - kBias)) * kLn2D;
    more = dense_next(a, w, walk, next);
    wait_d(S, &S.p_free, (n - 1) & 1u);
    tc_fence_after();
    if (g.whole) pdl_wait();   // own_out, own_lse
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
    // O as 16-bit rows through the warp's 8 KB of the P buffer and tensor
    // copies of 32 rows by 64 channels (stores from the registers, a row per
    // lane, or staged rows read back for coalesced stores keep the load / store
    // pipe, which is full anyway, 3.3 and 3.9 us a segment): bf16 if it is the
    // output, fp16 for a partial, whose rounding (2^-11 of a value) is below
    // the output's (2^-8)
    const float *own = g.whole && a.own_lse ? a.own_out + (tok_row + h) * D + 256 * kh : nullptr;
    const CUtensorMap *tm = g.whole ? &tm_out : &tm_part;
    const int32_t y = (int32_t)(g.whole ? tok_row : ((int64_t)g.slot * 2 + rank) * H) + 32 * (warp & 1);
#pragma unroll 1
    for (int c = 0; c < 256; c += 64) {
      uint8_t *stage = ps + warp * 8192 + (c & 64) * 64;
      if (c >= 128) {   // the copy out of this half two pieces ago has read it
        if (lane == 0) bulk_wait_read<1>();
        __syncwarp();
      }
#pragma unroll
      for (int e = 0; e < 64; e += 32) {
        uint32_t u[32];
        tmem_ld32(row + kColOut + c + e, u);
        tmem_ld_wait();
        float x[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = __uint_as_float(u[j]) * wd;
        if (own) {
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 o = *reinterpret_cast<const float4 *>(own + c + e + j);
            x[j] = fmaf(wo, o.x, x[j]);
            x[j + 1] = fmaf(wo, o.y, x[j + 1]);
            x[j + 2] = fmaf(wo, o.z, x[j + 2]);
            x[j + 3] = fmaf(wo, o.w, x[j + 3]);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t k[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            k[i] = g.whole ? bf16x2_bits(x[8 * j + 2 * i], x[8 * j + 2 * i + 1])
                           : half2_bits(x[8 * j + 2 * i], x[8 * j + 2 * i + 1]);
          *reinterpret_cast<uint4 *>(stage + lane * 128 + (((e / 8 + j) ^ (lane & 7)) << 4)) =
              make_uint4(k[0], k[1], k[2], k[3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d(tm, 256 * kh + c, y, stage);
        bulk_commit();
      }
    }
    if (lane == 0) bulk_wait_read<0>();   // the next P may be written (after the next maximum's barrier)
    __syncwarp();
    tc_fence_before();   // O is read before the next segment's products (ordered by p_full)
  }
  if (lane == 0) bulk_wait<0>();
  pdl_wait();   // the combine reads own_out too: this kernel's end is also the end of the one beside it
}

__global__ void __launch_bounds__(kThreadsD, 1)
    dense_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_out,
                      const __grid_constant__ CUtensorMap tm_part, const DenseArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *qs = base, *ps = qs + kQBytesD, *ring = ps + kPBytes;
  CtlD &S = *reinterpret_cast<CtlD *>(ring + kSlots * kSlotBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const int w = blockIdx.x >> 1;
  if (warp == kMmaWarpD && lane == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&S.full[s], 2 * kDeqWarps);
      for (int i = 0; i < kRingSets; ++i) mbar_init(&S.free[i][s], 1);
    }
    mbar_init(&S.q_raw, 1);
    mbar_init(&S.q_full, 2 * kDeqWarps);
    mbar_init(&S.q_free, 1);
    mbar_init(&S.s_full[0], 1);
    mbar_init(&S.s_full[1], 1);
    mbar_init(&S.p_full, 2 * kSoftWarps);
    mbar_init(&S.p_free, 1);
    mbar_init(&S.done, 1);
    S.abort = 0;
    fence_barrier_init();
    prefetch_tmap(&tm_q);
  }
  // Past pdl_wait the kernel before this one is complete (programmatic launch).
  // Behind the sparse readout of the same call (own_lse) only its results need
  // that wait, and it has itself waited for everything before it when it lets
  // this kernel start: the two run side by side, and the wait comes where a
  // whole pair's rows are merged with its own part, and at the kernel's end.
  // (Their CTAs cannot share an SM, whose shared memory each of them fills, so
  // neither can they share its tensor memory.)
  if (!a.own_lse) pdl_wait();
  int64_t total;
  int workers;
  const DenseWalk walk = dense_walk(a, w, lane, total, workers);
  if (warp < kSoftWarps) {
    dense_softmax(a, S, tm_out, tm_part, qs, ps, w, walk, rank, tid, lane, warp);
  } else if (warp < kMmaWarpD) {
    dense_dequant(a, S, qs, ring, w, walk, rank, tid - kSoftWarps * 32, lane);
  } else {
    __syncwarp();
    DenseWalk ahead = walk;
    DenseSegment g;
    const bool more = dense_next(a, w, ahead, g);
    if (more && lane == 0) load_q(a, S, tm_q, qs, g, rank);
    __syncwarp();
    tmem_alloc_pair(&S.tmem_base, 512);
    tmem_relinquish_pair();
    const uint32_t tmem = pair_ready(S);
    if (elect_one()) {
      if (rank == 0)
        dense_products(a, S, tm_q, qs, ps, ring, tmem, w, ahead, g, more);
      else
        dense_odd(a, S, tm_q, qs, w, ahead, g, more, total, workers);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // neither CTA reads or signals the other past here
  pdl_release();
  if (warp == kMmaWarpD) {
    tc_fence_after();
    tmem_dealloc_pair(S.tmem_base, 512);
  }
}

// Merges the pairs that several workers share, with the weights exp(lse_i -
// lse), lse the log-sum-exp over all their partials (and the other part of the
// softmax).  With fewer pairs than workers, a group of CTAs takes each pair;
// otherwise at most one shared pair starts in each range, and a group takes it;
// dense_odd says which and how many partials it has.  A CTA takes one token
// and 8 / a.split of its heads, a.split warps per head, each every a.split-th
// partial, four of them in flight (about as many warps as bring every partial
// in one or two rounds: a pair has workers / pairs partials).  The CTAs past
// the groups write the sequences without entries.
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

__global__ void __launch_bounds__(256, 3) dense_combine_kernel(const DenseArgs a) {
  __shared__ float red[8][D];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t pairs = (int64_t)a.seqs * ((a.n_q + 1) / 2);
  const bool by_pair = pairs < a.workers;
  const int groups = by_pair ? (int)pairs : a.workers;
  const int heads = 8 / a.split, ctas = 2 * (H / heads);   // per CTA, per group
  const int group = blockIdx.x / ctas, cta = blockIdx.x - group * ctas;
  if (group >= groups) {
    pdl_wait();
    // every warps-th token's length per lane: neighbours go to different CTAs
    const int rest = gridDim.x - groups * ctas, warps = rest * 8, me = warp * rest + blockIdx.x - groups * ctas;
    const int64_t tokens = (int64_t)a.seqs * a.n_q;
    for (int64_t t0 = me; t0 < tokens; t0 += 32 * (int64_t)warps) {
      const int64_t t = t0 + (int64_t)lane * warps;
      uint32_t empty = __ballot_sync(0xffffffffu, t < tokens && dense_len(a, (int)((uint32_t)t / (uint32_t)a.n_q)) == 0);
      for (; empty; empty &= empty - 1)
        rest_rows(a, (t0 + (int64_t)(__ffs(empty) - 1) * warps) * H, H, 0, 1, lane);
    }
    return;
  }
  // (older than the dense kernel: read before the wait) a pair without entries
  if (by_pair && dense_len(a, group / ((a.n_q + 1) / 2)) == 0) return;
  pdl_wait();   // the dense kernel's partials
  const int4 d = *reinterpret_cast<const int4 *>(a.shared + group);   // DenseShared
  const int n = d.w, r = cta & 1;
  if (n == 0 || r >= d.y) return;
  const int hw = warp / a.split, part = warp - hw * a.split;
  const int head = (cta >> 1) * heads + hw;
  const int64_t row = ((int64_t)d.x + r) * H + head;
  // partial i's row: the first one's slot, then the even ones
  const int64_t row0 = ((int64_t)2 * (d.z & ~1) + r) * H + head, odd = (d.z & 1) * 2 * H;
  auto part_row = [&](int i) { return row0 + (int64_t)i * (4 * H) + (i == 0 ? odd : 0); };
  // this warp's partials, kMine loads in flight, the first ones beside the
  // log-sum-exps'
  constexpr int kPer = (kDenseWorkers + 31) / 32, kMine = 4;
  uint4 v[kMine][2];
  auto load = [&](int i0) {
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const int i = i0 + k * a.split;
      v[k][0] = v[k][1] = make_uint4(0, 0, 0, 0);
      if (i < n) {
        const uint4 *src = reinterpret_cast<const uint4 *>(a.part + part_row(i) * D + lane * 16);
        v[k][0] = src[0];
        v[k][1] = src[1];
      }
    }
  };
  load(part);
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
      const float4 o = src[i];
      acc[4 * i] = own * o.x;
      acc[4 * i + 1] = own * o.y;
      acc[4 * i + 2] = own * o.z;
      acc[4 * i + 3] = own * o.w;
    }
  }
#pragma unroll 1
  for (int i0 = part;;) {
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const int i = i0 + k * a.split;
      float f = 0.0f;   // partials past n: e = 0
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const float x = __shfl_sync(0xffffffffu, e[j], i & 31);
        if (i >> 5 == j) f = x;
      }
      const uint32_t u[8] = {v[k][0].x, v[k][0].y, v[k][0].z, v[k][0].w, v[k][1].x, v[k][1].y, v[k][1].z, v[k][1].w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 x = half2_floats(u[j]);
        acc[2 * j] = fmaf(f, x.x, acc[2 * j]);
        acc[2 * j + 1] = fmaf(f, x.y, acc[2 * j + 1]);
      }
    }
    i0 += kMine * a.split;
    if (i0 >= n) break;
    load(i0);
  }
  const float inv = 1.0f / sum;
  if (a.split == 1) {
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] *= inv;
    put_row16(a, row, lane, acc);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4 *>(&red[warp][lane * 16 + 4 * i]) =
          make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
    __syncthreads();   // (the exits above are taken by the whole CTA)
    // the head's warps add up a share of its channels each
    for (int c = 2 * (32 * part + lane); c < D; c += 64 * a.split) {
      float x = 0.0f, y = 0.0f;
      for (int p = 0; p < a.split; ++p) {
        const float2 u = *reinterpret_cast<const float2 *>(&red[hw * a.split + p][c]);
        x += u.x;
        y += u.y;
      }
      *reinterpret_cast<uint32_t *>(a.out + row * D + c) = bf16x2_bits(x * inv, y * inv);
    }
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
  return (size_t)dense_workers(tokens, n_max) *
         (2 * 2 * H * (D * sizeof(__half) + sizeof(float)) + sizeof(DenseShared));
}

cudaError_t launch_dense_attn(const void *q, const uint8_t *kv, const int32_t *n_vis, int64_t n_max, int64_t cap,
                              int32_t seqs, int32_t n_q, void *out, float *lse, const float *own_out,
                              const float *own_lse, int own_ctas, void *scratch, int num_sms, cudaStream_t stream,
                              int *launches) {
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
  // Beside the own part's kernel: the workers that fit next to its CTAs, if
  // fewer of them end sooner than all of them after it.  Its latency is between
  // three and four units of theirs (in graphs, beside it against after it: no
  // units more, 1 sequence over 65,536 entries, 32.7 us against 43.6; three more,
  // 16 over 10,001 47.1 against 52.3, 8 over 20,000 46.9 against 50.1; four more, 4
  // over 131,072 85.1 against 82.2; eight more, 7 over 65,536 100.0 against 83.3).
  constexpr int64_t kOwnUnits = 3;
  const int64_t beside = (num_sms - own_ctas) / 2;
  if (own_ctas > 0 && beside >= 1 && beside < workers &&
      (most + beside - 1) / beside <= (most + workers - 1) / workers + kOwnUnits)
    workers = beside;
  a.workers = (int32_t)(workers < 1 ? 1 : workers);
  const int64_t pairs = (int64_t)seqs * ((n_q + 1) / 2), groups = pairs < a.workers ? pairs : a.workers;
  a.split = 1;   // warps per head of the combine: about four partials each
  while (a.split < 8 && groups * a.split * 4 < a.workers) a.split *= 2;
  a.out = static_cast<__nv_bfloat16 *>(out);
  a.lse = lse;
  a.own_out = own_out;
  a.own_lse = own_lse;
  a.part = static_cast<__half *>(scratch);
  a.part_lse = reinterpret_cast<float *>(a.part + (size_t)2 * a.workers * 2 * H * D);
  a.shared = reinterpret_cast<DenseShared *>(a.part_lse + (size_t)2 * a.workers * 2 * H);
  if (most == 0) {
    const int64_t rest = (int64_t)seqs * n_q * H;
    const cudaError_t e = launch_pdl(dense_rest_kernel, dim3((unsigned)(rest < 4096 ? (rest + 7) / 8 : 512)), dim3(256), 0,
                                     stream, 0u, a);
    if (e == cudaSuccess) ++*launches;
    return e;
  }
  const int64_t rows = (int64_t)seqs * n_q * H;
  CUtensorMap tm_q, tm_out, tm_part;   // (the partials' fp16 are copied as any 16-bit type)
  if (!make_tmap_bf16(&tm_q, q, D, rows, H) || !make_tmap_bf16(&tm_out, out, D, rows, 32) ||
      !make_tmap_bf16(&tm_part, a.part, D, (int64_t)a.workers * 4 * H, 32))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(dense_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemD);
  if (e != cudaSuccess) return e;
  e = launch_pdl(dense_attn_kernel, dim3((unsigned)(2 * a.workers)), dim3(kThreadsD), kSmemD, stream, 2u, tm_q, tm_out,
                 tm_part, a);
  if (e != cudaSuccess) return e;
  ++*launches;
  e = launch_pdl(dense_combine_kernel, dim3((unsigned)(groups * 2 * (H / (8 / a.split)) + (n_vis ? kEmptyCtas : 0))),
                 dim3(256), 0, stream, 0u, a);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace csa2
