// The step form of the readout, one CTA per token: a token's listed main-KV
// entries, its window rows and its extra rows (csa2_tree_attn; csa2_window_attn
// when its rows do not fit in the tiles of window_attn.cu), in one softmax:
//   o_h = sum_k softmax_k(q_h . v_k f_k / sqrt(512)) v_k f_k,
// v_k f_k an entry's 512 values (E2M1 x E4M3) or a row's E4M3 codes times its scale,
// f_k a power of two, or a row's scale times one, of their size (step_rows.cuh), so
// that the v_k are exact in fp16.
//
// No two tokens list the same entries, so a token's 64 heads are all that share a
// key: 4 x 64 x 512 flop for 288 bytes, which the tensor cores take as products of
// 64 rows at a quarter of their rate.  What bounds it is the SM's shared-memory
// pipe: a step of 64 keys passes 512 wavefronts of fp16 stores, some 580 of
// arriving entry sectors, 1,024 of operands of S and 768 of the second product.
// So the keys go through in steps of 64 in two slots of 64 KB, every part of the
// work on warps of its own, a step's rows being converted while the step before is
// in its softmax and products:
//   rows     8 warps: four lanes on 128 contiguous bytes of an entry, loaded a
//            step ahead into registers, written as fp16 into the slot [8 x 64
//            channels][64 keys][128 B], 128B-swizzled;
//   S        M = 64 heads, N = 64 keys, K = 512, in two accumulators in turn
//            (products into one wait for each other), two S buffers;
//   softmax  4 warps, a head's 64 logits on two lanes; the reference maximum (over
//            logit + log2(f_k)) is raised only past 2^8, O^T then rescaled; P to
//            shared memory as fp16;
//   O^T += V^T P^T  M = 128 channels (four blocks), N = 64 heads, K = 64 keys, V^T
//            from the same slot; its end frees the slot;
//   rows out O^T through shared memory, as bf16, while the next
//            token's first steps are converted and multiplied.
// Measured: 2,048 tokens of 512 + 128 keys 310 us, 41,600 wavefronts and some 43,000
// clocks a token, ten steps of 3,400 and 8,000 between tokens (Q's reload and
// conversion, beside them the rows out); 256 tokens 52 us, two rounds; 93 tokens of
// up to 168 keys 11.0 in a graph, 11.8 to 13.2 called one by one.  Both products issued by one thread, a tile of 128 keys and
// softmax on the rows' warps, as in the sparse readout: 637 us for the 2,048.
// Keys that the token does not see take no place: the list (whose -1 are masked),
// the window's visible rows, then the named extra rows.
//
// Warps: 0-3 softmax, 4-11 rows, 12 S, 13 second product.  Every wait is bounded;
// after one runs out every role falls through its waits and the output is
// undefined (CSA2_DEV_ERR_TIMEOUT).
#include "gather_q.h"
#include "step_rows.cuh"

namespace csa2 {

namespace {

constexpr int kSoftG = 4, kRowG = 8;
constexpr int kScoreWarpG = kSoftG + kRowG, kValueWarpG = kScoreWarpG + 1;
constexpr int kThreadsG = (kValueWarpG + 1) * 32;   // 128 registers a thread
constexpr int kStep = 64;                    // keys of a step
constexpr int kSlotG = kStep * D * 2;
constexpr int kBlockG = kStep * 128;         // a column block of 64 channels: of a slot, of Q, a buffer of P
constexpr uint32_t kColOG = 256;             // tensor memory: S at 128 slot + 64 accumulator, O^T at 256
constexpr float kLogitG = 0.06375871295460785f;   // log2(e) / sqrt(512)
constexpr float kLn2G = 0.69314718055994531f;
constexpr float kLazyG = 8.0f;               // log2 margin before the reference is raised
constexpr uint32_t kIdescSG = idesc_f16(0, 0, 0, kStep, H);
constexpr uint32_t kIdescOG = idesc_f16(0, /*A MN-major*/ 1, 0, H, 128);

struct __align__(16) CtlG {
  uint64_t rows_full[2], slot_free[2], s_full[2], p_full[2], q_raw, q_ready, q_free, o_free, done[2];
  uint32_t tmem_base;
  volatile uint32_t abort;
  float fac[H];
  __align__(16) float inv_l[H];
  __align__(16) uint32_t none[kSoftG];   // a softmax warp has found that the token sees nothing
  // per key of a slot: log2(e) / sqrt(512) x f, log2(f) (-inf: no key), 1 / f
  __align__(16) float rs[2][kStep];
  __align__(16) float lg[2][kStep];
  __align__(16) float inv[2][kStep];
};

constexpr size_t kSmemG = 1024 + (size_t)2 * kSlotG + H * D * 2 + 2 * kBlockG + sizeof(CtlG);
static_assert(kSmemG <= 232448, "gathered attention exceeds the shared-memory limit");

__device__ __forceinline__ void wait_g(CtlG &S, uint64_t *bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity) || S.abort) return;
  if (!mbar_wait(bar, parity)) S.abort = 1;
}

// A token's keys: its list, window rows at ring places place, place + 1, .. (around
// the ring's end), named extra rows.  By whole warps.
struct Keys {
  int64_t gp;
  int64_t ring_row0, extra_row0, entry_row0;   // first rows of the token's sequence
  int64_t place;
  uint64_t extra;
  int rows, named, steps;   // window rows, extra rows; steps of 64 keys (0: no token)
};

__device__ __forceinline__ Keys keys_of(const AttnArgs &a, int64_t gp) {
  Keys k;
  k.gp = gp;
  k.steps = 0;
  StepToken t;
  if (!step_token(a.step, gp, t)) return k;
  const int64_t first = max(t.end - t.left, (int64_t)0);
  k.rows = (int)(t.end - first);
  k.place = first % a.step.ring;
  k.extra = t.extra;
  k.named = __popcll(t.extra);
  k.ring_row0 = t.seq * a.step.ring;
  k.extra_row0 = t.seq * a.step.extras;
  k.entry_row0 = t.seq * a.cap;
  const int n = k.rows + k.named + a.K;
  k.steps = n > kStep ? (n + kStep - 1) / kStep : 1;
  return k;
}

// Whether a token sees any key (by whole warps).
__device__ __noinline__ bool has_keys(const AttnArgs &a, int64_t gp, int lane) {
  const Keys k = keys_of(a, gp);
  bool any = k.rows + k.named > 0;
  for (int e = lane; e < a.K; e += 32) {
    const int32_t id = __ldg(a.idx + gp * a.K + e);
    any |= id >= 0 && id < a.cap;
  }
  return __any_sync(0xffffffffu, any);
}

// The CTA's tokens that have steps, by whole warps; the next one is looked up while
// the one before is worked on.
struct Tokens {
  int64_t next;
  int steps;   // of the token `next`
  __device__ __forceinline__ void seek(const AttnArgs &a) {
    for (steps = 0; next < a.problems; next += gridDim.x) {
      steps = keys_of(a, next).steps;
      if (steps) break;
    }
  }
  __device__ __forceinline__ void start(const AttnArgs &a) {
    next = blockIdx.x;
    seek(a);
  }
  __device__ __forceinline__ bool take(const AttnArgs &a, int64_t &token, int &n) {
    token = next;
    n = steps;
    if (!n) return false;
    next += gridDim.x;
    seek(a);
    return true;
  }
};

// The place of set bit n of m.
__device__ __forceinline__ int nth_bit(uint64_t m, int n) {
  int at = 0;
#pragma unroll
  for (int w = 32; w > 0; w >>= 1) {
    const int c = __popcll(m & low_bits(w));
    if (n >= c) {
      n -= c;
      at += w;
      m >>= w;
    }
  }
  return at;
}

// ------------------------------------------------------------------- rows
// A warp has 8 keys of a step: lane l key l % 8, of which it takes 64 channels (a
// column block of the slot) twice, blocks l / 8 and l / 8 + 4.  Four lanes of a key
// read 128 contiguous bytes of an entry, and the eight lanes that a store serves at
// once are eight keys, whose swizzled chunks cover the eight bank groups.
struct KeyData {
  uint4 v[2][4];      // [block]: an entry's codes in the first two, or a row's 64
  uint32_t sc[2];     // [block]: an entry's four scales
  float scale;        // of a row
  int kind;           // 0 none, 1 entry, 2 row of codes
};

__device__ __forceinline__ void st_chunk(uint32_t at, int chunk, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at ^ (uint32_t)(chunk << 4)), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

__device__ __forceinline__ uint32_t or_words(const uint4 (&v)[4], int n) {
  uint32_t any = 0;
#pragma unroll
  for (int u = 0; u < n; ++u) any |= v[u].x | v[u].y | v[u].z | v[u].w;
  return any;
}

// The key's scale f, and what its values are multiplied by, by the four lanes that
// hold it.
__device__ __forceinline__ float scale_of(const KeyData &d, int lane, uint32_t &norm) {
  uint32_t size = 0, codes = 0;
  if (d.kind == 1) {
    size = larger_half(scales_size(d.sc[0], scales_size(d.sc[1], __half2(0.0f, 0.0f))));
    codes = (or_words(d.v[0], 2) | or_words(d.v[1], 2)) & 0x77777777u;
  } else if (d.kind == 2) {
    codes = (or_words(d.v[0], 4) | or_words(d.v[1], 4)) & 0x7F7F7F7Fu;
  }
  size = max(size, __shfl_xor_sync(0xffffffffu, size, 8));
  size = max(size, __shfl_xor_sync(0xffffffffu, size, 16));
  const uint32_t any = __ballot_sync(0xffffffffu, codes) & (0x01010101u << (lane & 7));
  return key_scale(d.kind == 1, size, d.scale, any == 0, norm);
}

// 64 channels into the 128-byte row whose chunk 0 is at `at` (chunk i at ^ 16 i).
__device__ __forceinline__ void put_entry(uint32_t at, const uint4 (&v)[4], uint32_t sc, uint32_t norm) {
  const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
  const uint32_t e[2] = {hmul2_u32(e4m3x2_to_half2((uint16_t)sc), norm), hmul2_u32(e4m3x2_to_half2((uint16_t)(sc >> 16)), norm)};
#pragma unroll
  for (int i = 0; i < 8; ++i) {   // 8 channels, of scale i / 2
    uint32_t h[4];
    e2m1x8_to_half2x4(w[i], h);
    const uint32_t s = __byte_perm(e[i >> 2], 0, i & 2 ? 0x3232 : 0x1010);
    st_chunk(at, i, hmul2_u32(h[0], s), hmul2_u32(h[1], s), hmul2_u32(h[2], s), hmul2_u32(h[3], s));
  }
}

__device__ __forceinline__ void put_codes(uint32_t at, const uint4 (&v)[4], uint32_t norm) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int j = 0; j < 2; ++j)
      st_chunk(at, 2 * i + j, hmul2_u32(e4m3x2_to_half2((uint16_t)w[2 * j]), norm),
               hmul2_u32(e4m3x2_to_half2((uint16_t)(w[2 * j] >> 16)), norm),
               hmul2_u32(e4m3x2_to_half2((uint16_t)w[2 * j + 1]), norm),
               hmul2_u32(e4m3x2_to_half2((uint16_t)(w[2 * j + 1] >> 16)), norm));
  }
}

// List place of key e, or -1 (past the list).
__device__ __forceinline__ int32_t list_id(const AttnArgs &a, const Keys &k, int e) {
  return k.steps && e < a.K ? __ldg(a.idx + k.gp * a.K + e) : -1;
}

// 32 bytes of a key; `wide`: the caches are 32-byte aligned (entries are 9 x 32 bytes).
__device__ __forceinline__ void load32(const uint8_t *p, bool wide, uint4 &x, uint4 &y) {
  if (wide) {
    ld_nc_v8(p, x, y);
  } else {
    x = ld_nc_v4(p);
    y = ld_nc_v4(p + 16);
  }
}

__device__ __forceinline__ void load_key(const AttnArgs &a, const Keys &k, int e, int32_t id, int block, bool wide, KeyData &d) {
  d.kind = 0;
  d.scale = 1.0f;
  if (e < a.K) {
    if (id < 0) return;
    if (id >= a.cap) {
      set_error(CSA2_DEV_ERR_INDEX);
      return;
    }
    const uint8_t *p = a.kv + (k.entry_row0 + id) * ENTRY_BYTES;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      load32(p + 128 * h + 32 * block, wide, d.v[h][0], d.v[h][1]);
      d.sc[h] = ld_nc_u32(p + 256 + 16 * h + 4 * block);
    }
    d.kind = 1;
    return;
  }
  const uint8_t *p;
  const float *s;
  e -= a.K;
  if (e >= k.rows + k.named) return;
  if (e < k.rows) {
    const int64_t at = k.place + e, row = k.ring_row0 + (at >= a.step.ring ? at - a.step.ring : at);
    p = a.swa + row * D;
    s = a.swa_scale + row;
  } else {
    const int64_t row = k.extra_row0 + nth_bit(k.extra, e - k.rows);
    p = a.step.extra + row * D;
    s = a.step.extra_scale + row;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int u = 0; u < 4; u += 2) load32(p + 256 * h + 64 * block + 16 * u, wide, d.v[h][u], d.v[h][u + 1]);
  d.scale = __uint_as_float(ld_nc_u32(s));
  d.kind = 2;
}

// Q in place from bf16 to fp16, by kThreads threads.
template <int kThreads>
__device__ __forceinline__ void convert_q(uint8_t *qs, int t) {
  uint4 *q = reinterpret_cast<uint4 *>(qs) + t;
  constexpr int kAtOnce = 8;   // loads before the first store
#pragma unroll 1
  for (int i = 0; i < H * D * 2 / 16; i += kAtOnce * kThreads) {
    uint4 v[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) v[u] = q[i + u * kThreads];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const uint32_t x[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
      uint32_t h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __half2 f = __floats2half2_rn(__uint_as_float(x[j] << 16), __uint_as_float(x[j] & 0xFFFF0000u));
        h[j] = *reinterpret_cast<const uint32_t *>(&f);
      }
      q[i + u * kThreads] = make_uint4(h[0], h[1], h[2], h[3]);
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
}

__device__ void row_warps_g(const AttnArgs &a, CtlG &S, uint8_t *slots, uint8_t *qs, int w, int lane) {
  const int key = 8 * w + (lane & 7), block = lane >> 3;
  const bool wide = ((reinterpret_cast<uintptr_t>(a.kv) | reinterpret_cast<uintptr_t>(a.swa) |
                      reinterpret_cast<uintptr_t>(a.step.extra)) & 31) == 0;
  int64_t token = blockIdx.x;
  // the step in registers (its token's keys k), the one after it (kn, list places idn)
  Keys k, kn;
  int s = 0, sn = 0;
  int64_t tn = token;
  KeyData d;
  int32_t idn;
  // the next token with steps from `tn` on
  auto seek = [&]() {
    kn.steps = 0;
    for (; tn < a.problems; tn += gridDim.x) {
      kn = keys_of(a, tn);
      if (kn.steps) break;
    }
  };
  auto ids = [&]() { idn = list_id(a, kn, sn * kStep + key); };
  auto load = [&]() {   // the next step becomes the one in registers
    k = kn;
    s = sn;
    if (!k.steps) return;
    load_key(a, k, s * kStep + key, idn, block, wide, d);
    if (++sn == kn.steps) {
      sn = 0;
      tn += gridDim.x;
      seek();
    }
    ids();
  };
  seek();
  ids();
  load();
  uint32_t n = 0;
  for (uint32_t g = 0; k.steps; ++g) {
    const uint32_t b = g & 1;
    const bool first = s == 0;
    uint32_t norm;
    const float f = scale_of(d, lane, norm);
    if (g > 1) wait_g(S, &S.slot_free[b], ((g >> 1) - 1) & 1);
    if (block == 0) {
      S.rs[b][key] = kLogitG * f;
      S.lg[b][key] = d.kind ? log2f(f) : -INFINITY;
      S.inv[b][key] = d.kind ? 1.0f / f : 1.0f;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t at = smem_u32(slots) + b * kSlotG + (4 * h + block) * kBlockG + key * 128 + ((key & 7) << 4);
      if (d.kind == 1) {
        put_entry(at, d.v[h], d.sc[h], norm);
      } else if (d.kind == 2) {
        put_codes(at, d.v[h], norm);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) st_chunk(at, i, 0, 0, 0, 0);
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.rows_full[b]);
    load();
    if (first) {   // the token's Q, which lands about now (the first token's is the softmax warps')
      if (n) {
#pragma unroll
        for (int i = 0; i < kQWaits; ++i) {
          const QWait q = q_wait(n, i);
          wait_g(S, q.ready ? &S.q_ready : &S.q_raw, q.phase & 1);
        }
        convert_q<kRowG * 32>(qs, w * 32 + lane);
        if (lane == 0) mbar_arrive(&S.q_ready);
      }
      ++n;
    }
  }
}

// ---------------------------------------------------------------- softmax
__device__ void softmax_warps_g(const AttnArgs &a, CtlG &S, uint8_t *qs, uint8_t *ps, uint32_t tmem, int w, int lane) {
  const uint32_t lanes = tmem + ((uint32_t)(32 * w) << 16);
  const int th = lane >> 4, h = 16 * w + (lane & 15);
  uint32_t g = 0;
  wait_g(S, &S.q_raw, 0);
  convert_q<kSoftG * 32>(qs, w * 32 + lane);
  if (lane < kRowG / kSoftG) mbar_arrive(&S.q_ready);
  Tokens tokens;
  tokens.start(a);
  int64_t token;
  for (int steps; tokens.take(a, token, steps);) {
    float m = -INFINITY, l = 0.0f;
#pragma unroll 1
    for (int s = 0; s < steps; ++s, ++g) {
      const uint32_t b = g & 1, ph = (g >> 1) & 1;
      wait_g(S, &S.rows_full[b], ph);   // the keys' scales
      wait_g(S, &S.s_full[b], ph);
      tc_fence_after();
      float x[2][16];
      float mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t u0[16], u1[16];
        tmem_ld16x2(lanes + b * 128 + 32 * i, u0);
        tmem_ld16x2(lanes + b * 128 + 64 + 32 * i, u1);
        tmem_ld_wait();
        const float4 *r4 = reinterpret_cast<const float4 *>(&S.rs[b][32 * i + 16 * th]);
        const float4 *g4 = reinterpret_cast<const float4 *>(&S.lg[b][32 * i + 16 * th]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 r = r4[q], e = g4[q];
          x[i][4 * q] = fmaf(__uint_as_float(u0[4 * q]) + __uint_as_float(u1[4 * q]), r.x, e.x);
          x[i][4 * q + 1] = fmaf(__uint_as_float(u0[4 * q + 1]) + __uint_as_float(u1[4 * q + 1]), r.y, e.y);
          x[i][4 * q + 2] = fmaf(__uint_as_float(u0[4 * q + 2]) + __uint_as_float(u1[4 * q + 2]), r.z, e.z);
          x[i][4 * q + 3] = fmaf(__uint_as_float(u0[4 * q + 3]) + __uint_as_float(u1[4 * q + 3]), r.w, e.w);
        }
#pragma unroll
        for (int q = 0; q < 16; ++q) mx = fmaxf(mx, x[i][q]);
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
      // a head that saw no key so far has nothing in O^T: its reference is set, not
      // raised; once one is raised, all are that can be
      if (m == -INFINITY) m = mx;
      if (bar_named_or(1, kSoftG * 32, mx > m + kLazyG)) {
        const float f = mx > m ? ex2_approx(m - mx) : 1.0f;
        m = fmaxf(m, mx);
        if (th == 0) S.fac[h] = f;
        l *= f;
        bar_named(1, kSoftG * 32);
        wait_g(S, &S.slot_free[(g - 1) & 1], ((g - 1) >> 1) & 1);   // the products so far
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < 256; c += 32) {
          uint32_t v[32];
          tmem_ld32(lanes + kColOG + c, v);
          tmem_ld_wait();
#pragma unroll
          for (int q = 0; q < 32; ++q) v[q] = __float_as_uint(__uint_as_float(v[q]) * S.fac[(c & 63) + q]);
          tmem_st32(lanes + kColOG + c, v);
        }
        tmem_st_wait();
        bar_named(1, kSoftG * 32);   // fac may be written again
      }
      const float ms = m == -INFINITY ? 0.0f : m;
      // P of two steps ago has been read
      if (g > 1) wait_g(S, &S.slot_free[b], ((g >> 1) - 1) & 1);
      uint8_t *prow = ps + b * kBlockG + h * 128;
      float l2 = 0.0f;
      uint32_t pk[2][8];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 *v4 = reinterpret_cast<const float4 *>(&S.inv[b][32 * i + 16 * th]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 v = v4[q];
          const float p0 = ex2_approx(x[i][4 * q] - ms), p1 = ex2_approx(x[i][4 * q + 1] - ms),
                      p2 = ex2_approx(x[i][4 * q + 2] - ms), p3 = ex2_approx(x[i][4 * q + 3] - ms);
          l = fmaf(p0, v.x, fmaf(p1, v.y, l));
          l2 = fmaf(p2, v.z, fmaf(p3, v.w, l2));
          const __half2 a2 = __floats2half2_rn(p0, p1), b2 = __floats2half2_rn(p2, p3);
          pk[i][2 * q] = *reinterpret_cast<const uint32_t *>(&a2);
          pk[i][2 * q + 1] = *reinterpret_cast<const uint32_t *>(&b2);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c0 = 4 * i + 2 * th;
        *reinterpret_cast<uint4 *>(prow + ((c0 ^ (h & 7)) << 4)) = make_uint4(pk[i][0], pk[i][1], pk[i][2], pk[i][3]);
        *reinterpret_cast<uint4 *>(prow + (((c0 + 1) ^ (h & 7)) << 4)) = make_uint4(pk[i][4], pk[i][5], pk[i][6], pk[i][7]);
      }
      l += l2;
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(&S.p_full[b]);
    }
    // ---------------------------------------------------------- token's end
    l += __shfl_xor_sync(0xffffffffu, l, 16);
    // a query of infinities or NaNs makes NaNs of the zeros in place of masked keys:
    // without a key nothing of them counts
    bool none = false;
    if (__any_sync(0xffffffffu, l != l)) {
      none = !has_keys(a, token, lane);
      if (none) l = 0.0f;
    }
    if (lane == 0) S.none[w] = none;
    if (th == 0) {
      S.inv_l[h] = l > 0.0f && !S.abort ? 1.0f / l : l;   // (0 stays 0, a NaN a NaN)
      if (a.lse) a.lse[token * H + h] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2G;
    }
    bar_named(1, kSoftG * 32);
    wait_g(S, &S.slot_free[(g - 1) & 1], ((g - 1) >> 1) & 1);
    tc_fence_after();
    const uint4 nw = *reinterpret_cast<const uint4 *>(S.none);
    none = nw.x | nw.y | nw.z | nw.w;   // (one head's warp has found it out for all)
    // 32 heads x 32 channels at a time: a lane's channel, heads in pairs, through the
    // P buffers (which the last products have read) as rows [channel][32 heads], and
    // back transposed, 8 channels of a head a lane, for 64 contiguous bytes a head.
    // (Few shared-memory instructions: pairs of channels by shuffles and 4-byte
    // stores took 9,000 clocks a token beside the row warps' stores.)
    const int mr = lane & 7, md = 8 * (mr >> 1) + 2 * (lane >> 3) + (mr & 1);   // the lane's matrix row: a channel
    const uint32_t sw = (lane >> 3 ^ lane >> 1) & 3, mw = (md >> 3 ^ md >> 1) & 3;
#pragma unroll 1
    for (int h0 = 0; h0 < H; h0 += 32) {
      float il[32];
#pragma unroll
      for (int q = 0; q < 32; q += 4) {
        const float4 f = *reinterpret_cast<const float4 *>(S.inv_l + h0 + q);
        il[q] = f.x;
        il[q + 1] = f.y;
        il[q + 2] = f.z;
        il[q + 3] = f.w;
      }
#pragma unroll 1
      for (int t = 0; t < 4; ++t) {
        uint32_t v[32];
        tmem_ld32(lanes + kColOG + 64 * t + h0, v);
        tmem_ld_wait();
        if (h0 && t == 3) {   // O^T is read: the next token's products may start
          tc_fence_before();
          mbar_arrive(&S.o_free);
        }
        if (none) {
#pragma unroll
          for (int q = 0; q < 32; ++q) v[q] = 0;
        }
        const uint32_t stage = smem_u32(ps + w * 4096 + (t & 1) * 2048);   // (two in turn: one barrier a time)
        uint32_t o[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const __nv_bfloat162 f =
              __floats2bfloat162_rn(__uint_as_float(v[2 * q]) * il[2 * q], __uint_as_float(v[2 * q + 1]) * il[2 * q + 1]);
          o[q] = *reinterpret_cast<const uint32_t *>(&f);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) st_chunk(stage + lane * 64 + (sw << 4), q, o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        __syncwarp();
        __nv_bfloat16 *out = a.step.out + (token * H + h0 + (lane >> 2)) * D + t * 128 + 32 * w + 8 * (lane & 3);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint4 u;
          ldmatrix_x4_trans((stage + md * 64 + (mw << 4)) ^ (uint32_t)(q << 4), u);
          *reinterpret_cast<uint4 *>(out + 8 * q * D) = u;
        }
      }
    }
    bar_named(1, kSoftG * 32);   // inv_l and the other warps' stages may be written again
  }
}

// --------------------------------------------------------------- products
__device__ __forceinline__ void load_q_g(CtlG &S, const CUtensorMap &tm_q, uint8_t *qs, int64_t token) {
  mbar_arrive_expect_tx(&S.q_raw, (uint32_t)(H * D * 2));
#pragma unroll 1
  for (int c = 0; c < 8; ++c) tma_load_2d(qs + c * kBlockG, &tm_q, 64 * c, (int32_t)(token * H), &S.q_raw);
}

// Every product that a warp's elected thread has issued has completed before the
// teardown, also after a wait ran out (a commit tells of its own thread's products
// only).
__device__ __forceinline__ void drain(uint64_t *done) {
  if (elect_one()) mma_commit(done);
  __syncwarp();
  mbar_wait(done, 0);
}

// (both by whole warps, an elected thread issuing)
__device__ void score_warp_g(const AttnArgs &a, CtlG &S, const CUtensorMap &tm_q, uint8_t *slots, uint8_t *qs, uint32_t tmem) {
  const uint64_t qd = smem_desc(smem_u32(qs), 16, 1024), kd = smem_desc(smem_u32(slots), 16, 1024);
  uint32_t g = 0, n = 0, copies = 1;
  Tokens tokens;
  tokens.start(a);
  int64_t token;
  for (int steps; tokens.take(a, token, steps);) {
    // (the first token's Q is on its way; a later one's last reader was the token before's last S)
    if (n) {
      wait_g(S, &S.q_free, (n - 1) & 1);
      if (!__any_sync(0xffffffffu, S.abort != 0)) {
        if (elect_one()) load_q_g(S, tm_q, qs, token);
        ++copies;
      }
      __syncwarp();
    }
    wait_g(S, &S.q_ready, n & 1);
    ++n;
#pragma unroll 1
    for (int s = 0; s < steps; ++s, ++g) {
      const uint32_t b = g & 1, d = tmem + b * 128;
      wait_g(S, &S.rows_full[b], (g >> 1) & 1);
      if (g > 1) wait_g(S, &S.p_full[b], ((g >> 1) - 1) & 1);   // S of two steps ago has been read
      tc_fence_after();
      if (elect_one()) {
        uint64_t qa = qd, kb = kd + (uint64_t)(b * kSlotG >> 4);
#pragma unroll 1
        for (int c = 0; c < 8; c += 2) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            mma_f16(d, qa + 2 * i, kb + 2 * i, kIdescSG, (c | i) ? 1u : 0u);
            mma_f16(d + 64, qa + (kBlockG >> 4) + 2 * i, kb + (kBlockG >> 4) + 2 * i, kIdescSG, (c | i) ? 1u : 0u);
          }
          qa += 2 * (kBlockG >> 4);
          kb += 2 * (kBlockG >> 4);
        }
        mma_commit(&S.s_full[b]);
        if (s == steps - 1) mma_commit(&S.q_free);
      }
      __syncwarp();
    }
  }
  drain(&S.done[0]);
  // a copy still in flight lands before the CTA's memory goes, also after a wait ran
  // out or when the CTA's first token is behind the last sequence
  mbar_wait(&S.q_raw, (copies - 1) & 1);
}

__device__ void value_warp_g(const AttnArgs &a, CtlG &S, uint8_t *slots, uint8_t *ps, uint32_t tmem) {
  const uint64_t vd = smem_desc(smem_u32(slots), kBlockG, 1024), pd = smem_desc(smem_u32(ps), 16, 1024);
  uint32_t g = 0, n = 0;
  Tokens tokens;
  tokens.start(a);
  int64_t token;
  for (int steps; tokens.take(a, token, steps);) {
    if (n) wait_g(S, &S.o_free, (n - 1) & 1);
    ++n;
#pragma unroll 1
    for (int s = 0; s < steps; ++s, ++g) {
      const uint32_t b = g & 1;
      wait_g(S, &S.p_full[b], (g >> 1) & 1);
      tc_fence_after();
      if (elect_one()) {
        uint64_t va = vd + (uint64_t)(b * kSlotG >> 4), pb = pd + (uint64_t)(b * kBlockG >> 4);
#pragma unroll 1
        for (int i = 0; i < kStep / 16; ++i) {   // 16 keys; the accumulators in turn
          const uint32_t acc = (s | i) ? 1u : 0u;
#pragma unroll
          for (int t = 0; t < 4; ++t) mma_f16(tmem + kColOG + 64 * t, va + (uint64_t)(2 * t * kBlockG >> 4), pb, kIdescOG, acc);
          va += 128;
          pb += 2;
        }
        mma_commit(&S.slot_free[b]);
      }
      __syncwarp();
    }
  }
  drain(&S.done[1]);
}

__global__ void __launch_bounds__(kThreadsG, 1)
    gather_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ AttnArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *slots = base, *qs = slots + 2 * kSlotG, *ps = qs + H * D * 2;
  CtlG &S = *reinterpret_cast<CtlG *>(ps + 2 * kBlockG);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == kScoreWarpG && lane == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.rows_full[i], kRowG);
      mbar_init(&S.slot_free[i], 1);
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.p_full[i], kSoftG * 32);
    }
    mbar_init(&S.q_raw, 1);
    mbar_init(&S.q_ready, kRowG);
    mbar_init(&S.q_free, 1);
    mbar_init(&S.o_free, kSoftG * 32);
    for (int i = 0; i < 2; ++i) mbar_init(&S.done[i], 1);
    S.abort = 0;
    fence_barrier_init();
    prefetch_tmap(&tm_q);
  }
  __syncwarp();
  pdl_enter();
  if (warp == kScoreWarpG && lane == 0) load_q_g(S, tm_q, qs, blockIdx.x);   // before its keys are known
  __syncwarp();
  if (warp == kValueWarpG) {
    tmem_alloc(&S.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;
  if (warp < kSoftG)
    softmax_warps_g(a, S, qs, ps, tmem, warp, lane);
  else if (warp < kScoreWarpG)
    row_warps_g(a, S, slots, qs, warp - kSoftG, lane);
  else if (warp == kScoreWarpG)
    score_warp_g(a, S, tm_q, slots, qs, tmem);
  else
    value_warp_g(a, S, slots, ps, tmem);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kValueWarpG) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

cudaError_t launch_gather_attn(const AttnArgs &a, int num_sms, cudaStream_t stream, int *launches) {
  CUtensorMap tm_q;
  if (!make_tmap_bf16(&tm_q, a.q, D, (int64_t)a.problems * H, H)) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(gather_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemG);
  if (e != cudaSuccess) return e;
  const int grid = a.problems < num_sms ? a.problems : num_sms;
  e = launch_pdl(gather_attn_kernel, dim3((unsigned)grid), dim3(kThreadsG), kSmemG, stream, 0u, tm_q, a);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace csa2
