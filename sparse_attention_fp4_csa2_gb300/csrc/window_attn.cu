// Attention over rows that neighbouring tokens share: a causal sliding window
// with the first tokens as sinks (csa2_window_attn), and the drafted tokens of a
// tree over their window and each other when they list no entries (csa2_tree_attn).
//   o_h = sum_k softmax_k(q_h . v_k s_k / sqrt(512)) v_k s_k,
// v_k a row's 512 E4M3 codes, s_k its scale.
//
// A token's query and output are 128 KB for 4 x 64 x 512 flop on each of some 130
// rows: 132 flop a byte, so many tokens are bound by HBM as long as the rows are
// read and converted once, not once a token.  A CTA takes a run of consecutive
// tokens and keeps the rows it needs as bf16 in shared memory (E4M3 is exact in
// bf16, and the queries then go to the tensor core as they are): the window of
// two tokens in R = W + 3 slots, position p in slot p mod R, and the sinks behind
// them.  A step from one pair of tokens to the next converts two rows, while the
// slots that the running products read stay; rows that a token does not see
// (another token's, stale ones) are masked in its softmax.
//
// A tile is two tokens: M = 128 (64 heads of each), N = up to 144 slots.
//   S = Q K^T      tcgen05, Q streamed through a ring of four 16 KB pieces of 64
//                  channels as it arrives (used once: no room and no need for all
//                  of it), two S buffers in tensor memory;
//   softmax        two threads per row of S; the weights are written back in place
//                  of S as the A operand of the second product;
//   O = P V        P from tensor memory, V^T from the same slots (MN-major), in
//                  pieces of 128, 64, 128, 64, 128 channels through two buffers;
//   rows out       bf16 through shared memory and tensor copies.
// What bounds it: HBM in a long run (2 x 8,192 tokens, window 128: 356 us in a graph,
// 6.1 TB/s, 0.91 of a plain copy's rate, and 377 to 389 called one by one; a tile takes 12,000 clocks, of which HBM needs
// 11,650), the latency of the fill and of a tile's chain in a short one (9 prompts
// of 3,139 tokens, 22 a CTA: 89 us, 4.6 TB/s; 64 trees of five tokens 23 us): rows 10,000
// clocks, S 3,000 to 5,000 (Q's arrival), softmax 3,500, the second product and the
// rows out 7,500.
// P is kept as two bf16 numbers, its rounding and the rest (16 bits together:
// bf16 alone would cost 2^-9 of a weight, fp16 would need the rows and the
// queries in fp16 too).  The reference is over logit + log2(s_k), so that P =
// 2^(logit - m) s_k is at most 1 when m is set (2^40 before it is raised) whatever the
// rows' scales are; the row sum takes it times 1 / s_k.  References are whole numbers:
// what a raise multiplies the weights written so far by is then a power of two, and
// both parts keep their bits.
//
// Warps: 0-7 softmax, 8-15 output, 16 rows, 17 copies of Q, 18 first product, 19
// second product.  Every wait is bounded; after one runs out every role falls
// through its waits and the output is undefined (CSA2_DEV_ERR_TIMEOUT).
#include "step_rows.cuh"

namespace csa2 {

namespace {

constexpr int kOutWarp = 8, kOutWarps = 8;   // softmax warps 0 .. 7
constexpr int kRowWarp = kOutWarp + kOutWarps;   // one warp
constexpr int kCopyWarp = kRowWarp + 1, kScoreWarp = kCopyWarp + 1, kValueWarp = kCopyWarp + 2;
constexpr int kThreadsW = (kValueWarp + 1) * 32;   // 96 registers a thread
constexpr int kMaxSlots = 144;
constexpr int kQPiece = 128 * 128;               // [128 rows][64 channels]
constexpr int kQRing = 4;
constexpr int kStage = 32 * 64;                  // [32 rows][32 channels] bf16, one per output warp
constexpr uint32_t kColS = 0, kColsS = 144;      // two S / P buffers
constexpr uint32_t kColO = 288;                  // pieces of 128 channels; of 64 channels behind it
constexpr uint32_t kColL = 480;                  // 1 / row sum, a column per S buffer
constexpr uint32_t kColX = 482;                  // what a row's two softmax threads tell each other: [half] maximum, reference, sum
constexpr float kLogitW = 0.06375871295460785f;  // log2(e) / sqrt(512)
constexpr float kLn2W = 0.69314718055994531f;

struct __align__(16) CtlW {
  uint64_t q_full[kQRing], q_free[kQRing];
  uint64_t fresh_full, rows_full[2], s_full[2], p_full[2], pv_done[2], o_full[2], o_free[2], done[2];
  uint32_t tmem_base;
  volatile uint32_t abort;
  __align__(16) float rs[kMaxSlots];         // per slot: log2(e) / sqrt(512) x scale
  __align__(16) float lg[kMaxSlots];         // log2(scale)
  __align__(16) float inv[kMaxSlots];        // 1 / scale
};

constexpr size_t kSmemW = 1024 + (size_t)kMaxSlots * D * 2 + kQRing * kQPiece + kOutWarps * kStage + sizeof(CtlW);
static_assert(kSmemW <= 232448, "window attention exceeds the shared-memory limit");

struct WindowArgs {
  StepRows s;
  const uint8_t *swa;
  const float *swa_scale;
  float *lse;
  int64_t n_tokens;
  int32_t slots;     // of a tile, a multiple of 16
  int32_t ring;      // R: slots of the window (window form)
  int32_t parts;     // CTAs per sequence (tree form)
};

__device__ __forceinline__ void wait_w(CtlW &S, uint64_t *bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity) || S.abort) return;
  if (!mbar_wait(bar, parity)) S.abort = 1;
}

// A tile: tokens tok and, with n = 2, tok + 1 of sequence seq.  fresh: the slots
// hold nothing of this sequence yet.  pos: the first token's position (window).
struct Tile {
  int64_t tok, pos;
  int seq, n;
  bool fresh;
};

// The tiles of a CTA, in order.  Window form: an equal share of the packed tokens
// (even, so that pairs stay pairs), cut at the sequences' ends.  Tree form: a part
// of a sequence's tokens, every gridDim-th such part.  What the device memory
// holds never makes a tile without tokens or past the call's tokens.
template <bool kTree>
struct Walk {
  int64_t tok = 0, end = 0, seq_end = 0, pos = 0;
  int64_t item = 0;
  int seq = 0;
  bool fresh = true;

  // by whole warps
  __device__ __forceinline__ void start(const WindowArgs &a) {
    if constexpr (kTree) {
      item = blockIdx.x;
    } else {
      int64_t total = a.s.cu[a.s.batch];
      total = total < 0 ? 0 : total < a.n_tokens ? total : a.n_tokens;
      int64_t per = (total + gridDim.x - 1) / gridDim.x;
      if (per > 2) per += per & 1;
      tok = (int64_t)blockIdx.x * per;
      end = min(tok + per, total);
      if (tok < end) {
        find_sequence(a.s.cu, a.s.batch, tok, seq);
        enter(a);
      }
    }
  }
  __device__ __forceinline__ void enter(const WindowArgs &a) {
    const int64_t at = a.s.cu[seq], last = a.s.cu[seq + 1];
    seq_end = seq + 1 < a.s.batch ? max(min(last, end), tok + 1) : end;
    pos = max((int64_t)max(a.s.ctx_len[seq], 0) + tok - at, (int64_t)0);
    fresh = true;
  }
  __device__ __forceinline__ bool next(const WindowArgs &a, Tile &t) {
    if constexpr (kTree) {
      while (tok == end) {   // (a sequence's last parts may be empty)
        if (item >= (int64_t)a.s.batch * a.parts) return false;
        const int T = a.s.extras;
        seq = (int)(item / a.parts);
        const int part = (int)(item - (int64_t)seq * a.parts);
        int per = (T + a.parts - 1) / a.parts;
        per += per & 1;
        const int lo = min(part * per, T), hi = min(lo + per, T);
        tok = (int64_t)seq * T + lo;
        end = (int64_t)seq * T + hi;
        fresh = true;
        item += gridDim.x;
      }
      t.n = end - tok > 1 ? 2 : 1;
    } else {
      if (tok >= end) return false;
      if (tok == seq_end) {
        // the next one with tokens: the neighbour, or by binary search (a run of empty ones)
        ++seq;
        if (seq + 1 < a.s.batch && a.s.cu[seq + 1] <= tok) seq = last_not_above(a.s.cu, seq, a.s.batch - seq, tok);
        enter(a);
      }
      t.n = seq_end - tok > 1 ? 2 : 1;
    }
    t.tok = tok;
    t.pos = pos;
    t.seq = seq;
    t.fresh = fresh;
    fresh = false;
    tok += t.n;
    pos += t.n;
    return true;
  }
};

// ------------------------------------------------------------------- rows
// A row's codes as bf16 in a slot: a lane takes channels 8 lane .. + 7 and those 256
// behind them, a 16-byte chunk of the 128B-swizzled row in column blocks lane / 8
// and lane / 8 + 4 each (eight lanes a whole 128-byte row).
// Two E4M3 codes (bytes 0 and 1, or 2 and 3, of w: `sel`) as bf16: exponent and
// fraction moved to bf16's places are the value times 2^-120, subnormals too.
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t w, uint32_t sel) {
  const uint32_t t = __byte_perm(w, 0, sel);   // the codes in the upper bytes of the halves
  const uint32_t b = (t & 0x80008000u) | ((t >> 4) & 0x07F007F0u);
  const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&b), __nv_bfloat162(
      __ushort_as_bfloat16(0x7B80), __ushort_as_bfloat16(0x7B80)));   // 2^120
  return *reinterpret_cast<const uint32_t *>(&v);
}

// True when the row holds a NaN, which the slot has as 480: it becomes a NaN weight
// (slot_scale: the row's logit is a NaN, so every channel of a token that sees it
// is), and a token that does not see it multiplies the slot by a weight of zero.
__device__ __forceinline__ bool put_row(uint8_t *at, uint32_t half, int slot, const uint4 &v, bool tiny, int lane) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t nan = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) nan |= (w[i] & 0x7F7F7F7Fu) + 0x01010101u;
  if (tiny) w[0] = w[1] = w[2] = w[3] = 0;
  uint8_t *dst = at + slot * 128 + (((lane ^ slot) & 7) << 4);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    *reinterpret_cast<uint4 *>(dst + i * half) =
        make_uint4(e4m3x2_to_bf16x2(w[2 * i], 0x1404), e4m3x2_to_bf16x2(w[2 * i], 0x3424),
                   e4m3x2_to_bf16x2(w[2 * i + 1], 0x1404), e4m3x2_to_bf16x2(w[2 * i + 1], 0x3424));
  return __any_sync(0xffffffffu, nan & 0x80808080u);
}

// What the softmax has to know of a slot (one thread).
__device__ __forceinline__ void slot_scale(CtlW &S, int slot, float scale, bool bad) {
  const float f = scale < kTinyScale ? kTinyScale : scale;
  S.rs[slot] = kLogitW * f;
  S.lg[slot] = bad ? __int_as_float(0x7FFFFFFF) : log2f(f);
  S.inv[slot] = f <= 3.0e38f ? 1.0f / f : 1.0f;   // finite: it multiplies the weights of masked slots (0) too
}

// The codes of n rows that a warp's first n lanes name (NULL: zeros): a lane's 16
// of each.
template <int kRows>
__device__ __forceinline__ void get_rows(uint4 (&v)[kRows], const uint8_t *row, int lane) {
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const uint8_t *p = reinterpret_cast<const uint8_t *>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(row), j));
    v[j] = make_uint4(0, 0, 0, 0);
    if (p) {
      const uint2 a = ld_nc_v2(p + 8 * lane), b = ld_nc_v2(p + 256 + 8 * lane);
      v[j] = make_uint4(a.x, a.y, b.x, b.y);
    }
  }
}

// Which of the barriers says that a tile's rows are in their slots: a sequence's
// first tile has one of its own, the others use two in turn.  (Neither can be a
// phase ahead of a waiting role: a fill comes after every product before it, and
// rows that follow after those of two tiles before.)
struct RowsReady {
  uint32_t fresh = 0, more = 0;
  __device__ __forceinline__ void wait(CtlW &S, const Tile &t) {
    if (t.fresh) {
      wait_w(S, &S.fresh_full, fresh & 1);
      ++fresh;
    } else {
      wait_w(S, &S.rows_full[more & 1], (more >> 1) & 1);
      ++more;
    }
  }
};

// Every slot of a sequence's first tile (tile i of the CTA): the window's rows, the
// extra rows, zeros elsewhere, once the products of tile i - 1 are done.  The
// softmax, output and row warps fill them together.
constexpr int kFillWarps = kRowWarp + 1;

template <bool kTree>
__device__ void fill_slots(const WindowArgs &a, CtlW &S, uint8_t *tile, const Tile &cur, uint32_t i, int w, int lane) {
  const StepRows &s = a.s;
  int64_t first, last, place;   // positions held, the ring place of `last`
  const int32_t len = s.ctx_len[cur.seq];
  const int64_t ctx = max(len, 0);
  if constexpr (kTree) {
    if (len < 0 && w == 0 && lane == 0) set_error(CSA2_DEV_ERR_INDEX);
    last = ctx - 1;
    first = max(ctx - s.win, (int64_t)0);
  } else {
    last = cur.pos + cur.n - 1;
    first = max(cur.pos - s.win + 1, (int64_t)0);
    if (w == 0 && lane == 0 &&
        (len < 0 || (s.win > 0 && min(ctx, (int64_t)s.win - 1) + s.cu[cur.seq + 1] - s.cu[cur.seq] > s.ring)))
      set_error(CSA2_DEV_ERR_INDEX);
  }
  place = last >= 0 ? last % s.ring : 0;
  const int held = kTree ? s.win : a.ring;           // slots of window rows
  const int at = kTree ? 0 : (int)(last % a.ring);   // (window form) the slot of `last`
  constexpr int warps = kFillWarps, kBatch = (kMaxSlots + warps - 1) / warps;   // all of a warp's rows at once
  // lane j names the warp's row j
  const int mine = w + lane * warps;
  const uint8_t *row = nullptr;
  float scale = 1.0f;
  if (lane < kBatch && mine < held) {
    const int back = kTree ? s.win - 1 - mine : (at >= mine ? at - mine : at - mine + a.ring);   // positions before `last`
    if (s.win > 0 && last - back >= first) {
      const int64_t r = (int64_t)cur.seq * s.ring + (place >= back ? place - back : place - back + s.ring);
      row = a.swa + r * D;
      scale = __uint_as_float(ld_nc_u32(a.swa_scale + r));
    }
  } else if (lane < kBatch && mine < held + s.extras) {
    const int64_t r = (int64_t)cur.seq * s.extras + mine - held;
    row = s.extra + r * D;
    scale = __uint_as_float(ld_nc_u32(s.extra_scale + r));
  }
  uint4 v[kBatch];
  get_rows(v, row, lane);
  const uint32_t tiny = __ballot_sync(0xffffffffu, scale < kTinyScale);
  if (i > 0) wait_w(S, &S.pv_done[(i - 1) & 1], ((i - 1) >> 1) & 1);
  uint32_t bad = 0;
  const uint32_t half = 4 * a.slots * 128;
  tile += (lane >> 3) * a.slots * 128;
#pragma unroll
  for (int j = 0; j < kBatch; ++j)
    if (w + j * warps < a.slots) bad |= (uint32_t)put_row(tile, half, w + j * warps, v[j], tiny >> j & 1, lane) << j;
  if (lane < kBatch && mine < a.slots) slot_scale(S, mine, scale, bad >> lane & 1);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(&S.fresh_full);
}

// The rows that the later tiles of a sequence add (window form), two at most, each
// loaded a tile ahead.
template <bool kTree>
__device__ void row_warp(const WindowArgs &a, CtlW &S, uint8_t *tile, Walk<kTree> walk, int lane) {
  const StepRows &s = a.s;
  Tile t;
  uint32_t more = 0, fresh = 0;
  bool filling = false;
  uint4 ahead[2];
  float scale = 1.0f;   // lane k: of row k
  bool next = walk.next(a, t);
  for (uint32_t i = 0; next; ++i) {
    if (t.fresh) {
      fill_slots<kTree>(a, S, tile, t, i, kRowWarp, lane);
      filling = true;
      ++fresh;
    } else {
      // (tree form too, which adds no rows: no role may be two phases behind)
      if (i > 1) wait_w(S, &S.pv_done[i & 1], ((i >> 1) - 1) & 1);
      if constexpr (!kTree) {
        // (a slot written below may be another warp's in the fill before)
        if (filling) wait_w(S, &S.fresh_full, (fresh - 1) & 1);
        filling = false;
        if (s.win > 0) {
          const uint32_t tiny = __ballot_sync(0xffffffffu, scale < kTinyScale);
          const int slot = (int)(t.pos % a.ring), second = slot + 1 == a.ring ? 0 : slot + 1;
          uint8_t *at = tile + (lane >> 3) * a.slots * 128;
          bool bad = put_row(at, 4 * a.slots * 128, slot, ahead[0], tiny & 1, lane);
          if (t.n > 1) {
            const bool b = put_row(at, 4 * a.slots * 128, second, ahead[1], tiny >> 1 & 1, lane);
            if (lane == 1) bad = b;
          }
          if (lane < t.n) slot_scale(S, lane ? second : slot, scale, bad);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(&S.rows_full[more & 1]);
      ++more;
    }
    next = walk.next(a, t);
    if constexpr (!kTree) {
      if (next && !t.fresh && s.win > 0) {
        const int64_t r = (int64_t)t.seq * s.ring + (t.pos + lane) % s.ring;
        scale = lane < t.n ? __uint_as_float(ld_nc_u32(a.swa_scale + r)) : 1.0f;
        get_rows(ahead, lane < t.n ? a.swa + r * D : nullptr, lane);
      }
    }
  }
}

// ---------------------------------------------------------------- softmax
// The slots that a token sees.
template <bool kTree>
struct Seen {
  int at, len, held;   // window slots at, at + 1, .. (around the ring's end) of len rows
  uint64_t extra;

  __device__ __forceinline__ void set(const WindowArgs &a, const Tile &t, int j) {
    const StepRows &s = a.s;
    if constexpr (kTree) {
      const int64_t ctx = max(s.ctx_len[t.seq], 0);
      extra = s.mask[t.tok + j] & low_bits(s.extras);
      len = (int)min((int64_t)max(s.win - __popcll(extra), 0), ctx);
      held = s.win;
      at = held - len;
    } else {
      const int64_t p = t.pos + j, before = p - s.win + 1, first = max(before, (int64_t)0);
      len = (int)(p - first) + 1;
      held = a.ring;
      at = (int)(first % a.ring);
      extra = low_bits((int)(before < s.extras ? (before > 0 ? before : 0) : s.extras));
    }
  }
  // slots 16 c .. + 15, a bit each, by whole warps
  __device__ __forceinline__ uint32_t word(int c, int lane) const {
    const int slot = 16 * c + (lane & 15), e = slot - held;
    const int d = slot - at;
    const bool ok = e < 0 ? (kTree || d >= 0 ? d : d + held) < len && (!kTree || d >= 0) : e < 64 && ((extra >> e) & 1);
    return __ballot_sync(0xffffffffu, ok) & 0xFFFFu;
  }
};

// 2^d of a whole number d <= 0 (0 below fp32's range).
__device__ __forceinline__ float pow2_whole(float d) { return d < -126.0f ? 0.0f : __int_as_float((127 + (int)d) << 23); }

// Weights already written (chunks c0 .. c1 - 1 of 16 slots) times f, a power of two or
// 0: the words of a chunk are 8 of upper halves and 8 of the rest.
__device__ __noinline__ void scale_weights(uint32_t st, int c0, int c1, float f) {
  tmem_st_wait();
#pragma unroll 1
  for (int c = c0; c < c1; ++c) {
    uint32_t u[16];
    tmem_ld16(st + 16 * c, u);
    tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(u[k] << 16) * f, __uint_as_float(u[k] & 0xFFFF0000u) * f);
      u[k] = *reinterpret_cast<const uint32_t *>(&v);
    }
    tmem_st16(st + 16 * c, u);
  }
  tmem_st_wait();
}

// Two threads a row, each on half of its chunks of 16 slots, in one pass: the
// reference is the maximum over both threads' first chunks (rounded up), raised only when a
// logit exceeds it by 2^kLazyW (bf16 has fp32's exponents, so weights above 1 cost
// nothing), which hardly ever happens; the weights written until then are then
// scaled in place, and the other thread's at the end.
constexpr float kLazyW = 40.0f;

// v of this thread's row to the other one of the row (the other half's warp of the
// same 32 rows), and its back.
__device__ __forceinline__ float swap_row(uint32_t lanes, int what, int half, int quarter, float v) {
  tmem_st1(lanes + kColX + 2 * what + half, __float_as_uint(v));
  tmem_st_wait();
  tc_fence_before();
  bar_named(1 + quarter, 64);
  tc_fence_after();
  return __uint_as_float(tmem_ld1(lanes + kColX + 2 * what + (half ^ 1)));
}

template <bool kTree>
__device__ void softmax_warps(const WindowArgs &a, CtlW &S, uint8_t *tile, Walk<kTree> walk, uint32_t tmem, int w, int lane) {
  const int quarter = w & 3, half = w >> 2;
  const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16);
  const int j = quarter >> 1, h = 32 * (quarter & 1) + lane;   // token of the tile, head
  const int chunks = a.slots >> 4, mid = (chunks + 1) >> 1;
  const int c0 = half ? mid : 0, c1 = half ? chunks : mid;
  Tile t;
  RowsReady rows;
  for (uint32_t i = 0; walk.next(a, t); ++i) {
    if (t.fresh) fill_slots<kTree>(a, S, tile, t, i, w, lane);
    const uint32_t b = i & 1, st = lanes + kColS + b * kColsS;
    Seen<kTree> see;
    if (j < t.n) {
      see.set(a, t, j);
    } else {
      see.at = see.len = see.held = 0;
      see.extra = 0;
    }
    rows.wait(S, t);   // the slots' scales
    wait_w(S, &S.s_full[b], (i >> 1) & 1);
    tc_fence_after();
    float m = -INFINITY, l = 0.0f;
#pragma unroll 1
    for (int c = c0; c < c1; ++c) {
      uint32_t u[16];
      tmem_ld16(st + 16 * c, u);
      const uint32_t seen = see.word(c, lane);
      float4 r[4], g[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        r[q] = *reinterpret_cast<const float4 *>(S.rs + 16 * c + 4 * q);
        g[q] = *reinterpret_cast<const float4 *>(S.lg + 16 * c + 4 * q);
      }
      tmem_ld_wait();
      float x[16];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        x[4 * q] = fmaf(__uint_as_float(u[4 * q]), r[q].x, g[q].x);
        x[4 * q + 1] = fmaf(__uint_as_float(u[4 * q + 1]), r[q].y, g[q].y);
        x[4 * q + 2] = fmaf(__uint_as_float(u[4 * q + 2]), r[q].z, g[q].z);
        x[4 * q + 3] = fmaf(__uint_as_float(u[4 * q + 3]), r[q].w, g[q].w);
      }
      if (seen != 0xFFFFu) {
#pragma unroll
        for (int q = 0; q < 16; ++q)
          if (!(seen >> q & 1)) x[q] = -INFINITY;
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int q = 0; q < 16; ++q) mx[q & 3] = fmaxf(mx[q & 3], x[q]);
      float cm = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      if (c == c0) {
        m = ceilf(fmaxf(cm, swap_row(lanes, 0, half, quarter, cm)));
      } else {
        const bool up = cm > m + kLazyW;
        if (__any_sync(0xffffffffu, up)) {
          cm = ceilf(cm);
          const float f = !up ? 1.0f : m == -INFINITY ? 0.0f : pow2_whole(m - cm);
          if (__any_sync(0xffffffffu, up && m != -INFINITY)) scale_weights(st, c0, c, f);
          l *= f;
          if (up) m = cm;
        }
      }
      const float ms = m == -INFINITY ? 0.0f : m;
      uint32_t o[16];
      float l2 = 0.0f;
#pragma unroll
      for (int q = 0; q < 16; q += 4) {
        const float4 v = *reinterpret_cast<const float4 *>(S.inv + 16 * c + q);
        const float p0 = ex2_approx(x[q] - ms), p1 = ex2_approx(x[q + 1] - ms), p2 = ex2_approx(x[q + 2] - ms),
                    p3 = ex2_approx(x[q + 3] - ms);
        l = fmaf(p0, v.x, fmaf(p1, v.y, l));
        l2 = fmaf(p2, v.z, fmaf(p3, v.w, l2));
        // the upper halves, and what they leave, rounded
        const uint32_t b0 = __float_as_uint(p0), b1 = __float_as_uint(p1), b2 = __float_as_uint(p2), b3 = __float_as_uint(p3);
        o[q >> 1] = __byte_perm(b0, b1, 0x7632);
        o[(q >> 1) + 1] = __byte_perm(b2, b3, 0x7632);
        const __nv_bfloat162 r0 = __floats2bfloat162_rn(p0 - __uint_as_float(b0 & 0xFFFF0000u), p1 - __uint_as_float(b1 & 0xFFFF0000u));
        const __nv_bfloat162 r1 = __floats2bfloat162_rn(p2 - __uint_as_float(b2 & 0xFFFF0000u), p3 - __uint_as_float(b3 & 0xFFFF0000u));
        o[8 + (q >> 1)] = *reinterpret_cast<const uint32_t *>(&r0);
        o[8 + (q >> 1) + 1] = *reinterpret_cast<const uint32_t *>(&r1);
      }
      l += l2;
      tmem_st16(st + 16 * c, o);
    }
    if (c0 == c1) m = ceilf(swap_row(lanes, 0, half, quarter, m));   // (16 slots in all: none of them this thread's)
    // one reference and one sum for the row
    tmem_st1(lanes + kColX + 4 + half, __float_as_uint(l));
    const float mo = swap_row(lanes, 1, half, quarter, m), mm = fmaxf(m, mo);
    const float lo = __uint_as_float(tmem_ld1(lanes + kColX + 4 + (half ^ 1)));
    if (__any_sync(0xffffffffu, m < mm)) {
      const float f = m < mm ? (m == -INFINITY ? 0.0f : pow2_whole(m - mm)) : 1.0f;
      scale_weights(st, c0, c1, f);
      l *= f;
    }
    l += mo < mm ? (mo == -INFINITY ? 0.0f : lo * pow2_whole(mo - mm)) : lo;
    if (half == 0) tmem_st1(lanes + kColL + b, __float_as_uint(l > 0.0f && !S.abort ? 1.0f / l : l));   // (0 stays 0, a NaN a NaN)
    tmem_st_wait();
    tc_fence_before();
    mbar_arrive(&S.p_full[b]);
    if (half == 0 && a.lse && j < t.n) a.lse[(t.tok + j) * H + h] = l == 0.0f ? -INFINITY : (mm + log2f(l)) * kLn2W;
  }
}

// ----------------------------------------------------------------- output
// The five pieces of a tile's channels: even ones 128 channels in the first
// buffer, odd ones 64 in the second.  Two warps for each 32 rows take every other
// 32 channels.
template <bool kTree>
__device__ void output_warps(const WindowArgs &a, CtlW &S, const CUtensorMap &tm_out, uint8_t *tile, uint8_t *stage,
                             Walk<kTree> walk, uint32_t tmem, int w, int lane) {
  const int quarter = w & 3, half = w >> 2, j = quarter >> 1;
  const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16);
  stage += w * kStage;
  uint32_t use[2] = {0, 0};
  Tile t;
  for (uint32_t i = 0; walk.next(a, t); ++i) {
    if (t.fresh) fill_slots<kTree>(a, S, tile, t, i, kOutWarp + w, lane);
    wait_w(S, &S.p_full[i & 1], (i >> 1) & 1);
    tc_fence_after();
    const float inv = __uint_as_float(tmem_ld1(lanes + kColL + (i & 1)));
    const int32_t y = (int32_t)((t.tok + j) * H + 32 * (quarter & 1));
#pragma unroll 1
    for (int piece = 0; piece < 5; ++piece) {
      const int buf = piece & 1, c0 = 192 * (piece >> 1) + 128 * buf, n = buf ? 2 : 4;
      wait_w(S, &S.o_full[buf], use[buf] & 1);
      ++use[buf];
      tc_fence_after();
#pragma unroll 1
      for (int e = half; e < n; e += 2) {
        uint32_t u[32];
        tmem_ld32(lanes + kColO + 128 * buf + 32 * e, u);
        tmem_ld_wait();
        if (e + 2 >= n) {   // the buffer is free for the next piece
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.o_free[buf]);
        }
        if (j >= t.n) continue;
        uint32_t o[16];
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(u[2 * x]) * inv, __uint_as_float(u[2 * x + 1]) * inv);
          o[x] = *reinterpret_cast<const uint32_t *>(&v);
        }
        if (lane == 0) bulk_wait_read<0>();   // the copy out of the stage before has read it
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<uint4 *>(stage + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)) =
              make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&tm_out, c0 + 32 * e, y, stage);
          bulk_commit();
        }
      }
    }
  }
  if (lane == 0) bulk_wait<0>();
}

// --------------------------------------------------------------- products
template <bool kTree>
__device__ void copy_warp(const WindowArgs &a, CtlW &S, const CUtensorMap &tm_q, uint8_t *ring, Walk<kTree> walk) {
  uint32_t n = 0;
  Tile t;
  while (walk.next(a, t)) {
#pragma unroll 1
    for (int c = 0; c < 8; ++c, ++n) {
      const uint32_t slot = n % kQRing, round = n / kQRing;
      if (round) wait_w(S, &S.q_free[slot], (round - 1) & 1);
      if (S.abort) break;
      mbar_arrive_expect_tx(&S.q_full[slot], (uint32_t)t.n * (kQPiece / 2));
      for (int j = 0; j < t.n; ++j)
        tma_load_2d(ring + slot * kQPiece + j * (kQPiece / 2), &tm_q, 64 * c, (int32_t)((t.tok + j) * H), &S.q_full[slot]);
    }
    if (S.abort) break;
  }
  // copies still in flight land before the CTA's memory goes, also after a wait ran out
  for (uint32_t k = n > kQRing ? n - kQRing : 0; k < n; ++k) mbar_wait(&S.q_full[k % kQRing], (k / kQRing) & 1);
}

// Every product that this thread has issued has completed before the teardown, also
// after a wait ran out (a commit tells of its own thread's products only).
__device__ __forceinline__ void drain(uint64_t *done) {
  mma_commit(done);
  mbar_wait(done, 0);
}

template <bool kTree>
__device__ void score_warp(const WindowArgs &a, CtlW &S, uint8_t *tile, uint8_t *ring, Walk<kTree> walk, uint32_t tmem) {
  const uint32_t idesc = idesc_f16(/*bf16*/ 1, 0, 0, (uint32_t)a.slots, 128);
  const uint64_t kd = smem_desc(smem_u32(tile), 16, 1024), qd = smem_desc(smem_u32(ring), 16, 1024);
  const uint64_t col = (uint64_t)a.slots * 128 >> 4;
  uint32_t n = 0;
  Tile t;
  RowsReady rows;
  for (uint32_t i = 0; walk.next(a, t); ++i) {
    const uint32_t b = i & 1, d = tmem + kColS + b * kColsS;
    rows.wait(S, t);
    if (i > 1) wait_w(S, &S.pv_done[b], ((i >> 1) - 1) & 1);   // P of two tiles ago has been read
#pragma unroll 1
    for (int c = 0; c < 8; ++c, ++n) {
      const uint32_t slot = n % kQRing;
      wait_w(S, &S.q_full[slot], (n / kQRing) & 1);
      tc_fence_after();
      const uint64_t qa = qd + (uint64_t)(slot * kQPiece >> 4), kb = kd + c * col;
#pragma unroll
      for (int k = 0; k < 4; ++k) mma_f16(d, qa + 2 * k, kb + 2 * k, idesc, (c | k) ? 1u : 0u);
      mma_commit(&S.q_free[slot]);
    }
    mma_commit(&S.s_full[b]);
  }
  drain(&S.done[0]);
}

template <bool kTree>
__device__ void value_warp(const WindowArgs &a, CtlW &S, uint8_t *tile, Walk<kTree> walk, uint32_t tmem) {
  const uint64_t col = (uint64_t)a.slots * 128 >> 4;
  const uint64_t vd = smem_desc(smem_u32(tile), (uint32_t)a.slots * 128, 1024);
  const int steps = a.slots / 16;
  uint32_t use[2] = {0, 0};
  Tile t;
  for (uint32_t i = 0; walk.next(a, t); ++i) {
    const uint32_t b = i & 1, p = tmem + kColS + b * kColsS;
    wait_w(S, &S.p_full[b], (i >> 1) & 1);
    tc_fence_after();
#pragma unroll 1
    for (int piece = 0; piece < 5; ++piece) {
      const int buf = piece & 1;
      const uint32_t idesc = idesc_f16(/*bf16*/ 1, 0, /*B MN-major*/ 1, buf ? 64 : 128, 128);
      const uint32_t d = tmem + kColO + 128 * buf;
      if (use[buf]) wait_w(S, &S.o_free[buf], (use[buf] - 1) & 1);
      ++use[buf];
      tc_fence_after();
      uint64_t vb = vd + (uint64_t)(3 * (piece >> 1) + 2 * buf) * col;
#pragma unroll 1
      for (int k = 0; k < steps; ++k, vb += 128) {
        // 16 slots: 8 columns of upper halves, 8 of the rest
        mma_f16_ts(d, p + 16 * k, vb, idesc, k ? 1u : 0u);
        mma_f16_ts(d, p + 16 * k + 8, vb, idesc, 1u);
      }
      mma_commit(&S.o_full[buf]);
    }
    mma_commit(&S.pv_done[b]);
  }
  drain(&S.done[1]);
}

template <bool kTree>
__global__ void __launch_bounds__(kThreadsW, 1)
    window_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_out,
                       const WindowArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *tile = base, *ring = tile + (size_t)kMaxSlots * D * 2, *stage = ring + kQRing * kQPiece;
  CtlW &S = *reinterpret_cast<CtlW *>(stage + kOutWarps * kStage);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kQRing; ++i) {
      mbar_init(&S.q_full[i], 1);
      mbar_init(&S.q_free[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.rows_full[i], 1);
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.p_full[i], kOutWarp * 32);
      mbar_init(&S.pv_done[i], 1);
      mbar_init(&S.o_full[i], 1);
      mbar_init(&S.o_free[i], kOutWarps);
    }
    mbar_init(&S.fresh_full, kFillWarps);
    for (int i = 0; i < 2; ++i) mbar_init(&S.done[i], 1);
    S.abort = 0;
    fence_barrier_init();
  }
  if (warp == kCopyWarp && lane == 0) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_out);
  }
  pdl_enter();
  if (warp == kValueWarp) {
    tmem_alloc(&S.tmem_base, 512);
    tmem_relinquish();
  }
  Walk<kTree> walk;
  walk.start(a);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;
  if (warp < kOutWarp) {
    softmax_warps<kTree>(a, S, tile, walk, tmem, warp, lane);
  } else if (warp < kRowWarp) {
    output_warps<kTree>(a, S, tm_out, tile, stage, walk, tmem, warp - kOutWarp, lane);
  } else if (warp == kRowWarp) {
    row_warp<kTree>(a, S, tile, walk, lane);
  } else if (elect_one()) {
    if (warp == kCopyWarp)
      copy_warp<kTree>(a, S, tm_q, ring, walk);
    else if (warp == kScoreWarp)
      score_warp<kTree>(a, S, tile, ring, walk, tmem);
    else
      value_warp<kTree>(a, S, tile, walk, tmem);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kValueWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

bool window_rows_fit(const StepRows &s) {
  return (s.cu ? s.win + 3 : s.win) + s.extras <= kMaxSlots;
}

cudaError_t launch_window_attn(const void *q, const uint8_t *swa, const float *swa_scale, const StepRows &s, int64_t tokens,
                               float *lse, int num_sms, cudaStream_t stream, int *launches) {
  WindowArgs a;
  a.s = s;
  a.swa = swa;
  a.swa_scale = swa_scale;
  a.lse = lse;
  a.n_tokens = tokens;
  a.ring = s.win + 3;
  const int rows = (s.cu ? a.ring : s.win) + s.extras;
  a.slots = (rows + 15) / 16 * 16;
  if (a.slots < 16) a.slots = 16;
  int64_t grid;
  if (s.cu) {
    a.parts = 0;
    grid = num_sms;   // (there are more tokens: csrc/api.cu)
  } else {
    // as many CTAs for each sequence as fit, at least a pair of tokens each
    const int pairs = (s.extras + 1) / 2, fit = num_sms / s.batch;
    a.parts = fit < 1 ? 1 : fit < pairs ? fit : pairs;
    const int64_t items = (int64_t)s.batch * a.parts;
    grid = items < num_sms ? items : num_sms;
  }
  CUtensorMap tm_q, tm_out;
  if (!make_tmap_bf16(&tm_q, q, D, tokens * H, H) || !make_tmap_bf16_half(&tm_out, s.out, D, tokens * H, 32))
    return cudaErrorInvalidValue;
  auto kern = s.cu ? window_attn_kernel<false> : window_attn_kernel<true>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemW);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3((unsigned)grid), dim3(kThreadsW), kSmemW, stream, 0u, tm_q, tm_out, a);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace csa2
