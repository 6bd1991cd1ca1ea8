// fa_score.cuh -- attention forward with modified scores, on grouped heads.
// sm_103a.
//
// The scores x_ij = scale <q_i, k_j> of a row at key position p = i + Skv - Sq
// become cap tanh(x / cap), minus slope_h |p - j|, and are visible where
// (not causal, or j <= p, or j < prefix_b) and the row's document is the
// key's.  The softmax, the products and the pipeline around them are those of
// the single-CTA prefill kernel (fa_prefill.cuh): a persistent CTA per SM,
// items of 256 rows in two ping-pong stages, S and O in tensor memory, P over
// S, one TMA producer, one MMA warp, an epilogue warpgroup.  What differs:
//
//   rows     Up to 128 query tokens: the group's heads of a kv head are
//            consecutive rows in memory, so they are taken together and K and
//            V are read once for the group.
//   halves   Where 256-row items would leave SMs idle, an item is 128 rows, both
//            stages have them, and the key tiles go to the stages in turn; the
//            epilogue joins the two states.  Every tile is then a K and a V
//            tile of its own, but a stage's softmax still hides behind the other's
//            products: 1.0 us a tile, 1.6 with the 128 rows in one stage alone.
//   tiles    An item walks the key tiles [t0, t0 + nT1): up to the last key
//            that a row sees, and with documents only those that hold ids of
//            the item's rows.  Tiles inside that range without a visible key
//            are computed and masked (documents that do not lie together).
//   scores   Tiles where every key is visible to every row of a warp are not
//            masked.  tanh is an odd polynomial of four terms where |x / cap|
//            is at most 0.5 (off by 1.0e-6 of the value at most; 5 FMA-pipe
//            operations a score), else 1 - 2 / (1 + e^2x) (an exponential and a
//            reciprocal on the XU: measured 1.4 times the whole kernel's time),
//            which only tiles with such a score meet.  The bias is linear in the column
//            on either side of the diagonal; tiles across it take |p - j|.
//            Document masks are built as 128 bits a row, by one ballot per
//            distinct document of the warp's rows.
//
// Like the prefill kernel it is bound by the chain softmax -> PV -> QK ->
// softmax of a stage; the cap adds FMA work to its softmax.
#pragma once
#include "fa_prefill.cuh"
#include "fa_score.h"

namespace fa {

// Packed pair of fp32 products (one mul.rn.f32x2).
__device__ __forceinline__ void fmul2(float& d0, float& d1, float a0, float a1, float b0,
                                      float b1) {
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

// How a call caps its scores: not; with the running reference maximum; without
// a reference, where the cap bounds every score enough.
enum CapForm { kCapNone = 0, kCapRunning = 1, kCapFixed = 2 };

// Registers a thread of the softmax, epilogue and control warpgroups: as in the
// prefill kernel for unmodified scores, more for the softmax of modified ones (the
// sums are the launch's allocation).  Measured on B4 H16 S4096 D128, bf16, us, for
// 176, 184 and 192: plain 371, 384, 384; cap 50 491, 470, 466; cap 100, causal,
// 301, 300, 290; a bias at B8 H16 S2048 D64 in fp16 124, 120, 127.
constexpr int kRegsLaunch = kThreads * 128;
template <int kCap, bool kBias>
struct ScoreRegs {
  static constexpr bool kMore = kCap != kCapNone || kBias;
  static constexpr int kSoftmax = kCap == kCapRunning ? 192 : kMore ? 184 : 176;
  static constexpr int kEpilogue = kCap == kCapRunning ? 56 : kMore ? 64 : 72;
  static constexpr int kControl = kCap == kCapRunning ? 72 : kMore ? 80 : 88;
  static_assert(128 * (2 * kSoftmax + kEpilogue + kControl) == kRegsLaunch,
                "register split must equal the launch allocation");
};

// One work item, worked out by the producer and handed to the other roles
// through a ring in shared memory (worked out by each of them, its divisions
// took 10 % of the kernel's time, 18 % at D = 64).
struct ScoreItem {
  int valid;       // 0: no more items
  int rh, b, kvh;  // row head, its batch row, its kv head [B * Hkv]
  int h0;          // its query head (packed: the group's first)
  int row0, nT0, nT1, t0, split;  // nT_s: stage s's tiles
  int turn;                       // >= 0: both stages' first tile is t0 + turn
};

// Key tiles that an item loads.
template <bool kHalves>
__device__ __forceinline__ int item_tiles(const ScoreItem& it) {
  return kHalves ? it.nT0 + it.nT1 : it.nT1;
}

// The q-th tile of an item that walks n tiles backwards: from the last to the
// first or, with `turn`, from t0 + turn to the first and then from the last.
template <bool kTurns>
__device__ __forceinline__ int tile_back(const ScoreItem& it, int n, int q) {
  if (kTurns && it.turn >= 0)
    return it.t0 + (q <= it.turn ? it.turn - q : it.turn + n - q);
  return it.t0 + n - 1 - q;
}

// Keys on both sides of the rows, with a bias: the tile next to the rows, whose
// scores are the largest (B4 H16 S4096 D128: 432 us, 527 from the last tile on).
template <bool kHalves>
__device__ __forceinline__ int item_turn(const ScoreParams& p, const ScoreItem& it) {
  const int n = item_tiles<kHalves>(it);
  if (!p.slopes || p.causal || (!kHalves && it.nT0 != it.nT1)) return -1;
  const int i = p.packed ? p.Sq - 1 : min(it.row0 + (kHalves ? kBM : kRowsPerCta), p.rows) - 1;
  return min(max(max(i + (p.Skv - p.Sq), 0) / kBN - it.t0, 0), n - 1);
}

template <int D>
struct ScoreLayout : PrefillLayout<D> {
  static constexpr int kOffRing = PrefillLayout<D>::kOffMisc + PrefillLayout<D>::kMiscBytes;
  static constexpr int kSmemBytes = kOffRing + kItemRing * static_cast<int>(sizeof(ScoreItem)) + 1024;
  // halves: [2][2][128] reference maxima and sums, where stage 1's Q would be
  static constexpr int kOffStates = PrefillLayout<D>::kOffQ + PrefillLayout<D>::kQBytes;
  static_assert(kOffRing % 4 == 0 && kSmemBytes <= 232448, "shared memory budget");
};

// First row of stage s of an item; p.rows where the stage has none.
template <bool kHalves>
__device__ __forceinline__ int stage_row(const ScoreParams& p, int row0, int s) {
  return kHalves ? row0 : min(row0 + s * kBM, p.rows);
}

// The key tiles [x, y) that the 128 rows from `row` of batch row b need.
__device__ __forceinline__ int2 stage_range(const ScoreParams& p, int b, int row) {
  if (row >= p.rows) return make_int2(0, 0);
  const int n_all = (p.Skv + kBN - 1) / kBN;
  int lo = 0, hi = n_all;
  if (p.causal) {
    const int last = min(row + kBM, p.rows) - 1;
    // the last query token among the rows (packed rows run through the heads)
    int i = last;
    if (p.packed) i = row / p.Sq == last / p.Sq ? last % p.Sq : p.Sq - 1;
    int keys = i + 1 + (p.Skv - p.Sq);
    if (p.prefix) keys = max(keys, p.prefix[b]);
    keys = min(max(keys, 0), p.Skv);
    hi = (keys + kBN - 1) / kBN;
  }
  if (p.doc_k) {
    const int2 d = p.stage_tiles[static_cast<size_t>(b) * p.n_stages + row / kBM];
    lo = max(lo, d.x);
    hi = min(hi, d.y);
  }
  return make_int2(lo, max(lo, hi));
}

template <bool kHalves>
__device__ __forceinline__ ScoreItem get_score_item(const ScoreParams& p, int idx) {
  ScoreItem it;
  it.valid = 1;
  const int qi = p.n_splits == 1 ? idx : idx / p.n_splits;
  it.split = idx - qi * p.n_splits;
  int qtile;
  if (p.causal) {  // heaviest first
    const int back = qi / p.row_heads;
    qtile = p.n_qtiles - 1 - back;
    it.rh = qi - back * p.row_heads;
  } else {
    it.rh = qi / p.n_qtiles;
    qtile = qi - it.rh * p.n_qtiles;
  }
  if (p.packed) {
    it.b = it.rh / p.Hkv;
    it.kvh = it.rh;
    it.h0 = (it.rh - it.b * p.Hkv) * p.group;
  } else {
    it.b = it.rh / p.H;
    it.h0 = it.rh - it.b * p.H;
    it.kvh = it.b * p.Hkv + it.h0 / p.group;
  }
  it.row0 = qtile * (kHalves ? kBM : kRowsPerCta);
  int2 r0 = stage_range(p, it.b, stage_row<kHalves>(p, it.row0, 0));
  int2 r1 = stage_range(p, it.b, stage_row<kHalves>(p, it.row0, 1));
  const int s0 = it.split * p.tiles_per_split, s1 = s0 + p.tiles_per_split;
  r0.x = max(r0.x, s0);
  r1.x = max(r1.x, s0);
  r0.y = min(r0.y, s1);
  r1.y = min(r1.y, s1);
  if constexpr (kHalves) {
    const int n = max(r0.y - r0.x, 0);
    it.t0 = r0.x;
    it.nT0 = (n + 1) >> 1;
    it.nT1 = n >> 1;
    it.turn = item_turn<kHalves>(p, it);
    return it;
  }
  const bool h0 = r0.x < r0.y, h1 = r1.x < r1.y;
  it.t0 = h0 ? (h1 ? min(r0.x, r1.x) : r0.x) : (h1 ? r1.x : 0);
  it.nT0 = h0 ? r0.y - it.t0 : 0;
  // the MMA warp steps through stage 1's tiles: stage 0 never has more
  it.nT1 = max(h1 ? r1.y - it.t0 : 0, it.nT0);
  it.turn = item_turn<kHalves>(p, it);
  return it;
}

__device__ __forceinline__ int claim_score_item(const ScoreParams& p) {
  const unsigned long long ticket = atomicAdd(p.sched, 1ull);
  const unsigned long long idx = gridDim.x + ticket;
  return idx < static_cast<unsigned long long>(p.n_items) ? static_cast<int>(idx) : -1;
}

// The k-th item of this CTA, as published by the producer.
template <unsigned kSleepNs>
__device__ __forceinline__ ScoreItem take_score_item(const ScoreItem* ring, uint32_t full,
                                                     uint32_t empty, uint32_t k, const Ctl& c,
                                                     bool& ok) {
  const uint32_t slot = k % kItemRing;
  ok = wait_bar_warp<kSleepNs>(full + 8u * slot, (k / kItemRing) & 1, c);
  ScoreItem it{};
  if (ok) it = ring[slot];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(empty + 8u * slot);
  return it;
}

// What a softmax thread knows of its row during an item, and its warp of all 32.
struct ScoreRow {
  int lim;         // keys below it are visible (documents apart)
  int lim_warp;    // the least of the warp's
  int doc;         // its document (< 0: sees nothing)
  int doc_warp;    // the warp's one document, or kDocSeveral
  int pos;         // the row's own key position
  float slope;     // slope * log2(e)
};
// No tile has this "document": a warp whose rows have several.
constexpr int kDocSeveral = kDocMixed + 1;

// The exponential form of a capped score, for |s scale / cap| past the
// polynomial's range: off by about 1e-7 of the cap.
__device__ __forceinline__ float cap_far(float t, const ScoreParams& p) {
  const float ex = ex2_approx(t * p.cap_arg);
  return fmaf(-2.f * p.cap_log2, __fdividef(1.f, 1.f + ex), p.cap_log2);
}

// Two capped scores, each by the form that holds for it.  Within the polynomial's
// range they have the bits of a tile without scores past it, so that no other
// score, of whatever row or of a key that none sees, changes them; there the
// exponential form would be off by the cap's last digits (0.1 in a score near 0
// under a cap of 1e6).
__device__ __forceinline__ void cap_pair(float& x0, float& x1, float a, float b,
                                         const ScoreParams& p) {
  const float c0 = p.cap_poly[0], c1 = p.cap_poly[1], c2 = p.cap_poly[2], c3 = p.cap_poly[3];
  float t0, t1, u0, u1, y0, y1;
  fmul2(t0, t1, a, b, p.cap_mul, p.cap_mul);
  fmul2(u0, u1, t0, t1, t0, t1);
  ffma2(y0, y1, u0, u1, c3, c3, c2, c2);
  ffma2(y0, y1, y0, y1, u0, u1, c1, c1);
  ffma2(y0, y1, y0, y1, u0, u1, c0, c0);
  fmul2(y0, y1, y0, y1, t0, t1);
  const float f0 = cap_far(t0, p), f1 = cap_far(t1, p);
  x0 = u0 <= p.cap_u_max ? y0 : f0;
  x1 = u1 <= p.cap_u_max ? y1 : f1;
}

// Scores of one tile in log2 units after the cap: x = cap log2(e) tanh(s scale
// / cap).  The polynomial runs over the registers first; a warp with a score
// past its range takes its tile through tensor memory once more, each score by
// its own form.
__device__ __forceinline__ void cap_tile(uint32_t (&sr)[8][16], uint32_t tS, const ScoreParams& p) {
  float top = 0.f;
  const float c0 = p.cap_poly[0], c1 = p.cap_poly[1], c2 = p.cap_poly[2], c3 = p.cap_poly[3];
#pragma unroll
  for (int cc = 0; cc < 8; ++cc)
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      const float a = __uint_as_float(sr[cc][e]), b = __uint_as_float(sr[cc][e + 1]);
      float u0, u1, y0, y1;
      fmul2(u0, u1, a, b, a, b);
      top = fmax3(top, u0, u1);
      ffma2(y0, y1, u0, u1, c3, c3, c2, c2);
      ffma2(y0, y1, y0, y1, u0, u1, c1, c1);
      ffma2(y0, y1, y0, y1, u0, u1, c0, c0);
      fmul2(y0, y1, y0, y1, a, b);
      sr[cc][e] = __float_as_uint(y0);
      sr[cc][e + 1] = __float_as_uint(y1);
    }
  if (!__any_sync(0xffffffffu, !(top <= p.cap_u_fast))) return;
#pragma unroll 1
  for (int c = 0; c < kBN; c += 16) {
    uint32_t v[16];
    tmem_ld16(tS + c, v);
    tmem_wait_ld();
    reg_fence16(v);
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      float x0, x1;
      cap_pair(x0, x1, __uint_as_float(v[e]), __uint_as_float(v[e + 1]), p);
      v[e] = __float_as_uint(x0);
      v[e + 1] = __float_as_uint(x1);
    }
    tmem_st16(tS + c, v);
  }
  tmem_wait_st();
#pragma unroll
  for (int cc = 0; cc < 8; cc += 2) tmem_ld32(tS + cc * 16, sr[cc], sr[cc + 1]);
  tmem_wait_ld();
#pragma unroll
  for (int cc = 0; cc < 8; ++cc) reg_fence16(sr[cc]);
}

// The bits of the columns below the row's limit.
__device__ __forceinline__ void limit_columns(int lim, int key0, uint32_t (&bits)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int n = lim - key0 - 32 * k;
    bits[k] &= n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u);
  }
}

// The bit mask of the tile's columns that the row sees, its document's below its
// limit.  Lane l holds the ids of columns l, l + 32, l + 64, l + 96; each distinct
// document of the warp's rows is one round of ballots.  Made while the warp would
// wait for the scores.
__device__ __forceinline__ void doc_columns(const ScoreParams& p, int b, int key0,
                                            const ScoreRow& row, uint32_t (&bits)[4]) {
  const int my_doc = row.doc;
  const int lane = static_cast<int>(lane_id());
  int id[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int key = key0 + 32 * k + lane;
    id[k] = key < p.Skv ? p.doc_k[static_cast<size_t>(b) * p.Skv + key] : -1;
    bits[k] = 0u;
  }
  uint32_t todo = 0xffffffffu;
  while (todo) {
    const int d = __shfl_sync(0xffffffffu, my_doc, __ffs(static_cast<int>(todo)) - 1);
    const bool mine = my_doc == d;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t v = __ballot_sync(0xffffffffu, id[k] == d && d >= 0);
      if (mine) bits[k] = v;
    }
    todo &= ~__ballot_sync(0xffffffffu, mine);
  }
  limit_columns(row.lim, key0, bits);
}

// One key tile of one stage's softmax for this thread's row: softmax_tile of
// fa_prefill.cuh with the scores modified first.  docs: only the columns in `seen`
// are visible (made by doc_columns).
template <int D, bool BF16, int kCap, bool kBias>
__device__ __forceinline__ void score_tile(uint32_t tS, uint32_t tO, int key0,
                                           const ScoreRow& row, const ScoreParams& p, bool docs,
                                           const uint32_t (&seen)[4], bool may_rescale, float& m,
                                           float& l) {
  constexpr float kTau = 8.f;
  uint32_t sr[8][16];
#pragma unroll
  for (int cc = 0; cc < 8; cc += 2) tmem_ld32(tS + cc * 16, sr[cc], sr[cc + 1]);
  tmem_wait_ld();
#pragma unroll
  for (int cc = 0; cc < 8; ++cc) reg_fence16(sr[cc]);

  // the factor of the scores in registers: with a cap or a bias they are in
  // log2 units already
  const float c = kCap != kCapNone || kBias ? 1.f : p.scale_log2;
  if constexpr (kCap != kCapNone) cap_tile(sr, tS, p);
  if constexpr (kBias) {
    // x = s c - slope |p - j|, linear in the column away from the diagonal
    const float cs = kCap != kCapNone ? 1.f : p.scale_log2;
    const int d0 = key0 - row.pos;
    const bool left = d0 + kBN - 1 <= 0, right = d0 >= 0;
    if (__all_sync(0xffffffffu, left) || __all_sync(0xffffffffu, right)) {
      // the bias of 16 columns by steps of two from their first: seven
      // additions' rounding at most
      const float step = right ? -row.slope : row.slope, step2 = 2.f * step;
      const float base = step * static_cast<float>(d0);
#pragma unroll
      for (int cc = 0; cc < 8; ++cc) {
        float b0 = fmaf(step, static_cast<float>(cc * 16), base), b1 = b0 + step;
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          float x0, x1;
          ffma2(x0, x1, __uint_as_float(sr[cc][e]), __uint_as_float(sr[cc][e + 1]), cs, cs, b0, b1);
          sr[cc][e] = __float_as_uint(x0);
          sr[cc][e + 1] = __float_as_uint(x1);
          if (e < 14) fadd2(b0, b1, b0, b1, step2, step2);
        }
      }
    } else {
      const float f0 = static_cast<float>(d0);
#pragma unroll
      for (int cc = 0; cc < 8; ++cc)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          sr[cc][e] = __float_as_uint(fmaf(__uint_as_float(sr[cc][e]), cs,
                                           -row.slope * fabsf(f0 + static_cast<float>(cc * 16 + e))));
    }
  }

  if (docs) {
#pragma unroll
    for (int cc = 0; cc < 8; ++cc)
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (!((seen[cc >> 1] >> ((cc & 1) * 16 + e)) & 1u)) sr[cc][e] = __float_as_uint(-INFINITY);
  } else if (key0 + kBN > row.lim_warp) {
    const int lim = row.lim - 1 - key0;
#pragma unroll
    for (int cc = 0; cc < 8; ++cc)
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (cc * 16 + e > lim) sr[cc][e] = __float_as_uint(-INFINITY);
  }

  float mx[16];
#pragma unroll
  for (int g = 0; g < 16; ++g) {
    const uint32_t* v = &sr[g >> 1][(g & 1) * 8];
    float a = fmax3(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]));
    a = fmax3(a, __uint_as_float(v[3]), __uint_as_float(v[4]));
    a = fmax3(a, __uint_as_float(v[5]), __uint_as_float(v[6]));
    mx[g] = fmaxf(a, __uint_as_float(v[7]));
  }
  const float r0 = fmax3(mx[0], mx[1], mx[2]), r1 = fmax3(mx[3], mx[4], mx[5]);
  const float r2 = fmax3(mx[6], mx[7], mx[8]), r3 = fmax3(mx[9], mx[10], mx[11]);
  const float r4 = fmax3(mx[12], mx[13], mx[14]);
  const float t_max = fmaxf(fmax3(r0, r1, r2), fmax3(r3, r4, mx[15])) * c;
  // raise the reference max only past the threshold (m = -inf: always)
  const float m_new = t_max > m + kTau ? t_max : m;
  const float m_use = m_new == -INFINITY ? 0.f : m_new;
  const float alpha = m_new == m ? 1.f : ex2_approx(m - m_use);
  const float neg_m = -m_use;
  const bool rescale = may_rescale && __any_sync(0xffffffffu, alpha != 1.f);
  float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    uint32_t pk[16];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int col = h * 32 + q * 4;
      uint32_t* v = &sr[col >> 4][col & 15];
      float x0, x1, x2, x3;
      ffma2(x0, x1, __uint_as_float(v[0]), __uint_as_float(v[1]), c, c, neg_m, neg_m);
      ffma2(x2, x3, __uint_as_float(v[2]), __uint_as_float(v[3]), c, c, neg_m, neg_m);
      const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
      const float p2 = ex2_approx(x2), p3 = ex2_approx(x3);
      fadd2(l0, l1, l0, l1, p0, p1);
      fadd2(l2, l3, l2, l3, p2, p3);
      pk[2 * q] = pack2<BF16>(p0, p1);
      pk[2 * q + 1] = pack2<BF16>(p2, p3);
    }
    tmem_st16(tS + h * 16, pk);
  }
  l = l * alpha + ((l0 + l1) + (l2 + l3));
  m = m_new;
  if (rescale) {
    uint32_t v[D / 16][16];
#pragma unroll
    for (int cc = 0; cc < D / 32; ++cc) tmem_ld32(tO + cc * 32, v[2 * cc], v[2 * cc + 1]);
    tmem_wait_ld();
#pragma unroll
    for (int cc = 0; cc < D / 16; ++cc) {
      reg_fence16(v[cc]);
#pragma unroll
      for (int e = 0; e < 16; ++e)
        v[cc][e] = __float_as_uint(__uint_as_float(v[cc][e]) * alpha);
      tmem_st16(tO + cc * 16, v[cc]);
    }
  }
  tmem_wait_st();
}

// The exponentials of 32 columns without a reference: p = 2^x of the capped
// scores x, to their 16 columns of P.
template <bool BF16, bool kMasked>
__device__ __forceinline__ void fixed_columns(const uint32_t (&v)[2][16], uint32_t tP,
                                              uint32_t visible, const ScoreParams& p, float& l0,
                                              float& l1) {
  const float c0 = p.cap_poly[0], c1 = p.cap_poly[1], c2 = p.cap_poly[2], c3 = p.cap_poly[3];
  float x[32], top = 0.f;
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    const float a = __uint_as_float(v[e >> 4][e & 15]), b = __uint_as_float(v[e >> 4][(e & 15) + 1]);
    float u0, u1, y0, y1;
    fmul2(u0, u1, a, b, a, b);
    top = fmax3(top, u0, u1);
    ffma2(y0, y1, u0, u1, c3, c3, c2, c2);
    ffma2(y0, y1, y0, y1, u0, u1, c1, c1);
    ffma2(y0, y1, y0, y1, u0, u1, c0, c0);
    fmul2(x[e], x[e + 1], y0, y1, a, b);
  }
  // (each score by its form here too: 250 us at B4 H16 S4096 D128 causal, 245
  // with the exponential form for all of the 32 columns)
  if (__any_sync(0xffffffffu, !(top <= p.cap_u_max))) {
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const float s = __uint_as_float(v[e >> 4][e & 15]);
      const float far = cap_far(s, p);
      if (!(fabsf(s) <= p.cap_t_max)) x[e] = far;
    }
  }
  if constexpr (kMasked) {
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (!((visible >> e) & 1u)) x[e] = -INFINITY;
  }
  uint32_t pk[16];
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    const float p0 = ex2_approx(x[e]), p1 = ex2_approx(x[e + 1]);
    fadd2(l0, l1, l0, l1, p0, p1);
    pk[e / 2] = pack2<BF16>(p0, p1);
  }
  tmem_st16(tP, pk);
}

// One key tile of one stage's softmax under a cap that bounds every score:
// p = 2^x, so there is no maximum to find, nothing to rescale, and 32 columns at
// a time go from S to P, the next 32 loading meanwhile (P's columns 16 h ... lie
// below those still to be read).  At |x| <= 72.5 bf16 holds p as exactly as
// around 1, and the fp32 sums l (2^96 with 2^24 keys) and p v (values of 2^-50
// ... 2^30) stay normal numbers; fp16 does not hold p, and takes the running
// maximum.
template <bool BF16>
__device__ __forceinline__ void score_tile_fixed(uint32_t tS, int key0, const ScoreRow& row,
                                                 const ScoreParams& p, bool docs,
                                                 const uint32_t (&seen)[4], float& l) {
  uint32_t va[2][16], vb[2][16];
  tmem_ld32(tS, va[0], va[1]);
  float l0 = 0.f, l1 = 0.f;
  if (docs || key0 + kBN > row.lim_warp) {
    uint32_t bits[4] = {~0u, ~0u, ~0u, ~0u};
    if (docs) {
#pragma unroll
      for (int k = 0; k < 4; ++k) bits[k] = seen[k];
    } else {
      limit_columns(row.lim, key0, bits);
    }
#pragma unroll 1
    for (int h = 0; h < 4; ++h) {
      tmem_wait_ld();
      reg_fence16(va[0]);
      reg_fence16(va[1]);
      fixed_columns<BF16, true>(va, tS + 16 * h, bits[0], p, l0, l1);
      bits[0] = bits[1];
      bits[1] = bits[2];
      bits[2] = bits[3];
      if (h < 3) tmem_ld32(tS + 32 * h + 32, va[0], va[1]);
    }
  } else {
#pragma unroll 1
    for (int h = 0; h < 4; h += 2) {
      tmem_wait_ld();
      reg_fence16(va[0]);
      reg_fence16(va[1]);
      tmem_ld32(tS + 32 * h + 32, vb[0], vb[1]);
      fixed_columns<BF16, false>(va, tS + 16 * h, 0u, p, l0, l1);
      tmem_wait_ld();
      reg_fence16(vb[0]);
      reg_fence16(vb[1]);
      if (h == 0) tmem_ld32(tS + 64, va[0], va[1]);
      fixed_columns<BF16, false>(vb, tS + 16 * h + 16, 0u, p, l0, l1);
    }
  }
  l += l0 + l1;
  tmem_wait_st();
}

template <int D, bool BF16, int kCap, bool kBias, bool kDocs, bool kHalves>
__global__ void __launch_bounds__(kThreads, 1)
    fa_score_kernel(const __grid_constant__ CUtensorMap tmQ,
                    const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV,
                    const __grid_constant__ CUtensorMap tmO,
                    const ScoreParams p) {
  using L = ScoreLayout<D>;
  using Regs = ScoreRegs<kCap, kBias>;
  // Modified scores: an item's key tiles run from the last to the first, and
  // stage 0, which lacks the last ones of a causal item, joins late.  With a bias
  // the keys next to the rows have the largest scores, and what comes after them
  // raises no reference maximum; all gain from the stages' start one tile apart.
  // B4 H16 S4096 D128 causal: bias 238 us, 280 from the first tile on; cap 50: 251
  // and 257; documents of 1000: 99 and 103.  (Unmodified scores keep the order,
  // and with it the bits, of the prefill kernel.)
  constexpr bool kBack = kBias || kCap != kCapNone || kDocs;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t sQ = sbase + L::kOffQ;
  const uint32_t sKV = sbase + L::kOffKV;
  const uint32_t sOut = sbase + L::kOffOut;
  const uint32_t bars = sbase + L::kOffBars;
  float* inv_l_smem = reinterpret_cast<float*>(smem + L::kOffInvL);
  float* m_smem = reinterpret_cast<float*>(smem + L::kOffStates);  // halves only
  float* l_smem = m_smem + 2 * kBM;
  ScoreItem* item_ring = reinterpret_cast<ScoreItem*>(smem + L::kOffRing);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffTmemSlot);
  volatile uint32_t* abort_flag =
      reinterpret_cast<volatile uint32_t*>(smem + L::kOffAbort);
  auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  // ---- setup (once per CTA; every barrier's phase runs on across items) ----
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(L::Q_FULL + s), 1);
      mbar_init(bar(L::Q_EMPTY + s), 1);
      mbar_init(bar(L::S_FULL + s), 1);
      mbar_init(bar(L::PV_READY + s), 4);  // the stage's 4 softmax warps
      mbar_init(bar(L::O_READY + s), 1);
      mbar_init(bar(L::ML_FULL + s), 4);
      mbar_init(bar(L::O_FREE + s), 4);    // the 4 epilogue warps
    }
    mbar_init(bar(L::DRAIN), 1);
    for (int i = 0; i < kItemRing; ++i) {
      mbar_init(bar(L::ITEM_FULL + i), 1);
      mbar_init(bar(L::ITEM_EMPTY + i), kItemTakers);
    }
    for (int i = 0; i < L::kSlots; ++i) {
      mbar_init(bar(L::KV_FULL + i), 1);
      mbar_init(bar(L::KV_EMPTY + i), 1);
    }
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(smem_u32(tmem_slot), L::kTmemCols);
    tmem_relinquish();
  }
  if (warp == 13 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmO);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();
  grid_launch_dependents();  // the merge of split keys waits for this grid's end
  const Ctl ctl{abort_flag, p.status, p.timeout_ns};

  const int wg = warp >> 2;
  if (wg < 2) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Regs::kSoftmax));
  } else if (wg == 2) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs::kEpilogue));
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs::kControl));
  }

  if (wg < 2) {
    // =========================== softmax, stage s ===========================
    const int s = wg;
    const int rq = warp & 3;                 // lane quarter of TMEM
    const int r = rq * 32 + lane;            // row within the stage
    const uint32_t t_lane = static_cast<uint32_t>(rq * 32) << 16;
    const uint32_t tS = tmem + t_lane + static_cast<uint32_t>(s * kBN);
    const uint32_t tO = tmem + t_lane + static_cast<uint32_t>(L::kTmemO + s * D);
    uint32_t n_s = 0;  // tiles of this stage so far (S_FULL / O_READY phase)
    bool ok = true;

#pragma unroll 1
    for (uint32_t k = 0; ok; ++k) {
      const ScoreItem it =
          take_score_item<0>(item_ring, bar(L::ITEM_FULL), bar(L::ITEM_EMPTY), k, ctl, ok);
      if (!ok || !it.valid) break;
      const int nT = s == 0 ? it.nT0 : it.nT1;
      const int row_g = stage_row<kHalves>(p, it.row0, s) + r;  // row of the row head
      const bool stored = row_g < p.rows;
      ScoreRow row{};
      // this stage's j-th tile
      auto tile_of = [&](int j) {
        const int q = kHalves ? s + 2 * j : j;
        return kBack ? tile_back<kBias>(it, kHalves ? it.nT0 + it.nT1 : nT, q) : it.t0 + q;
      };
      // the id that all keys of a tile have, of the tile to come
      const int* docs_of = nullptr;
      int doc = 0;
      if constexpr (kDocs) {
        docs_of = p.tile_doc + it.b * p.n_key_tiles;
        if (nT > 0) doc = docs_of[tile_of(0)];
      }
      {
        const int h_in = p.packed ? row_g / p.Sq : 0;  // the head within its group
        const int i = row_g - h_in * p.Sq;
        row.pos = i + (p.Skv - p.Sq);
        row.lim = p.Skv;
        if (stored) {
          if (p.causal) {
            row.lim = row.pos + 1;
            if (p.prefix) row.lim = max(row.lim, p.prefix[it.b]);
            row.lim = min(max(row.lim, 0), p.Skv);
          }
          if constexpr (kBias)
            row.slope = p.slopes[it.h0 + h_in] * 1.4426950408889634f;
        }
        row.lim_warp = __reduce_min_sync(0xffffffffu, row.lim);
        if constexpr (kDocs) {
          row.doc = stored ? p.doc_q[static_cast<size_t>(it.b) * p.Sq + i] : -1;
          // rows past the last are not stored: any document is theirs
          const int lo = __reduce_min_sync(0xffffffffu, stored ? row.doc : 0x7fffffff);
          const int hi = __reduce_max_sync(0xffffffffu, stored ? row.doc : kDocMixed);
          row.doc_warp = lo == hi && lo >= 0 ? lo : kDocSeveral;
        }
      }
      // (worked out here: its parts would be more to keep in registers)
      float* const lse_at =
          p.n_splits > 1
              ? p.part_lse + (static_cast<size_t>(it.split) * p.row_heads + it.rh) * p.rows + row_g
              : p.lse + static_cast<size_t>(it.rh) * p.rows + row_g;
      // reference of the scores (log2 units)
      float m = kCap == kCapFixed ? 0.f : -INFINITY;
      float l = 0.f;        // running sum of 2^(c*s - m)

#pragma unroll 1
      for (int j = 0; j < nT; ++j, ++n_s) {
        const int key0 = tile_of(j) * kBN;
        bool docs = false;
        uint32_t seen[4] = {};
        if constexpr (kDocs) {
          docs = row.doc_warp != doc;
          if (docs) doc_columns(p, it.b, key0, row, seen);
          if (j + 1 < nT) doc = docs_of[tile_of(j + 1)];  // in flight during the tile
        }
        if (!wait_bar_warp(bar(L::S_FULL + s), n_s & 1, ctl)) { ok = false; break; }
        tc_fence_after();
        if constexpr (kCap == kCapFixed)
          score_tile_fixed<BF16>(tS, key0, row, p, docs, seen, l);
        else
          score_tile<D, BF16, kCap, kBias>(tS, tO, key0, row, p, docs, seen, j > 0, m, l);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::PV_READY + s));
      }
      if (!ok) break;

      // end of the item: LSE straight to global, 1/l to the epilogue warps
      // once the item's last PV_s has completed (then O_s is final)
      if (stored && !kHalves) {
        // l = 0: no visible key; a NaN stays one
        const float lse = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
        *lse_at = lse;
      }
      if (nT > 0) {
        if (!wait_bar_warp(bar(L::O_READY + s), (n_s - 1) & 1, ctl)) { ok = false; break; }
        if constexpr (kHalves) {
          m_smem[s * kBM + r] = m;
          l_smem[s * kBM + r] = l;
        } else {
          inv_l_smem[s * kBM + r] = l == 0.f ? 0.f : 1.f / l;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::ML_FULL + s));
      }
    }
    __syncwarp();
  } else if (wg == 2) {
    // =============================== epilogue ===============================
    // Per item and stage: O_s * (1/l), rounded to 16 bits, staged in this
    // warp's 32-row slice of shared memory and written by TMA.  The warp
    // arrives on O_FREE_s as soon as it has read O_s out of tensor memory,
    // which lets the next item's first PV_s overwrite it.
    const int rq = warp & 3;
    const int r = rq * 32 + lane;
    const uint32_t t_lane = static_cast<uint32_t>(rq * 32) << 16;
    const uint32_t stage_buf = sOut + static_cast<uint32_t>(rq * L::kOutWarpBytes);
    uint32_t n_t0 = 0, n_t1 = 0;  // tiles of stage s so far (O_READY phase)
    uint32_t n_e0 = 0, n_e1 = 0;  // ML_FULL phases
    bool ok = true;
#pragma unroll 1
    for (uint32_t k = 0; ok; ++k) {
      const ScoreItem it = take_score_item<kSleepEpilogueNs>(item_ring, bar(L::ITEM_FULL),
                                                             bar(L::ITEM_EMPTY), k, ctl, ok);
      if (!ok || !it.valid) break;
      if constexpr (kHalves) {
        // the two stages' states of the same rows: O = sum_s f_s O_s
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int nT = s == 0 ? it.nT0 : it.nT1;
          uint32_t& n_t = s == 0 ? n_t0 : n_t1;
          uint32_t& n_e = s == 0 ? n_e0 : n_e1;
          if (!ok || nT == 0) continue;
          n_t += static_cast<uint32_t>(nT);
          if (!wait_bar_warp<kSleepEpilogueNs>(bar(L::ML_FULL + s), n_e & 1, ctl)) { ok = false; continue; }
          ++n_e;
          m[s] = m_smem[s * kBM + r];
          l[s] = l_smem[s * kBM + r];
          if (!wait_bar_warp<kSleepEpilogueNs>(bar(L::O_READY + s), (n_t - 1) & 1, ctl)) { ok = false; continue; }
        }
        if (!ok) break;
        tc_fence_after();
        const float top = fmaxf(m[0], m[1]), base = top == -INFINITY ? 0.f : top;
        float f0 = ex2_approx(m[0] - base), f1 = ex2_approx(m[1] - base);
        const float sum = fmaf(l[0], f0, l[1] * f1), inv = sum == 0.f ? 0.f : 1.f / sum;
        f0 *= inv;
        f1 *= inv;
        const int row_g = it.row0 + r;
        const bool stored = row_g < p.rows;
        const size_t part = p.n_splits > 1 ? static_cast<size_t>(it.split) * p.row_heads : 0;
        const size_t at = (part + it.rh) * p.rows + static_cast<size_t>(row_g);
        if (stored)
          (p.n_splits > 1 ? p.part_lse : p.lse)[at] =
              sum == 0.f ? -INFINITY : (base + log2f(sum)) * 0.69314718055994530942f;
        const uint32_t tO = tmem + t_lane + static_cast<uint32_t>(L::kTmemO);
        if (p.n_splits == 1) {
          // the slice is free once the previous store has read it
          if (lane == 0) bulk_wait_group_read0();
          __syncwarp();
        }
#pragma unroll 1
        for (int cc = 0; cc < D / 16; ++cc) {
          float o[16] = {};
          if (it.nT0 > 0) {
            uint32_t v[16];
            tmem_ld16(tO + cc * 16, v);
            tmem_wait_ld();
            reg_fence16(v);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __uint_as_float(v[e]) * f0;
          }
          if (it.nT1 > 0) {
            uint32_t v[16];
            tmem_ld16(tO + D + cc * 16, v);
            tmem_wait_ld();
            reg_fence16(v);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = fmaf(__uint_as_float(v[e]), f1, o[e]);
          }
          if (p.n_splits > 1) {
            if (stored) {
              float4* prow = reinterpret_cast<float4*>(p.part_o + at * D) + cc * 4;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                prow[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            }
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float* x = o + 8 * h;
              const int box = cc >> 2, chunk = (cc & 3) * 2 + h;
              st_shared_v4(stage_buf + static_cast<uint32_t>(box * L::kOutBox + lane * 128 +
                                                             ((chunk ^ (lane & 7)) << 4)),
                           pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]),
                           pack2<BF16>(x[4], x[5]), pack2<BF16>(x[6], x[7]));
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (it.nT0 > 0) mbar_arrive(bar(L::O_FREE + 0));
          if (it.nT1 > 0) mbar_arrive(bar(L::O_FREE + 1));
        }
        if (p.n_splits == 1) {
          fence_proxy_async_smem();
          __syncwarp();
          const int warp_row0 = it.row0 + rq * 32;
          if (lane == 0 && warp_row0 < p.rows) {
#pragma unroll
            for (int box = 0; box < D / 64; ++box)
              tma_store_3d(&tmO, stage_buf + static_cast<uint32_t>(box * L::kOutBox), box * 64,
                           warp_row0, it.rh);
            bulk_commit_group();
          }
        }
      }
#pragma unroll
      for (int s = kHalves ? 2 : 0; s < 2; ++s) {
        if (!ok) continue;
        const int nT = s == 0 ? it.nT0 : it.nT1;
        const bool have_o = nT > 0;
        float inv_l = 0.f;
        if (have_o) {
          uint32_t& n_t = s == 0 ? n_t0 : n_t1;
          uint32_t& n_e = s == 0 ? n_e0 : n_e1;
          n_t += static_cast<uint32_t>(nT);
          if (!wait_bar_warp<kSleepEpilogueNs>(bar(L::ML_FULL + s), n_e & 1, ctl)) { ok = false; continue; }
          ++n_e;
          inv_l = inv_l_smem[s * kBM + r];
          if (!wait_bar_warp<kSleepEpilogueNs>(bar(L::O_READY + s), (n_t - 1) & 1, ctl)) { ok = false; continue; }
          tc_fence_after();
        }
        const uint32_t tO = tmem + t_lane + static_cast<uint32_t>(L::kTmemO + s * D);
        if (p.n_splits > 1) {
          // a key range: O / l of this range in fp32, one row per thread
          const int row_g = stage_row<kHalves>(p, it.row0, s) + r;
          float4* prow = reinterpret_cast<float4*>(
              p.part_o + ((static_cast<size_t>(it.split) * p.row_heads + it.rh) * p.rows +
                          static_cast<size_t>(row_g)) * D);
#pragma unroll 1
          for (int cc = 0; cc < D / 16; ++cc) {
            uint32_t v[16];
            if (have_o) {
              tmem_ld16(tO + cc * 16, v);
              tmem_wait_ld();
              reg_fence16(v);
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] = 0u;
            }
            if (row_g < p.rows) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                prow[cc * 4 + e] = make_float4(__uint_as_float(v[4 * e]) * inv_l,
                                               __uint_as_float(v[4 * e + 1]) * inv_l,
                                               __uint_as_float(v[4 * e + 2]) * inv_l,
                                               __uint_as_float(v[4 * e + 3]) * inv_l);
            }
          }
          if (have_o) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::O_FREE + s));
          }
          continue;
        }
        // the slice is free once the previous store has read it
        if (lane == 0) bulk_wait_group_read0();
        __syncwarp();
        stage_o_rows<D, BF16>(tO, have_o, inv_l, stage_buf, L::kOutBox, lane);
        if (have_o) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::O_FREE + s));
        }
        fence_proxy_async_smem();
        __syncwarp();
        const int warp_row0 = stage_row<kHalves>(p, it.row0, s) + rq * 32;
        if (lane == 0 && warp_row0 < p.rows) {
#pragma unroll
          for (int box = 0; box < D / 64; ++box)
            tma_store_3d(&tmO, stage_buf + static_cast<uint32_t>(box * L::kOutBox), box * 64,
                         warp_row0, it.rh);
          bulk_commit_group();
        }
      }
    }
    if (lane == 0) bulk_wait_group0();  // every store has landed before exit
    __syncwarp();
  } else if (warp == 12) {
    // ============================== MMA issuer ==============================
    // the whole warp runs this loop in lockstep; each MMA / commit wrapper
    // elects the issuing lane itself
    {
      constexpr uint32_t kIdescQK = idesc_f16(BF16, false, false, kBM, kBN);
      constexpr uint32_t kIdescPV = idesc_f16(BF16, false, true, kBM, D);
      const uint32_t tS0 = tmem, tS1 = tmem + kBN;
      const uint32_t tO0 = tmem + L::kTmemO, tO1 = tmem + L::kTmemO + D;
      bool issued = false;

      auto slot_of = [&](int fill) { return fill % L::kSlots; };
      auto par_of = [&](int fill) { return static_cast<uint32_t>((fill / L::kSlots) & 1); };
      // QK_s with K from fill fk: one asm block, K = D, both operands K-major
      // in smem; commits S_FULL_s, and Q_EMPTY_s after the item's last QK_s
      auto qk = [&](int s, int fk, bool last_of_stage) {
        const uint64_t da = smem_desc_sw128(
            sQ + static_cast<uint32_t>(kHalves ? 0 : s * L::kQBytes), 16, 1024);
        const uint64_t db = smem_desc_sw128(sKV + static_cast<uint32_t>(slot_of(fk) * L::kKVBytes), 16, 1024);
        if constexpr (D == 128) {
          umma_f16_ss_k128(s == 0 ? tS0 : tS1, da, db, kIdescQK, 0u);
        } else {
          umma_f16_ss_k64(s == 0 ? tS0 : tS1, da, db, kIdescQK, 0u);
        }
        umma_commit(bar(L::S_FULL + s));
        if (last_of_stage) umma_commit(bar(L::Q_EMPTY + (kHalves ? 0 : s)));
      };
      // PV_s: K = 128 keys, A = P_s from tensor memory, B = V MN-major
      auto pv = [&](int s, int fv, bool acc) {
        umma_f16_ts_k128(s == 0 ? tO0 : tO1, s == 0 ? tS0 : tS1,
                         smem_desc_sw128(sKV + static_cast<uint32_t>(slot_of(fv) * L::kKVBytes),
                                         L::kBox, 1024),
                         kIdescPV, acc ? 1u : 0u);
        umma_commit(bar(L::O_READY + s));
      };
      // Stage 0's tiles are an item's steps first0 ... end0 - 1
      auto first0 = [](const ScoreItem& it) { return kBack ? it.nT1 - it.nT0 : 0; };
      auto end0 = [](const ScoreItem& it) { return kBack ? it.nT1 : it.nT0; };
      auto begin0 = [&](const ScoreItem& it, int f) {
        if (it.nT0 == 0)
          umma_commit(bar(L::Q_EMPTY + 0));
        else if (first0(it) == 0)
          qk(0, f, it.nT0 == 1);
      };
      // First QKs of an item whose Q is in buffer phase kq and whose K_0 is
      // fill f (used for the CTA's first item and after an item without keys)
      auto begin = [&](const ScoreItem& it, int kq, int f) -> bool {
        if (!wait_bar_warp<kSleepMmaNs>(bar(L::Q_FULL + 0), kq & 1, ctl) ||
            !wait_bar_warp<kSleepMmaNs>(bar(L::Q_FULL + 1), kq & 1, ctl))
          return false;
        if (it.nT1 > 0 && !wait_bar_warp<kSleepMmaNs>(bar(L::KV_FULL + slot_of(f)), par_of(f), ctl)) return false;
        tc_fence_after();
        begin0(it, f);
        if (it.nT1 > 0) {
          qk(1, f, it.nT1 == 1);
          umma_commit(bar(L::KV_EMPTY + slot_of(f)));
        } else {
          umma_commit(bar(L::Q_EMPTY + 1));
        }
        issued = true;
        return true;
      };

      // Tensor-core order within an item: QK_0(0) QK_1(0), then per key tile
      //   PV_0(j) QK_0(j+1) PV_1(j) QK_1(j+1)
      // and at an item's last tile the next item's QK_s(0) take the place of
      // QK_s(j+1), so the tensor core moves on while this item's epilogue
      // runs; the next item's PV_s(0) also waits for O_FREE_s.
      uint32_t n_pv0 = 0, n_pv1 = 0;  // PV_s issued so far (PV_READY phase)
      uint32_t n_o0 = 0, n_o1 = 0;    // items so far with a PV_s (O_FREE phase)
      int kq = 0;                     // items begun (Q_FULL phase)
      int fK = 0;                     // fill of the current item's K_0
      bool ok = true;
      ScoreItem cur = take_score_item<kSleepMmaNs>(item_ring, bar(L::ITEM_FULL),
                                                   bar(L::ITEM_EMPTY), 0, ctl, ok);
      if (!cur.valid) ok = false;
      if constexpr (!kHalves) {
        if (ok) ok = begin(cur, 0, 0);
      } else {
        // Halves: tile q, fills f + 2 q and f + 2 q + 1, is stage q & 1's.  The
        // order is QK(0) QK(1), then per tile PV(q) QK(q + 2).  Q_0 serves both
        // stages: the item's last QK frees it.  (The next item begins after
        // this one's last PV: SMs seldom take a second one.)
        auto start = [&](const ScoreItem& it, int s, int kq, int f) -> bool {
          const int n = it.nT0 + it.nT1;
          if (s >= n) {
            if (n == 0 && s == 0) {  // no tile: Q, once here, is free again
              if (!wait_bar_warp<kSleepMmaNs>(bar(L::Q_FULL), kq & 1, ctl)) return false;
              umma_commit(bar(L::Q_EMPTY));
              issued = true;
            }
            return true;
          }
          const int fk = f + 2 * s;
          if (!wait_bar_warp<kSleepMmaNs>(bar(L::Q_FULL), kq & 1, ctl) ||
              !wait_bar_warp<kSleepMmaNs>(bar(L::KV_FULL + slot_of(fk)), par_of(fk), ctl))
            return false;
          tc_fence_after();
          qk(s, fk, s + 1 == n);
          umma_commit(bar(L::KV_EMPTY + slot_of(fk)));
          issued = true;
          return true;
        };
        if (ok) ok = start(cur, 0, 0, 0) && start(cur, 1, 0, 0);
#pragma unroll 1
        while (ok) {
          const int n = cur.nT0 + cur.nT1, fN = fK + 2 * n;
#pragma unroll 1
          for (int q = 0; q < n && ok; ++q) {
            const int s = q & 1, fv = fK + 2 * q + 1, fk2 = fK + 2 * q + 4;
            uint32_t& n_pv = s == 0 ? n_pv0 : n_pv1;
            const uint32_t n_o = s == 0 ? n_o0 : n_o1;
            if (!wait_bar_warp<kSleepMmaNs>(bar(L::KV_FULL + slot_of(fv)), par_of(fv), ctl) ||
                !wait_bar_warp<kSleepMmaNs>(bar(L::PV_READY + s), n_pv & 1, ctl) ||
                (q < 2 && n_o > 0 &&
                 !wait_bar_warp<kSleepMmaNs>(bar(L::O_FREE + s), (n_o - 1) & 1, ctl))) {
              ok = false;
              break;
            }
            ++n_pv;
            tc_fence_after();
            pv(s, fv, q >= 2);
            umma_commit(bar(L::KV_EMPTY + slot_of(fv)));
            if (q + 2 < n) {
              if (!wait_bar_warp<kSleepMmaNs>(bar(L::KV_FULL + slot_of(fk2)), par_of(fk2), ctl)) {
                ok = false;
                break;
              }
              tc_fence_after();
              qk(s, fk2, q + 3 == n);
              umma_commit(bar(L::KV_EMPTY + slot_of(fk2)));
            }
          }
          if (!ok) break;
          const ScoreItem nxt = take_score_item<kSleepMmaNs>(
              item_ring, bar(L::ITEM_FULL), bar(L::ITEM_EMPTY), kq + 1, ctl, ok);
          if (!ok || !nxt.valid) break;
          if (cur.nT0 > 0) ++n_o0;
          if (cur.nT1 > 0) ++n_o1;
          ++kq;
          cur = nxt;
          fK = fN;
          ok = start(cur, 0, kq, fK) && start(cur, 1, kq, fK);
        }
        ok = false;  // done
      }
#pragma unroll 1
      while (ok) {
        // the next item is taken at this item's last key tile, once the
        // producer has claimed it (it does so after the last K/V fill)
        bool taken = false, has_next = false;
        ScoreItem nxt{};
        auto take_next = [&]() {
          if (taken) return;
          taken = true;
          nxt = take_score_item<kSleepMmaNs>(item_ring, bar(L::ITEM_FULL), bar(L::ITEM_EMPTY),
                                             kq + 1, ctl, ok);
          has_next = ok && nxt.valid;
        };
        const int fN = fK + 2 * cur.nT1;  // the next item's K_0
        const int f0 = first0(cur), e0 = end0(cur);
#pragma unroll 1
        for (int j = 0; j < cur.nT1; ++j) {
          const bool last = j + 1 == cur.nT1;
          if (last) {
            take_next();
            if (!ok) break;
          }
          const int fv = fK + 2 * j + 1, fk1 = fK + 2 * j + 2;
          // V_j and PV_READY_0 first, probed together (usually both are
          // complete; the bounded waits only when one is not); K_(j+1) only
          // once PV_0(j) is issued, so that its wait is off the path from
          // the softmax's arrival to the next PV
          bool rdy = mbar_try_wait(bar(L::KV_FULL + slot_of(fv)), par_of(fv));
          const bool on0 = j >= f0 && j < e0;
          if (on0) rdy &= mbar_try_wait(bar(L::PV_READY + 0), n_pv0 & 1);
          if (!__all_sync(0xffffffffu, rdy)) {
            if (!wait_bar_warp<kSleepMmaNs>(bar(L::KV_FULL + slot_of(fv)), par_of(fv), ctl)) { ok = false; break; }
            if (on0 && !wait_bar_warp<kSleepMmaNs>(bar(L::PV_READY + 0), n_pv0 & 1, ctl)) { ok = false; break; }
          }
          if (on0) {  // PV_0(j), then QK_0 over P_0(j)
            if (j == f0 && n_o0 > 0 && !wait_bar_warp<kSleepMmaNs>(bar(L::O_FREE + 0), (n_o0 - 1) & 1, ctl)) {
              ok = false;
              break;
            }
            ++n_pv0;
            tc_fence_after();
            pv(0, fv, j > f0);
          }
          if (!last && !wait_bar_warp<kSleepMmaNs>(bar(L::KV_FULL + slot_of(fk1)), par_of(fk1), ctl)) {
            ok = false;
            break;
          }
          if (!last) {
            if (j + 1 >= f0 && j + 1 < e0) qk(0, fk1, j + 2 == e0);
          } else if (has_next) {
            if (!wait_bar_warp<kSleepMmaNs>(bar(L::Q_FULL + 0), (kq + 1) & 1, ctl)) { ok = false; break; }
            if (nxt.nT1 > 0 && !wait_bar_warp<kSleepMmaNs>(bar(L::KV_FULL + slot_of(fN)), par_of(fN), ctl)) {
              ok = false;
              break;
            }
            tc_fence_after();
            begin0(nxt, fN);
          }
          // PV_1(j), then QK_1 over P_1(j)
          if (!wait_bar_warp<kSleepMmaNs>(bar(L::PV_READY + 1), n_pv1 & 1, ctl)) { ok = false; break; }
          if (j == 0 && n_o1 > 0 && !wait_bar_warp<kSleepMmaNs>(bar(L::O_FREE + 1), (n_o1 - 1) & 1, ctl)) {
            ok = false;
            break;
          }
          ++n_pv1;
          tc_fence_after();
          pv(1, fv, j > 0);
          umma_commit(bar(L::KV_EMPTY + slot_of(fv)));
          if (!last) {
            qk(1, fk1, j + 2 == cur.nT1);
            umma_commit(bar(L::KV_EMPTY + slot_of(fk1)));
          } else if (has_next) {
            if (!wait_bar_warp<kSleepMmaNs>(bar(L::Q_FULL + 1), (kq + 1) & 1, ctl)) { ok = false; break; }
            tc_fence_after();
            if (nxt.nT1 > 0) {
              qk(1, fN, nxt.nT1 == 1);
              umma_commit(bar(L::KV_EMPTY + slot_of(fN)));
            } else {
              umma_commit(bar(L::Q_EMPTY + 1));
            }
          }
        }
        if (ok) take_next();  // an item without key tiles
        if (!ok || !has_next) break;
        if (cur.nT0 > 0) ++n_o0;
        if (cur.nT1 > 0) ++n_o1;
        if (cur.nT1 == 0) ok = begin(nxt, kq + 1, fN);  // no tile above began it
        ++kq;
        cur = nxt;
        fK = fN;
      }
      if (issued) {  // every MMA issued so far completes before TMEM is freed
        umma_commit(bar(L::DRAIN));
        wait_drain(bar(L::DRAIN), 0, p.timeout_ns);
      }
    }
    __syncwarp();
  } else if (warp == 13) {
    // ============================== TMA producer =============================
    // Per item: Q_0, K_0, Q_1, V_0, then K_j V_j.  The Q of the next item
    // waits for the current item's last QK on that stage, the K/V ring for
    // the tiles of the previous round of the ring.
    if (lane == 0) {
      int fill = 0;
      int last_fill[L::kSlots];
#pragma unroll
      for (int i = 0; i < L::kSlots; ++i) last_fill[i] = -1;
      int nq[2] = {0, 0};  // Q loads issued per stage
      bool ok = true;
      auto load_q = [&](const ScoreItem& it, int s) -> bool {
        if (nq[s] > 0 && !wait_bar<kSleepProducerNs>(bar(L::Q_EMPTY + s), (nq[s] - 1) & 1, ctl)) return false;
        mbar_arrive_expect_tx(bar(L::Q_FULL + s), L::kQBytes);
#pragma unroll
        for (int box = 0; box < D / 64; ++box)
          tma_load_3d(sQ + static_cast<uint32_t>(s * L::kQBytes + box * L::kBox), &tmQ,
                      bar(L::Q_FULL + s), box * 64, stage_row<kHalves>(p, it.row0, s), it.rh);
        ++nq[s];
        return true;
      };
      auto load_kv = [&](const ScoreItem& it, int kv, int j) -> bool {
        const int slot = fill % L::kSlots;
        const uint32_t par = static_cast<uint32_t>(((fill / L::kSlots) & 1) ^ 1);
        if (!wait_bar<kSleepProducerNs>(bar(L::KV_EMPTY + slot), par, ctl)) return false;
        mbar_arrive_expect_tx(bar(L::KV_FULL + slot), L::kKVBytes);
        const CUtensorMap* tm = kv == 0 ? &tmK : &tmV;
#pragma unroll
        for (int box = 0; box < D / 64; ++box)
          tma_load_3d(sKV + static_cast<uint32_t>(slot * L::kKVBytes + box * L::kBox), tm,
                      bar(L::KV_FULL + slot), box * 64,
                      (kBack ? tile_back<kBias>(it, item_tiles<kHalves>(it), j) : it.t0 + j) * kBN, it.kvh);
        last_fill[slot] = fill;
        ++fill;
        return true;
      };
      int idx = static_cast<int>(blockIdx.x);  // the grid never exceeds the items
#pragma unroll 1
      for (uint32_t k = 0; ok; ++k) {
        // publish item k (or the end) once every role has taken item k - 4
        const uint32_t slot = k % kItemRing;
        if (k >= kItemRing &&
            !wait_bar<kSleepProducerNs>(bar(L::ITEM_EMPTY + slot), (k / kItemRing - 1) & 1, ctl)) {
          ok = false;
          break;
        }
        const ScoreItem it = idx < 0 ? ScoreItem{} : get_score_item<kHalves>(p, idx);
        item_ring[slot] = it;
        mbar_arrive(bar(L::ITEM_FULL + slot));
        if (idx < 0) break;
        ok = load_q(it, 0);
#pragma unroll 1
        for (int j = 0; ok && j < item_tiles<kHalves>(it); ++j) {
          ok = load_kv(it, 0, j);
          if (ok && j == 0 && !kHalves) ok = load_q(it, 1);
          if (ok) ok = load_kv(it, 1, j);
        }
        if (ok && !kHalves && it.nT1 == 0) ok = load_q(it, 1);
        idx = claim_score_item(p);
      }
      // drain: every load issued lands before shared memory goes away
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (nq[s] > 0) wait_drain(bar(L::Q_FULL + s), (nq[s] - 1) & 1, p.timeout_ns);
#pragma unroll 1
      for (int i = 0; i < L::kSlots; ++i)
        if (last_fill[i] >= 0)
          wait_drain(bar(L::KV_FULL + i), static_cast<uint32_t>((last_fill[i] / L::kSlots) & 1),
                     p.timeout_ns);
    }
    __syncwarp();
  }

  // ---- teardown ----
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmemCols);
  }
  if (threadIdx.x == 0) {
    // the launch's last CTA clears the scheduler slot (claims are over: a
    // CTA claims only from its producer, which has finished)
    __threadfence();
    if (atomicAdd(&p.sched[1], 1ull) == gridDim.x - 1) {
      p.sched[0] = 0ull;
      p.sched[1] = 0ull;
      __threadfence();
    }
  }
}

}  // namespace fa
