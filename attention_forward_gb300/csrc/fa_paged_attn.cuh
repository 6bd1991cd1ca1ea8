// fa_paged_attn.cuh -- attention of a few query rows per kv head over a 16-bit
// paged cache, split over the keys: keys and values of a head (64 or 128
// channels), or latent rows of 576 channels whose first 512 are the value too.
// sm_103a.
//
// A kv head's query rows (its H / Hkv heads times Sq tokens; all heads of a latent
// row) share every key.  A CTA takes up to N of them over one range of keys, 64 keys
// a tile.  The keys are the tensor core's M side, so that few query rows cost few
// columns and a latent tile, once in shared memory, serves both products:
//   S^T [64 keys, N]       = K Q^T        A = K (K-major),  B = Q
//   O^T [channels, N]     += V^T P^T      A = V (MN-major: the rows as they lie),
//                                         B = P, N rows of 64 keys
// Scores, sums and O are fp32 in tensor memory; a probability is rounded to the
// type of V for its product.
//
// Warps:
//   0-3  softmax: a warp's 16 keys of the tile as mma fragments (16x256b loads),
//        one reference maximum a row, raised for the whole CTA when a score passes it
//        by 15 (log2 units; then O is rescaled in place), set 8 below the maximum so
//        that fp16 holds p over 2^-24 ... 2^15 around it; p goes to shared memory
//        transposed (stmatrix).  At a segment's end they write O.
//   4    MMA issue, the queries' load, tensor memory
//   5    TMA producer: a ring of tiles, by boxes of 8 rows (all channels): any page
//        size is a multiple of them.  A box past the sequence or of a page that does
//        not exist is fetched from past the pool's end, as zeros.
// The tensor core runs S(j + 1) while the softmax works on S(j), when the tile is
// there: warp 4 takes whichever of S(j + 1) and O(j) is ready first.
//
// Every wait is bounded by the watchdog, as in the prefill kernels.
#pragma once
#include "fa_keys.cuh"
#include "fa_merge.cuh"
#include "fa_paged.h"
#include "fa_prefill.cuh"

namespace fa {

constexpr int kPagedThreads = 192;
constexpr int kPagedKeys = kCacheAttnKeys;  // 64 keys: a tile, and a chunk of the deal

// kKC, kVC: 64-channel chunks of a key and of a value; kShared: the value is the
// key's first chunks.  kN: query rows of a CTA.
template <int kKC_, int kVC_, bool kShared_, int kN_, int kStages_, int kCtas_>
struct PagedShape {
  static constexpr int kKC = kKC_, kVC = kVC_, kN = kN_, kStages = kStages_, kCtas = kCtas_;
  static constexpr bool kShared = kShared_;
  static constexpr int kDv = 64 * kVC;
  static constexpr int kTileK = kPagedKeys * 128 * kKC;
  static constexpr int kTileV = kShared ? 0 : kPagedKeys * 128 * kVC;
  static constexpr int kStageBytes = kTileK + kTileV;
  static constexpr int kVStride = (kShared ? kKC : kVC) * 1024;  // from 8 keys to the next 8
  static constexpr int kQBytes = kN * 128 * kKC;
  static constexpr int kPBytes = kN * 128;
  static constexpr int kBlocks = kVC == 1 ? 1 : kVC / 2;  // O^T in blocks of 128 channels (64)
  static constexpr int kColO = 2 * kN;
  static constexpr int kCols = kColO + kBlocks * kN;
  static constexpr int kTmemCols =
      kCols <= 32 ? 32 : kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static constexpr int kOffP = kQBytes, kOffRing = kOffP + kPBytes;
  static constexpr int kOffMisc = kOffRing + kStages * kStageBytes;
  static_assert(kVC == 1 || kVC % 2 == 0, "values of 64 channels, or of 128 a block");
  static_assert(kOffP % 1024 == 0 && kOffRing % 1024 == 0, "128-byte swizzled tiles");
  static_assert(kCols <= 512 && kCtas * kTmemCols <= 512, "tensor memory");
};

struct PagedMiscBars {
  static constexpr int kMaxStages = 12;
  alignas(8) unsigned long long kv_full[kMaxStages], kv_empty[kMaxStages];
  unsigned long long s_full[2], p_ready, o_done, q_full, q_empty, drain;
};

template <int kN, bool kSlopes>
struct PagedMisc {
  PagedMiscBars bars;
  KeyScan<kPagedThreads / 32> scan;
  uint32_t tmem, abort;
  uint32_t bad[PagedMiscBars::kMaxStages];  // a bit for each 8 keys whose page does not exist
  float red[4][kN];
  float factor[kN];  // a rescale's, then a row's 1 / l
  union {
    int limit[kN];   // keys below it are visible
    float top[kN];   // after the tiles: reference maxima
  };
  float slope[kSlopes ? kN : 1];
};

template <class S>
constexpr int paged_smem_bytes() {
  return S::kOffMisc + static_cast<int>(sizeof(PagedMisc<S::kN, !S::kShared>)) + 1024;  // + alignment
}

// The CTA's segments: ranges of one unit's keys.
struct PagedWalk {
  int cur, first, last;  // chunks, or units where they are not split
  int b, len, before;    // the sequence, its length, the chunks of those before it
};
struct PagedSeg {
  int hk, row0, n_rows, len, k_begin, k_end, n_tiles, part;
  bool whole;
  long long out_row0;
  const int* pages;
};

template <int kN>
__device__ __forceinline__ bool paged_next(const PagedAttnParams& p, PagedWalk& w, PagedSeg& s) {
  if (w.cur >= w.last) return false;
  const int units = p.Hkv * p.n_row_blocks;
  if (p.whole) w.b = w.cur / units;
  if (p.whole || w.cur != w.first) w.len = cache_length(p, w.b);
  const int seq_chunks = cache_chunks(w.len);
  const int unit = p.whole ? w.cur - w.b * units : (w.cur - w.before) / seq_chunks;
  const int chunk0 = p.whole ? 0 : w.cur - w.before - unit * seq_chunks;
  const int n_chunks = p.whole ? seq_chunks : min(seq_chunks - chunk0, w.last - w.cur);
  s.whole = n_chunks == seq_chunks;
  s.part = 2 * static_cast<int>(blockIdx.x) + (w.cur == w.first ? 0 : 1);
  s.hk = unit / p.n_row_blocks;
  const int rb = unit - s.hk * p.n_row_blocks;
  s.row0 = rb * kN;
  s.n_rows = min(kN, p.rows - s.row0);
  s.out_row0 = (static_cast<long long>(w.b) * p.Hkv + s.hk) * p.rows + s.row0;
  s.len = w.len;
  s.k_begin = chunk0 * kPagedKeys;
  s.k_end = min(w.len, s.k_begin + n_chunks * kPagedKeys);
  s.n_tiles = (s.k_end - s.k_begin + kPagedKeys - 1) / kPagedKeys;
  s.pages = p.page_table + static_cast<long long>(w.b) * p.max_pages;
  if (p.whole) {
    w.cur += static_cast<int>(gridDim.x);
  } else {
    w.cur += n_chunks;
    if (chunk0 + n_chunks == seq_chunks && unit == units - 1) {
      w.before += seq_chunks * units;
      ++w.b;
    }
  }
  return true;
}

template <class S, bool BF16, bool kMod>
__global__ void __launch_bounds__(kPagedThreads, S::kCtas)
    fa_paged_attn_kernel(const __grid_constant__ CUtensorMap tmQ,
                         const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const PagedAttnParams p) {
  constexpr int kN = S::kN, kNB = kN / 8, kStages = S::kStages;
  constexpr float kLog2e = 1.4426950408889634f;
  constexpr float kBelow = 8.f, kTau = 15.f;
  constexpr float kNone = -3.0e38f;  // below every score that counts; -inf - kNone is -inf
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sQ = smem_u32(smem), sP = sQ + S::kOffP, sRing = sQ + S::kOffRing;
  using Misc = PagedMisc<kN, !S::kShared>;
  Misc& sm = *reinterpret_cast<Misc*>(smem + S::kOffMisc);
  const uint32_t kv_full = smem_u32(sm.bars.kv_full), kv_empty = smem_u32(sm.bars.kv_empty);
  const uint32_t s_full = smem_u32(sm.bars.s_full), p_ready = smem_u32(&sm.bars.p_ready);
  const uint32_t o_done = smem_u32(&sm.bars.o_done), q_full = smem_u32(&sm.bars.q_full);
  const uint32_t q_empty = smem_u32(&sm.bars.q_empty), drain = smem_u32(&sm.bars.drain);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(kv_full + 8 * i, 1);
      mbar_init(kv_empty + 8 * i, 1);
    }
    mbar_init(s_full, 1);
    mbar_init(s_full + 8, 1);
    mbar_init(p_ready, 4);
    mbar_init(o_done, 1);
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(drain, 1);
    sm.abort = 0u;
    fence_mbar_init();
  }
  if (warp == 4) {
    tmem_alloc(smem_u32(&sm.tmem), S::kTmemCols);
    tmem_relinquish();
  }
  if (warp == 5 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    if constexpr (!S::kShared) tma_prefetch_desc(&tmV);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  const Ctl ctl{&sm.abort, p.status, p.timeout_ns};
  grid_dependency_wait();
  grid_launch_dependents();  // this grid's CTAs have their tensor memory

  PagedWalk walk{};
  if (p.whole) {
    walk.first = static_cast<int>(blockIdx.x);
    walk.last = p.B * p.Hkv * p.n_row_blocks;
  } else {
    int upto;
    const int all = cache_scan(p, sm.scan, blockIdx.x == 0, upto);
    const CacheDeal deal = cache_deal(all, static_cast<int>(gridDim.x));
    if (static_cast<int>(blockIdx.x) < deal.n) {
      walk.first = deal.begin(static_cast<int>(blockIdx.x));
      walk.last = deal.begin(static_cast<int>(blockIdx.x) + 1);
      cache_find(p, sm.scan, upto, walk.first, walk.b, walk.len, walk.before);
    }
  }
  walk.cur = walk.first;
  PagedSeg seg;

  if (warp < 4) {
    // ================================ softmax ================================
    const int g = lane >> 2, t4 = lane & 3;
    const uint32_t t_lane = static_cast<uint32_t>(warp * 32) << 16;
    // this lane's address of a transposed store of two blocks of 8 rows: row (lane /
    // 16) * 8 + lane % 8, keys 16 warp + 8 (lane / 8 % 2)
    const uint32_t p_at = sP + static_cast<uint32_t>(((lane >> 4) * 8 + (lane & 7)) * 128 +
                                                     (((2 * warp + ((lane >> 3) & 1)) ^ (lane & 7)) << 4));
    const float fac = kMod && p.cap > 0.f ? p.scale : p.scale * kLog2e;
    uint32_t t = 0;  // tiles so far
    bool ok = true;
#pragma unroll 1
    while (ok && paged_next<kN>(p, walk, seg)) {
      if (p.whole && threadIdx.x == 0 && seg.len != p.length[walk.b])
        atomicMax(p.status, kStatusBadIndex);
      for (int n = threadIdx.x; n < kN; n += 128) {
        const int rr = min(n, seg.n_rows - 1) + seg.row0;
        const int h = rr / p.Sq, i = rr - h * p.Sq;
        sm.limit[n] = n < seg.n_rows ? seg.len - (p.Sq - 1 - i) : seg.len;
        if constexpr (kMod)
          sm.slope[n] = p.slopes ? p.slopes[seg.hk * (p.H / p.Hkv) + h] * kLog2e : 0.f;
      }
      named_bar_sync(1, 128);
      const int least = seg.len - (p.Sq - 1);
      float m[kNB][2], l[kNB][2];
#pragma unroll
      for (int n = 0; n < kNB; ++n) m[n][0] = m[n][1] = kNone, l[n][0] = l[n][1] = 0.f;

#pragma unroll 1
      for (int j = 0; j < seg.n_tiles; ++j, ++t) {
        const uint32_t stage = t % kStages, buf = t & 1u;
        const int key0 = seg.k_begin + j * kPagedKeys;
        ok = ok && wait_bar_warp(s_full + 8 * buf, (t >> 1) & 1u, ctl);
        // (long since complete: makes the producer's note of bad pages visible)
        ok = ok && wait_bar_warp(kv_full + 8 * stage, (t / kStages) & 1u, ctl);
        tc_fence_after();
        uint32_t raw[kNB][4];
        tmem_ld_frag(tmem + t_lane + buf * kN, raw);
        const uint32_t bad = sm.bad[stage];
        tmem_wait_ld();
        float s[kNB][4];
#pragma unroll
        for (int n = 0; n < kNB; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            asm volatile("" : "+r"(raw[n][e]));  // not before the wait
            s[n][e] = __uint_as_float(raw[n][e]) * fac;
          }
        const int k0 = key0 + 16 * warp + g;  // this lane's keys: k0, k0 + 8
        if constexpr (kMod) {
#pragma unroll
          for (int n = 0; n < kNB; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (p.cap > 0.f) s[n][e] = cap_score(s[n][e], p) * kLog2e;
              if (p.slopes) {
                const int row = 8 * n + 2 * t4 + (e & 1);
                s[n][e] = fmaf(-sm.slope[row],
                               static_cast<float>(abs(sm.limit[row] - 1 - k0 - 8 * (e >> 1))), s[n][e]);
              }
            }
        }
        if (key0 + kPagedKeys > least || bad != 0u) {
          const bool off[2] = {((bad >> (2 * warp)) & 1u) != 0u, ((bad >> (2 * warp + 1)) & 1u) != 0u};
#pragma unroll
          for (int n = 0; n < kNB; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (off[e >> 1] || k0 + 8 * (e >> 1) >= sm.limit[8 * n + 2 * t4 + (e & 1)])
                s[n][e] = -INFINITY;
          // slots past the sequence may hold anything: zeros where they share 8
          // rows with its last (their scores are read, whose operand they were)
          const int tail = (key0 + kPagedKeys > seg.len ? seg.len - key0 : 0) & 7;
          if (tail != 0) {
            const uint32_t rows = sRing + stage * S::kStageBytes + (S::kShared ? 0 : S::kTileK) +
                                  static_cast<uint32_t>((seg.len - key0) >> 3) * S::kVStride;
            for (int i = threadIdx.x; i < (8 - tail) * S::kVC * 8; i += 128) {
              const int r = tail + i / (S::kVC * 8), c = i % (S::kVC * 8);
              st_shared_v4(rows + static_cast<uint32_t>((c >> 3) * 1024 + r * 128 + (c & 7) * 16), 0u,
                           0u, 0u, 0u);
            }
          }
        }
        bool over = false;
#pragma unroll
        for (int n = 0; n < kNB; ++n)
          over = over || fmaxf(s[n][0], s[n][2]) > m[n][0] + kTau ||
                 fmaxf(s[n][1], s[n][3]) > m[n][1] + kTau;
        if (named_bar_or(1, 128, over || !ok)) {
          // rare: a row's reference rises, or a wait ran out somewhere
          if (named_bar_or(1, 128, !ok)) {
            ok = false;
            break;
          }
#pragma unroll
          for (int n = 0; n < kNB; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float top = fmaxf(s[n][c], s[n][c + 2]);
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
              if (g == 0) sm.red[warp][8 * n + 2 * t4 + c] = top;
            }
          named_bar_sync(1, 128);
#pragma unroll
          for (int n = 0; n < kNB; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int row = 8 * n + 2 * t4 + c;
              const float top = fmaxf(fmaxf(sm.red[0][row], sm.red[1][row]),
                                      fmaxf(sm.red[2][row], sm.red[3][row]));
              float a = 1.f;
              if (top > m[n][c] + kTau) {
                a = ex2_approx(m[n][c] - (top - kBelow));
                m[n][c] = top - kBelow;
                l[n][c] *= a;
              }
              if (warp == 0 && g == 0) sm.factor[row] = a;
            }
          named_bar_sync(1, 128);
          if (j > 0) {
            ok = wait_bar_warp(o_done, (t - 1) & 1u, ctl);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < S::kBlocks * kN; c += 16) {
              uint32_t v[16];
              tmem_ld16(tmem + t_lane + S::kColO + c, v);
              tmem_wait_ld();
              reg_fence16(v);
#pragma unroll
              for (int e = 0; e < 16; ++e)
                v[e] = __float_as_uint(__uint_as_float(v[e]) * sm.factor[(c + e) % kN]);
              tmem_st16(tmem + t_lane + S::kColO + c, v);
            }
            tmem_wait_st();
          }
        }
        uint32_t pk[kNB][2];
#pragma unroll
        for (int n = 0; n < kNB; ++n) {
          float e[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            e[k] = ex2_approx(s[n][k] - m[n][k & 1]);
            l[n][k & 1] += e[k];
          }
          pk[n][0] = pack2<BF16>(e[0], e[1]);
          pk[n][1] = pack2<BF16>(e[2], e[3]);
        }
        // the product before has read its P (a segment's first: its end waited)
        if (j > 0) ok = ok && wait_bar_warp(o_done, (t - 1) & 1u, ctl);
#pragma unroll
        for (int n = 0; n < kNB; n += 2)
          stmatrix_trans4(p_at + n * 1024, pk[n][0], pk[n][1], pk[n + 1][0], pk[n + 1][1]);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_ready);
      }

      // ---- the segment's end: sums over the keys, then O^T out ----
      ok = !named_bar_or(1, 128, !ok);
      if (!ok) break;
#pragma unroll
      for (int n = 0; n < kNB; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float sum = l[n][c];
          sum += __shfl_xor_sync(0xffffffffu, sum, 4);
          sum += __shfl_xor_sync(0xffffffffu, sum, 8);
          sum += __shfl_xor_sync(0xffffffffu, sum, 16);
          if (g == 0) {
            sm.red[warp][8 * n + 2 * t4 + c] = sum;
            if (warp == 0) sm.top[8 * n + 2 * t4 + c] = m[n][c];
          }
        }
      named_bar_sync(1, 128);
      for (int n = threadIdx.x; n < kN; n += 128) {
        const float sum = (sm.red[0][n] + sm.red[1][n]) + (sm.red[2][n] + sm.red[3][n]);
        sm.factor[n] = sum == 0.f ? 0.f : 1.f / sum;  // no visible key: 0; a NaN stays one
        if (n < seg.n_rows) {
          const float lse = sum == 0.f ? -INFINITY : (sm.top[n] + log2f(sum)) * 0.69314718055994530942f;
          if (seg.whole)
            p.lse[seg.out_row0 + n] = lse;
          else
            p.part_lse[static_cast<long long>(seg.part) * kN + n] = lse;
        }
      }
      named_bar_sync(1, 128);
      if (seg.n_tiles > 0) {
        ok = wait_bar_warp(o_done, (t - 1) & 1u, ctl);
        tc_fence_after();
      }
      // a lane's channel of each block; with 64 channels a warp has 16
      const int ch = S::kVC == 1 ? 16 * warp + lane : 32 * warp + lane;
#pragma unroll 1
      for (int blk = 0; blk < S::kBlocks; ++blk)
#pragma unroll 1
        for (int c = 0; c < kN; c += 16) {
          uint32_t v[16];
          if (seg.n_tiles > 0) {
            tmem_ld16(tmem + t_lane + S::kColO + blk * kN + c, v);
            tmem_wait_ld();
            reg_fence16(v);
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = 0u;
          }
          if (ok && (S::kVC > 1 || lane < 16)) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float x = sm.factor[c + e] == 0.f ? 0.f : __uint_as_float(v[e]) * sm.factor[c + e];
              if (c + e < seg.n_rows) {
                if (seg.whole) {
                  const uint32_t w = pack2<BF16>(x, x);
                  reinterpret_cast<uint16_t*>(p.o)[(seg.out_row0 + c + e) * S::kDv + blk * 128 + ch] =
                      static_cast<uint16_t>(w);
                } else {
                  p.part_o[(static_cast<long long>(seg.part) * kN + c + e) * S::kDv + blk * 128 + ch] = x;
                }
              }
            }
          }
        }
      tc_fence_before();
      ok = !named_bar_or(1, 128, !ok);
    }
  } else if (warp == 4) {
    // =============================== MMA issue ===============================
    constexpr uint32_t kIdescS = idesc_f16(BF16, false, false, 64, kN);
    constexpr uint32_t kIdescO = idesc_f16(BF16, true, false, S::kVC == 1 ? 64 : 128, kN);
    uint32_t t0 = 0, nq = 0;  // tiles, and segments with tiles, before this one
    bool ok = true, issued = false;
#pragma unroll 1
    while (ok && paged_next<kN>(p, walk, seg)) {
      const uint32_t n = static_cast<uint32_t>(seg.n_tiles);
      if (n == 0) continue;
      // the queries, once the scores of the segment before are done
      if (nq > 0 && !wait_bar_warp<kSleepMmaNs>(q_empty, (nq - 1) & 1u, ctl)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(q_full, S::kQBytes);
        tma_load_3d(sQ, &tmQ, q_full, 0, static_cast<int>(seg.out_row0), 0);
      }
      __syncwarp();
      issued = true;
      const bool q_ok = wait_bar_warp<kSleepMmaNs>(q_full, nq & 1u, ctl);
      ++nq;
      if (!q_ok) break;
      uint32_t s = 0, o = 0;  // products issued in this segment
      uint64_t since = 0;
      uint32_t polls = 0;
#pragma unroll 1
      while (o < n) {
        if (o < s && __all_sync(0xffffffffu, mbar_test_wait(p_ready, (t0 + o) & 1u))) {
          tc_fence_after();
          const uint32_t stage = (t0 + o) % kStages;
          const uint64_t a = smem_desc_sw128(
              sRing + stage * S::kStageBytes + (S::kShared ? 0 : S::kTileK), 1024, S::kVStride);
          const uint64_t b = smem_desc_sw128(sP, 16, 1024);
#pragma unroll
          for (int blk = 0; blk < S::kBlocks; ++blk)
#pragma unroll
            for (int k = 0; k < kPagedKeys / 16; ++k)
              umma_f16_ss(tmem + S::kColO + blk * kN, a + blk * (2048 >> 4) + k * (2 * S::kVStride >> 4),
                          b + 2 * k, kIdescO, (o > 0 || k > 0) ? 1u : 0u);
          umma_commit(kv_empty + 8 * stage);
          umma_commit(o_done);
          ++o;
          since = 0;
          continue;
        }
        const uint32_t ts = t0 + s;
        if (s < n && s < o + 2 &&
            __all_sync(0xffffffffu, mbar_test_wait(kv_full + 8 * (ts % kStages), (ts / kStages) & 1u))) {
          tc_fence_after();
          const uint64_t a = smem_desc_sw128(sRing + (ts % kStages) * S::kStageBytes, 16, S::kKC * 1024);
          const uint64_t b = smem_desc_sw128(sQ, 16, 1024);
#pragma unroll
          for (int c = 0; c < S::kKC; ++c)
            umma_f16_ss_k64(tmem + (ts & 1u) * kN, a + c * (1024 >> 4), b + c * (kN * 128 >> 4), kIdescS,
                            c > 0 ? 1u : 0u);
          umma_commit(s_full + 8 * (ts & 1u));
          if (s + 1 == n) umma_commit(q_empty);
          ++s;
          since = 0;
          continue;
        }
        if ((++polls & 31u) == 0) {
          const uint64_t now = globaltimer_ns();
          bool stop = *ctl.abort != 0u;
          if (since == 0) {
            since = now;
          } else if (now - since > p.timeout_ns) {
            *ctl.abort = 1u;
            atomicExch(p.status, kStatusTimeout);
            stop = true;
          }
          if (__any_sync(0xffffffffu, stop)) {
            ok = false;
            break;
          }
        }
        __nanosleep(kSleepMmaNs);
      }
      t0 += n;
    }
    if (nq > 0) wait_drain(q_full, (nq - 1) & 1u, p.timeout_ns);
    if (issued) {  // every MMA issued completes before tensor memory is freed
      umma_commit(drain);
      wait_drain(drain, 0, p.timeout_ns);
    }
    __syncwarp();
  } else {
    // =============================== producer ================================
    uint32_t t = 0;
    bool ok = true;
#pragma unroll 1
    while (ok && paged_next<kN>(p, walk, seg)) {
      // four tiles' places at a time, a lane for each 8 keys, the next four's fetched
      // ahead
      const int page_keys = 1 << p.page_shift;
      auto page_of = [&](int key) { return key < seg.k_end ? seg.pages[key >> p.page_shift] : 0; };
      int ahead = page_of(seg.k_begin + 8 * lane);
#pragma unroll 1
      for (int j0 = 0; ok && j0 < seg.n_tiles; j0 += 4) {
        const int key = seg.k_begin + j0 * kPagedKeys + 8 * lane;
        const int page = ahead;
        ahead = page_of(key + 4 * kPagedKeys);
        const bool here = key < seg.k_end;
        const bool is_bad = here && (page < 0 || page >= p.num_pages);
        if (is_bad) atomicMax(p.status, kStatusBadIndex);
        const uint32_t bad = __ballot_sync(0xffffffffu, is_bad);
        const int row = here && !is_bad
                            ? ((page * p.Hkv + seg.hk) << p.page_shift) + (key & (page_keys - 1))
                            : p.pool_rows;
#pragma unroll 1
        for (int k = 0; k < 4 && j0 + k < seg.n_tiles; ++k, ++t) {
          const uint32_t stage = t % kStages, full = kv_full + 8 * stage;
          if (!wait_bar_warp<kSleepProducerNs>(kv_empty + 8 * stage, ((t / kStages) & 1u) ^ 1u, ctl)) {
            ok = false;
            break;
          }
          if (lane == 0) {
            sm.bad[stage] = (bad >> (8 * k)) & 0xffu;
            mbar_arrive_expect_tx(full, S::kStageBytes);
          }
          __syncwarp();
          if ((lane >> 3) == k) {
            const uint32_t dst = sRing + stage * S::kStageBytes;
            tma_load_3d(dst + (lane & 7) * (S::kKC * 1024), &tmK, full, 0, row, 0);
            if constexpr (!S::kShared)
              tma_load_3d(dst + S::kTileK + (lane & 7) * (S::kVC * 1024), &tmV, full, 0, row, 0);
          }
          __syncwarp();
        }
      }
    }
    // every load issued lands before shared memory goes away
    for (uint32_t i = t > kStages ? t - kStages : 0u; i < t; ++i)
      wait_drain(kv_full + 8 * (i % kStages), (i / kStages) & 1u, p.timeout_ns);
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmemCols);
  }
}

// The units that several CTAs shared, as the 4-bit cache's merge: a slice of 128
// channels (64) of a row by the four warps of a block (few units of many parts), or
// by one warp, the rows of a unit eight to a block (many units of few parts).
constexpr int kPagedMergeRows = 8;

template <class S, bool BF16, bool kByUnit>
__global__ void __launch_bounds__(32 * kMergeWarps)
    fa_paged_merge_kernel(const PagedAttnParams p, int attn_grid) {
  constexpr int kN = S::kN, kSlice = S::kVC == 1 ? 64 : 128, kSlices = S::kDv / kSlice;
  __shared__ KeyScan<kMergeWarps> scan;
  const int slice = static_cast<int>(blockIdx.y);
  int b, hk, rb, r;  // r: the block's first row within the kv head's
  if constexpr (kByUnit) {
    const int units = p.Hkv * p.n_row_blocks;
    const int groups = (min(kN, p.rows) + kPagedMergeRows - 1) / kPagedMergeRows;
    const int all = static_cast<int>(blockIdx.x) / groups;
    b = all / units;
    const int unit = all - b * units;
    hk = unit / p.n_row_blocks;
    rb = unit - hk * p.n_row_blocks;
    r = rb * kN + (static_cast<int>(blockIdx.x) - all * groups) * kPagedMergeRows;
  } else {
    const int bh = static_cast<int>(blockIdx.x) / p.rows;
    r = static_cast<int>(blockIdx.x) - bh * p.rows;
    b = bh / p.Hkv;
    hk = bh - b * p.Hkv;
    rb = r / kN;
  }
  int upto;
  const int all = cache_scan(p, scan, false, upto);
  const CacheDeal deal = cache_deal(all, attn_grid);
  // chunks per unit of the sequences before b: the thread with b in its run
  const int run = (p.B + 32 * kMergeWarps - 1) / (32 * kMergeWarps);
  if (b / run == static_cast<int>(threadIdx.x)) {
    for (int k = static_cast<int>(threadIdx.x) * run; k < b; ++k)
      upto += cache_chunks(cache_length(p, k));
    scan.before = upto;
  }
  __syncthreads();
  const int chunks = cache_chunks(cache_length(p, b));
  const int start = scan.before * (p.Hkv * p.n_row_blocks) + (hk * p.n_row_blocks + rb) * chunks;
  const int x0 = deal.cta_of(start), x1 = deal.cta_of(start + chunks - 1);
  grid_dependency_wait();  // all blocks: this grid's end is then the attention's too
  if (x0 == x1) return;
  // a CTA's first segment, except where the unit begins inside x0
  const int inside = deal.begin(x0) < start ? 1 : 0;
  const long long row0 = (static_cast<long long>(b) * p.Hkv + hk) * p.rows;
  const float* part_o = p.part_o + slice * kSlice;
  void* o = static_cast<uint16_t*>(p.o) + slice * kSlice;
  float* lse = slice == 0 ? p.lse : nullptr;
  const int n_parts = x1 - x0 + 1;
  if constexpr (kByUnit) {
    const int end = min(min(p.rows, (rb + 1) * kN), r + kPagedMergeRows);
    for (int row = r + (static_cast<int>(threadIdx.x) >> 5); row < end; row += kMergeWarps)
      merge_row_warp<kSlice, BF16, S::kDv>(
          part_o, p.part_lse, n_parts,
          [&](int s) -> long long {
            return (2ll * (x0 + s) + (s == 0 ? inside : 0)) * kN + row - rb * kN;
          },
          o, lse, row0 + row);
  } else {
    __shared__ MergeSmem<kSlice> sm;
    merge_row<kSlice, BF16, S::kDv>(
        part_o, p.part_lse, n_parts,
        [&](int s) -> long long { return (2ll * (x0 + s) + (s == 0 ? inside : 0)) * kN + r - rb * kN; },
        o, lse, row0 + r, sm);
  }
  static_assert(kSlices * kSlice == S::kDv, "slices");
}

}  // namespace fa
