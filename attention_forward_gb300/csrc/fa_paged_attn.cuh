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
//   4 softmax, a group, or 8, two groups with half of 64 rows each (one group: 64 latent
//        heads over 1024 keys 13.7 us, two 12.2): a warp's 16 keys of the tile as mma
//        fragments (16x256b loads), one reference maximum a row, raised for the whole
//        group when a score passes it by 15 (log2 units; then O is rescaled in place),
//        set 8 below the maximum so that fp16 holds p over 2^-24 ... 2^15 around it; p
//        goes to shared memory transposed (stmatrix).  They also send for a segment's
//        queries (TMA: by the warps themselves 128 rows of 576 channels took 9 us) and
//        write its O.
//   1 MMA issue, tensor memory
//   1 or 2 TMA producers, of K and of V (one for latent rows): rings of tiles, by boxes
//        of 8 rows (all channels): any page size is a multiple of them.  A box past the
//        sequence or of a page that does not exist is fetched from past the pool's end,
//        as zeros.
// The tensor core runs S(j + 1) while the softmax works on S(j), when the tile is
// there: the issuing warp takes whichever of S(j + 1) and O(j) is ready first.
//
// Bound, and measured (in a CUDA graph, merge included): 32 sequences of 8192 keys, 8 kv
// heads of 128 channels, by HBM: 139 us, 6.4 TB/s; latent rows, 64 sequences of 4096 and
// 16 heads, by HBM between 13 us of start, end and merge: 54.5 us; 32 of up to
// 8192 and 128 heads 96 us: a tile of 64 keys takes 2700 cycles where its products take 2040,
// for two tiles and the queries fill shared memory, and a tile is reloaded only behind its
// product.
//
// More than 64 rows of latent attention are dealt to pairs of CTAs, neighbours in the grid,
// which go through the same keys at about the same time, each for 64 rows and each with
// loads of its own: the second to ask finds a tile in L2.  Nothing makes them wait for one
// another (started as a cluster of two they are no faster).
//
// Every wait is bounded by the watchdog, as in the prefill kernels.
#pragma once
#include "fa_keys.cuh"
#include "fa_paged.h"
#include "fa_prefill.cuh"

namespace fa {

constexpr int kPagedKeys = kCacheAttnKeys;  // 64 keys: a tile, and a chunk of the deal

// kKC, kVC: 64-channel chunks of a key and of a value; kShared: the value is the
// key's first chunks.  kN: query rows of a CTA.
// kPeers: CTAs, next to each other in the grid, that take the same keys, each for a block of
// query rows (latent rows only).
template <int kKC_, int kVC_, bool kShared_, int kN_, int kStages_, int kCtas_, int kPs_ = 2,
          int kPeers_ = 1>
struct PagedShape {
  static constexpr int kKC = kKC_, kVC = kVC_, kN = kN_, kStages = kStages_, kCtas = kCtas_;
  static constexpr int kPs = kPs_;  // buffers for P
  static constexpr int kPeers = kPeers_;
  static constexpr bool kShared = kShared_;
  // groups of four softmax warps, each with its share of the query rows
  static constexpr int kGroups = kN == 64 ? 2 : 1, kRows = kN / kGroups;
  static constexpr int kMmaWarp = 4 * kGroups;
  static constexpr int kWarps = kMmaWarp + (kShared ? 2 : 3), kThreads = 32 * kWarps;
  static constexpr int kDv = 64 * kVC;
  static constexpr int kTileK = kPagedKeys * 128 * kKC;
  static constexpr int kTileV = kShared ? 0 : kPagedKeys * 128 * kVC;
  static constexpr int kStageBytes = kTileK + kTileV;
  static constexpr int kVTile = kShared ? kTileK : kTileV;       // from a tile's V to the next
  static constexpr int kVStride = (kShared ? kKC : kVC) * 1024;  // from 8 keys to the next 8
  static constexpr int kSegment = paged_segment(kPeers);
  static constexpr int kQBytes = kN * 128 * kKC;
  static constexpr int kPBytes = kN * 128;
  static constexpr int kBlocks = kVC == 1 ? 1 : kVC / 2;  // O^T in blocks of 128 channels (64)
  static constexpr int kColO = 2 * kN;
  static constexpr int kCols = kColO + kBlocks * kN;
  static constexpr int kTmemCols =
      kCols <= 32 ? 32 : kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static constexpr int kOffP = kQBytes, kOffRing = kOffP + kPs * kPBytes;
  static constexpr int kOffMisc = kOffRing + kStages * kStageBytes;
  static_assert(kPeers == 1 || (kPeers == 2 && kShared), "pairs over latent rows");
  static_assert(kVC == 1 || kVC % 2 == 0, "values of 64 channels, or of 128 a block");
  static_assert(kOffP % 1024 == 0 && kOffRing % 1024 == 0, "128-byte swizzled tiles");
  static_assert(kCols <= 512 && kCtas * kTmemCols <= 512, "tensor memory");
};

// K and V have rings of their own.  A latent stage is given back 16 keys at a time:
// k_empty[4 stage + 16-key block].
struct PagedMiscBars {
  static constexpr int kMaxStages = 8;
  alignas(8) unsigned long long k_full[kMaxStages], k_empty[kMaxStages];
  unsigned long long v_full[kMaxStages], v_empty[kMaxStages];
  unsigned long long s_full[2], p_ready[2], o_done[2], q_full, drain;
};

constexpr int kPagedBad = 16;
static_assert(kPagedBad >= PagedMiscBars::kMaxStages + 3, "notes of the tiles in flight");

template <int kN, int kWarps, bool kSlopes>
struct PagedMisc {
  PagedMiscBars bars;
  KeyScan<kWarps> scan;
  uint32_t tmem, abort;
  // of a tile, a bit for each 8 keys whose page does not exist: written before its keys
  // are sent for, read after their scores, at most a ring and three tiles later
  volatile uint32_t bad[kPagedBad];
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
  return S::kOffMisc + static_cast<int>(sizeof(PagedMisc<S::kN, S::kWarps, !S::kShared>)) + 1024;  // + alignment
}

// The row of place i of a channel's in the parts.  A lane of the attention holds rows
// 2 t4, 2 t4 + 1 of every 8: those of 32 rows (of 16) lie next to each other, so that
// four lanes write a line (half) with one store each.  Parts of 4 or 8 rows: in order.
template <int kN>
__device__ __forceinline__ int paged_part_row(int i, int part_rows) {
  if constexpr (kN >= 32)
    return (i & ~31) + ((i >> 1) & 3) * 8 + ((i >> 3) & 3) * 2 + (i & 1);
  else
    return part_rows < 16 ? i : ((i >> 1) & 1) * 8 + (i >> 2) * 2 + (i & 1);
}

// The CTA's segments: ranges of one unit's keys.
struct PagedWalk {
  int cta, ctas, rank;   // of the deal: a CTA, or a pair; the CTA's rank in it
  int cur, first, last;  // chunks, or units where they are not split
  int b, len, before;    // the sequence, its length, the chunks of those before it
};
struct PagedSeg {
  int seq, hk, row0, n_rows, len, k_begin, k_end, n_tiles, part;
  bool whole;
  long long out_row0;
  const int* pages;
};

template <class S>
__device__ __forceinline__ bool paged_next(const PagedAttnParams& p, PagedWalk& w, PagedSeg& s) {
  constexpr int kN = S::kN, kPeers = S::kPeers;
  const int units = p.Hkv * p.n_row_blocks;
  int seq_chunks, unit, chunk0;
  while (true) {
    if (w.cur >= w.last) return false;
    if (p.whole) w.b = w.cur / units;
    if (p.whole || w.cur != w.first) w.len = cache_length(p, w.b);
    seq_chunks = cache_chunks(w.len);
    if (p.whole) {
      unit = w.cur - w.b * units;
      chunk0 = 0;
      break;
    }
    const int dealt = seq_chunks + S::kSegment;
    unit = (w.cur - w.before) / dealt;
    chunk0 = w.cur - w.before - unit * dealt;
    if (chunk0 < seq_chunks) break;
    // nothing but what stands for the unit's end
    w.cur += dealt - chunk0;
    if (unit == units - 1) {
      w.before += dealt * units;
      ++w.b;
    }
  }
  const int n_chunks = p.whole ? seq_chunks : min(seq_chunks - chunk0, w.last - w.cur);
  s.whole = n_chunks == seq_chunks;
  s.part = (2 * w.cta + (w.cur == w.first ? 0 : 1)) * kPeers + w.rank;
  s.hk = unit / p.n_row_blocks;
  s.row0 = ((unit - s.hk * p.n_row_blocks) * kPeers + w.rank) * kN;
  s.n_rows = max(0, min(kN, p.rows - s.row0));  // a pair's last may have none
  s.out_row0 = (static_cast<long long>(w.b) * p.Hkv + s.hk) * p.rows + s.row0;
  s.seq = w.b;
  s.len = w.len;
  s.k_begin = chunk0 * kPagedKeys;
  s.k_end = min(w.len, s.k_begin + n_chunks * kPagedKeys);
  s.n_tiles = (s.k_end - s.k_begin + kPagedKeys - 1) / kPagedKeys;
  s.pages = p.page_table + static_cast<long long>(w.b) * p.max_pages;
  if (p.whole) {
    w.cur += w.ctas;
  } else if (chunk0 + n_chunks < seq_chunks) {
    w.cur += n_chunks;
  } else {
    w.cur += n_chunks + S::kSegment;
    if (unit == units - 1) {
      w.before += (seq_chunks + S::kSegment) * units;
      ++w.b;
    }
  }
  return true;
}

template <class S, bool BF16, bool kMod>
__global__ void __launch_bounds__(S::kThreads, S::kCtas)
    fa_paged_attn_kernel(const __grid_constant__ CUtensorMap tmQ,
                         const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const PagedAttnParams p) {
  constexpr int kN = S::kN, kRows = S::kRows, kNB = kRows / 8, kStages = S::kStages;
  constexpr float kLog2e = 1.4426950408889634f;
  constexpr float kBelow = 8.f, kTau = 15.f;
  constexpr float kNone = -3.0e38f;  // below every score that counts; -inf - kNone is -inf
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sQ = smem_u32(smem), sP = sQ + S::kOffP, sK = sQ + S::kOffRing;
  const uint32_t sV = S::kShared ? sK : sK + kStages * S::kTileK;  // V's ring
  using Misc = PagedMisc<kN, S::kWarps, !S::kShared>;
  Misc& sm = *reinterpret_cast<Misc*>(smem + S::kOffMisc);
  const uint32_t k_full = smem_u32(sm.bars.k_full), k_empty = smem_u32(sm.bars.k_empty);
  const uint32_t v_full = smem_u32(sm.bars.v_full), v_empty = smem_u32(sm.bars.v_empty);
  const uint32_t s_full = smem_u32(sm.bars.s_full), p_ready = smem_u32(sm.bars.p_ready);
  const uint32_t o_done = smem_u32(sm.bars.o_done), q_full = smem_u32(&sm.bars.q_full);
  const uint32_t drain = smem_u32(&sm.bars.drain);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < PagedMiscBars::kMaxStages; ++i) {
      mbar_init(k_full + 8 * i, 1);
      mbar_init(k_empty + 8 * i, 1);
      mbar_init(v_full + 8 * i, 1);
      mbar_init(v_empty + 8 * i, 1);
    }
    mbar_init(s_full, 1);
    mbar_init(s_full + 8, 1);
    mbar_init(p_ready, 4 * S::kGroups);
    mbar_init(p_ready + 8, 4 * S::kGroups);
    mbar_init(o_done, 1);
    mbar_init(o_done + 8, 1);
    mbar_init(q_full, 1);
    mbar_init(drain, 1);
    sm.abort = 0u;
    fence_mbar_init();
  }
  if (warp == S::kMmaWarp) {
    tmem_alloc(smem_u32(&sm.tmem), S::kTmemCols);
    tmem_relinquish();
  }
  if (warp == S::kMmaWarp + 1 && lane == 0) {
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
  walk.cta = static_cast<int>(blockIdx.x) / S::kPeers;
  walk.ctas = static_cast<int>(gridDim.x) / S::kPeers;
  walk.rank = static_cast<int>(blockIdx.x) % S::kPeers;
  if (p.whole) {
    walk.first = walk.cta;
    walk.last = p.B * p.Hkv * p.n_row_blocks;
  } else {
    int upto;
    const int all = cache_scan(p, sm.scan, blockIdx.x == 0, upto, S::kSegment);
    const CacheDeal deal = cache_deal(all, walk.ctas, kPagedMinChunks);
    if (walk.cta < deal.n) {
      walk.first = deal.begin(walk.cta);
      walk.last = deal.begin(walk.cta + 1);
      cache_find(p, sm.scan, upto, walk.first, walk.b, walk.len, walk.before,
                 S::kSegment);
    }
  }
  walk.cur = walk.first;
  PagedSeg seg;

  if (warp < S::kMmaWarp) {
    // ================================ softmax ================================
    // rows row0 ... row0 + kRows of the CTA's are this group's; they meet at its barrier
    const int g = lane >> 2, t4 = lane & 3;
    const int wq = warp & 3, tid = static_cast<int>(threadIdx.x) & 127, row0 = (warp >> 2) * kRows;
    const uint32_t group_bar = 1u + static_cast<uint32_t>(warp >> 2);
    const uint32_t t_lane = static_cast<uint32_t>(wq * 32) << 16;
    // this lane's address of a transposed store of two blocks of 8 rows: row (lane /
    // 16) * 8 + lane % 8, keys 16 wq + 8 (lane / 8 % 2)
    const uint32_t p_at = sP + static_cast<uint32_t>((row0 + (lane >> 4) * 8 + (lane & 7)) * 128 +
                                                     (((2 * wq + ((lane >> 3) & 1)) ^ (lane & 7)) << 4));
    const float fac = kMod && p.cap > 0.f ? p.scale : p.scale * kLog2e;
    uint32_t t = 0, nq = 0;  // tiles, and loads of queries, so far
    bool ok = true;
    // a segment's queries (the rows behind them, where it has fewer than kN, are nobody's);
    // the scores of the segment before are all there
    auto load_q = [&](const PagedSeg& s) {
      if (s.n_tiles == 0) return;
      ++nq;
      if (threadIdx.x == 0) {
        mbar_arrive_expect_tx(q_full, S::kQBytes);
        tma_load_3d(sQ, &tmQ, q_full, 0, static_cast<int>(s.out_row0), 0);
      }
      __syncwarp();
    };
    PagedSeg next;
    bool more = paged_next<S>(p, walk, seg);
    if (more) load_q(seg);
#pragma unroll 1
    while (more) {
      if (p.whole && threadIdx.x == 0 && seg.len != p.length[seg.seq])
        atomicMax(p.status, kStatusBadIndex);
      for (int n = row0 + tid; n < row0 + kRows; n += 128) {
        const int rr = min(min(n, seg.n_rows - 1) + seg.row0, p.rows - 1);
        const int h = rr / p.Sq, i = rr - h * p.Sq;
        sm.limit[n] = n < seg.n_rows ? seg.len - (p.Sq - 1 - i) : seg.len;
        if constexpr (kMod)
          sm.slope[n] = p.slopes ? p.slopes[seg.hk * (p.H / p.Hkv) + h] * kLog2e : 0.f;
      }
      named_bar_sync(group_bar, 128);
      const int least = seg.len - (p.Sq - 1);
      float m[kNB][2], l[kNB][2];
#pragma unroll
      for (int n = 0; n < kNB; ++n) m[n][0] = m[n][1] = kNone, l[n][0] = l[n][1] = 0.f;

#pragma unroll 1
      for (int j = 0; j < seg.n_tiles; ++j, ++t) {
        const uint32_t stage = t % kStages, buf = t & 1u;
        const int key0 = seg.k_begin + j * kPagedKeys;
        ok = ok && wait_bar_warp(s_full + 8 * buf, (t >> 1) & 1u, ctl);
        tc_fence_after();
        uint32_t raw[kNB][4];
        tmem_ld_frag(tmem + t_lane + buf * kN + row0, raw);
        const uint32_t bad = sm.bad[t % kPagedBad];
        tmem_wait_ld();
        float s[kNB][4];
#pragma unroll
        for (int n = 0; n < kNB; ++n)
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            asm volatile("" : "+r"(raw[n][e]), "+r"(raw[n][e + 1]));  // not before the wait
            ffma2(s[n][e], s[n][e + 1], __uint_as_float(raw[n][e]), __uint_as_float(raw[n][e + 1]), fac,
                  fac, 0.f, 0.f);
          }
        const int k0 = key0 + 16 * wq + g;  // this lane's keys: k0, k0 + 8
        if constexpr (kMod) {
#pragma unroll
          for (int n = 0; n < kNB; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (p.cap > 0.f) s[n][e] = cap_score(s[n][e], p) * kLog2e;
              if (p.slopes) {
                const int row = row0 + 8 * n + 2 * t4 + (e & 1);
                s[n][e] = fmaf(-sm.slope[row],
                               static_cast<float>(abs(sm.limit[row] - 1 - k0 - 8 * (e >> 1))), s[n][e]);
              }
            }
        }
        if (key0 + kPagedKeys > least || bad != 0u) {
          const bool off[2] = {((bad >> (2 * wq)) & 1u) != 0u, ((bad >> (2 * wq + 1)) & 1u) != 0u};
#pragma unroll
          for (int n = 0; n < kNB; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (off[e >> 1] || k0 + 8 * (e >> 1) >= sm.limit[row0 + 8 * n + 2 * t4 + (e & 1)])
                s[n][e] = -INFINITY;
          // slots past the sequence may hold anything: zeros where they share 8
          // rows with its last (their scores are read, whose operand they were)
          const int tail = (key0 + kPagedKeys > seg.len ? seg.len - key0 : 0) & 7;
          if (tail != 0) {
            if constexpr (!S::kShared) ok = ok && wait_bar_warp(v_full + 8 * stage, (t / kStages) & 1u, ctl);
            const uint32_t rows = sV + stage * S::kVTile +
                                  static_cast<uint32_t>((seg.len - key0) >> 3) * S::kVStride;
            for (int i = threadIdx.x; i < (8 - tail) * S::kVC * 8; i += 128 * S::kGroups) {
              const int r = tail + i / (S::kVC * 8), c = i % (S::kVC * 8);
              st_shared_v4(rows + static_cast<uint32_t>((c >> 3) * 1024 + r * 128 + (c & 7) * 16), 0u,
                           0u, 0u, 0u);
            }
          }
        }
        // above the references, and the largest of this lane's
        float x[kNB][4], over = -INFINITY;
        auto above = [&]() {
#pragma unroll
          for (int n = 0; n < kNB; ++n)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              fadd2(x[n][e], x[n][e + 1], s[n][e], s[n][e + 1], -m[n][0], -m[n][1]);
              over = fmax3(over, x[n][e], x[n][e + 1]);
            }
        };
        above();
        // whether the product that had P's buffer has read it, asked before the
        // exponentials (a segment's first ones: its end waited)
        const uint32_t p_free = o_done + 8 * ((t - S::kPs) & 1u), p_par = ((t - S::kPs) >> 1) & 1u;
        const bool free_now = j < S::kPs || mbar_test_wait(p_free, p_par);
        if (named_bar_or(group_bar, 128, over > kTau || !ok)) {
          // rare: a row's reference rises, or a wait ran out somewhere
          if (named_bar_or(group_bar, 128, !ok)) {
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
              if (g == 0) sm.red[wq][row0 + 8 * n + 2 * t4 + c] = top;
            }
          named_bar_sync(group_bar, 128);
#pragma unroll
          for (int n = 0; n < kNB; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int row = row0 + 8 * n + 2 * t4 + c;
              const float top = fmaxf(fmaxf(sm.red[0][row], sm.red[1][row]),
                                      fmaxf(sm.red[2][row], sm.red[3][row]));
              float a = 1.f;
              if (top > m[n][c] + kTau) {
                a = ex2_approx(m[n][c] - (top - kBelow));
                m[n][c] = top - kBelow;
                l[n][c] *= a;
              }
              if (wq == 0 && g == 0) sm.factor[row] = a;
            }
          named_bar_sync(group_bar, 128);
          if (j > 0) {
            ok = wait_bar_warp(o_done + 8 * ((t - 1) & 1u), ((t - 1) >> 1) & 1u, ctl);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < S::kBlocks * kRows; c += 16) {
              const int row = row0 + c % kRows;
              const uint32_t at = tmem + t_lane + S::kColO + c / kRows * kN + row;
              uint32_t v[16];
              tmem_ld16(at, v);
              tmem_wait_ld();
              reg_fence16(v);
#pragma unroll
              for (int e = 0; e < 16; ++e)
                v[e] = __float_as_uint(__uint_as_float(v[e]) * sm.factor[row + e]);
              tmem_st16(at, v);
            }
            tmem_wait_st();
          }
          above();
        }
        uint32_t pk[kNB][2];
#pragma unroll
        for (int n = 0; n < kNB; ++n) {
          float e[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) e[k] = ex2_approx(x[n][k]);
          fadd2(l[n][0], l[n][1], l[n][0], l[n][1], e[0], e[1]);
          fadd2(l[n][0], l[n][1], l[n][0], l[n][1], e[2], e[3]);
          pk[n][0] = pack2<BF16>(e[0], e[1]);
          pk[n][1] = pack2<BF16>(e[2], e[3]);
        }
        if (!__all_sync(0xffffffffu, free_now)) ok = ok && wait_bar_warp(p_free, p_par, ctl);
        const uint32_t p_buf = p_at + (S::kPs > 1 ? buf * S::kPBytes : 0u);
#pragma unroll
        for (int n = 0; n < kNB; n += 2)
          stmatrix_trans4(p_buf + n * 1024, pk[n][0], pk[n][1], pk[n + 1][0], pk[n + 1][1]);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_ready + 8 * buf);
      }

      // ---- the segment's end: sums over the keys, then O^T out ----
      ok = !named_bar_or(group_bar, 128, !ok);
      if (!ok) break;
      // the next segment's queries first: its scores run beside what follows
      more = paged_next<S>(p, walk, next);
      if (more) load_q(next);
#pragma unroll
      for (int n = 0; n < kNB; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float sum = l[n][c];
          sum += __shfl_xor_sync(0xffffffffu, sum, 4);
          sum += __shfl_xor_sync(0xffffffffu, sum, 8);
          sum += __shfl_xor_sync(0xffffffffu, sum, 16);
          if (g == 0) {
            sm.red[wq][row0 + 8 * n + 2 * t4 + c] = sum;
            if (wq == 0) sm.top[row0 + 8 * n + 2 * t4 + c] = m[n][c];
          }
        }
      named_bar_sync(group_bar, 128);
      for (int n = row0 + tid; n < row0 + kRows; n += 128) {
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
      named_bar_sync(group_bar, 128);
      if (seg.n_tiles > 0) {
        ok = wait_bar_warp(o_done + 8 * ((t - 1) & 1u), ((t - 1) >> 1) & 1u, ctl);
        tc_fence_after();
      }
      // 16 channels at a time as fragments.  O: transposed through the warp's share of
      // P's memory, 32 bytes a row; parts: as they are, [channel, row].
      float inv[kNB][2];
#pragma unroll
      for (int n = 0; n < kNB; ++n) {
        inv[n][0] = sm.factor[row0 + 8 * n + 2 * t4];
        inv[n][1] = sm.factor[row0 + 8 * n + 2 * t4 + 1];
      }
      const uint32_t out_at = sP + static_cast<uint32_t>(warp * kRows * 32);
      constexpr int kHalves = S::kVC == 1 ? 1 : 2;  // with 64 channels a warp has 16
#pragma unroll 1
      for (int i = 0; i < S::kBlocks * kHalves; ++i) {
        const int blk = i / kHalves, half = i % kHalves;
        const int ch0 = blk * 128 + 16 * (kHalves * wq + half);
        uint32_t v[kNB][4];
        if (seg.n_tiles > 0) {
          tmem_ld_frag(tmem + t_lane + (static_cast<uint32_t>(half) << 20) + S::kColO + blk * kN + row0, v);
          tmem_wait_ld();
        }
        float x[kNB][4];
#pragma unroll
        for (int n = 0; n < kNB; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            asm volatile("" : "+r"(v[n][e]));  // not before the wait
            x[n][e] = inv[n][e & 1] == 0.f ? 0.f : __uint_as_float(v[n][e]) * inv[n][e & 1];
          }
        if (!ok) continue;
        if (seg.whole) {
          const uint32_t row8 = static_cast<uint32_t>((lane >> 4) * 8 + (lane & 7));
          const uint32_t to = out_at + row8 * 32 + ((((lane >> 3) ^ (row8 >> 2)) & 1u) << 4);
#pragma unroll
          for (int n = 0; n < kNB; n += 2)
            stmatrix_trans4(to + n * 256, pack2<BF16>(x[n][0], x[n][1]), pack2<BF16>(x[n][2], x[n][3]),
                            pack2<BF16>(x[n + 1][0], x[n + 1][1]), pack2<BF16>(x[n + 1][2], x[n + 1][3]));
          __syncwarp();
#pragma unroll
          for (int k = 0; k < kRows / 16; ++k) {
            const int row = 16 * k + (lane >> 1), c = lane & 1;
            uint32_t w[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(out_at + row * 32 + ((c ^ ((row >> 2) & 1)) << 4)));
            if (row0 + row < seg.n_rows)
              *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) +
                                        (seg.out_row0 + row0 + row) * S::kDv + ch0 + 8 * c) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          __syncwarp();
        } else {
          // a lane's values of a channel next to each other (paged_part_row)
          float* part =
              p.part_o + (static_cast<long long>(seg.part) * S::kDv + ch0 + g) * p.part_rows + row0;
          const int down = 8 * p.part_rows;
          if constexpr (kN >= 32) {
#pragma unroll
            for (int n = 0; n < kNB; n += 4)
              if (row0 + 8 * n < p.part_rows) {
                st_global_v8(part + 8 * n + 8 * t4, x[n][0], x[n][1], x[n + 1][0], x[n + 1][1],
                             x[n + 2][0], x[n + 2][1], x[n + 3][0], x[n + 3][1]);
                st_global_v8(part + down + 8 * n + 8 * t4, x[n][2], x[n][3], x[n + 1][2], x[n + 1][3],
                             x[n + 2][2], x[n + 2][3], x[n + 3][2], x[n + 3][3]);
              }
          } else if (p.part_rows == 16) {
            *reinterpret_cast<float4*>(part + 4 * t4) = make_float4(x[0][0], x[0][1], x[1][0], x[1][1]);
            *reinterpret_cast<float4*>(part + down + 4 * t4) =
                make_float4(x[0][2], x[0][3], x[1][2], x[1][3]);
          } else if (2 * t4 < p.part_rows) {
            *reinterpret_cast<float2*>(part + 2 * t4) = make_float2(x[0][0], x[0][1]);
            *reinterpret_cast<float2*>(part + down + 2 * t4) = make_float2(x[0][2], x[0][3]);
          }
        }
      }
      tc_fence_before();
      if (named_bar_or(group_bar, 128, !ok)) break;
      seg = next;
    }
    // queries sent for land before shared memory goes away
    if (nq > 0) wait_drain(q_full, (nq - 1) & 1u, p.timeout_ns);
  } else if (warp == S::kMmaWarp) {
    // =============================== MMA issue ===============================
    constexpr uint32_t kIdescS = idesc_f16(BF16, false, false, 64, kN);
    constexpr uint32_t kIdescO = idesc_f16(BF16, true, false, S::kVC == 1 ? 64 : 128, kN);
    uint32_t t0 = 0, nq = 0;  // tiles, and segments with tiles, before this one
    bool ok = true, issued = false;
#pragma unroll 1
    while (ok && paged_next<S>(p, walk, seg)) {
      const uint32_t n = static_cast<uint32_t>(seg.n_tiles);
      if (n == 0) continue;
      if (!wait_bar_warp(q_full, nq & 1u, ctl)) break;
      ++nq;
      issued = true;
      uint32_t s = 0, o = 0;  // products issued in this segment
      auto score = [&]() {
        const uint32_t ts = t0 + s;
        tc_fence_after();
        const uint64_t a = smem_desc_sw128(sK + (ts % kStages) * S::kTileK, 16, S::kKC * 1024);
        const uint64_t b = smem_desc_sw128(sQ, 16, 1024);
#pragma unroll
        for (int c = 0; c < S::kKC; ++c)
          umma_f16_ss_k64(tmem + (ts & 1u) * kN, a + c * (1024 >> 4), b + c * (kN * 128 >> 4), kIdescS,
                          c > 0 ? 1u : 0u);
        umma_commit(s_full + 8 * (ts & 1u));
        if constexpr (!S::kShared) umma_commit(k_empty + 8 * (ts % kStages));
        ++s;
      };
      auto output = [&]() {
        const uint32_t stage = (t0 + o) % kStages;
        if constexpr (!S::kShared) {
          ok = wait_bar_warp(v_full + 8 * stage, ((t0 + o) / kStages) & 1u, ctl);
          if (!ok) return;
        }
        tc_fence_after();
        const uint64_t a = smem_desc_sw128(sV + stage * S::kVTile, 1024, S::kVStride);
        const uint64_t b =
            smem_desc_sw128(sP + (S::kPs > 1 ? ((t0 + o) & 1u) * S::kPBytes : 0u), 16, 1024);
#pragma unroll
        for (int k = 0; k < kPagedKeys / 16; ++k) {
#pragma unroll
          for (int blk = 0; blk < S::kBlocks; ++blk)
            umma_f16_ss(tmem + S::kColO + blk * kN, a + blk * (2048 >> 4) + k * (2 * S::kVStride >> 4),
                        b + 2 * k, kIdescO, (o > 0 || k > 0) ? 1u : 0u);
          if constexpr (S::kShared) umma_commit(k_empty + 8 * (4 * stage + k));
        }
        if constexpr (!S::kShared) umma_commit(v_empty + 8 * stage);
        umma_commit(o_done + 8 * ((t0 + o) & 1u));
        ++o;
      };
#pragma unroll 1
      while (ok && o < n) {
        const uint32_t full = k_full + 8 * ((t0 + s) % kStages), full_par = ((t0 + s) / kStages) & 1u;
        const uint32_t ready = p_ready + 8 * ((t0 + o) & 1u), p_par = ((t0 + o) >> 1) & 1u;
        if (s == n || s == o + 2) {  // nothing but the product with P can come next
          ok = wait_bar_warp(ready, p_par, ctl);
          if (ok) output();
        } else if (s == o) {  // nothing but scores
          ok = wait_bar_warp(full, full_par, ctl);
          if (ok) score();
        } else {  // whichever is ready first
          uint64_t since = 0;
#pragma unroll 1
          for (uint32_t polls = 1;; ++polls) {
            if (__all_sync(0xffffffffu, mbar_test_wait(ready, p_par))) {
              output();
              break;
            }
            if (__all_sync(0xffffffffu, mbar_test_wait(full, full_par))) {
              score();
              break;
            }
            if ((polls & 31u) == 0) {
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
          }
        }
      }
      t0 += n;
    }
    if (issued) {  // every MMA issued completes before tensor memory is freed
      umma_commit(drain);
      wait_drain(drain, 0, p.timeout_ns);
    }
    __syncwarp();
  } else {
    // =============================== producers ===============================
    // the first the keys, the second the values
    const bool is_k = warp == S::kMmaWarp + 1;
    const uint32_t full0 = is_k ? k_full : v_full, empty0 = is_k ? k_empty : v_empty;
    const uint32_t bytes = is_k ? S::kTileK : S::kTileV;
    const uint32_t ring = (is_k ? sK : sV) + (lane & 7) * ((is_k ? S::kKC : S::kVC) * 1024);
    const CUtensorMap* tm = is_k ? &tmK : &tmV;
    const int at = is_k ? p.k_at : p.v_at;
    uint32_t t = 0;
    bool ok = true;
#pragma unroll 1
    while (ok && paged_next<S>(p, walk, seg)) {
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
        // the row of this lane's keys, past the pool where there are none
        auto row_of = [&](int k, int pg) {
          return k < seg.k_end && pg >= 0 && pg < p.num_pages
                     ? ((pg * p.Hkv + seg.hk) << p.page_shift) + (k & (page_keys - 1))
                     : p.pool_rows;
        };
        const int row = row_of(key, page);
        const bool is_bad = key < seg.k_end && row == p.pool_rows;
        if (is_bad) atomicMax(p.status, kStatusBadIndex);
        const uint32_t bad = __ballot_sync(0xffffffffu, is_bad);
#pragma unroll 1
        for (int k = 0; ok && k < 4 && j0 + k < seg.n_tiles; ++k, ++t) {
          const uint32_t stage = t % kStages, full = full0 + 8 * stage, par = ((t / kStages) & 1u) ^ 1u;
          const uint32_t dst = ring + stage * bytes;
          // a latent stage 16 keys at a time
          constexpr int kBlocks = S::kShared ? 4 : 1;
#pragma unroll 1
          for (int block = 0; ok && block < kBlocks; ++block) {
            ok = wait_bar_warp(empty0 + 8 * (kBlocks * stage + block), par, ctl);
            if (!ok) break;
            if (block == 0 && lane == 0) {
              if (is_k) sm.bad[t % kPagedBad] = (bad >> (8 * k)) & 0xffu;
              mbar_arrive_expect_tx(full, bytes);
            }
            __syncwarp();
            if ((lane >> 3) == k && (!S::kShared || ((lane & 7) >> 1) == block))
              tma_load_4d(dst, tm, full, 0, row, 0, at);
            __syncwarp();
          }
          // two latent tiles in flight are not enough for HBM's latency: the next four come
          // to L2 meanwhile.  (128 heads, 32 sequences of up to 8192 rows: 96.2 us, without
          // 102.6; half of them by each of a pair, whose CTAs may have drifted apart, 96.9.)
          if constexpr (S::kPeers > 1)
            if (k == 1) {
              const int next_row = row_of(key + 4 * kPagedKeys, ahead);
              if (next_row != p.pool_rows) tma_prefetch_l2_4d(tm, 0, next_row, 0, at);
              __syncwarp();
            }
        }
      }
    }
    // every load issued lands before shared memory goes away (an abort may have left
    // the last tile's unsent: the wait is bounded)
    for (uint32_t i = t > kStages ? t - kStages : 0u; i < t; ++i)
      wait_drain(full0 + 8 * (i % kStages), (i / kStages) & 1u, p.timeout_ns);
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == S::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmemCols);
  }
}

// The units that several CTAs shared: O = sum_s w_s O_s / sum_s w_s over their parts,
// w_s = exp(LSE_s - max LSE).  A block takes kCh channels of a unit: it makes the
// weights of all the unit's rows once, then its threads take four rows of a channel
// each, which lie together in the parts, the parts dealt to groups of threads where
// those are few.  As many channels as leave every multiprocessor a block.
constexpr int kPagedMergeThreads = 256;  // 128: H 128 slower by 6 us

// Four blocks an SM (three: 32 sequences of 8192 keys 138 to 141 us), or no limit for the
// narrow slices that few units have.
template <class S, bool BF16, int kCh>
__global__ void __launch_bounds__(kPagedMergeThreads, kCh > 8 ? 4 : 1)
    fa_paged_merge_kernel(const PagedAttnParams p, int attn_grid) {
  constexpr int kN = S::kN, kThr = kPagedMergeThreads, kWarps = kThr / 32;
  constexpr int kParts = 64;                                // whose weights are held at once
  constexpr int kItems = (kCh * kN / 4 + kThr - 1) / kThr;  // of a thread
  constexpr int kAhead = kItems == 1 ? 4 : 2;               // its parts fetched before the weights
  constexpr int kPer = kThr / kN;                           // threads that share a row's weights
  constexpr int kW = kN + 4;
  constexpr float kLog2e = 1.4426950408889634f;
  __shared__ KeyScan<kWarps> scan;
  __shared__ alignas(16) float w[kParts * kW];
  __shared__ alignas(16) float old[kN];
  __shared__ float sums[kN];
  __shared__ union {
    float4 acc[kThr];
    alignas(16) uint16_t out[kN * (kCh + 8) + kN / 2];
  } end;
  const int tid = static_cast<int>(threadIdx.x);
  // a unit of the deal and, in pairs, the rank of the CTA whose rows these are
  const int units = p.Hkv * p.n_row_blocks, rank = static_cast<int>(blockIdx.z);
  const int b = static_cast<int>(blockIdx.x) / units, unit = static_cast<int>(blockIdx.x) - b * units;
  const int hk = unit / p.n_row_blocks;
  const int rb = (unit - hk * p.n_row_blocks) * S::kPeers + rank;
  const int ch0 = static_cast<int>(blockIdx.y) * kCh;
  int upto;
  const int all = cache_scan(p, scan, false, upto, S::kSegment);
  const CacheDeal deal = cache_deal(all, attn_grid, kPagedMinChunks);
  // chunks per unit of the sequences before b: the thread with b in its run
  const int run = (p.B + kThr - 1) / kThr;
  if (b / run == tid) {
    for (int k = tid * run; k < b; ++k) upto += cache_chunks(cache_length(p, k)) + S::kSegment;
    scan.before = upto;
  }
  __syncthreads();
  const int chunks = cache_chunks(cache_length(p, b));
  const int start = scan.before * units + unit * (chunks + S::kSegment);
  const int x0 = deal.cta_of(start), x1 = deal.cta_of(start + chunks - 1);
  grid_dependency_wait();  // all blocks: this grid's end is then the attention's too
  if (x0 == x1) return;
  // a CTA's first segment, except where the unit begins inside x0
  const int inside = deal.begin(x0) < start ? 1 : 0;
  auto part_of = [&](int s) { return (2 * (x0 + s) + (s == 0 ? inside : 0)) * S::kPeers + rank; };
  const int n_parts = x1 - x0 + 1, n_rows = max(0, min(kN, p.rows - rb * kN));
  const int quads = p.part_rows / 4, items = kCh * quads;  // four rows of a channel each
  const int groups = items < kThr ? kThr / items : 1;
  const int group = items < kThr ? tid / items : 0;
  const int item0 = items < kThr ? tid - group * items : tid;
  const bool busy = group < groups && item0 < items;
  const float* from = p.part_o + static_cast<long long>(ch0) * p.part_rows;
  const long long step = static_cast<long long>(S::kDv) * p.part_rows;
  auto load = [&](int s, int item) {
    return *reinterpret_cast<const float4*>(from + part_of(s) * step + 4 * item);
  };
  float4 acc[kItems];
#pragma unroll
  for (int i = 0; i < kItems; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  const int row = tid / kPer, j = tid % kPer;  // a row by its place in the parts
  // the output's rows, so that the threads that write a channel's meet few banks twice
  auto out_at = [](int r) { return r * (kCh + 8) + (r >> 4) * 8; };
  float top = -INFINITY, sum = 0.f;  // the row's, over the parts so far

#pragma unroll 1
  for (int s0 = 0; s0 < n_parts; s0 += kParts) {
    const int now = min(kParts, n_parts - s0);
    float4 ahead[kItems][kAhead];
#pragma unroll
    for (int i = 0; i < kItems; ++i)
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (busy && item0 + i * kThr < items && group + k * groups < now)
          ahead[i][k] = load(s0 + group + k * groups, item0 + i * kThr);
    if (s0 > 0) __syncthreads();  // the weights before are done with
    for (int i = tid; i < now * kN; i += kThr) {
      const int s = i / kN, at = i % kN, n = paged_part_row<kN>(at, p.part_rows);
      w[s * kW + at] = n < n_rows ? p.part_lse[static_cast<long long>(part_of(s0 + s)) * kN + n] * kLog2e
                                  : -INFINITY;
    }
    __syncthreads();
    float m = top, part_sum = 0.f;
    for (int s = j; s < now; s += kPer) m = fmaxf(m, w[s * kW + row]);
#pragma unroll
    for (int k = kPer / 2; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
    const float base = m == -INFINITY ? 0.f : m;
    for (int s = j; s < now; s += kPer) {
      const float x = ex2_approx(w[s * kW + row] - base);
      w[s * kW + row] = x;
      part_sum += x;
    }
#pragma unroll
    for (int k = kPer / 2; k > 0; k >>= 1) part_sum += __shfl_xor_sync(0xffffffffu, part_sum, k);
    const float f = ex2_approx(top - base);
    sum = fmaf(sum, f, part_sum);
    top = m;
    if (j == 0) {
      old[row] = f;
      sums[row] = sum;
    }
    __syncthreads();
    if (busy) {
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        const int item = item0 + i * kThr;
        if (item >= items) break;
        const int r = 4 * (item % quads);
        const float4 q = *reinterpret_cast<const float4*>(old + r);
        acc[i].x *= q.x, acc[i].y *= q.y, acc[i].z *= q.z, acc[i].w *= q.w;
        auto add = [&](int s, const float4& v) {
          const float4 x = *reinterpret_cast<const float4*>(w + s * kW + r);
          acc[i].x = fmaf(x.x, v.x, acc[i].x);
          acc[i].y = fmaf(x.y, v.y, acc[i].y);
          acc[i].z = fmaf(x.z, v.z, acc[i].z);
          acc[i].w = fmaf(x.w, v.w, acc[i].w);
        };
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
          if (group + k * groups < now) add(group + k * groups, ahead[i][k]);
#pragma unroll 4
        for (int s = group + kAhead * groups; s < now; s += groups) add(s, load(s0 + s, item));
      }
    }
  }
  if (groups > 1) {
    end.acc[tid] = acc[0];
    __syncthreads();
    if (group == 0 && busy)
      for (int k = 1; k < groups; ++k) {
        const float4 v = end.acc[k * items + item0];
        acc[0].x += v.x, acc[0].y += v.y, acc[0].z += v.z, acc[0].w += v.w;
      }
    __syncthreads();  // the memory is the output's
  }
  if (group == 0 && busy) {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int item = item0 + i * kThr;
      if (item >= items) break;
      const int r = 4 * (item % quads), c = item / quads;
      const float v[4] = {acc[i].x, acc[i].y, acc[i].z, acc[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        // no part has a key: 0; a NaN stays one
        const float x = sums[r + k] == 0.f ? 0.f : v[k] / sums[r + k];
        end.out[out_at(paged_part_row<kN>(r + k, p.part_rows)) + c] = static_cast<uint16_t>(pack2<BF16>(x, x));
      }
    }
  }
  __syncthreads();
  const long long row0 = (static_cast<long long>(b) * p.Hkv + hk) * p.rows + rb * kN;
  for (int i = tid; i < n_rows * (kCh / 8); i += kThr) {
    const int r = i / (kCh / 8), c = i % (kCh / 8);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + (row0 + r) * S::kDv + ch0 + 8 * c) =
        *reinterpret_cast<const uint4*>(end.out + out_at(r) + 8 * c);
  }
  const int out_row = paged_part_row<kN>(row, p.part_rows);
  if (blockIdx.y == 0 && j == 0 && out_row < n_rows)
    p.lse[row0 + out_row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994530942f;
}

}  // namespace fa
