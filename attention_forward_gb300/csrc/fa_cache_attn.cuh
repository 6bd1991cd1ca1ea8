// fa_cache_attn.cuh -- attention of a few query rows per head over a paged
// cache held in 4 bits, split over the keys.  sm_103a.
//
// Each kv head's query rows (its H / Hkv heads times Sq tokens) share every
// key, so a CTA takes up to 8 NT of them over one range of keys.  A warp walks
// the range 16 keys at a time and holds everything in registers:
//
//   scores, keys x rows (m16n8k16, fp16 in, fp32 out): A is the raw codes.  A
//     nibble c masked in place in a 16-bit half is the fp16 subnormal
//     c 2^-24 (bits 0-3) or c 2^-20 (bits 4-7), exact, so a word of 8 codes
//     becomes four A registers with one shift and four ANDs.  B is the query
//     row, scaled by a power of two that puts its largest element in
//     [2^13, 2^14), times 2^-4 opposite the 2^-20 codes.  (Exact down to 2^-26 of
//     the row's largest channel in bf16 and 2^-23 in fp16, off by at most 2^-34 of
//     that below.)  A group's 32 channels are two such products; its scale
//     multiplies their fp32 sums.  The minima come from one more product:
//     A = the stored (scale, minimum) pairs, B = (0, sum of the group's query
//     channels), that sum in two fp16 parts, to 2^-22 of itself.
//   softmax: fp32, log2 domain, one reference maximum per row, raised when a
//     score passes it by 15: p = 2^(t - m) <= 2^15 with m set 8 below the
//     maximum, so that fp16 holds p over 2^-24 ... 2^15 around it.
//   output, channels x rows: A = the values, dequantised to fp16 pairs of two
//     tokens ((1024 + c) - 1024 or (64 + c) - 64, then one fma with scale and
//     minimum: a rounding of 2^-11 of the value, an eighth of bf16's), B = p
//     in fp16 (2^-11), turned from the score layout by movmatrix.  Both are what
//     the product's 16-bit operands hold; the sums are fp32.
//
// A warp copies its tiles (16 keys: 2560 bytes at D = 128) into a ring of its own
// in shared memory with 16-byte asynchronous copies, kCacheAttnStages tiles
// ahead, and reads them from there in the order its lanes need: lane (g, t) =
// (lane / 4, lane % 4) takes the words of two keys that hold its channels 8 t
// ... 8 t + 7 of every group, and the words 2 g, 2 g + 1 of four value tokens.
// Nothing is shared between the warps until the end, where their states meet
// in shared memory and the CTA writes O and LSE, or the range's partials for
// the merge kernel.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "fa_cache.cuh"
#include "fa_cache.h"
#include "fa_keys.cuh"
#include "fa_merge.cuh"
#include "sm103_ptx.cuh"

namespace fa {

// D += A B, m16n8k16, fp16 operands, fp32 accumulators.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// D = A B.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Transpose of an 8 x 8 matrix of 16-bit elements held two per lane.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// 16 bytes global -> shared, past L1.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int N>
__device__ __forceinline__ void lds(uint32_t (&v)[N], uint32_t addr) {
  static_assert(N == 1 || N == 2 || N == 4, "one load");
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(addr));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(addr));
  else
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v[0]) : "r"(addr));
}

__device__ __forceinline__ __half2 as_half2(uint32_t w) { return *reinterpret_cast<__half2*>(&w); }
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// (a & mask) | bits in one instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t bits) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(a), "r"(mask), "r"(bits));
  return d;
}

// A 16-key tile in shared memory: the 16 rows' codes and parameters of K, then
// of V, as they lie in the pool.
template <int D>
struct CacheTile {
  static constexpr int kRow = D / 2, kPar = D / kCacheGroup * 4;
  static constexpr int kKCodes = 0, kKParams = 16 * kRow;
  static constexpr int kVCodes = kKParams + 16 * kPar, kVParams = kVCodes + 16 * kRow;
  static constexpr int kBytes = kVParams + 16 * kPar;
};

// Score row r (0 ... 15) of a tile, and value slot r of its product, is token
// tile_token(r): lane t's value tokens (rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9) are
// then t, 4 + (t ^ 1), 8 + t, 12 + (t ^ 1), so that the four lanes of a load
// read four neighbouring rows (with 2 t they would all fall on one half of the
// banks), and rows g, g + 1 of the keys still fall on both halves.
__device__ __forceinline__ int tile_token(int r) {
  return (r & 8) + ((r & 1) ? 4 + (((r >> 1) & 3) ^ 1) : ((r >> 1) & 3));
}

// What a lane copies of a tile: 16 bytes at these places, at 512-byte steps of
// the codes; the low lanes take K's parameters, the high lanes V's.
struct CacheLane {
  const uint8_t *kc, *vc, *par;
  uint32_t par_dst;
  bool has_par;
};

template <int D>
__device__ __forceinline__ CacheLane cache_lane(const CacheAttnParams& p, int lane) {
  using T = CacheTile<D>;
  CacheLane c;
  c.kc = p.pool.codes[0] + 16 * lane;
  c.vc = p.pool.codes[1] + 16 * lane;
  const int l = lane & 15;
  c.par = reinterpret_cast<const uint8_t*>(lane < 16 ? p.pool.params[0] : p.pool.params[1]) + 16 * l;
  c.par_dst = (lane < 16 ? T::kKParams : T::kVParams) + 16 * l;
  c.has_par = l < T::kPar;  // 16 rows of kPar bytes, 16 at a time
  return c;
}

template <int D>
__device__ __forceinline__ void copy_tile(uint32_t dst, const CacheLane& c, long long row, int lane) {
  using T = CacheTile<D>;
  const long long off = row * T::kRow;
  const uint32_t d = dst + 16u * static_cast<uint32_t>(lane);
#pragma unroll
  for (int k = 0; k < 16 * T::kRow / 512; ++k) {
    cp_async16(d + T::kKCodes + 512 * k, c.kc + off + 512 * k);
    cp_async16(d + T::kVCodes + 512 * k, c.vc + off + 512 * k);
  }
  if (c.has_par) cp_async16(dst + c.par_dst, c.par + row * T::kPar);
}

constexpr int kCacheAttnThreads = kCacheAttnWarps * 32;
using CacheScan = KeyScan<kCacheAttnWarps>;

template <int D, int NT>
struct CacheAttnSmem {
  static constexpr int kRows = 8 * NT;
  static constexpr int kRowFloats = D + 1;
  long long rows[kCachePiece / 16];  // a tile's first row in the pool, or -1
  CacheScan scan;
  union {
    // the warps' rings
    alignas(16) uint8_t ring[kCacheAttnWarps][kCacheAttnStages][CacheTile<D>::kBytes];
    // at a segment's end, per warp: reference maximum and sum of each row, then
    // O by (row, channel); a row's D channels are followed by one pad word
    struct {
      float m[kCacheAttnWarps][kRows];
      float l[kCacheAttnWarps][kRows];
      float o[kCacheAttnWarps][kRows][kRowFloats];
    } end;
  };
};

// Persistent CTAs.  Short caches (p.whole) are dealt in whole units, a row block
// of a kv head of a sequence each.  Otherwise the work is counted in chunks of
// kCacheAttnKeys keys of a unit, units in the order (sequence, kv head, row
// block), and the CTAs have equal shares of them (CacheDeal), whatever the
// lengths, which are read here.  A unit that lies within one CTA is written
// out; the parts of the others go to the workspace, the CTA's first segment to
// part 2 x, its last to 2 x + 1, where the merge kernel finds them by the same
// arithmetic.  kMod: the scores are capped or biased (without it those
// instructions, issued and predicated off, were a quarter of the loop).
//
// Bound: HBM by its bytes, but the instructions that cut the codes out come
// close: 320 a tile and warp, 504 of an SM sub-partition's cycles a tile against
// 441 of HBM time.  Measured at 32 sequences x 8 kv heads, 4 rows, D = 128: each
// further 8192 keys at 6.0 TB/s of 6.8 (88 %), behind 10 us to start, look the
// lengths and pages up and merge, and 3.4 us where a CTA has two segments; 59.6
// us for the ragged 280 MB of 8192 (4.7 TB/s).  What did not pay: tiles in
// registers two ahead (89 us: too few bytes in flight), 3 or 5 CTAs an SM
// instead of 4 (even, 6 % slower), 4 tiles ahead (even), the next segment's first
// tiles fetched while this one's warps meet (62.7 us).
template <int D, bool BF16, int NT, bool kMod>
__global__ void __launch_bounds__(kCacheAttnThreads, cache_attn_occupancy(8 * NT))
    fa_cache_attn_kernel(const CacheAttnParams p) {
  constexpr int G = D / kCacheGroup;
  constexpr int kWords = D / 64;   // value words per lane and token
  constexpr int kMmas = D / 16;    // output products: 8 per value word pair
  constexpr float kLog2e = 1.4426950408889634f;
  constexpr float kBelow = 8.f, kTau = 15.f;
  // a reference below every score that counts: -inf - kNone is -inf, so masked
  // keys get 0 from the first tile on
  constexpr float kNone = -3.0e38f;
  using T = CacheTile<D>;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  CacheAttnSmem<D, NT>& sm = *reinterpret_cast<CacheAttnSmem<D, NT>*>(smem_raw);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;

  grid_dependency_wait();
  grid_launch_dependents();  // the merge, and the next kernel, wait for this grid's end
  const int x_cta = static_cast<int>(blockIdx.x);
  const int units = p.Hkv * p.n_row_blocks;  // of a sequence
  // the sequence, its length, the chunks of those before it, the CTA's chunks
  int b, len, before, first, last;
  if (p.whole) {  // units x, x + grid, ...: `first` and `last` count units here
    b = len = before = 0;
    first = x_cta;
    last = p.B * units;
  } else {
    int upto;
    const int all_chunks = cache_scan(p, sm.scan, blockIdx.x == 0, upto);
    const CacheDeal deal = cache_deal(all_chunks, static_cast<int>(gridDim.x));
    if (x_cta >= deal.n) return;
    first = deal.begin(x_cta);
    last = deal.begin(x_cta + 1);
    cache_find(p, sm.scan, upto, first, b, len, before);
  }

  // this lane's places in the ring's tiles and in the pool
  const uint32_t ring = smem_u32(sm.ring[warp]);
  const CacheLane from = cache_lane<D>(p, lane);
  const int tok = tile_token(g);  // and tok + 8: its keys
  const uint32_t at_kc = T::kKCodes + tok * T::kRow + t * (4 * G);
  const uint32_t at_kp = T::kKParams + tok * T::kPar;
  const uint32_t at_kz = at_kp + 4 * (t & (G - 1));
  // D = 128: words 2 g, 2 g + 1, of groups 2 (g & 1), 2 (g & 1) + 1; D = 64: word
  // g, of group g & 1
  const uint32_t at_vc = T::kVCodes + g * (4 * kWords);
  const uint32_t at_vp = T::kVParams + (g & 1) * (4 * kWords);
  const int vtok[2] = {t, 4 + (t ^ 1)};  // and these + 8: its value tokens

#pragma unroll 1
  for (int cur = first; cur < last;) {
  if (p.whole) b = cur / units;
  if (p.whole || cur != first) len = cache_length(p, b);
  if (p.whole && threadIdx.x == 0 && len != p.length[b]) atomicMax(p.status, kStatusBadIndex);
  const int seq_chunks = cache_chunks(len);
  const int unit = p.whole ? cur - b * units : (cur - before) / seq_chunks;
  const int chunk0 = p.whole ? 0 : cur - before - unit * seq_chunks;
  const int n_chunks = p.whole ? seq_chunks : min(seq_chunks - chunk0, last - cur);
  const bool whole = n_chunks == seq_chunks;
  const int part = 2 * x_cta + (cur == first ? 0 : 1);
  const int hk = unit / p.n_row_blocks, rb = unit - hk * p.n_row_blocks;
  const int row0 = rb * 8 * NT;
  const long long out_row0 = (static_cast<long long>(b) * p.Hkv + hk) * p.rows + row0;
  const int n_rows = min(8 * NT, p.rows - row0);
  const int k_begin = chunk0 * kCacheAttnKeys;
  const int k_end = min(len, k_begin + n_chunks * kCacheAttnKeys);
  const int* pages = p.page_table + static_cast<long long>(b) * p.max_pages;
  // on to the next segment
  if (p.whole) {
    cur += static_cast<int>(gridDim.x);
  } else {
    cur += n_chunks;
    if (chunk0 + n_chunks == seq_chunks && unit == units - 1) {
      before += seq_chunks * units;
      ++b;
    }
  }

  // The segment's tiles in pieces whose places fit in shared memory: all the
  // threads look the places of a piece up, then every warp starts its copies.
  // The ring runs kCacheAttnStages - 1 tiles ahead; every turn commits one
  // group of copies, empty past the end and for a tile that does not exist, so
  // that the group to wait for is always the same number back.
  int n_tiles = 0;
  auto fetch = [&](int i, int stage) {
    const long long row = i < n_tiles ? sm.rows[i] : -1;
    if (row >= 0) copy_tile<D>(ring + stage * T::kBytes, from, row, lane);
    cp_async_commit();
  };
  auto start_piece = [&](int piece) {
    n_tiles = (min(k_end - piece, kCachePiece) + 15) >> 4;
    for (int i = threadIdx.x; i < n_tiles; i += kCacheAttnThreads) {
      const int key = piece + 16 * i;  // a 16-key tile lies within one page
      const int pg = pages[key >> p.page_shift];
      const bool bad = pg < 0 || pg >= p.num_pages;
      if (bad) atomicMax(p.status, kStatusBadIndex);
      sm.rows[i] = bad ? -1
                       : ((static_cast<long long>(pg) * p.Hkv + hk) << p.page_shift) +
                             (key & ((1 << p.page_shift) - 1));
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kCacheAttnStages - 1; ++k) fetch(warp + k * kCacheAttnWarps, k);
  };
  start_piece(k_begin);  // in flight while the queries are made ready

  // ---- the query rows: B operands, and per-row constants of the columns
  // this lane's accumulators hold (rows 2 t, 2 t + 1 of each block of 8)
  uint32_t qb[NT][G][4];   // [group][product 0: b0, b1; product 1: b0, b1]
  uint32_t qs[NT][2];      // (0, sum) of group t: high part, low part
  float fac[NT][2];        // score = sum * fac
  float slope[NT][2];
  int limit[NT][2];        // keys below it are visible
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = 8 * n + g;  // the row of this lane's B column
    float q[G][8];
    float top = 0.f;
#pragma unroll
    for (int gr = 0; gr < G; ++gr) {
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (r < n_rows)
        w = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.q) +
                                            ((out_row0 + r) * D + 32 * gr + 8 * t) * 2);
      const float2 a = cache_unpack<BF16>(w.x), b2 = cache_unpack<BF16>(w.y);
      const float2 c = cache_unpack<BF16>(w.z), d = cache_unpack<BF16>(w.w);
      q[gr][0] = a.x; q[gr][1] = a.y; q[gr][2] = b2.x; q[gr][3] = b2.y;
      q[gr][4] = c.x; q[gr][5] = c.y; q[gr][6] = d.x; q[gr][7] = d.y;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(q[gr][e]));
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // up = 2^e with top * up in [2^13, 2^14); e is at least 13 - 127, and at most
    // 120, as for an all-zero row, so that 1 / up is a float and its scores are 0
    // under any scale
    int e2 = top > 0.f ? (top < INFINITY ? 13 - ilogbf(top) : 0) : 120;
    e2 = min(e2, 120);
    const float up = __int_as_float((127 + e2) << 23);
    float part[G];
#pragma unroll
    for (int gr = 0; gr < G; ++gr) {
      part[gr] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        q[gr][e] *= up;
        part[gr] += q[gr][e];
      }
      part[gr] += __shfl_xor_sync(0xffffffffu, part[gr], 1);
      part[gr] += __shfl_xor_sync(0xffffffffu, part[gr], 2);
      // channels (0, 4), (1, 5), (2, 6), (3, 7) of the word: the nibbles that
      // share a register; the odd pairs' codes are 2^4 larger
      qb[n][gr][0] = as_u32(__floats2half2_rn(q[gr][0], q[gr][4]));
      qb[n][gr][1] = as_u32(__floats2half2_rn(q[gr][1] * 0.0625f, q[gr][5] * 0.0625f));
      qb[n][gr][2] = as_u32(__floats2half2_rn(q[gr][2], q[gr][6]));
      qb[n][gr][3] = as_u32(__floats2half2_rn(q[gr][3] * 0.0625f, q[gr][7] * 0.0625f));
    }
    // the group sums at 2^-8 of the rows' scale: |sum| < 2^19 fits fp16
    float sum = 0.f;
#pragma unroll
    for (int gr = 0; gr < G; ++gr)
      if (t == gr) sum = part[gr] * 0.00390625f;
    const __half hi = __float2half_rn(sum);
    const __half lo = __float2half_rn(sum - __half2float(hi));
    qs[n][0] = static_cast<uint32_t>(__half_as_ushort(hi)) << 16;
    qs[n][1] = static_cast<uint32_t>(__half_as_ushort(lo)) << 16;
    // what a sum is multiplied by: 1 / up, the scale, then 2^24 (the codes') and
    // log2(e) unless the cap comes between; in this order it overflows only where
    // the scores do
    const float down = __int_as_float((127 - e2) << 23);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int rc = 8 * n + 2 * t + c;
      fac[n][c] = __shfl_sync(0xffffffffu, down, (2 * t + c) * 4) * p.scale *
                  (kMod && p.cap > 0.f ? 16777216.f : 16777216.f * kLog2e);
      const int rr = min(rc, n_rows - 1) + row0;
      const int h = hk * (p.H / p.Hkv) + rr / p.Sq, i = rr % p.Sq;
      slope[n][c] = kMod && p.slopes ? p.slopes[h] * kLog2e : 0.f;
      limit[n][c] = rc < n_rows ? len - (p.Sq - 1 - i) : len;  // rows past n_rows are not stored
      m[n][c] = kNone;
      l[n][c] = 0.f;
    }
  }
  float acc[NT][kMmas][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < kMmas; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[n][i][e] = 0.f;

  int least_limit = limit[0][0];  // over this lane's rows
#pragma unroll
  for (int n = 0; n < NT; ++n) least_limit = min(least_limit, min(limit[n][0], limit[n][1]));
  least_limit = __reduce_min_sync(0xffffffffu, least_limit);

  // edge: some row does not see some key of the tile
  auto compute = [&](uint32_t tile, int key0, auto edge) {
    // ------------------------------ scores ------------------------------
    float s[NT][4];
    uint32_t kc[2][G], kp[2][G];
    lds(kc[0], tile + at_kc);
    lds(kc[1], tile + at_kc + 8 * T::kRow);
    lds(kp[0], tile + at_kp);
    lds(kp[1], tile + at_kp + 8 * T::kPar);
    {
      uint32_t z0[1], z1[1];  // group t's pair (D = 64: lanes 2, 3 take weights of 0)
      lds(z0, tile + at_kz);
      lds(z1, tile + at_kz + 8 * T::kPar);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float z[4];
        mma_f16_first(z, z0[0], z1[0], z0[0], z1[0], qs[n][0], qs[n][1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = z[e] * 1.52587890625e-5f;  // 2^8 / 2^24
      }
    }
#pragma unroll
    for (int gr = 0; gr < G; ++gr) {
      const uint32_t w0 = kc[0][gr], w1 = kc[1][gr];
      const uint32_t y0 = w0 >> 8, y1 = w1 >> 8;
      const float s0 = __low2float(as_half2(kp[0][gr])), s1 = __low2float(as_half2(kp[1][gr]));
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float d[4];
        mma_f16_first(d, w0 & 0x000f000fu, w1 & 0x000f000fu, w0 & 0x00f000f0u, w1 & 0x00f000f0u,
                qb[n][gr][0], qb[n][gr][1]);
        mma_f16(d, y0 & 0x000f000fu, y1 & 0x000f000fu, y0 & 0x00f000f0u, y1 & 0x00f000f0u,
                qb[n][gr][2], qb[n][gr][3]);
        s[n][0] = fmaf(d[0], s0, s[n][0]);
        s[n][1] = fmaf(d[1], s0, s[n][1]);
        s[n][2] = fmaf(d[2], s1, s[n][2]);
        s[n][3] = fmaf(d[3], s1, s[n][3]);
      }
    }

    // ------------------------------ softmax -----------------------------
    uint32_t pb[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = e & 1, key = key0 + tok + 8 * (e >> 1);
        float v = s[n][e] * fac[n][c];
        if (kMod && p.cap > 0.f) v = cap_score(v, p) * kLog2e;
        if (kMod && p.slopes) v = fmaf(-slope[n][c], static_cast<float>(abs(limit[n][c] - 1 - key)), v);
        if constexpr (decltype(edge)::value) v = key < limit[n][c] ? v : -INFINITY;
        s[n][e] = v;
      }
      const bool over = fmaxf(s[n][0], s[n][2]) > m[n][0] + kTau ||
                        fmaxf(s[n][1], s[n][3]) > m[n][1] + kTau;
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float top = fmaxf(s[n][c], s[n][c + 2]);
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
          if (top > m[n][c] + kTau) {
            const float m_new = top - kBelow;
            const float a = ex2_approx(m[n][c] - m_new);
            m[n][c] = m_new;
            l[n][c] *= a;
#pragma unroll
            for (int k = 0; k < kMmas; ++k) {
              acc[n][k][c] *= a;
              acc[n][k][c + 2] *= a;
            }
          }
        }
      }
      float pr[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // before the first visible key m is below every finite reference
        pr[e] = ex2_approx(s[n][e] - m[n][e & 1]);
        l[n][e & 1] += pr[e];
      }
      pb[n][0] = movmatrix_trans(as_u32(__floats2half2_rn(pr[0], pr[1])));
      pb[n][1] = movmatrix_trans(as_u32(__floats2half2_rn(pr[2], pr[3])));
    }

    // ------------------------------ output ------------------------------
    uint32_t vc[4][kWords], vp[4][kWords];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t r = vtok[k & 1] + 8 * (k >> 1);
      lds(vc[k], tile + at_vc + r * T::kRow);
      lds(vp[k], tile + at_vp + r * T::kPar);
    }
    if constexpr (decltype(edge)::value) {  // slots past the sequence may hold anything
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (key0 + vtok[k & 1] + 8 * (k >> 1) >= len)
#pragma unroll
          for (int w = 0; w < kWords; ++w) vp[k][w] = 0u;
    }
    // scale and minimum pairs of the token pairs
    __half2 sc[kWords][2], mn[kWords][2];
#pragma unroll
    for (int w = 0; w < kWords; ++w)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        sc[w][k] = as_half2(__byte_perm(vp[2 * k][w], vp[2 * k + 1][w], 0x5410));
        mn[w][k] = as_half2(__byte_perm(vp[2 * k][w], vp[2 * k + 1][w], 0x7632));
      }
    // registers of half a word's channels (4 of 8) for both token pairs:
    // a[pair][channel]
    auto dequant = [&](int w, int half, uint32_t (&a)[2][4]) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t c = __byte_perm(vc[2 * k][w], vc[2 * k + 1][w], half ? 0x7632 : 0x5410);
        const uint32_t y = c >> 8;
        const __half2 k1024 = as_half2(0x64006400u), k64 = as_half2(0x54005400u);
        const __half2 h0 = __hsub2(as_half2(and_or(c, 0x000f000fu, 0x64006400u)), k1024);
        const __half2 h1 = __hsub2(as_half2(and_or(c, 0x00f000f0u, 0x54005400u)), k64);
        const __half2 h2 = __hsub2(as_half2(and_or(y, 0x000f000fu, 0x64006400u)), k1024);
        const __half2 h3 = __hsub2(as_half2(and_or(y, 0x00f000f0u, 0x54005400u)), k64);
        a[k][0] = as_u32(__hfma2(h0, sc[w][k], mn[w][k]));
        a[k][1] = as_u32(__hfma2(h1, sc[w][k], mn[w][k]));
        a[k][2] = as_u32(__hfma2(h2, sc[w][k], mn[w][k]));
        a[k][3] = as_u32(__hfma2(h3, sc[w][k], mn[w][k]));
      }
    };
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t a0[2][4];
      dequant(0, half, a0);
      if constexpr (D == 128) {
        uint32_t a1[2][4];
        dequant(1, half, a1);
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma_f16(acc[n][4 * half + k], a0[0][k], a1[0][k], a0[1][k], a1[1][k], pb[n][0], pb[n][1]);
      } else {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma_f16(acc[n][2 * half + k], a0[0][k], a0[0][k + 2], a0[1][k], a0[1][k + 2], pb[n][0],
                    pb[n][1]);
      }
    }
  };

#pragma unroll 1
  for (int piece = k_begin; piece < k_end; piece += kCachePiece) {
    if (piece > k_begin) {
      __syncthreads();  // every warp is done with the places before
      start_piece(piece);
    }
    int stage = 0;
#pragma unroll 1
    for (int i = warp; i < n_tiles; i += kCacheAttnWarps) {
      cp_async_wait<kCacheAttnStages - 2>();
      __syncwarp();  // every lane's copies have landed, every lane is done with the stage before
      fetch(i + (kCacheAttnStages - 1) * kCacheAttnWarps,
            stage == 0 ? kCacheAttnStages - 1 : stage - 1);
      if (sm.rows[i] >= 0) {
        const int key0 = piece + 16 * i;
        if (key0 + 16 <= least_limit)
          compute(ring + stage * T::kBytes, key0, std::false_type{});
        else
          compute(ring + stage * T::kBytes, key0, std::true_type{});
      }
      stage = stage == kCacheAttnStages - 1 ? 0 : stage + 1;
    }
    cp_async_wait<0>();
    __syncwarp();
  }
  __syncthreads();  // the rings' memory is the end's

  // ---- the warps' states meet in shared memory ----
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float sum = l[n][c];
      sum += __shfl_xor_sync(0xffffffffu, sum, 4);
      sum += __shfl_xor_sync(0xffffffffu, sum, 8);
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      const int r = 8 * n + 2 * t + c;
      if (g == 0) {
        sm.end.m[warp][r] = m[n][c];
        sm.end.l[warp][r] = sum;
      }
#pragma unroll
      for (int k = 0; k < kMmas; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // accumulator row g (e = 0) or g + 8 (e = 1) of product k
          int word, nib;
          if constexpr (D == 128) {
            word = 2 * g + e;
            nib = k;
          } else {
            word = g;
            nib = 4 * (k >> 1) + (k & 1) + 2 * e;
          }
          const int ch = 32 * (word % G) + 8 * (word / G) + nib;
          sm.end.o[warp][r][ch] = acc[n][k][2 * e + c];
        }
    }
  __syncthreads();
  // two channels per thread, rows in turn
  constexpr int kPer = D / 2;
  for (int i = threadIdx.x; i < n_rows * kPer; i += kCacheAttnWarps * 32) {
    const int r = i / kPer, ch = 2 * (i - r * kPer);
    float M = kNone;
#pragma unroll
    for (int w = 0; w < kCacheAttnWarps; ++w) M = fmaxf(M, sm.end.m[w][r]);
    float L = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
    for (int w = 0; w < kCacheAttnWarps; ++w) {
      const float a = ex2_approx(sm.end.m[w][r] - M);
      L = fmaf(sm.end.l[w][r], a, L);
      o0 = fmaf(sm.end.o[w][r][ch], a, o0);
      o1 = fmaf(sm.end.o[w][r][ch + 1], a, o1);
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const float lse = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994530942f;
    if (whole) {
      reinterpret_cast<uint32_t*>(p.o)[((out_row0 + r) * D + ch) / 2] = cache_pack<BF16>(o0 * inv, o1 * inv);
      if (ch == 0) p.lse[out_row0 + r] = lse;
    } else {
      const long long at = static_cast<long long>(part) * (8 * NT) + r;
      *reinterpret_cast<float2*>(p.part_o + at * D + ch) = make_float2(o0 * inv, o1 * inv);
      if (ch == 0) p.part_lse[at] = lse;
    }
  }
  __syncthreads();  // the end's memory is the rings' again
  }
}

// The units that several CTAs shared: O = sum_s w_s O_s / sum_s w_s over their
// parts, w_s = exp(LSE_s - max LSE).  kByUnit: a block per unit, its warps taking
// rows in turn (many units of few parts each); else a block per row, its warps
// sharing the parts (few units of many).  A block per row of 128 x 8 x 4 rows
// cost 6 us, mostly of finding the parts.
template <int D, bool BF16, int NT, bool kByUnit>
__global__ void __launch_bounds__(kCacheAttnThreads)
    fa_cache_merge_kernel(const CacheAttnParams p, int attn_grid) {
  __shared__ CacheScan scan;
  int b, hk, rb, r = 0;  // r: the row within the kv head's
  if constexpr (kByUnit) {
    const int units = p.Hkv * p.n_row_blocks;
    b = static_cast<int>(blockIdx.x) / units;
    const int unit = static_cast<int>(blockIdx.x) - b * units;
    hk = unit / p.n_row_blocks;
    rb = unit - hk * p.n_row_blocks;
  } else {
    const int bh = static_cast<int>(blockIdx.x / static_cast<unsigned>(p.rows));
    r = static_cast<int>(blockIdx.x) - bh * p.rows;
    b = bh / p.Hkv;
    hk = bh - b * p.Hkv;
    rb = r / (8 * NT);
  }
  int upto;
  const int all = cache_scan(p, scan, false, upto);
  const CacheDeal deal = cache_deal(all, attn_grid);
  // chunks per unit of the sequences before b: the thread with b in its run
  const int run = (p.B + kCacheAttnThreads - 1) / kCacheAttnThreads;
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
  auto merge = [&](int row, auto&& with) {
    with([&](int s) -> long long {
      return (2ll * (x0 + s) + (s == 0 ? inside : 0)) * (8 * NT) + row % (8 * NT);
    });
  };
  const int n_parts = x1 - x0 + 1;
  if constexpr (kByUnit) {
    const int end = min(p.rows, (rb + 1) * 8 * NT);
    for (int row = rb * 8 * NT + (static_cast<int>(threadIdx.x) >> 5); row < end; row += kMergeWarps)
      merge(row, [&](auto part_row) {
        merge_row_warp<D, BF16>(p.part_o, p.part_lse, n_parts, part_row, p.o, p.lse, row0 + row);
      });
  } else {
    __shared__ MergeSmem<D> sm;
    merge(r, [&](auto part_row) {
      merge_row<D, BF16>(p.part_o, p.part_lse, n_parts, part_row, p.o, p.lse, row0 + r, sm);
    });
  }
}

}  // namespace fa
