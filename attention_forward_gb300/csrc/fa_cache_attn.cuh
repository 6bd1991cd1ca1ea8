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
//     [2^13, 2^14) (bf16 queries become fp16 exactly), times 2^-4 opposite the
//     2^-20 codes.  A group's 32 channels are two such products; its scale
//     multiplies their fp32 sums.  The minima come from one more product:
//     A = the stored (scale, minimum) pairs, B = (0, sum of the group's query
//     channels), that sum in two fp16 parts.  The scores lose nothing to
//     rounding before the fp32 sums.
//   softmax: fp32, log2 domain, one reference maximum per row, raised when a
//     score passes it by 15: p = 2^(t - m) <= 2^15 with m set 8 below the
//     maximum, so that fp16 holds p over 2^-24 ... 2^15 around it.
//   output, channels x rows: A = the values, dequantised to fp16 pairs of two
//     tokens ((1024 + c) - 1024 or (64 + c) - 64, then one fma with scale and
//     minimum: a rounding of 2^-11 of the value, an eighth of bf16's), B = p
//     in fp16 (2^-11), turned from the score layout by movmatrix.
//
// Codes and parameters go from global memory straight to the registers of the
// lane that needs them: lane (g, t) = (lane / 4, lane % 4) reads the 16 bytes
// of keys g and g + 8 that hold its channels 8 t ... 8 t + 7 of every group, and
// the words 2 g, 2 g + 1 of its four value tokens.  Every warp's loads cover
// whole sectors; the next 16 keys' loads are in flight while these are
// computed.  At the end the warps' states merge in shared memory and the CTA
// writes O and LSE, or the split's partials for the combine kernel.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_cache.h"
#include "fa_cache.cuh"
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

// Transpose of an 8 x 8 matrix of 16-bit elements held two per lane.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ uint4 ldg_stream(const uint4* p) {
  uint4 v;
  asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
      : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ldg_stream(const uint2* p) {
  uint2 v;
  asm("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ldg_stream(const uint32_t* p) {
  uint32_t v;
  asm("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

__device__ __forceinline__ __half2 as_half2(uint32_t w) { return *reinterpret_cast<__half2*>(&w); }
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// (a & mask) | bits in one instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t bits) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(a), "r"(mask), "r"(bits));
  return d;
}

// cap tanh(x / cap): for |y| = |x / cap| < 1/4 the odd series through y^7 (its
// next term is 3e-7 of the value), else 1 - 2 / (1 + e^(2 y)), which is off by
// a few 2^-24 of the cap and saturates to +-cap as the exponential reaches
// infinity or 0.
__device__ __forceinline__ float cap_score(float x, const CacheAttnParams& p) {
  const float y = x * p.inv_cap, u = y * y;
  const float small = fmaf(u, fmaf(u, fmaf(u, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f), 1.f) * x;
  const float e = ex2_approx(x * p.cap_arg);
  const float large = fmaf(-2.f * p.cap, __fdividef(1.f, 1.f + e), p.cap);
  return u < 0.0625f ? small : large;
}

// What a lane holds of 16 keys.
template <int D>
struct CacheTile {
  static constexpr int G = D / kCacheGroup;
  uint32_t kc[2][G];   // keys g, g + 8: channels 8 t ... of every group
  uint32_t kp[2][G];   // their (scale, minimum) pairs
  uint32_t vc[4][D / 64];  // tokens 2 t, 2 t + 1, 2 t + 8, 2 t + 9: words of lane g
  uint32_t vp[4][D / 64];  // the pairs of those words' groups
};

template <int D>
__device__ __forceinline__ void load_tile(CacheTile<D>& x, const CacheAttnParams& p,
                                          long long row0, int g, int t) {
  constexpr int G = D / kCacheGroup;
  const uint32_t* kc = reinterpret_cast<const uint32_t*>(p.pool.codes[0]);
  const uint32_t* vc = reinterpret_cast<const uint32_t*>(p.pool.codes[1]);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const long long row = row0 + g + 8 * i;
    if constexpr (D == 128) {
      const uint4 c = ldg_stream(reinterpret_cast<const uint4*>(kc + row * (D / 8) + G * t));
      const uint4 s = ldg_stream(reinterpret_cast<const uint4*>(p.pool.params[0] + row * G));
      x.kc[i][0] = c.x; x.kc[i][1] = c.y; x.kc[i][2] = c.z; x.kc[i][3] = c.w;
      x.kp[i][0] = s.x; x.kp[i][1] = s.y; x.kp[i][2] = s.z; x.kp[i][3] = s.w;
    } else {
      const uint2 c = ldg_stream(reinterpret_cast<const uint2*>(kc + row * (D / 8) + G * t));
      const uint2 s = ldg_stream(reinterpret_cast<const uint2*>(p.pool.params[0] + row * G));
      x.kc[i][0] = c.x; x.kc[i][1] = c.y;
      x.kp[i][0] = s.x; x.kp[i][1] = s.y;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long row = row0 + 2 * t + (i & 1) + 8 * (i >> 1);
    if constexpr (D == 128) {  // words 2 g, 2 g + 1: groups 2 (g & 1), 2 (g & 1) + 1
      const uint2 c = ldg_stream(reinterpret_cast<const uint2*>(vc + row * (D / 8) + 2 * g));
      const uint2 s = ldg_stream(reinterpret_cast<const uint2*>(p.pool.params[1] + row * G + 2 * (g & 1)));
      x.vc[i][0] = c.x; x.vc[i][1] = c.y;
      x.vp[i][0] = s.x; x.vp[i][1] = s.y;
    } else {  // word g: group g & 1
      x.vc[i][0] = ldg_stream(vc + row * (D / 8) + g);
      x.vp[i][0] = ldg_stream(p.pool.params[1] + row * G + (g & 1));
    }
  }
}

template <int D, int NT>
struct CacheAttnSmem {
  // per warp: reference maximum and sum of each row, then O by (row, channel);
  // a row's D channels are followed by one pad word
  static constexpr int kRows = 8 * NT;
  static constexpr int kRowFloats = D + 1;
  float m[kCacheAttnWarps][kRows];
  float l[kCacheAttnWarps][kRows];
  float o[kCacheAttnWarps][kRows][kRowFloats];
  int pages[kCacheAttnMaxKeys / 16];
};

// p.n_splits ranges x p.n_row_blocks x (B * Hkv), row blocks fastest (they
// read the same keys).
template <int D, bool BF16, int NT>
__global__ void __launch_bounds__(kCacheAttnWarps * 32, NT == 1 ? 4 : 3)
    fa_cache_attn_kernel(const CacheAttnParams p) {
  constexpr int G = D / kCacheGroup;
  constexpr int kWords = D / 64;   // value words per lane and token
  constexpr int kMmas = D / 16;    // output products: 8 per value word pair
  constexpr float kLog2e = 1.4426950408889634f;
  constexpr float kBelow = 8.f, kTau = 15.f;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  CacheAttnSmem<D, NT>& sm = *reinterpret_cast<CacheAttnSmem<D, NT>*>(smem_raw);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  int id = static_cast<int>(blockIdx.x);
  const int rb = id % p.n_row_blocks;
  id /= p.n_row_blocks;
  const int split = id % p.n_splits;
  const int bh = id / p.n_splits;
  const int b = bh / p.Hkv, hk = bh - b * p.Hkv;
  const int row0 = rb * 8 * NT;
  const long long total_rows = static_cast<long long>(p.B) * p.H * p.Sq;
  const long long out_row0 = static_cast<long long>(bh) * p.rows + row0;
  const int n_rows = min(8 * NT, p.rows - row0);

  const int len_raw = p.length[b];
  const int len = max(0, min(len_raw, p.max_length));  // max_length <= max_pages * page_size
  if (len != len_raw && threadIdx.x == 0) atomicExch(p.status, kStatusBadIndex);
  const int k_begin = min(len, split * p.keys_per_split);  // both below 2^25
  const int k_end = min(len, k_begin + p.keys_per_split);

  // this range's pages, by 16-key tile: the first row of the tile's 16 slots
  // as a page number; -1 marks a page that does not exist
  const int n_tiles = (k_end - k_begin + 15) >> 4;
  for (int i = threadIdx.x; i < n_tiles; i += kCacheAttnWarps * 32) {
    const int pg = p.page_table[static_cast<long long>(b) * p.max_pages + ((k_begin + 16 * i) >> p.page_shift)];
    const bool bad = pg < 0 || pg >= p.num_pages;
    if (bad) atomicExch(p.status, kStatusBadIndex);
    sm.pages[i] = bad ? -1 : pg;
  }

  // ---- the query rows: B operands, and per-row constants of the columns
  // this lane's accumulators hold (rows 2 t, 2 t + 1 of each block of 8)
  uint32_t qb[NT][G][4];   // [group][product 0: b0, b1; product 1: b0, b1]
  uint32_t qs[NT][2];      // (0, sum) of group t: high part, low part
  float fac[NT][2];        // score = 2^24 (the codes') * sum * fac
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
    // up = 2^e with top * up in [2^13, 2^14); its exponent stays within what
    // one float holds for every finite row (an all-zero row takes 1)
    int e2 = top > 0.f && top < INFINITY ? 13 - ilogbf(top) : 0;
    e2 = min(max(e2, -120), 120);
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
    const float down = __int_as_float((127 - e2) << 23);  // 1 / up
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int rc = 8 * n + 2 * t + c;
      fac[n][c] = __shfl_sync(0xffffffffu, down, (2 * t + c) * 4) * p.scale;
      const int rr = min(rc, n_rows - 1) + row0;
      const int h = hk * (p.H / p.Hkv) + rr / p.Sq, i = rr % p.Sq;
      slope[n][c] = p.slopes ? p.slopes[h] * kLog2e : 0.f;
      limit[n][c] = rc < n_rows ? len - (p.Sq - 1 - i) : 0;
      m[n][c] = -INFINITY;
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
  __syncthreads();
  grid_launch_dependents();  // the merge waits for this grid's end

  const int slot_mask = (1 << p.page_shift) - 1;
  // the first pool row of a 16-key tile, or -1
  auto tile_row = [&](int i) -> long long {
    if (i >= n_tiles) return -1;
    const int pg = sm.pages[i];
    if (pg < 0) return -1;
    return ((static_cast<long long>(pg) * p.Hkv + hk) << p.page_shift) + ((k_begin + 16 * i) & slot_mask);
  };

  CacheTile<D> next;
  long long next_row = tile_row(warp);
  if (next_row >= 0) load_tile<D>(next, p, next_row, g, t);
#pragma unroll 1
  for (int i = warp; i < n_tiles; i += kCacheAttnWarps) {
    CacheTile<D> x = next;
    const bool have = next_row >= 0;
    next_row = tile_row(i + kCacheAttnWarps);
    if (next_row >= 0) load_tile<D>(next, p, next_row, g, t);
    if (!have) continue;
    const int key0 = k_begin + 16 * i;

    // ------------------------------ scores ------------------------------
    float s[NT][4];
    {
      uint32_t z0 = x.kp[0][0], z1 = x.kp[1][0];
#pragma unroll
      for (int gr = 1; gr < G; ++gr) {
        z0 = t == gr ? x.kp[0][gr] : z0;
        z1 = t == gr ? x.kp[1][gr] : z1;
      }
      if (G < 4 && t >= G) z0 = z1 = 0u;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float z[4] = {0.f, 0.f, 0.f, 0.f};
        mma_f16(z, z0, z1, z0, z1, qs[n][0], qs[n][1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = z[e] * 1.52587890625e-5f;  // 2^8 / 2^24
      }
    }
#pragma unroll
    for (int gr = 0; gr < G; ++gr) {
      const uint32_t w0 = x.kc[0][gr], w1 = x.kc[1][gr];
      const uint32_t y0 = w0 >> 8, y1 = w1 >> 8;
      const float s0 = __low2float(as_half2(x.kp[0][gr])), s1 = __low2float(as_half2(x.kp[1][gr]));
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        mma_f16(d, w0 & 0x000f000fu, w1 & 0x000f000fu, w0 & 0x00f000f0u, w1 & 0x00f000f0u,
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
      bool over = false;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = e & 1, key = key0 + g + 8 * (e >> 1);
        float v = (s[n][e] * 16777216.f) * fac[n][c];
        if (p.cap > 0.f) v = cap_score(v, p);
        v *= kLog2e;
        if (p.slopes) v = fmaf(-slope[n][c], static_cast<float>(abs(limit[n][c] - 1 - key)), v);
        v = key < limit[n][c] ? v : -INFINITY;
        s[n][e] = v;
        over |= v > m[n][c] + kTau;
      }
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
        const float mm = m[n][e & 1];
        pr[e] = ex2_approx(s[n][e] - (mm == -INFINITY ? 0.f : mm));
        l[n][e & 1] += pr[e];
      }
      pb[n][0] = movmatrix_trans(as_u32(__floats2half2_rn(pr[0], pr[1])));
      pb[n][1] = movmatrix_trans(as_u32(__floats2half2_rn(pr[2], pr[3])));
    }

    // ------------------------------ output ------------------------------
    if (key0 + 16 > len) {  // slots past the sequence may hold anything
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (key0 + 2 * t + (k & 1) + 8 * (k >> 1) >= len)
#pragma unroll
          for (int w = 0; w < kWords; ++w) x.vp[k][w] = 0u;
    }
    // registers of half a word's channels (4 of 8) for both token pairs:
    // a[pair][channel]
    auto dequant = [&](int w, int half, uint32_t (&a)[2][4]) {
#pragma unroll
      for (int pr2 = 0; pr2 < 2; ++pr2) {
        const uint32_t c01 = __byte_perm(x.vc[2 * pr2][w], x.vc[2 * pr2 + 1][w], half ? 0x7632 : 0x5410);
        const __half2 sc = as_half2(__byte_perm(x.vp[2 * pr2][w], x.vp[2 * pr2 + 1][w], 0x5410));
        const __half2 mn = as_half2(__byte_perm(x.vp[2 * pr2][w], x.vp[2 * pr2 + 1][w], 0x7632));
        const uint32_t y = c01 >> 8;
        const __half2 k1024 = as_half2(0x64006400u), k64 = as_half2(0x54005400u);
        const __half2 h0 = __hsub2(as_half2(and_or(c01, 0x000f000fu, 0x64006400u)), k1024);
        const __half2 h1 = __hsub2(as_half2(and_or(c01, 0x00f000f0u, 0x54005400u)), k64);
        const __half2 h2 = __hsub2(as_half2(and_or(y, 0x000f000fu, 0x64006400u)), k1024);
        const __half2 h3 = __hsub2(as_half2(and_or(y, 0x00f000f0u, 0x54005400u)), k64);
        a[pr2][0] = as_u32(__hfma2(h0, sc, mn));
        a[pr2][1] = as_u32(__hfma2(h1, sc, mn));
        a[pr2][2] = as_u32(__hfma2(h2, sc, mn));
        a[pr2][3] = as_u32(__hfma2(h3, sc, mn));
      }
    };
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t a0[2][4], a1[2][4];
      dequant(0, half, a0);
      if constexpr (D == 128) {
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
  }

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
        sm.m[warp][r] = m[n][c];
        sm.l[warp][r] = sum;
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
          sm.o[warp][r][ch] = acc[n][k][2 * e + c];
        }
    }
  __syncthreads();
  // two channels per thread, rows in turn
  constexpr int kPer = D / 2;
  for (int i = threadIdx.x; i < n_rows * kPer; i += kCacheAttnWarps * 32) {
    const int r = i / kPer, ch = 2 * (i - r * kPer);
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kCacheAttnWarps; ++w) M = fmaxf(M, sm.m[w][r]);
    const float mu = M == -INFINITY ? 0.f : M;
    float L = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
    for (int w = 0; w < kCacheAttnWarps; ++w) {
      const float a = ex2_approx(sm.m[w][r] - mu);
      L = fmaf(sm.l[w][r], a, L);
      o0 = fmaf(sm.o[w][r][ch], a, o0);
      o1 = fmaf(sm.o[w][r][ch + 1], a, o1);
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const float lse = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994530942f;
    if (p.n_splits == 1) {
      reinterpret_cast<uint32_t*>(p.o)[((out_row0 + r) * D + ch) / 2] = cache_pack<BF16>(o0 * inv, o1 * inv);
      if (ch == 0) p.lse[out_row0 + r] = lse;
    } else {
      const long long at = static_cast<long long>(split) * total_rows + out_row0 + r;
      *reinterpret_cast<float2*>(p.part_o + at * D + ch) = make_float2(o0 * inv, o1 * inv);
      if (ch == 0) p.part_lse[at] = lse;
    }
  }
}

}  // namespace fa
