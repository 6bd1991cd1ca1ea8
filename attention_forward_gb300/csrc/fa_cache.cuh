// fa_cache.cuh -- the 4-bit key/value cache: write (quantise) and read back.
//
// A token's row of one kv head is D codes of 4 bits in groups of 32 channels
// with a scale s and a minimum z in fp16: value = s * code + z.
//   z = fp16(min x), s = fp16((max x - min x) / 15),
//   code = clamp(floor((x - z) / s + 1/2), 0, 15), 0 where s is 0.
// Word (D/32) * t + g of a row holds channels 32 g + 8 t ... + 7, lowest
// first, so that the attention's lane t finds its words of all groups side
// by side.
//
// Both kernels only move bytes (write: 4 D in, 2 (D/2 + D/8) out per token
// and head; read the reverse).  The read is bound by HBM: a thread takes 8
// channels of K and of V, a word each on the packed side and 16 bytes on the
// other, so that a row's lanes cover whole sectors on both.  The write is bound
// by its instructions (16 a value at first, most of them of the ALU pipe): a
// thread takes 16 channels, so that two lanes share a group's parameters.
// 32 x 8 heads of 4096 tokens, D = 128, 705 MB: write 144 us in bf16 (4.9 TB/s of
// 6.8), 126 in fp16, whose grid has fewer ties; read 112 us (6.3 TB/s), 108 in fp16.  With 8
// channels a lane, every tie and limit looked at in place: 218 us.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_cache.h"
#include "sm103_ptx.cuh"

namespace fa {

template <bool BF16>
__device__ __forceinline__ float2 cache_unpack(uint32_t w) {
  if constexpr (BF16) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
  } else {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
}

template <bool BF16>
__device__ __forceinline__ uint32_t cache_pack(float lo, float hi) {
  if constexpr (BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

// The pool's row of the token at position `pos` of sequence b, for kv head hk
// (pages, then heads, then slots); -1 when its place does not exist.  A
// position below 0 is past every page table as an unsigned number.
__device__ __forceinline__ long long cache_row(const CacheCopyParams& p, int b, int hk,
                                               uint32_t pos) {
  const uint32_t n = pos >> p.page_shift;
  if (n >= static_cast<uint32_t>(p.max_pages)) return -1;
  const int page = p.page_table[static_cast<size_t>(b) * p.max_pages + n];
  if (page < 0 || page >= p.num_pages) return -1;
  return ((static_cast<long long>(page) * p.Hkv + hk) << p.page_shift) +
         (pos & ((1u << p.page_shift) - 1u));
}

// min / max that a NaN goes through.
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float min3_nan(float a, float b, float c) {
  float d;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// The codes of a group are floor((x - z) / s + 1/2), decided exactly.  With
// d = x - z and inv = 1 / s, both rounded, q = d inv + 1.5 2^23 leaves the nearest
// integer c to d / s in the low bits of q, and r = d - c s is exact in one FMA
// (c s has 15 bits, and d is within a scale of it).  |r| < 0.499998 s says that c
// is the code wherever d is x - z to 2^-23.  A value beside a tie, a code outside
// 0 ... 15, a value past the limit, a NaN and s = 0 go to cache_codes_slow, as ties
// of bf16 values often do.

// The word of 8 channels when any of the group's lanes found such a value.  r >=
// s / 2, a tie that went down, adds one.  Only beside a tie can the bits that d
// lost decide: there the lane looks for them (two-sum), and with any of them goes
// through its channels with err, the lost part, added to r.
// (Out of line: its registers are not the kernel's.  A template, for the linker.)
template <int kUnused = 0>
__device__ __noinline__ uint32_t cache_codes_slow(float x0, float x1, float x2, float x3, float x4,
                                                  float x5, float x6, float x7, float z, float s) {
  const float x[8] = {x0, x1, x2, x3, x4, x5, x6, x7};
  constexpr float kMagic = 12582912.f;  // 1.5 2^23
  if (s == 0.f) return 0u;
  const float inv = __fdividef(1.f, s);  // q may miss by one: r shows it
  const float half_s = 0.5f * s;
  float far = 0.f;
  uint32_t word = 0u;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float d = x[e] - z;
    float q = fmaf(d, inv, kMagic);
    const float r = fmaf(-(q - kMagic), s, d);
    far = fmaxf(far, fabsf(r));
    q += r >= half_s ? 1.f : 0.f;
    // each q's bits are the magic's and the code: the magic's share of the
    // sum is taken off below
    word += __float_as_uint(fminf(fmaxf(q, kMagic), kMagic + 15.f)) << (4 * e);
  }
  constexpr uint32_t kMagicBits = 0x4b400000u;
  word -= kMagicBits * 0x11111111u;
  if (!(far < s * 0.499998f)) {  // a tie or next to one, or a value past the limit
    bool lost = !(far <= half_s);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float d = x[e] - z, bb = d - x[e];
      lost |= (x[e] - (d - bb)) + (-z - bb) != 0.f;
    }
    if (lost) {
      word = 0u;
#pragma unroll 1
      for (int e = 0; e < 8; ++e) {
        float v = x[0];
#pragma unroll
        for (int k = 1; k < 8; ++k) v = e == k ? x[k] : v;
        v = fminf(fmaxf(v, -kCacheLimit), kCacheLimit);
        const float d = v - z;
        const float bb = d - v;
        const float err = (v - (d - bb)) + (-z - bb);
        float c = rintf(d * inv);
        const float r = fmaf(-c, s, d);
        if ((r - half_s) + err >= 0.f) c += 1.f;
        if ((r + half_s) + err < 0.f) c -= 1.f;
        word |= static_cast<uint32_t>(fminf(fmaxf(c, 0.f), 15.f)) << (4 * e);
      }
    }
  }
  return word;
}

// (scale, minimum) of the values lo ... hi.
__device__ __forceinline__ void cache_params(float lo, float hi, __half& sh, __half& zh) {
  zh = __float2half_rn(lo);
  // (hi - lo) / 15, correctly rounded: a product by 1/15 and its residual
  const float range = hi - lo, near15 = range * (1.f / 15.f);
  sh = __float2half_rn(fmaf(fmaf(-15.f, near15, range), 1.f / 15.f, near15));
}

// One group's codes from 16 of its channels per lane (the 2 lanes of a pair hold
// the group): the two words of codes and the (scale, minimum) pair.  What takes a
// group's time is the ALU pipe (minima, maxima, comparisons, shifts), so codes
// are put together by FMAs, c0 + 16 c1 + 256 c2 + 4096 c3 at a time, exactly.
__device__ __forceinline__ void cache_quantise(const float (&x)[2][8], uint32_t (&word)[2],
                                               uint32_t& param) {
  constexpr float kMagic = 12582912.f;  // 1.5 2^23
  float lo = x[0][0], hi = x[0][0];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      lo = min3_nan(lo, x[h][e], x[h][e + 1]);
      hi = fmax3(hi, x[h][e], x[h][e + 1]);
    }
  }
  lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, 1));
  hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, 1));
  __half sh, zh;
  cache_params(lo, hi, sh, zh);
  float z = __half2float(zh), s = __half2float(sh);
  const float inv = __fdividef(1.f, s);
  // both words at once, in packed pairs
  float far[2] = {0.f, 0.f}, sum[2][2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float c[4][2], r[4][2];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float d0, d1;
      fadd2(d0, d1, x[0][4 * k + e], x[1][4 * k + e], -z, -z);
      ffma2(c[e][0], c[e][1], d0, d1, inv, inv, kMagic, kMagic);
      fadd2(c[e][0], c[e][1], c[e][0], c[e][1], -kMagic, -kMagic);
      ffma2(r[e][0], r[e][1], c[e][0], c[e][1], -s, -s, d0, d1);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      far[h] = fmax3(far[h], fabsf(r[0][h]), fabsf(r[1][h]));
      far[h] = fmax3(far[h], fabsf(r[2][h]), fabsf(r[3][h]));
    }
    fadd2(sum[k][0], sum[k][1], c[0][0], c[0][1], 8388608.f, 8388608.f);
    ffma2(sum[k][0], sum[k][1], c[1][0], c[1][1], 16.f, 16.f, sum[k][0], sum[k][1]);
    ffma2(sum[k][0], sum[k][1], c[2][0], c[2][1], 256.f, 256.f, sum[k][0], sum[k][1]);
    ffma2(sum[k][0], sum[k][1], c[3][0], c[3][1], 4096.f, 4096.f, sum[k][0], sum[k][1]);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)  // 2^23 + 16 bits of codes each
    word[h] = __byte_perm(__float_as_uint(sum[0][h]), __float_as_uint(sum[1][h]), 0x5410);
  param = static_cast<uint32_t>(__half_as_ushort(sh)) |
          (static_cast<uint32_t>(__half_as_ushort(zh)) << 16);
  // the extremes' codes are within 0 ... 15 (a NaN fails every comparison)
  const bool plain = lo - z > -0.49f * s && hi - z < 15.49f * s && lo >= -kCacheLimit &&
                     hi <= kCacheLimit;
  if (!plain) {
    if (lo != lo) {  // a NaN makes its whole group NaN: the parameters carry it
      word[0] = word[1] = 0u;
      param = 0x7fff7fffu;
      return;
    }
    // values past the limit take the codes at the ends
    cache_params(fminf(fmaxf(lo, -kCacheLimit), kCacheLimit),
                 fminf(fmaxf(hi, -kCacheLimit), kCacheLimit), sh, zh);
    z = __half2float(zh);
    s = __half2float(sh);
#pragma unroll
    for (int h = 0; h < 2; ++h)
      word[h] = cache_codes_slow<>(x[h][0], x[h][1], x[h][2], x[h][3], x[h][4], x[h][5], x[h][6],
                                 x[h][7], z, s);
    param = static_cast<uint32_t>(__half_as_ushort(sh)) |
            (static_cast<uint32_t>(__half_as_ushort(zh)) << 16);
    return;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (!(far[h] < s * 0.499998f))
      word[h] = cache_codes_slow<>(x[h][0], x[h][1], x[h][2], x[h][3], x[h][4], x[h][5], x[h][6],
                                 x[h][7], z, s);
}

// Two codes at a time are cut out as fp16 pairs (channels e, e + 4): a code
// masked into the low or high nibble of a fp16 mantissa is 1024 or 64 too large.
__device__ __forceinline__ __half2 cache_code_pair(uint32_t word, int e) {
  const uint32_t w = e & 2 ? word >> 8 : word;
  const uint32_t bits = e & 1 ? (w & 0x00f000f0u) | 0x54005400u : (w & 0x000f000fu) | 0x64006400u;
  return __hsub2(*reinterpret_cast<const __half2*>(&bits), __float2half2_rn(e & 1 ? 64.f : 1024.f));
}

// Pairs (e, e + 4) in the order of their channels.
__device__ __forceinline__ uint4 cache_in_order(const uint32_t (&v)[4]) {
  return make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                    __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632));
}

// c s + z rounded to odd: rounded again to bf16, that is c s + z rounded once,
// where rounding it to nearest first could make a tie of it.
__device__ __forceinline__ float fma_odd(float c, float s, float z) {
  const float lo = __fmaf_rd(c, s, z), hi = __fmaf_ru(c, s, z);
  return (__float_as_uint(lo) & 1u) ? lo : hi;
}

// cache_values in bf16 where fp32 does not hold the sums.  (Out of line: its
// registers are not the kernel's.  A template, for the linker.)
template <int kUnused = 0>
__device__ __noinline__ uint4 cache_values_odd(uint32_t word, float s, float z) {
  uint32_t v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __half2 c = cache_code_pair(word, e);
    v[e] = cache_pack<true>(fma_odd(__low2float(c), s, z), fma_odd(__high2float(c), s, z));
  }
  return cache_in_order(v);
}

// The 8 values of a word, rounded once to 16 bits, in the order of their
// channels.
template <bool BF16>
__device__ __forceinline__ uint4 cache_values(uint32_t word, uint32_t param) {
  const __half2 sz = *reinterpret_cast<const __half2*>(&param);
  uint32_t v[4];  // channels (e, e + 4)
  if constexpr (BF16) {
    const float s = __low2float(sz), z = __high2float(sz);
    // c s + z is exact in fp32 where its last place, at least 2^-11 of the smaller
    // of s and |z|, is within 2^-23 of |z| + 16 s: nearly always (705 MB in 112 us;
    // 121 with every group by fma_odd, 114 with both in line, 110 rounding twice)
    if (fminf(s, fabsf(z)) * 4096.f < fmaf(16.f, s, fabsf(z))) return cache_values_odd<>(word, s, z);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __half2 c = cache_code_pair(word, e);
      v[e] = cache_pack<true>(fmaf(__low2float(c), s, z), fmaf(__high2float(c), s, z));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __half2 r = __hfma2(cache_code_pair(word, e), __low2half2(sz), __high2half2(sz));
      v[e] = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
  return cache_in_order(v);
}

// Rows per block: the lanes of a row lie side by side.  blockIdx.y is the
// (sequence, kv head), blockIdx.x the block of its tokens.  A write thread takes 4
// tokens one after the other, which spreads its 64-bit addresses (us for the 705
// MB: 1 token 181, 2 162, 4 154, 8 151 with a longer tail where tokens are few),
// 8 blocks an SM (64 registers; 144 us, 7 blocks 152, 10 151).  A read thread takes
// 2, whose loads go out together (1 ... 8 measured within 6 %).
constexpr int kCacheCopyThreads = 128;
constexpr int kCacheWriteTurns = 4, kCacheReadTurns = 2, kCacheWriteBlocks = 8;

template <int D>
constexpr int kCacheWriteRows = kCacheCopyThreads / (D / 16);
template <int D>
constexpr int kCacheReadRows = kCacheCopyThreads / (D / 8);

template <int D, bool BF16>
__global__ void __launch_bounds__(kCacheCopyThreads, kCacheWriteBlocks)
    fa_cache_write_kernel(const CacheCopyParams p) {
  constexpr int kLanes = D / 16, kGroups = D / kCacheGroup, kRows = kCacheWriteRows<D>;
  constexpr int kTurns = kCacheWriteTurns;
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = static_cast<int>(threadIdx.x) % kLanes;  // channels 16 lane ... + 15
  const int bh = static_cast<int>(blockIdx.y);
  const int b = bh / p.Hkv, hk = bh - b * p.Hkv;
  const int first = static_cast<int>(blockIdx.x) * kRows * kTurns;
  const int start = p.start ? p.start[b] : 0;
  const int count = p.count ? min(p.count[b], p.S) : p.S;
  if (first >= count) return;
  const int g = lane >> 1, t = 2 * (lane & 1);
  const uint4* in[2];
  uint32_t *codes[2], *params[2];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    in[n] = reinterpret_cast<const uint4*>(p.rows[n]) + static_cast<size_t>(bh) * p.S * (2 * kLanes) +
            2 * lane;
    codes[n] = reinterpret_cast<uint32_t*>(p.pool.codes[n]) + kGroups * t + g;
    params[n] = p.pool.params[n] + g;
  }

#pragma unroll 1
  for (int i = first + static_cast<int>(threadIdx.x) / kLanes, end = min(first + kRows * kTurns, count);
       __any_sync(0xffffffffu, i < end); i += kRows) {
    uint4 w[2][2];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        w[n][h] = i < end ? __ldcs(in[n] + static_cast<size_t>(i) * (2 * kLanes) + h)
                          : make_uint4(0u, 0u, 0u, 0u);
    const long long row =
        i < end ? cache_row(p, b, hk, static_cast<uint32_t>(start) + static_cast<uint32_t>(i)) : -1;
    if (i < end && row < 0 && lane == 0) atomicMax(p.status, kStatusBadIndex);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      float x[2][8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float2 a = cache_unpack<BF16>(w[n][h].x), b2 = cache_unpack<BF16>(w[n][h].y);
        const float2 c = cache_unpack<BF16>(w[n][h].z), d = cache_unpack<BF16>(w[n][h].w);
        x[h][0] = a.x; x[h][1] = a.y; x[h][2] = b2.x; x[h][3] = b2.y;
        x[h][4] = c.x; x[h][5] = c.y; x[h][6] = d.x; x[h][7] = d.y;
      }
      uint32_t word[2], param;
      cache_quantise(x, word, param);
      if (row >= 0) {
        codes[n][row * (D / 8)] = word[0];
        codes[n][row * (D / 8) + kGroups] = word[1];
        if (t == 0) params[n][row * kGroups] = param;
      }
    }
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kCacheCopyThreads) fa_cache_read_kernel(const CacheCopyParams p) {
  constexpr int kLanes = D / 8, kGroups = D / kCacheGroup, kRows = kCacheReadRows<D>;
  constexpr int kTurns = kCacheReadTurns;
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = static_cast<int>(threadIdx.x) % kLanes;  // channels 8 lane ... + 7
  const int bh = static_cast<int>(blockIdx.y);
  const int b = bh / p.Hkv, hk = bh - b * p.Hkv;
  const int start = p.start ? p.start[b] : 0;
  const int count = p.count ? min(p.count[b], p.S) : p.S;
  const int i0 = static_cast<int>(blockIdx.x) * kRows * kTurns +
                 static_cast<int>(threadIdx.x) / kLanes;
  if (i0 >= count) return;
  const int g = lane >> 2, t = lane & 3;

  uint32_t word[kTurns][2], param[kTurns][2];
#pragma unroll
  for (int k = 0; k < kTurns; ++k) {
    const int i = i0 + k * kRows;
    const long long row =
        i < count ? cache_row(p, b, hk, static_cast<uint32_t>(start) + static_cast<uint32_t>(i)) : -1;
    if (i < count && row < 0 && lane == 0) atomicMax(p.status, kStatusBadIndex);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      word[k][n] = param[k][n] = 0u;  // a place that does not exist reads as zeros
      if (row >= 0) {
        // from L2: the kernel may have started while the write before it ran
        word[k][n] = __ldcg(reinterpret_cast<const uint32_t*>(p.pool.codes[n]) + row * kLanes +
                            kGroups * t + g);
        param[k][n] = __ldcg(p.pool.params[n] + row * kGroups + g);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kTurns; ++k) {
    const int i = i0 + k * kRows;
    if (i >= count) return;
#pragma unroll
    for (int n = 0; n < 2; ++n)
      reinterpret_cast<uint4*>(p.rows[n])[(static_cast<size_t>(bh) * p.S + i) * kLanes + lane] =
          cache_values<BF16>(word[k][n], param[k][n]);
  }
}

}  // namespace fa
