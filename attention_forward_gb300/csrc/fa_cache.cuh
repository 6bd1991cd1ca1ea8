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
// and head; read the reverse) and are bound by HBM: one thread takes 8
// channels of K and of V, 16 bytes each on the 16-bit side and a word each on
// the packed side, so that a row's lanes cover whole sectors on both.
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

// One group's codes from 8 of its channels per lane (4 lanes of a quad hold
// the group): the word of codes and the (scale, minimum) pair.
//
// A code is floor((x - z) / s + 1/2), decided exactly.  q = d inv + 1.5 2^23
// leaves the nearest integer c to d / s (d = x - z, inv = 1 / s, both
// rounded) in the low bits of q, and r = d - c s is exact in one FMA (c s has
// 15 bits, and d is within a scale of it); r >= s / 2 (a tie that went down)
// adds one.  That is the code wherever d is x - z exactly, as it is unless x
// has bits 2^24 below z.  Only beside a tie can the lost bits decide: there
// the lane looks for them (two-sum), and with any of them goes through its
// channels with err, the lost part, added to r.
__device__ __forceinline__ void cache_quantise(const float (&x)[8], uint32_t& word,
                                               uint32_t& param) {
  constexpr float kMagic = 12582912.f;  // 1.5 2^23
  float lo = min3_nan(x[0], x[1], x[2]), hi = fmax3(x[0], x[1], x[2]);
  lo = min3_nan(lo, x[3], x[4]);
  hi = fmax3(hi, x[3], x[4]);
  lo = min3_nan(lo, x[5], x[6]);
  hi = fmax3(hi, x[5], x[6]);
  lo = min_nan(lo, x[7]);
  hi = fmaxf(hi, x[7]);
#pragma unroll
  for (int m = 1; m <= 2; m <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, m));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
  }
  if (lo != lo) {  // a NaN makes its whole group NaN: the parameters carry it
    word = 0u;
    param = 0x7fff7fffu;
    return;
  }
  // values past the limit take the codes at the ends
  lo = fminf(fmaxf(lo, -kCacheLimit), kCacheLimit);
  hi = fminf(fmaxf(hi, -kCacheLimit), kCacheLimit);
  const __half zh = __float2half_rn(lo);
  // (hi - lo) / 15, correctly rounded: a product by 1/15 and its residual
  const float range = hi - lo, near15 = range * (1.f / 15.f);
  const __half sh = __float2half_rn(fmaf(fmaf(-15.f, near15, range), 1.f / 15.f, near15));
  param = static_cast<uint32_t>(__half_as_ushort(sh)) |
          (static_cast<uint32_t>(__half_as_ushort(zh)) << 16);
  const float z = __half2float(zh), s = __half2float(sh);
  if (s == 0.f) {
    word = 0u;
    return;
  }
  const float inv = __fdividef(1.f, s);  // q may miss by one: r shows it
  const float half_s = 0.5f * s;
  float far = 0.f;
  word = 0u;
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
}

// The 8 values of a word, rounded once to 16 bits, in the order of their
// channels.  Two codes at a time are cut out as fp16 pairs (channels e, e + 4):
// a code masked into the low or high nibble of a fp16 mantissa is 1024 or 64
// too large.
template <bool BF16>
__device__ __forceinline__ uint4 cache_values(uint32_t word, uint32_t param) {
  const __half2 sz = *reinterpret_cast<const __half2*>(&param);
  const uint32_t y = word >> 8;
  const uint32_t bits[4] = {(word & 0x000f000fu) | 0x64006400u, (word & 0x00f000f0u) | 0x54005400u,
                            (y & 0x000f000fu) | 0x64006400u, (y & 0x00f000f0u) | 0x54005400u};
  uint32_t v[4];  // channels (e, e + 4)
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __half2 c = __hsub2(*reinterpret_cast<const __half2*>(&bits[e]),
                              __float2half2_rn(e & 1 ? 64.f : 1024.f));
    if constexpr (BF16) {
      const float s = __low2float(sz), z = __high2float(sz);
      v[e] = cache_pack<true>(fmaf(__low2float(c), s, z), fmaf(__high2float(c), s, z));
    } else {
      const __half2 r = __hfma2(c, __low2half2(sz), __high2half2(sz));
      v[e] = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
  return make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                    __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632));
}

// Rows per block: the lanes of a row lie side by side.  blockIdx.y is the
// (sequence, kv head), blockIdx.x the block of its tokens; a thread takes
// a few tokens in turn, whose loads go out together.
constexpr int kCacheCopyThreads = 128;
constexpr int kCacheWriteTurns = 2, kCacheReadTurns = 2;  // 1 ... 8 measured within 6 %

template <int D>
constexpr int kCacheCopyRows = kCacheCopyThreads / (D / 8);

template <int D, bool BF16>
__global__ void __launch_bounds__(kCacheCopyThreads) fa_cache_write_kernel(const CacheCopyParams p) {
  constexpr int kLanes = D / 8, kGroups = D / kCacheGroup, kRows = kCacheCopyRows<D>;
  constexpr int kTurns = kCacheWriteTurns;
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = static_cast<int>(threadIdx.x) % kLanes;  // channels 8 lane ... + 7
  const int bh = static_cast<int>(blockIdx.y);
  const int b = bh / p.Hkv, hk = bh - b * p.Hkv;
  const int first = static_cast<int>(blockIdx.x) * kRows * kTurns;
  const int start = p.start ? p.start[b] : 0;
  const int count = p.count ? min(p.count[b], p.S) : p.S;
  if (first >= count) return;
  const int i0 = first + static_cast<int>(threadIdx.x) / kLanes;
  const int g = lane >> 2, t = lane & 3;

  uint4 w[kTurns][2];
  long long row[kTurns];
#pragma unroll
  for (int k = 0; k < kTurns; ++k) {
    const int i = i0 + k * kRows;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      w[k][n] = make_uint4(0u, 0u, 0u, 0u);
      if (i < count)
        w[k][n] = __ldcs(reinterpret_cast<const uint4*>(p.rows[n]) +
                         (static_cast<size_t>(bh) * p.S + i) * kLanes + lane);
    }
    row[k] = i < count ? cache_row(p, b, hk, static_cast<uint32_t>(start) + static_cast<uint32_t>(i)) : -1;
    if (i < count && row[k] < 0 && lane == 0) atomicExch(p.status, kStatusBadIndex);
  }
#pragma unroll
  for (int k = 0; k < kTurns; ++k) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const float2 a = cache_unpack<BF16>(w[k][n].x), b2 = cache_unpack<BF16>(w[k][n].y);
      const float2 c = cache_unpack<BF16>(w[k][n].z), d = cache_unpack<BF16>(w[k][n].w);
      const float x[8] = {a.x, a.y, b2.x, b2.y, c.x, c.y, d.x, d.y};
      uint32_t word, param;
      cache_quantise(x, word, param);
      if (row[k] >= 0) {
        reinterpret_cast<uint32_t*>(p.pool.codes[n])[row[k] * kLanes + kGroups * t + g] = word;
        if (t == 0) p.pool.params[n][row[k] * kGroups + g] = param;
      }
    }
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kCacheCopyThreads) fa_cache_read_kernel(const CacheCopyParams p) {
  constexpr int kLanes = D / 8, kGroups = D / kCacheGroup, kRows = kCacheCopyRows<D>;
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
    if (i < count && row < 0 && lane == 0) atomicExch(p.status, kStatusBadIndex);
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
