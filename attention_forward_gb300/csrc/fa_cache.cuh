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

// Where row `row` of [B, Hkv, S] lies in the pool: its (page, kv head, slot)
// index, or -1 when the row is not in the call (past the sequence's count) and
// -2 when its place does not exist (a position or page out of range).
__device__ __forceinline__ long long cache_place(const CacheCopyParams& p, long long row) {
  if (row >= p.n_rows) return -1;
  const long long bh = row / p.S;
  const int i = static_cast<int>(row - bh * p.S);
  const int b = static_cast<int>(bh / p.Hkv);
  const int hk = static_cast<int>(bh - static_cast<long long>(b) * p.Hkv);
  if (p.count && i >= p.count[b]) return -1;
  const long long pos = (p.start ? static_cast<long long>(p.start[b]) : 0ll) + i;
  if (pos < 0) return -2;
  const long long n = pos >> p.page_shift;
  if (n >= p.max_pages) return -2;
  const int page = p.page_table[static_cast<long long>(b) * p.max_pages + n];
  if (page < 0 || page >= p.num_pages) return -2;
  return ((static_cast<long long>(page) * p.Hkv + hk) << p.page_shift) +
         (pos & ((1ll << p.page_shift) - 1));
}

// One group's codes from 8 of its channels per lane (4 lanes of a quad hold
// the group): the word of codes and the (scale, minimum) pair.
__device__ __forceinline__ void cache_quantise(const float (&in)[8], uint32_t& word,
                                               uint32_t& param) {
  float x[8];
  bool bad = false;
  float lo = INFINITY, hi = -INFINITY;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    bad |= in[e] != in[e];
    x[e] = fminf(fmaxf(in[e], -kCacheLimit), kCacheLimit);
    lo = fminf(lo, x[e]);
    hi = fmaxf(hi, x[e]);
  }
#pragma unroll
  for (int m = 1; m <= 2; m <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
  }
  const uint32_t votes = __ballot_sync(0xffffffffu, bad);
  // a NaN makes its whole group NaN: the scale carries it
  bad = ((votes >> (threadIdx.x & 28u)) & 15u) != 0;
  const __half zh = __float2half_rn(lo);
  const __half sh = __float2half_rn(__fdiv_rn(hi - lo, 15.f));
  const float z = __half2float(zh), s = __half2float(sh);
  const float inv = s > 0.f ? __frcp_rn(s) : 0.f, half_s = 0.5f * s;
  word = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    // floor((x - z) / s + 1/2), decided exactly: d + err is x - z (two-sum),
    // c a nearest guess, r = d - c s exact by one FMA; r against half a
    // scale, the lost part err included, says whether c moves by one
    const float d = x[e] - z;
    const float bb = d - x[e];
    const float err = (x[e] - (d - bb)) + (-z - bb);
    float c = rintf(d * inv);
    const float r = fmaf(-c, s, d);
    if ((r - half_s) + err >= 0.f) c += 1.f;
    if ((r + half_s) + err < 0.f) c -= 1.f;
    c = s > 0.f ? fminf(fmaxf(c, 0.f), 15.f) : 0.f;
    word |= static_cast<uint32_t>(c) << (4 * e);
  }
  if (bad) word = 0;
  const uint32_t sz = static_cast<uint32_t>(__half_as_ushort(sh)) |
                      (static_cast<uint32_t>(__half_as_ushort(zh)) << 16);
  param = bad ? 0x7fff7fffu : sz;
}

constexpr int kCacheCopyThreads = 256;

template <int D, bool BF16>
__global__ void __launch_bounds__(kCacheCopyThreads) fa_cache_write_kernel(const CacheCopyParams p) {
  constexpr int kLanes = D / 8, kGroups = D / kCacheGroup;
  const long long idx = static_cast<long long>(blockIdx.x) * kCacheCopyThreads + threadIdx.x;
  const long long row = idx / kLanes;
  const int lane = static_cast<int>(idx - row * kLanes);  // 8 channels: group lane / 4, part lane % 4
  const long long at = cache_place(p, row);
  if (at == -2 && lane == 0) atomicExch(p.status, kStatusBadIndex);
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    float x[8] = {};
    if (at >= 0) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(p.rows[n]) + idx);
      const float2 a = cache_unpack<BF16>(w.x), b = cache_unpack<BF16>(w.y);
      const float2 c = cache_unpack<BF16>(w.z), d = cache_unpack<BF16>(w.w);
      x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
      x[4] = c.x; x[5] = c.y; x[6] = d.x; x[7] = d.y;
    }
    uint32_t word, param;
    cache_quantise(x, word, param);
    if (at >= 0) {
      reinterpret_cast<uint32_t*>(p.pool.codes[n])[at * kLanes + kGroups * t + g] = word;
      if (t == 0) p.pool.params[n][at * kGroups + g] = param;
    }
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kCacheCopyThreads) fa_cache_read_kernel(const CacheCopyParams p) {
  constexpr int kLanes = D / 8, kGroups = D / kCacheGroup;
  const long long idx = static_cast<long long>(blockIdx.x) * kCacheCopyThreads + threadIdx.x;
  const long long row = idx / kLanes;
  const int lane = static_cast<int>(idx - row * kLanes);  // the row's word
  const long long at = cache_place(p, row);
  if (at == -2 && lane == 0) atomicExch(p.status, kStatusBadIndex);
  if (at == -1) return;
  const int t = lane / kGroups, g = lane - t * kGroups;
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    uint4 out = make_uint4(0u, 0u, 0u, 0u);  // a place that does not exist reads as zeros
    if (at >= 0) {
      const uint32_t word = __ldg(reinterpret_cast<const uint32_t*>(p.pool.codes[n]) + at * kLanes + lane);
      const uint32_t param = __ldg(p.pool.params[n] + at * kGroups + g);
      const float2 sz = __half22float2(*reinterpret_cast<const __half2*>(&param));
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[e] = fmaf(static_cast<float>((word >> (4 * e)) & 15u), sz.x, sz.y);
      out.x = cache_pack<BF16>(x[0], x[1]);
      out.y = cache_pack<BF16>(x[2], x[3]);
      out.z = cache_pack<BF16>(x[4], x[5]);
      out.w = cache_pack<BF16>(x[6], x[7]);
    }
    reinterpret_cast<uint4*>(p.rows[n])[row * kLanes + 4 * g + t] = out;
  }
}

}  // namespace fa
