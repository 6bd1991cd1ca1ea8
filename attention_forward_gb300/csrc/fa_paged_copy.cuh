// fa_paged_copy.cuh -- the 16-bit paged caches: rotating write, and read back.
//
// Rotation of a pair (x, y) of channels at position n with frequency f (radians a
// position):  (x cos a - y sin a, y cos a + x sin a),  a = n f.
// The angle is held in turns as a 64-bit fraction: f / 2 pi to 2^-61 of a turn, whose
// product with n is exact modulo a turn; its upper 32 bits, rounded to fp32, go to the sine
// and cosine.  All in integers: the GPU makes two double-precision products a cycle and
// multiprocessor.  That rounding is nearly all of the angle's error: half turns in [-1, 1)
// are off by 2^-25, which is 2^-23.3 radian; f's fraction adds 2^-35 f at n = 2^24.  n f in
// fp32 would be off by half a radian there.
//
// Both kernels only move bytes.  Write: a block takes 2^token_shift tokens of a
// sequence and a slice of their heads.  A thread keeps to 16 channels of one token:
// two 16-byte words of a row, the halves of 8 pairs (which lie apart by half of what is
// rotated, or side by side), and goes through the heads with the 8 sines and cosines in
// registers, made once by the block.
//
// Measured, 4 x 4096 tokens, in a graph: 32 + 8 + 8 heads of 128 channels written and read
// back in 54.1 us (5.6 TB/s), latent rows and 16 heads in 22.7 (3.6 TB/s: 1024 blocks,
// of which 608 run at once).  Rows in flight a thread, write and latent write: 2 at five
// and six blocks an SM 63 and 28 us, 3 at four and five 54.5 and 26, 4 at three and four
// 55.3 and 22.6.  A token of 32 sequences: 2.2 us, three loads one behind the other.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_cache.cuh"
#include "fa_paged.h"

namespace fa {

constexpr int kPagedCopyThreads = 256;
constexpr int kPagedMaxTokenShift = 4;
constexpr int kPagedAtOnce = 4;  // tasks of a thread whose loads go out together
constexpr int kPagedMaxPairs = 64;

// f / 2 pi as a fraction of a turn in 2^-64ths: f's 24 bits times 1 / 2 pi in 64.  Off
// by 2^-61 of f's power of two, or 2^-64.
__device__ __forceinline__ unsigned long long rope_step(float f) {
  const uint32_t bits = __float_as_uint(f);
  const int e = static_cast<int>((bits >> 23) & 0xffu) - 127;  // |f| = 1.m 2^e
  if (e < -64 || e > 63) return 0ull;  // no angle at 2^24 positions, or no fp32 angle
  const unsigned long long m = static_cast<unsigned long long>((bits & 0x7fffffu) | 0x800000u) << 40;
  // 2^64 / 2 pi; the product's upper half is 2^63 1.m / 2 pi
  const unsigned long long half = __umul64hi(m, 0x28be60db9391054aull);
  const unsigned long long step = e >= 0 ? half << 1 << e : half >> (-e - 1);
  return bits >> 31 ? 0ull - step : step;
}

// Cosine and sine of the angle n steps.
__device__ __forceinline__ float2 rope_unit(int n, unsigned long long step) {
  const unsigned long long at = step * static_cast<unsigned long long>(static_cast<long long>(n));
  // the upper half as a signed number: half turns in [-1, 1), rounded to 24 bits as sine and
  // cosine are
  const float half = static_cast<float>(static_cast<int>(at >> 32)) * 4.656612873077393e-10f;
  float2 u;
  sincospif(half, &u.y, &u.x);
  return u;
}

// Two 16-byte words of 16-bit channels: the pairs (e, e) of both words, or (2 e, 2 e
// + 1) of one, rotated by unit[0 ... 7].
template <bool BF16, bool kPairs>
__device__ __forceinline__ void rope_turn(uint4& a, uint4& b, const float2 (&unit)[8]) {
  uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
  auto turn = [](float& x, float& y, float2 u) {
    const float t = fmaf(x, u.x, -y * u.y);
    y = fmaf(y, u.x, x * u.y);
    x = t;
  };
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float2 x = cache_unpack<BF16>(wa[e]), y = cache_unpack<BF16>(wb[e]);
    if constexpr (kPairs) {
      turn(x.x, x.y, unit[e]);
      turn(y.x, y.y, unit[e + 4]);
    } else {
      turn(x.x, y.x, unit[2 * e]);
      turn(x.y, y.y, unit[2 * e + 1]);
    }
    wa[e] = cache_pack<BF16>(x.x, x.y);
    wb[e] = cache_pack<BF16>(y.x, y.y);
  }
  a = make_uint4(wa[0], wa[1], wa[2], wa[3]);
  b = make_uint4(wb[0], wb[1], wb[2], wb[3]);
}

// The slot of the token at position `pos` of sequence b as a row of kv head 0; -1
// when its place does not exist.
template <class P>
__device__ __forceinline__ long long paged_slot(const P& p, int b, uint32_t pos) {
  const uint32_t n = pos >> p.page_shift;
  if (n >= static_cast<uint32_t>(p.max_pages)) return -1;
  const int page = p.page_table[static_cast<size_t>(b) * p.max_pages + n];
  if (page < 0 || page >= p.num_pages) return -1;
  return ((static_cast<long long>(page) * p.Hkv) << p.page_shift) +
         (pos & ((1u << p.page_shift) - 1u));
}

template <bool kLat, bool BF16, bool kPairs>
__global__ void __launch_bounds__(kPagedCopyThreads, kLat ? 4 : 3)
    fa_paged_write_kernel(const PagedWriteParams p) {
  __shared__ float2 units[kPagedMaxPairs << kPagedMaxTokenShift];  // [token][pair]
  grid_dependency_wait();
  grid_launch_dependents();
  const int b = static_cast<int>(blockIdx.y), tid = static_cast<int>(threadIdx.x);
  const int ts = p.token_shift, first = static_cast<int>(blockIdx.x) << ts;
  // the thread's 16 channels of every row, its token, and the first of its heads
  const int d_shift = kLat ? 2 : (p.D == 128 ? 3 : 2), d = kLat ? kLatentRope : p.D;
  const int u = tid & ((1 << d_shift) - 1);
  const int token = first + ((tid >> d_shift) & ((1 << ts) - 1));
  const int step = kPagedCopyThreads >> (d_shift + ts);
  const int half = p.rot >> 1;
  const bool turned = 16 * u < p.rot, halves = turned && !kPairs;
  const int w0 = halves ? u : 2 * u, w1 = halves ? u + (half >> 3) : 2 * u + 1;
  // heads of q, of k, then of v (the latent as eight of 64 channels)
  constexpr int kLatHeads = kLatent / kLatentRope;
  const int h_v = p.H + p.Hkv, all = h_v + (kLat ? kLatHeads : p.Hkv);
  const int per = (all + static_cast<int>(gridDim.z) - 1) / static_cast<int>(gridDim.z);
  const int h1 = min(all, per * (static_cast<int>(blockIdx.z) + 1));
  int h = per * static_cast<int>(blockIdx.z) + (tid >> (d_shift + ts));
  auto source = [&](int i) -> const uint4* {
    const bool is_q = i < p.H, is_v = i >= h_v;
    const uint4* in = static_cast<const uint4*>(is_q ? p.q : (is_v ? p.v : p.k));
    if (kLat && is_v)
      return in + (static_cast<long long>(b) * p.S + token) * (kLatent / 8) + (i - h_v) * 8;
    const int heads = is_q ? p.H : p.Hkv, head = is_q ? i : i - (is_v ? h_v : p.H);
    return in + (((static_cast<long long>(b) * heads + head) * p.S + token) << (d_shift + 1));
  };

  uint4 x[kPagedAtOnce], y[kPagedAtOnce];
  // (rows past the count are there all the same: the first words need not wait for it.
  // From L2: the kernel may have started while the one that wrote them ran.)
  auto load = [&]() {
#pragma unroll
    for (int k = 0; k < kPagedAtOnce; ++k)
      if (h + k * step < h1 && token < p.S) {
        const uint4* in = source(h + k * step);
        x[k] = __ldcg(in + w0);
        y[k] = __ldcg(in + w1);
      }
  };
  load();
  const int start = p.start ? p.start[b] : 0;
  const int count = p.count ? min(p.count[b], p.S) : p.S;
  if (first >= count) return;
  // (before the angles, which its latency then hides)
  const long long slot =
      paged_slot(p, b, static_cast<uint32_t>(start) + static_cast<uint32_t>(token));
  float2 unit[8];
  if (half > 0) {
    for (int i = tid; i < half << ts; i += kPagedCopyThreads) {
      const int tok = i / half;
      units[i] = rope_unit(static_cast<int>(static_cast<uint32_t>(start) +
                                            static_cast<uint32_t>(first + tok)),
                           rope_step(p.freqs[i - tok * half]));
    }
    __syncthreads();
    if (turned) {
#pragma unroll
      for (int e = 0; e < 8; ++e) unit[e] = units[(token - first) * half + 8 * u + e];
    }
  }
  if (token >= count) return;
  if (slot < 0 && u == 0 && h == 0) atomicMax(p.status, kStatusBadIndex);
#pragma unroll 1
  for (;;) {
#pragma unroll
    for (int k = 0; k < kPagedAtOnce; ++k) {
      const int i = h + k * step;
      if (i >= h1) break;
      const bool is_q = i < p.H, is_v = i >= h_v;
      if (turned && !is_v) rope_turn<BF16, kPairs>(x[k], y[k], unit);
      uint4* out;
      if (is_q) {
        out = static_cast<uint4*>(p.q_out) +
              ((static_cast<long long>(b) * p.H + i) * p.S + token) * (p.q_width >> 3) +
              ((p.q_width - d) >> 3);
      } else if (slot < 0) {
        continue;
      } else if constexpr (kLat) {
        out = static_cast<uint4*>(p.pool[0]) + slot * (kLatentRow / 8) +
              (is_v ? 8 * (i - h_v) : kLatent / 8);
      } else {
        const long long head = i - (is_v ? h_v : p.H);
        out = static_cast<uint4*>(is_v ? p.pool[1] : p.pool[0]) +
              ((slot + (head << p.page_shift)) << (d_shift + 1));
      }
      out[w0] = x[k];
      out[w1] = y[k];
    }
    h += kPagedAtOnce * step;
    if (h >= h1) break;
    load();
  }
}

// A thread takes the same 16 bytes of kPagedAtOnce rows.  blockIdx.y: the (sequence,
// kv head), blockIdx.z: keys or values; latent rows (72 words) are taken whole.
template <bool kLat>
__global__ void __launch_bounds__(kPagedCopyThreads) fa_paged_read_kernel(const PagedReadParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int bh = static_cast<int>(blockIdx.y);
  const int b = bh / p.Hkv, hk = bh - b * p.Hkv;
  const int start = p.start ? p.start[b] : 0;
  const int count = p.count ? min(p.count[b], p.S) : p.S;
  const int words = kLat ? kLatentRow / 8 : p.D / 8;
  const int lanes = kPagedCopyThreads / words;  // rows at once
  const int row_of = static_cast<int>(threadIdx.x) / words;
  const int w = static_cast<int>(threadIdx.x) - row_of * words;
  const int i0 = static_cast<int>(blockIdx.x) * lanes * kPagedAtOnce + row_of;
  if (row_of >= lanes || i0 >= count) return;
  const uint4* pool = static_cast<const uint4*>(kLat || blockIdx.z == 0 ? p.pool[0] : p.pool[1]);
  uint4 x[kPagedAtOnce];
#pragma unroll
  for (int k = 0; k < kPagedAtOnce; ++k) {
    const int i = i0 + k * lanes;
    x[k] = make_uint4(0u, 0u, 0u, 0u);  // a place that does not exist reads as zeros
    if (i >= count) continue;
    const long long s = paged_slot(p, b, static_cast<uint32_t>(start) + static_cast<uint32_t>(i));
    if (s < 0) {
      if (w == 0) atomicMax(p.status, kStatusBadIndex);
    } else {
      // from L2: the kernel may have started while the write before it ran
      x[k] = __ldcg(pool + (s + (static_cast<long long>(hk) << p.page_shift)) * words + w);
    }
  }
#pragma unroll
  for (int k = 0; k < kPagedAtOnce; ++k) {
    const int i = i0 + k * lanes;
    if (i >= count) continue;
    const long long row = static_cast<long long>(bh) * p.S + i;
    if constexpr (kLat) {
      if (w < kLatent / 8)
        static_cast<uint4*>(p.out[0])[row * (kLatent / 8) + w] = x[k];
      else
        static_cast<uint4*>(p.out[1])[row * (kLatentRope / 8) + w - kLatent / 8] = x[k];
    } else {
      static_cast<uint4*>(blockIdx.z == 0 ? p.out[0] : p.out[1])[row * words + w] = x[k];
    }
  }
}

}  // namespace fa
