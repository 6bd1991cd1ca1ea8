// fa_expanded.cuh -- latent attention with its heads expanded (prompts): scores over
// 192 channels, of which 128 are a head's own and 64 the heads share, values of 128.
// sm_103a.
//
//   S = scale (Q[:, :128] K^T + Q[:, 128:] R^T),  O = softmax(S) V
// with K and V the halves of the head's rows of kv [Skv, 256], as one product with
// the expansion's weights leaves them, and R = k_rope [Skv, 64]: neither is ever put
// together with the other or repeated by heads in memory.
//
// The prefill kernel's pipeline (its header): items of two stages of 128 rows, the
// same warps, softmax, register split and tensor memory.  What differs follows from
// shared memory: Q takes 2 x 48 KB, a key tile 48 KB and a value tile 32 KB, so that
// two tiles do not fit.  Keys and values therefore go through one ring of eight
// 16 KB chunks, five a tile in the order of their use:
//   K chunk c (3): 128 keys x 64 channels;  V chunk h (2): 64 keys x 128 channels
// The ring runs 1.6 tiles ahead.  A tile's K, and its V, have one pair of barriers each:
// with a pair for every chunk, the issuing warp's waits and commits took 4430 cycles a
// tile of two stages, whose products take 2560.  Warps 12 and 13 issue a stage's products
// each, warp 14 claims the items and sends for the keys, warp 15 for queries and values:
// by one warp, a chunk took 860 cycles (4200 a tile).  O goes from
// registers to global memory (its staging's 32 KB are the ring's).
#pragma once
#include "fa_paged.h"
#include "fa_prefill.cuh"

namespace fa {

struct ExpandedParams {
  PrefillParams a;  // lse, scheduler, sizes, masks, split keys; o in a.o
  int H;
};

struct ExpandedLayout {
  static constexpr int kDq = kNope + kLatentRope;    // 192
  static constexpr int kChunk = 128 * 64 * 2;        // 16 KB
  static constexpr int kQBytes = 3 * kChunk;         // one stage of Q
  static constexpr int kSlots = 8;
  static constexpr int kPerTile = 5;                 // chunks: K 3, V 2
  static constexpr int kOffQ = 0;
  static constexpr int kOffRing = kStages * kQBytes;
  static constexpr int kOffBars = kOffRing + kSlots * kChunk;
  // mbarrier indices, as the prefill kernel's
  static constexpr int Q_FULL = 0, Q_EMPTY = 2, S_FULL = 4, PV_READY = 6, O_READY = 8, ML_FULL = 10,
                       O_FREE = 12, ITEM_FULL = 15, ITEM_EMPTY = 19,
                       // of the K and V of a tile, by the tile's parity
                       K_FULL = 23, K_EMPTY = 25, V_FULL = 27, V_EMPTY = 29, DRAIN = 31,
                       kNumBars = 33;
  static constexpr int kOffInvL = kOffBars + ((kNumBars * 8 + 15) / 16) * 16;
  static constexpr int kOffItems = kOffInvL + kStages * kBM * 4;
  static constexpr int kOffTmemSlot = kOffItems + kItemRing * 4;
  static constexpr int kOffAbort = kOffTmemSlot + 4;
  static constexpr int kSmemBytes = kOffAbort + 4 + 1024;  // + align
  static constexpr int kTmemCols = 512;
  static constexpr int kTmemO = 256;  // O_s at column 256 + 128 s
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

template <bool BF16, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    fa_expanded_kernel(const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV,
                       const __grid_constant__ CUtensorMap tmR, const ExpandedParams ep) {
  using L = ExpandedLayout;
  constexpr int D = kNope;
  const PrefillParams& p = ep.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t sQ = sbase + L::kOffQ, sRing = sbase + L::kOffRing, bars = sbase + L::kOffBars;
  float* inv_l_smem = reinterpret_cast<float*>(smem + L::kOffInvL);
  volatile int* item_ring = reinterpret_cast<volatile int*>(smem + L::kOffItems);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffTmemSlot);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + L::kOffAbort);
  auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

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
    for (int i = 0; i < kItemRing; ++i) {
      mbar_init(bar(L::ITEM_FULL + i), 1);
      mbar_init(bar(L::ITEM_EMPTY + i), kItemTakers + 2);  // two that issue, two that load
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(L::K_FULL + i), 1);
      mbar_init(bar(L::K_EMPTY + i), 2);  // both stages
      mbar_init(bar(L::V_FULL + i), 1);
      mbar_init(bar(L::V_EMPTY + i), 2);
      mbar_init(bar(L::DRAIN + i), 1);
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
    tma_prefetch_desc(&tmR);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Ctl ctl{abort_flag, p.status, p.timeout_ns};
  grid_dependency_wait();  // the setup overlapped the end of the kernel before

  const int wg = warp >> 2;
  if (wg < 2) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmaxSingle));
  } else if (wg == 2) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsEpilogueSingle));
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControlSingle));
  }

  if (wg < 2) {
    // =========================== softmax, stage s ===========================
    const int s = wg, rq = warp & 3, r = rq * 32 + lane;
    const uint32_t t_lane = static_cast<uint32_t>(rq * 32) << 16;
    const uint32_t tS = tmem + t_lane + static_cast<uint32_t>(s * kBN);
    const uint32_t tO = tmem + t_lane + static_cast<uint32_t>(L::kTmemO + s * D);
    uint32_t n_s = 0;  // tiles of this stage so far (S_FULL / O_READY phase)
    bool ok = true;
#pragma unroll 1
    for (uint32_t k = 0; ok; ++k) {
      const int idx = take_item<0>(item_ring, bar(L::ITEM_FULL), bar(L::ITEM_EMPTY), k, ctl, ok);
      if (!ok || idx < 0) break;
      const ItemT<kSplit> it = get_item<kSplit>(p, idx);
      const int nT = s == 0 ? it.nT0 : it.nT1;
      const int stage_row0 = it.row0 + s * kBM, row_g = stage_row0 + r;
      float m = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int j = 0; j < nT; ++j, ++n_s) {
        if (!wait_bar_warp(bar(L::S_FULL + s), n_s & 1, ctl)) { ok = false; break; }
        tc_fence_after();
        softmax_tile<D, BF16>(tS, tO, (it.t0 + j) * kBN, stage_row0, row_g, p, j > 0, m, l);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::PV_READY + s));
      }
      if (!ok) break;
      if (row_g < p.Sq) {
        const float lse = l > 0.f ? (m + log2f(l)) * 0.69314718055994530942f : l == 0.f ? -INFINITY : l;
        if constexpr (kSplit)
          p.part_lse[(static_cast<size_t>(it.split) * p.BH + it.bh) * p.Sq + row_g] = lse;
        else
          p.lse[static_cast<size_t>(it.bh) * p.Sq + row_g] = lse;
      }
      if (nT > 0) {
        if (!wait_bar_warp(bar(L::O_READY + s), (n_s - 1) & 1, ctl)) { ok = false; break; }
        inv_l_smem[s * kBM + r] = l == 0.f ? 0.f : 1.f / l;  // a NaN stays one
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::ML_FULL + s));
      }
    }
    __syncwarp();
  } else if (wg == 2) {
    // =============================== epilogue ===============================
    const int rq = warp & 3, r = rq * 32 + lane;
    const uint32_t t_lane = static_cast<uint32_t>(rq * 32) << 16;
    uint32_t n_t[2] = {0u, 0u}, n_e[2] = {0u, 0u};  // O_READY and ML_FULL phases
    bool ok = true;
#pragma unroll 1
    for (uint32_t k = 0; ok; ++k) {
      const int idx = take_item<kSleepEpilogueNs>(item_ring, bar(L::ITEM_FULL), bar(L::ITEM_EMPTY), k,
                                                  ctl, ok);
      if (!ok || idx < 0) break;
      const ItemT<kSplit> it = get_item<kSplit>(p, idx);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (!ok) continue;
        const int nT = s == 0 ? it.nT0 : it.nT1;
        float inv_l = 0.f;
        if (nT > 0) {
          n_t[s] += static_cast<uint32_t>(nT);
          ok = wait_bar_warp<kSleepEpilogueNs>(bar(L::ML_FULL + s), n_e[s] & 1, ctl);
          ++n_e[s];
          ok = ok && wait_bar_warp<kSleepEpilogueNs>(bar(L::O_READY + s), (n_t[s] - 1) & 1, ctl);
          if (!ok) continue;
          inv_l = inv_l_smem[s * kBM + r];
          tc_fence_after();
        }
        const uint32_t tO = tmem + t_lane + static_cast<uint32_t>(L::kTmemO + s * D);
        const int row_g = it.row0 + s * kBM + r;
        const size_t row = static_cast<size_t>(it.bh) * p.Sq + row_g;
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t v[2][16];
          if (nT > 0) {
            tmem_ld32(tO + cc * 32, v[0], v[1]);
            tmem_wait_ld();
            reg_fence16(v[0]);
            reg_fence16(v[1]);
          } else {  // no visible key: O = 0
#pragma unroll
            for (int e = 0; e < 16; ++e) v[0][e] = v[1][e] = 0u;
          }
          if (row_g >= p.Sq) continue;
          float x[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(v[e >> 4][e & 15]) * inv_l;
          if constexpr (kSplit) {
            float4* out = reinterpret_cast<float4*>(
                p.part_o + ((static_cast<size_t>(it.split) * p.BH) * p.Sq + row) * D + cc * 32);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              out[e] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
          } else {
            uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + row * D + cc * 32);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              out[e] = make_uint4(pack2<BF16>(x[8 * e], x[8 * e + 1]),
                                  pack2<BF16>(x[8 * e + 2], x[8 * e + 3]),
                                  pack2<BF16>(x[8 * e + 4], x[8 * e + 5]),
                                  pack2<BF16>(x[8 * e + 6], x[8 * e + 7]));
          }
        }
        if (nT > 0) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::O_FREE + s));
        }
      }
    }
    __syncwarp();
  } else if (warp < 14) {
    // ======================= MMA issuers, a warp a stage =====================
    // per key tile PV_s(j - 1), QK_s(j): in this order, for the scores overwrite P.  (By
    // one warp for both stages, its waits and commits left the tensor core idle for 1400
    // of a tile's 4000 cycles.)
    constexpr uint32_t kIdescQK = idesc_f16(BF16, false, false, kBM, kBN);
    constexpr uint32_t kIdescPV = idesc_f16(BF16, false, true, kBM, D);
    const int s = warp - 12;
    const uint32_t tS = tmem + static_cast<uint32_t>(s * kBN);
    const uint32_t tO = tmem + static_cast<uint32_t>(L::kTmemO + s * D);
    const uint64_t q = smem_desc_sw128(sQ + static_cast<uint32_t>(s * L::kQBytes), 16, 1024);
    // the chunk of fill `fill` as an operand
    auto at = [&](uint32_t fill) { return sRing + (fill % L::kSlots) * L::kChunk; };
    auto by_tile = [&](int first, uint32_t t) { return bar(first + static_cast<int>(t & 1u)); };
    auto wait = [&](bool asked, uint32_t b, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, asked) || wait_bar_warp<kSleepMmaNs>(b, parity & 1u, ctl);
    };
    uint32_t n_pv = 0, n_o = 0;  // PV_s so far, and items with one (PV_READY, O_FREE phases)
    uint32_t tile = 0;           // the item's first tile, counted over the CTA's items
    bool ok = true, issued = false;
#pragma unroll 1
    for (uint32_t k = 0; ok; ++k) {
      const int idx = take_item<kSleepMmaNs>(item_ring, bar(L::ITEM_FULL), bar(L::ITEM_EMPTY), k, ctl, ok);
      if (!ok || idx < 0) break;
      const ItemT<kSplit> it = get_item<kSplit>(p, idx);
      const int n = s == 0 ? it.nT0 : it.nT1;
      ok = wait(false, bar(L::Q_FULL + s), k);
      if (ok && n == 0) umma_commit(bar(L::Q_EMPTY + s));
      bool got_k = false;
#pragma unroll 1
      for (int j = 0; ok && j <= n && n > 0; ++j) {
        const uint32_t t = tile + static_cast<uint32_t>(j);
        if (j > 0) {
          // both probed together: usually both are there
          bool rdy = mbar_try_wait(by_tile(L::V_FULL, t - 1), ((t - 1) >> 1) & 1u);
          rdy &= mbar_try_wait(bar(L::PV_READY + s), n_pv & 1u);
          ok = __all_sync(0xffffffffu, rdy) ||
               (wait(false, by_tile(L::V_FULL, t - 1), (t - 1) >> 1) &&
                wait(false, bar(L::PV_READY + s), n_pv));
          ++n_pv;
          if (ok && j == 1 && n_o > 0) ok = wait(false, bar(L::O_FREE + s), n_o - 1);
          if (!ok) break;
          got_k = j < n && mbar_test_wait(by_tile(L::K_FULL, t), (t >> 1) & 1u);
          tc_fence_after();
          const uint32_t fill = L::kPerTile * (t - 1) + 3;
          umma_f16_ts_2k64(tO, tS, smem_desc_sw128(at(fill), L::kChunk / 2, 1024),
                           smem_desc_sw128(at(fill + 1), L::kChunk / 2, 1024), kIdescPV, j > 1 ? 1u : 0u);
          umma_commit(by_tile(L::V_EMPTY, t - 1));
          umma_commit(bar(L::O_READY + s));
        }
        if (j < n) {
          ok = wait(got_k, by_tile(L::K_FULL, t), t >> 1);
          if (!ok) break;
          tc_fence_after();
          const uint32_t fill = L::kPerTile * t;
          umma_f16_ss_3k64(tS, q, smem_desc_sw128(at(fill), 16, 1024), smem_desc_sw128(at(fill + 1), 16, 1024),
                           smem_desc_sw128(at(fill + 2), 16, 1024), kIdescQK);
          issued = true;
          umma_commit(bar(L::S_FULL + s));
          umma_commit(by_tile(L::K_EMPTY, t));
          if (j + 1 == n) umma_commit(bar(L::Q_EMPTY + s));
        }
      }
      if (n > 0) ++n_o;
      // tiles that the other stage alone uses
#pragma unroll 1
      for (int j = n; ok && j < it.nT1; ++j) {
        const uint32_t t = tile + static_cast<uint32_t>(j);
        ok = wait(false, by_tile(L::K_FULL, t), t >> 1) && wait(false, by_tile(L::V_FULL, t), t >> 1);
        if (ok && lane == 0) {
          mbar_arrive(by_tile(L::K_EMPTY, t));
          mbar_arrive(by_tile(L::V_EMPTY, t));
        }
        __syncwarp();
      }
      tile += static_cast<uint32_t>(it.nT1);
    }
    if (issued) {  // every MMA issued so far completes before TMEM is freed
      umma_commit(bar(L::DRAIN + s));
      wait_drain(bar(L::DRAIN + s), 0, p.timeout_ns);
    }
    __syncwarp();
  } else if (warp == 14) {
    // ================= scheduler, and TMA producer of the keys ================
    // A K chunk's slot was that of a chunk eight fills back: c 0 the last of K(T - 2), c 1
    // and 2 those of V(T - 2); V's were the first two of K(T - 1).  Barriers of two tiles
    // serve: K and V of a tile are done with before those of the next but one arrive.
    if (lane == 0) {
      uint32_t tile = 0;
      bool ok = true;
      int idx = static_cast<int>(blockIdx.x);  // the grid never exceeds the items
#pragma unroll 1
      for (uint32_t k = 0; ok; ++k) {
        const uint32_t slot = k % kItemRing;
        if (k >= kItemRing &&
            !wait_bar<kSleepProducerNs>(bar(L::ITEM_EMPTY + slot), (k / kItemRing - 1) & 1u, ctl)) {
          ok = false;
          break;
        }
        item_ring[slot] = idx;
        mbar_arrive(bar(L::ITEM_FULL + slot));
        if (idx < 0) break;
        const ItemT<kSplit> it = get_item<kSplit>(p, idx);
        const int batch = it.bh / ep.H;
        int key = it.t0 * kBN;
#pragma unroll 1
        for (int j = 0; j < it.nT1; ++j, ++tile, key += kBN) {
          const int odd = static_cast<int>(tile & 1u);
          const uint32_t free_par = ((tile >> 1) & 1u) ^ 1u, full = bar(L::K_FULL + odd);
          const uint32_t fill = L::kPerTile * tile;
          if (tile >= 2 && !wait_bar<kSleepProducerNs>(bar(L::K_EMPTY + odd), free_par, ctl)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(full, 3 * L::kChunk);
          tma_load_3d(sRing + (fill % L::kSlots) * L::kChunk, &tmK, full, 0, key, it.bh);
          if (tile >= 2 && !wait_bar<kSleepProducerNs>(bar(L::V_EMPTY + odd), free_par, ctl)) {
            ok = false;
            break;
          }
          tma_load_3d(sRing + ((fill + 1) % L::kSlots) * L::kChunk, &tmK, full, 64, key, it.bh);
          tma_load_3d(sRing + ((fill + 2) % L::kSlots) * L::kChunk, &tmR, full, 0, key, batch);
        }
        idx = claim_item(p);
        if (idx < 0) grid_launch_dependents();  // the next grid may take the SMs
      }
      // drain: every load issued lands before shared memory goes away (an abort may have
      // left a tile's last chunks unsent: the waits are bounded)
      for (uint32_t i = tile > 2 ? tile - 2 : 0u; i < tile + (ok ? 0u : 1u); ++i)
        wait_drain(bar(L::K_FULL + static_cast<int>(i & 1u)), (i >> 1) & 1u, p.timeout_ns);
    }
    __syncwarp();
  } else {
    // ================ TMA producer of the queries and the values ==============
    uint32_t tile = 0, items = 0;
    bool ok = true;
#pragma unroll 1
    for (uint32_t k = 0; ok; ++k) {
      const int idx = take_item<kSleepProducerNs>(item_ring, bar(L::ITEM_FULL), bar(L::ITEM_EMPTY), k, ctl, ok);
      if (!ok || idx < 0) break;
      const ItemT<kSplit> it = get_item<kSplit>(p, idx);
#pragma unroll 1
      for (int s = 0; ok && s < 2; ++s) {
        ok = items == 0 || wait_bar_warp<kSleepProducerNs>(bar(L::Q_EMPTY + s), (items - 1) & 1u, ctl);
        if (ok && lane == 0) {
          mbar_arrive_expect_tx(bar(L::Q_FULL + s), L::kQBytes);
#pragma unroll
          for (int c = 0; c < 3; ++c)
            tma_load_3d(sQ + static_cast<uint32_t>(s * L::kQBytes + c * L::kChunk), &tmQ,
                        bar(L::Q_FULL + s), c * 64, it.row0 + s * kBM, it.bh);
        }
        __syncwarp();
      }
      if (!ok) break;
      ++items;
      int key = it.t0 * kBN;
#pragma unroll 1
      for (int j = 0; j < it.nT1; ++j, ++tile, key += kBN) {
        const uint32_t before = tile - 1, fill = L::kPerTile * tile + 3;
        ok = tile == 0 || wait_bar_warp<kSleepProducerNs>(bar(L::K_EMPTY + static_cast<int>(before & 1u)),
                                                          (before >> 1) & 1u, ctl);
        if (!ok) break;
        if (lane == 0) {
          const uint32_t full = bar(L::V_FULL + static_cast<int>(tile & 1u));
          mbar_arrive_expect_tx(full, 2 * L::kChunk);
#pragma unroll
          for (uint32_t h = 0; h < 2; ++h) {
            const uint32_t dst = sRing + ((fill + h) % L::kSlots) * L::kChunk;
            tma_load_3d(dst, &tmV, full, kNope, key + static_cast<int>(h) * 64, it.bh);
            tma_load_3d(dst + L::kChunk / 2, &tmV, full, kNope + 64, key + static_cast<int>(h) * 64, it.bh);
          }
        }
        __syncwarp();
      }
    }
    // drain, as above
    if (items > 0)
      for (int s = 0; s < 2; ++s) wait_drain(bar(L::Q_FULL + s), (items - 1) & 1u, p.timeout_ns);
    for (uint32_t i = tile > 2 ? tile - 2 : 0u; i < tile; ++i)
      wait_drain(bar(L::V_FULL + static_cast<int>(i & 1u)), (i >> 1) & 1u, p.timeout_ns);
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
    // the launch's last CTA clears the scheduler slot
    __threadfence();
    if (atomicAdd(&p.sched[1], 1ull) == gridDim.x - 1) {
      p.sched[0] = 0ull;
      p.sched[1] = 0ull;
      __threadfence();
    }
  }
}

}  // namespace fa
