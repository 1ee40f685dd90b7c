// gated_mx.cuh -- the gated feed-forward block with many rows from MX operands
// (E4M3 activations, E4M3 or E2M1 weights, E8M0 scales per 32 inputs): 256-row
// tiles on pairs of SMs, cta_group::2 MMAs of M = 256, N = 256, 128 outputs a tile
// (lin_pair.cuh's layout: gate rows from the leader, up rows from its peer).
//
// The sums take 256 TMEM columns and the scales of 20 K blocks the rest: one set
// of sums, which the epilogue reads into registers and gives back before it goes
// on.  A thread of its own issues the scale copies to TMEM (tcgen05.cp), well
// ahead of the MMAs: between the MMAs they run in line with them, about 60 cycles
// each, three to a K block.
//
// Bound by the tensor pipe, MMAs and copies together: 4096 x 6144 x 1536 with the
// projections kept takes 77 us (2.0 PFLOP/s; 68 without), 0.42 us a K block where
// int8 tiles of the same size take 0.34, and some 1.2 us a tile to hand the sums over.
//
// Tried on 4096 x 6144 x 1536 and left: 96 outputs a tile and two sets of sums,
// with the scales laid out for any 32-row offset by four warps - stores to TMEM by
// those warps (tcgen05.st) wait for the MMAs' own traffic (107 us), larger copies
// (.128x256b) need a ring of replicated scales deeper than shared memory has room
// for (89 us).  MMAs of N = 128 for each weight, which would let one weight's first
// sums overlap the epilogue, are slower themselves (0.51 us a K block against 0.42).
#pragma once

#include "lin_pair.cuh"

namespace bq {

constexpr int kMxOut = 128;       // outputs of a tile
constexpr int kMxSfChunks = 4;    // K blocks of a scale stage, and of a set in TMEM

// Warps: 0 activation tile and scale copies, 1 TMEM and MMA issue, 2 weight tile
// copies, 3 scales to TMEM, 4-19 four epilogue groups.
constexpr int kMxThreads = 128 + 128 * kPairGroups;

struct GatedMxSmem {
  static constexpr int kBytesA = kBlockP * kBlockK;  // this CTA's 128 rows of A
  static constexpr int kBytesW = kMxOut * kBlockK;   // its 128 weight rows
  static constexpr int kStageTiles = kBytesA + kBytesW;
  static constexpr int kStages = 5;
  static constexpr int kSfBand = kMxSfChunks * kSfAtom;  // a band's atoms along K
  static constexpr int kSfBytes = 3 * kSfBand;           // A's band, both weights'
  static constexpr int kSfStages = 3;
  static constexpr int kSfCols = 12;  // TMEM columns of a K block
  static constexpr int kSfSet = kMxSfChunks * kSfCols;
  static constexpr int kSets = 5;
  static constexpr int kOffY = kStages * kStageTiles;
  static constexpr int kOffSf = kOffY + kPairGroups * kYChunkBytes;
  static constexpr int kOffBar = kOffSf + kSfStages * kSfBytes;
  static constexpr int kNumBars = 2 * kStages + 2 + 2 * kSfStages + 2 * kSets + 2;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kBytes = kOffMisc + 64 + 1024;  // + alignment slack
  static constexpr int kTmemCols = 512;
  static_assert(256 + kSets * kSfSet <= kTmemCols, "TMEM budget");
  static_assert(kBytes <= 232448, "shared memory budget");
};

__global__ void __launch_bounds__(kMxThreads, 1)
    gated_mx_kernel(const __grid_constant__ CUtensorMap tm_a,
                    const __grid_constant__ CUtensorMap tm_w0,
                    const __grid_constant__ CUtensorMap tm_w1,
                    const __grid_constant__ CUtensorMap tm_sfa,
                    const __grid_constant__ CUtensorMap tm_sf0,
                    const __grid_constant__ CUtensorMap tm_sf1,
                    const __grid_constant__ CUtensorMap tm_y,
                    const __grid_constant__ CUtensorMap tm_g,
                    const __grid_constant__ CUtensorMap tm_u, const FfnArgs a) {
  using L = GatedMxSmem;
  constexpr int kStages = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::kOffBar);
  uint64_t *empty = full + kStages;
  uint64_t *tfull = empty + kStages;
  uint64_t *tempty = tfull + 1;
  uint64_t *sf_full = tempty + 1;             // leader: a scale stage has landed in both CTAs
  uint64_t *sf_free = sf_full + L::kSfStages;  // it is in TMEM
  uint64_t *sf_tmem = sf_free + L::kSfStages;  // leader: a set is in both CTAs' TMEM
  uint64_t *sf_used = sf_tmem + L::kSets;      // leader: the MMAs have read it
  uint64_t *drain = sf_used + L::kSets;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kOffMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kOffMisc + 4);

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x / 2, num_pairs = gridDim.x / 2;
  const int total_units = a.tiles_p * a.tiles_q;

  if (threadIdx.x == 0) {
    for (int st = 0; st < kStages; ++st) {
      mbar_init(&full[st], 2);   // the leader's copy threads (bytes of both CTAs)
      mbar_init(&empty[st], 1);  // the leader's commit
    }
    mbar_init(tfull, 1);
    mbar_init(tempty, 8 * kPairGroups);  // every epilogue warp of both CTAs
    for (int i = 0; i < L::kSfStages; ++i) {
      mbar_init(&sf_full[i], 1);
      mbar_init(&sf_free[i], 1);
    }
    for (int i = 0; i < L::kSets; ++i) {
      mbar_init(&sf_tmem[i], 1);
      mbar_init(&sf_used[i], 1);
    }
    mbar_init(drain, 1);
    mbar_init(drain + 1, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(rank == 1 ? &tm_w1 : &tm_w0);
  }
  if (warp == 1) tmem_alloc2(tmem_slot, L::kTmemCols);
  tc_fence_before();
  __syncthreads();
  // Copies of both CTAs complete on the leader's barriers and its commits arrive
  // on both: everything is set up before anything crosses.
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t sf_cols = tmem_base + 256;

  if (warp == 0 || warp == 2) {
    // -------------------------------------------------------- tile copies --
    if (lane == 0) {
      if (warp == 0) {  // the activations may come from the kernel before
        griddep_wait();
        griddep_launch_dependents();
      }
      const uint32_t tx = 2 * (warp == 0 ? static_cast<uint32_t>(L::kBytesA) : a.w_tile_bytes);
      const CUtensorMap *map = warp == 0 ? &tm_a : rank == 1 ? &tm_w1 : &tm_w0;
      int stage = 0, sf_stage = 0;
      uint32_t phase = 0, sf_phase = 0;
      bool ok = true;
      for (int unit = pair; unit < total_units && ok; unit += num_pairs) {
        const UnitPos u = unit_pos(a, unit);
        const int band = 2 * u.tp + static_cast<int>(rank);  // this CTA's 128 rows of A
        const int row = warp == 0 ? band * 128 : u.tq * kMxOut;
        for (int kt = 0; kt < a.kt_total; ++kt) {
          if (warp == 0 && kt % kMxSfChunks == 0) {
            if (!mbar_wait(&sf_free[sf_stage], sf_phase ^ 1, a.err, abort_flag, kWaitProdEmpty)) {
              ok = false;
              break;
            }
            if (rank == 0)
              mbar_arrive_expect_tx(&sf_full[sf_stage], 2 * static_cast<uint32_t>(L::kSfBytes));
            const uint32_t bar = mapa_shared(smem_u32(&sf_full[sf_stage]), 0);
            uint8_t *sf = smem + L::kOffSf + sf_stage * L::kSfBytes;
            tma2_load_3d(sf, &tm_sfa, bar, 0, kt, band);
            tma2_load_3d(sf + L::kSfBand, &tm_sf0, bar, 0, kt, u.tq);
            tma2_load_3d(sf + 2 * L::kSfBand, &tm_sf1, bar, 0, kt, u.tq);
            if (++sf_stage == L::kSfStages) {
              sf_stage = 0;
              sf_phase ^= 1;
            }
          }
          if (!mbar_wait(&empty[stage], phase ^ 1, a.err, abort_flag, kWaitProdEmpty)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], tx);
          tma2_load_3d(smem + stage * L::kStageTiles + (warp == 0 ? 0 : L::kBytesA), map,
                       mapa_shared(smem_u32(&full[stage]), 0), kt * kBlockK, row, 0);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (!ok) sleep_ns(200000);  // copies already issued land before the CTA goes away
    }
  } else if (warp == 1) {
    // ------------------------------------------------- MMA issue (leader) --
    if (rank == 0 && lane == 0) {
      const uint32_t tiles0 = smem_u32(smem);
      int stage = 0, set = 0;
      uint32_t phase = 0, acc_phase = 0, set_phase = 0;
      bool ok = true;
      for (int unit = pair; unit < total_units && ok; unit += num_pairs) {
        if (!mbar_wait(tempty, acc_phase ^ 1, a.err, abort_flag, kWaitMmaTmemEmpty)) break;
        acc_phase ^= 1;
        tc_fence_after();
        for (int kt = 0; kt < a.kt_total; ++kt) {
          const int sc = kt % kMxSfChunks;  // this K block in its scale set
          if ((sc == 0 && !mbar_wait(&sf_tmem[set], set_phase, a.err, abort_flag, kWaitMmaFull)) ||
              !mbar_wait(&full[stage], phase, a.err, abort_flag, kWaitMmaFull)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t ta = tiles0 + stage * L::kStageTiles, tb = ta + L::kBytesA;
          const uint32_t sf = sf_cols + set * L::kSfSet + sc * L::kSfCols;
#pragma unroll
          for (int ks = 0; ks < kBlockK / kMmaK; ++ks)
            tc_mma2_mxf8f6f4(tmem_base, desc_kmajor_sw128(ta + ks * kMmaK),
                             desc_kmajor_sw128(tb + ks * kMmaK),
                             make_idesc_m(a.fmt_a, a.fmt_w, 256, 256, ks), sf, sf + 4,
                             (kt > 0 || ks > 0) ? 1u : 0u);
          tc_commit2_both(&empty[stage]);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
          if (sc == kMxSfChunks - 1 || kt == a.kt_total - 1) {
            tc_commit2(mapa_shared(smem_u32(&sf_used[set]), 0));
            if (++set == L::kSets) {
              set = 0;
              set_phase ^= 1;
            }
          }
        }
        if (!ok) break;
        tc_commit2_both(tfull);
      }
      tc_commit2(mapa_shared(smem_u32(drain), 0));
      if (!mbar_wait_timed(drain, 0, a.err, kWaitDrain)) sleep_ns(200000);
    }
  } else if (warp == 3) {
    // ------------------------------------------- scales to TMEM (leader) --
    if (rank == 0 && lane == 0) {
      const uint32_t sf0 = smem_u32(smem + L::kOffSf);
      int stage = 0, set = 0;
      uint32_t phase = 0, set_phase = 0;
      bool ok = true;
      for (int unit = pair; unit < total_units && ok; unit += num_pairs) {
        for (int kt = 0; kt < a.kt_total; kt += kMxSfChunks) {
          if (!mbar_wait(&sf_used[set], set_phase ^ 1, a.err, abort_flag, kWaitMmaFull) ||
              !mbar_wait(&sf_full[stage], phase, a.err, abort_flag, kWaitMmaFull)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int nv = min(kMxSfChunks, a.kt_total - kt);
#pragma unroll 1
          for (int c = 0; c < nv; ++c)
#pragma unroll
            for (int j = 0; j < 3; ++j)
              tc_cp_sf2(sf_cols + set * L::kSfSet + c * L::kSfCols + 4 * j,
                        desc_sf_32x128b(sf0 + stage * L::kSfBytes + j * L::kSfBand + c * kSfAtom));
          tc_commit2(mapa_shared(smem_u32(&sf_tmem[set]), 0));
          tc_commit2_both(&sf_free[stage]);
          if (++stage == L::kSfStages) {
            stage = 0;
            phase ^= 1;
          }
          if (++set == L::kSets) {
            set = 0;
            set_phase ^= 1;
          }
        }
      }
      tc_commit2(mapa_shared(smem_u32(drain + 1), 0));
      if (!mbar_wait_timed(drain + 1, 0, a.err, kWaitDrain)) sleep_ns(200000);
    }
  } else {
    // ---------------------------------------------- epilogue (both CTAs) --
    const int quad = warp % 4;  // TMEM lane quadrant this warp may access
    const int row = quad * 32 + lane;
    const int group = (warp - 4) / 4;
    const OutSlot out{smem + L::kOffY + group * kYChunkBytes, row, group,
                      static_cast<int>(threadIdx.x % 128)};
    const uint32_t lead_tempty = mapa_shared(smem_u32(tempty), 0);
    uint32_t acc_phase = 0;
    griddep_wait();  // the kernel before may still use the outputs' memory
    for (int unit = pair; unit < total_units; unit += num_pairs) {
      const UnitPos u = unit_pos(a, unit);
      const int m0 = (2 * u.tp + static_cast<int>(rank)) * 128;
      const int q0 = u.tq * kMxOut + group * 32;
      __syncwarp();
      if (!mbar_wait(tfull, acc_phase, a.err, abort_flag, kWaitEpiFull)) break;
      acc_phase ^= 1;
      __syncwarp();
      tc_fence_after();
      const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
      // all sums into registers, then their TMEM goes back to the MMAs
      uint32_t vg[32], vu[32];
      tmem_ld_32x32b_x32(t_row + group * 32, vg);
      tmem_ld_32x32b_x32(t_row + kMxOut + group * 32, vu);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_pair(lead_tempty);
      if (q0 < a.N)  // uniform
        gated_chunk(a, out, &tm_y, &tm_g, &tm_u, vg, vu, q0, m0);
    }
  }

  // The last stores are done, and neither CTA's barriers, shared memory or TMEM
  // are in use, when the pair leaves.
  if (warp >= 4 && threadIdx.x % 128 == 0) bulk_wait_group_all();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc2(tmem_base, L::kTmemCols);
  }
}

}  // namespace bq
