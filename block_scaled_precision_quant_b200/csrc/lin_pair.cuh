// lin_pair.cuh -- int8 products and gated feed-forward blocks with many rows:
// 256-row tiles on pairs of SMs (a cluster of 2), computed by tcgen05 MMAs of
// the cta_group::2 form with M = 256, N = 256.
//
// A pair's tile is 256 rows of A against 256 weight rows.  Each CTA loads its
// own 128 rows of A and 128 of the weight rows; the pair's MMAs, issued by the
// leader (rank 0), read both CTAs' shared memory and leave each CTA its own 128
// rows x 256 sums in TMEM.  Plain products take 256 consecutive weight rows:
// 256 outputs.  Gated ones take 128 rows of the gate's weight, loaded by the
// leader, and the same 128 rows of the up projection's, loaded by its peer:
// column j and column 128 + j of a sum row are g and u of one output, so the
// product is formed in the registers of one thread.
//
// Per 128 K an SM brings 32 KB into shared memory for 512 cycles of MMAs, a
// third less than a 128 x 256 tile of its own needs.  Int8 keeps two sets of
// sums (2 x 256 TMEM columns): the epilogue of one tile runs under the MMAs of
// the next.  MX tiles need TMEM for scales and keep one set, which the
// epilogue reads into registers and gives back before it goes on.
#pragma once

#include "ffn_args.cuh"
#include "gemm_pair.cuh"

namespace bq {

// Warps: 0 activation tile copies, 1 TMEM and MMA issue, 2 weight tile copies,
// 3 scale copies (MX), 4-7 and 8-11 two epilogue groups.
constexpr int kLinPairThreads = 384;

template <bool I8>
struct LinPairSmem {
  static constexpr int kBytesA = kBlockP * kBlockK;  // this CTA's 128 rows of A
  static constexpr int kBytesB = kBlockP * kBlockK;  // its 128 weight rows
  static constexpr int kStageTiles = kBytesA + kBytesB;
  static constexpr int kSfBytes = I8 ? 0 : 3 * kSfAtom;  // A's band, both weight bands
  static constexpr int kStages = I8 ? 6 : 5;
  static constexpr int kAcc = I8 ? 2 : 1;
  static constexpr int kSfCols = I8 ? 0 : 12;
  static constexpr int kSlots = I8 ? 2 : 3;  // 128 x 32 bf16 staging tiles of an epilogue group
  static constexpr int kOffY = kStages * kStageTiles;
  static constexpr int kOffSf = kOffY + 2 * kSlots * kYChunkBytes;
  static constexpr int kOffBar = kOffSf + kStages * kSfBytes;
  static constexpr int kNumBars = 2 * kStages + 2 * kAcc + 1;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kBytes = kOffMisc + 64 + 1024;  // + alignment slack
  static constexpr int kTmemCols = 512;
  static_assert(kAcc * 256 + kStages * kSfCols <= kTmemCols, "TMEM budget");
  static_assert(kBytes <= 232448, "shared memory budget");
};

__device__ __forceinline__ void tc_mma2_i8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t"
      "}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrive on the barrier at this shared-memory offset in both CTAs of the pair
// once every pair MMA and copy this thread issued has completed.
__device__ __forceinline__ void tc_commit2_both(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// Named barrier of one epilogue group's 128 threads.
__device__ __forceinline__ void group_sync(int group) {
  __syncwarp();
  asm volatile("barrier.sync %0, 128;" ::"r"(1 + group) : "memory");
}

// An epilogue group's way out: its ring of staging tiles and the next one's number.
template <int SLOTS>
struct OutRing {
  uint8_t *base;
  int row, group, tid;  // tid: 0 .. 127 in the group
  int next;
};

// One 128-row x 32-column chunk of bf16 outputs (thread = row) through the ring to
// the tensor behind `map` at column q0 of rows m0 ...: TMA stores leave out what
// lies outside the tensor.  A slot is written again once all but the latest
// SLOTS - 1 stores have read theirs.
template <int SLOTS>
__device__ __forceinline__ void store_chunk(OutRing<SLOTS> &ring, const CUtensorMap *map, int q0,
                                            int m0, int M, int b, const uint32_t (&o)[16]) {
  uint8_t *slot = ring.base + ring.next * kYChunkBytes;
  ring.next = ring.next + 1 == SLOTS ? 0 : ring.next + 1;
  if (ring.tid == 0) bulk_wait_group_read<SLOTS - 1>();
  group_sync(ring.group);
  const int row = ring.row;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint4 *>(slot + row * 64 + ((j ^ ((row >> 1) & 3)) << 4)) =
        make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
  fence_proxy_async_smem();
  group_sync(ring.group);
  if (ring.tid == 0) {
    if (m0 < M) tma_store_3d(map, slot, q0, m0, b);
    bulk_commit_group();
  }
}

// The fp32 values alpha * scale * sum of 32 columns n ... of one row.  Int8: `sa`
// is the row's scale, sw the columns' (n % 8 == 0 keeps each read of four inside).
template <bool I8>
__device__ __forceinline__ void scaled32(const uint32_t (&v)[32], float alpha, float sa,
                                         const float *sw, int n, int N, float (&f)[32]) {
  if constexpr (I8) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
      if (n + 4 * j < N) s = __ldg(reinterpret_cast<const float4 *>(sw + n) + j);
      const float s4[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        f[4 * j + i] = __int2float_rn(static_cast<int>(v[4 * j + i])) * (sa * (alpha * s4[i]));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j) f[j] = alpha * __uint_as_float(v[j]);
  }
}

template <bool I8, bool GATED>
__global__ void __launch_bounds__(kLinPairThreads, 1)
    lin_pair_kernel(const __grid_constant__ CUtensorMap tm_a,
                    const __grid_constant__ CUtensorMap tm_w0,
                    const __grid_constant__ CUtensorMap tm_w1,
                    const __grid_constant__ CUtensorMap tm_sfa,
                    const __grid_constant__ CUtensorMap tm_sf0,
                    const __grid_constant__ CUtensorMap tm_sf1,
                    const __grid_constant__ CUtensorMap tm_y,
                    const __grid_constant__ CUtensorMap tm_g,
                    const __grid_constant__ CUtensorMap tm_u, const FfnArgs a) {
  using L = LinPairSmem<I8>;
  constexpr int kStages = L::kStages, kAcc = L::kAcc;
  constexpr int kTileN = GATED ? 128 : 256;  // outputs of a tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::kOffBar);
  uint64_t *empty = full + kStages;
  uint64_t *tfull = empty + kStages;
  uint64_t *tempty = tfull + kAcc;
  uint64_t *drain = tempty + kAcc;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kOffMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kOffMisc + 4);

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x / 2, num_pairs = gridDim.x / 2;
  const int total_units = a.batch * a.tiles_p * a.tiles_q;

  if (threadIdx.x == 0) {
    for (int st = 0; st < kStages; ++st) {
      mbar_init(&full[st], I8 ? 2 : 3);  // the leader's copy threads (bytes of both CTAs)
      mbar_init(&empty[st], 1);          // the leader's commit
    }
    for (int i = 0; i < kAcc; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 16);  // every epilogue warp of both CTAs
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(rank == 1 && GATED ? &tm_w1 : &tm_w0);
    if (!I8) {
      tma_prefetch_desc(&tm_sfa);
      tma_prefetch_desc(&tm_sf0);
      tma_prefetch_desc(&tm_sf1);
    }
  }
  if (warp == 1) tmem_alloc2(tmem_slot, L::kTmemCols);
  tc_fence_before();
  __syncthreads();
  // Copies of both CTAs complete on the leader's barriers and its commits arrive
  // on both: everything is set up before anything crosses.
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0 || warp == 2 || (!I8 && warp == 3)) {
    // ------------------------------------------------------------- copies --
    if (lane == 0) {
      if (warp != 2) {  // activations and their scales may come from the kernel before
        griddep_wait();
        if (warp == 0) griddep_launch_dependents();
      }
      const uint32_t tx = warp == 0   ? 2 * L::kBytesA
                          : warp == 2 ? 2 * a.w_tile_bytes
                                      : 2 * static_cast<uint32_t>(L::kSfBytes);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int unit = pair; unit < total_units && ok; unit += num_pairs) {
        const UnitPos u = unit_pos(a, unit);
        const int band = 2 * u.tp + static_cast<int>(rank);  // this CTA's 128 rows of A
        const int brow = GATED ? u.tq * 128 : u.tq * 256 + static_cast<int>(rank) * 128;
        const int ba = a.q_batched ? u.b : 0, bw = a.p_batched ? u.b : 0;
        for (int kt = 0; kt < a.kt_total; ++kt) {
          if (!mbar_wait(&empty[stage], phase ^ 1, a.err, abort_flag, kWaitProdEmpty)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], tx);
          const uint32_t bar = mapa_shared(smem_u32(&full[stage]), 0);
          uint8_t *tiles = smem + stage * L::kStageTiles;
          if (warp == 0) {
            tma2_load_3d(tiles, &tm_a, bar, kt * kBlockK, band * 128, ba);
          } else if (warp == 2) {
            tma2_load_3d(tiles + L::kBytesA, GATED && rank == 1 ? &tm_w1 : &tm_w0, bar,
                         kt * kBlockK, brow, bw);
          } else {
            uint8_t *sf = smem + L::kOffSf + stage * L::kSfBytes;
            tma2_load_3d(sf, &tm_sfa, bar, 0, kt, band);
            tma2_load_3d(sf + kSfAtom, &tm_sf0, bar, 0, kt, u.tq);
            tma2_load_3d(sf + 2 * kSfAtom, &tm_sf1, bar, 0, kt, u.tq);
          }
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
      const uint32_t tiles0 = smem_u32(smem), sf0 = smem_u32(smem + L::kOffSf);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int unit = pair; unit < total_units && ok; unit += num_pairs) {
        if (!mbar_wait_cluster(&tempty[acc], acc_phase ^ 1, a.err, abort_flag, kWaitMmaTmemEmpty))
          break;
        tc_fence_after();
        const uint32_t d = tmem_base + acc * 256;
        for (int kt = 0; kt < a.kt_total; ++kt) {
          if (!mbar_wait(&full[stage], phase, a.err, abort_flag, kWaitMmaFull)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t ta = tiles0 + stage * L::kStageTiles, tb = ta + L::kBytesA;
          const uint32_t sf_t = tmem_base + kAcc * 256 + stage * L::kSfCols;
          if constexpr (!I8) {
#pragma unroll
            for (int j = 0; j < 3; ++j)
              tc_cp_sf2(sf_t + 4 * j,
                        desc_sf_32x128b(sf0 + stage * L::kSfBytes + j * kSfAtom));
          }
#pragma unroll
          for (int ks = 0; ks < kBlockK / kMmaK; ++ks) {
            const uint32_t acc_in = (kt > 0 || ks > 0) ? 1u : 0u;
            const uint64_t da = desc_kmajor_sw128(ta + ks * kMmaK);
            const uint64_t db = desc_kmajor_sw128(tb + ks * kMmaK);
            if constexpr (I8)
              tc_mma2_i8(d, da, db, idesc_i8(256, 256), acc_in);
            else
              tc_mma2_mxf8f6f4(d, da, db, make_idesc_m(a.fmt_a, a.fmt_w, 256, 256, ks), sf_t,
                               sf_t + 4, acc_in);
          }
          tc_commit2_both(&empty[stage]);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        tc_commit2_both(&tfull[acc]);
        if (++acc == kAcc) {
          acc = 0;
          acc_phase ^= 1;
        }
      }
      tc_commit2(mapa_shared(smem_u32(drain), 0));
      if (!mbar_wait_timed(drain, 0, a.err, kWaitDrain)) sleep_ns(200000);
    }
  } else if (warp >= 4) {
    // ---------------------------------------------- epilogue (both CTAs) --
    const int quad = warp % 4;  // TMEM lane quadrant this warp may access
    const int row = quad * 32 + lane;
    const int group = (warp - 4) / 4;
    OutRing<L::kSlots> ring{smem + L::kOffY + group * L::kSlots * kYChunkBytes, row, group,
                            static_cast<int>(threadIdx.x % 128), 0};
    const uint32_t lead_tempty = mapa_shared(smem_u32(tempty), 0);
    int acc = 0;
    uint32_t acc_phase = 0;
    griddep_wait();  // scales, bias and residual may come from the kernel before
    for (int unit = pair; unit < total_units; unit += num_pairs) {
      const UnitPos u = unit_pos(a, unit);
      const int m0 = (2 * u.tp + static_cast<int>(rank)) * 128, m = m0 + row;
      const int n0 = u.tq * kTileN;
      const bool mok = m < a.M;
      const float sa = I8 && mok ? __ldg(a.sa + u.b * a.sa_bstride + m) : 0.0f;
      __syncwarp();
      if (!mbar_wait_cluster(&tfull[acc], acc_phase, a.err, abort_flag, kWaitEpiFull)) break;
      tc_fence_after();
      const uint32_t t_row = tmem_base + acc * 256 + (static_cast<uint32_t>(quad * 32) << 16);
      const int nch = min(kTileN / 32, (a.N - n0 + 31) / 32);
      if constexpr (GATED) {
        // This group's two chunks of 32 outputs: first all sums into registers,
        // then the sums' TMEM goes back to the MMAs.
        uint32_t vg[2][32], vu[2][32];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int c = group + 2 * i;
          __syncwarp();
          tmem_ld_32x32b_x32(t_row + c * 32, vg[i]);
          tmem_ld_32x32b_x32(t_row + 128 + c * 32, vu[i]);
        }
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(lead_tempty + acc * 8);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int c = group + 2 * i;
          if (c >= nch) break;  // uniform
          const int q0 = n0 + c * 32;
          float g[32], up[32];
          scaled32<I8>(vg[i], a.alpha, sa, a.sw[0], q0, a.N, g);
          scaled32<I8>(vu[i], a.alpha, sa, a.sw[1], q0, a.N, up);
          uint32_t o[16];
          if (a.gu) {
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = pack_bf16(g[2 * j], g[2 * j + 1]);
            store_chunk(ring, &tm_g, q0, m0, a.M, 0, o);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = pack_bf16(up[2 * j], up[2 * j + 1]);
            store_chunk(ring, &tm_u, q0, m0, a.M, 0, o);
          }
          if (a.act == kGateSilu) {
#pragma unroll
            for (int j = 0; j < 32; ++j) g[j] = silu(g[j]) * up[j];
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) g[j] = gelu_erf(g[j]) * up[j];
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) o[j] = pack_bf16(g[2 * j], g[2 * j + 1]);
          if (a.q_out) quant_out_row32(a, 0, m, q0, o);
          if (a.y) store_chunk(ring, &tm_y, q0, m0, a.M, 0, o);
        }
      } else {
#pragma unroll 1
        for (int c = group; c < nch; c += 2) {
          const int q0 = n0 + c * 32;
          uint32_t v[32];
          __syncwarp();
          tmem_ld_32x32b_x32(t_row + c * 32, v);
          uint4 rv[4];
          if (a.res) {
            const __nv_bfloat16 *r =
                a.res + u.b * a.res_bstride + static_cast<int64_t>(m) * a.ldres + q0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              rv[j] = mok && q0 + 8 * j < a.N ? *reinterpret_cast<const uint4 *>(r + 8 * j)
                                              : make_uint4(0u, 0u, 0u, 0u);
          }
          tmem_ld_wait();
          float f[32];
          scaled32<I8>(v, a.alpha, sa, a.sw[0] + u.b * a.sw_bstride, q0, a.N, f);
          if (a.bias) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (q0 + 8 * j >= a.N) break;
              const uint4 bv = __ldg(reinterpret_cast<const uint4 *>(a.bias + q0 + 8 * j));
              const uint32_t w[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                f[8 * j + 2 * i] += bf16_bits_to_f32(w[i] & 0xFFFFu);
                f[8 * j + 2 * i + 1] += bf16_bits_to_f32(w[i] >> 16);
              }
            }
          }
          if (a.act == 1) {
#pragma unroll
            for (int j = 0; j < 32; ++j) f[j] = gelu_erf(f[j]);
          }
          if (a.res) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t w[4] = {rv[j].x, rv[j].y, rv[j].z, rv[j].w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                f[8 * j + 2 * i] += bf16_bits_to_f32(w[i] & 0xFFFFu);
                f[8 * j + 2 * i + 1] += bf16_bits_to_f32(w[i] >> 16);
              }
            }
          }
          uint32_t o[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) o[j] = pack_bf16(f[2 * j], f[2 * j + 1]);
          store_chunk(ring, &tm_y, q0, m0, a.M, u.b, o);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(lead_tempty + acc * 8);
      }
      if (++acc == kAcc) {
        acc = 0;
        acc_phase ^= 1;
      }
    }
  }

  // The last stores are done, and neither CTA's barriers, shared memory or TMEM
  // are in use, when the pair leaves.
  if (threadIdx.x == 128 || threadIdx.x == 256) bulk_wait_group_all();
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
