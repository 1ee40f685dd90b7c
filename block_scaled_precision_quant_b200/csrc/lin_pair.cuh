// lin_pair.cuh -- int8 products and gated feed-forward blocks with many rows:
// 256-row tiles on pairs of SMs (a cluster of 2), computed by tcgen05 MMAs of
// the cta_group::2 form with M = 256, N = 256.  (MX operands: gated_mx.cuh.)
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
// third less than a 128 x 256 tile of its own needs.  Two sets of sums (2 x 256
// TMEM columns): the epilogue of one tile runs under the MMAs of the next.
//
// Bound by the MMAs, and under a lasting load by the power cap on their clock: int8
// 8192^3 330 to 400 us (3.3 to 2.7 Pop/s; the tensor pipe busy 84 % of the cycles at
// 4096 x 8192 x 4096), gated 2048 x 8192 x 4096 94 us (2.9 Pop/s).
#pragma once

#include "ffn_args.cuh"
#include "gemm_pair.cuh"

namespace bq {

// Warps: 0 activation tile copies, 1 TMEM and MMA issue, 2 weight tile copies, 3
// none, 4-19 four epilogue groups of four, one warp to a quadrant of the TMEM
// lanes.
constexpr int kLinPairThreads = 640;
constexpr int kPairGroups = 4;

// RES: products with a residual, whose chunks come by TMA into the staging tiles
// before the sums stand; two tiles a group then, for one operand stage less.
template <bool RES>
struct LinPairSmem {
  static constexpr int kBytesA = kBlockP * kBlockK;  // this CTA's 128 rows of A
  static constexpr int kBytesB = kBlockP * kBlockK;  // its 128 weight rows
  static constexpr int kStageTiles = kBytesA + kBytesB;
  static constexpr int kStages = RES ? 5 : 6;
  static constexpr int kSlots = RES ? 2 : 1;           // 128 x 32 bf16 staging tiles a group
  static constexpr int kOffY = kStages * kStageTiles;
  static constexpr int kOffBar = kOffY + kPairGroups * kSlots * kYChunkBytes;
  static constexpr int kNumBars = 2 * kStages + 2 * 2 + 1 + (RES ? kPairGroups * kSlots : 0);
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kBytes = kOffMisc + 64 + 1024;  // + alignment slack
  static constexpr int kTmemCols = 512;
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

// Arrive on an mbarrier given by its shared::cluster address, ordering nothing but
// what tcgen05.fence::before_thread_sync has: no memory passes hands by it, and a
// release at cluster scope would wait for the epilogue's stores.
__device__ __forceinline__ void mbar_arrive_pair(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Named barrier of one epilogue group's 128 threads.
__device__ __forceinline__ void group_sync(int group) {
  __syncwarp();
  asm volatile("barrier.sync %0, 128;" ::"r"(1 + group) : "memory");
}

// An epilogue group's way out: its staging tile.
struct OutSlot {
  uint8_t *slot;
  int row, group, tid;  // tid: 0 .. 127 in the group
};

// One 128-row x 32-column chunk of bf16 outputs (thread = row) through the group's
// staging tile to the tensor behind `map` at column q0 of rows m0 ...: TMA stores
// leave out what lies outside the tensor.
__device__ __forceinline__ void store_chunk(const OutSlot &out, const CUtensorMap *map, int q0,
                                            int m0, int M, int b, const uint32_t (&o)[16]) {
  if (out.tid == 0) bulk_wait_group_read<0>();  // the group's previous store has read the tile
  group_sync(out.group);
  const int row = out.row;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint4 *>(out.slot + row * 64 + ((j ^ ((row >> 1) & 3)) << 4)) =
        make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
  fence_proxy_async_smem();
  group_sync(out.group);
  if (out.tid == 0 && m0 < M) {
    tma_store_3d(map, out.slot, q0, m0, b);
    bulk_commit_group();
  }
}

// The values sa sw[j] v[j] of 32 columns of one row; lane j holds the scale of
// column j (with so much shared memory in use there is no L1 to keep the scales
// in: every lane reading all of them went to L2 each time).
__device__ __forceinline__ void scaled32(const uint32_t (&v)[32], float sa, float sw,
                                         float (&f)[32]) {
#pragma unroll
  for (int j = 0; j < 32; ++j)
    f[j] = __int2float_rn(static_cast<int>(v[j])) * (sa * __shfl_sync(0xFFFFFFFFu, sw, j));
}

// 32 gated outputs of one row (columns q0 ...), from g and u: the projections on
// request, h = act(g) u, its codes and scales on request.
__device__ __forceinline__ void gated_out(const FfnArgs &a, const OutSlot &out,
                                          const CUtensorMap *tm_y, const CUtensorMap *tm_g,
                                          const CUtensorMap *tm_u, float (&g)[32],
                                          const float (&up)[32], int q0, int m0) {
  uint32_t o[16];
  if (a.gu) {
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j] = pack_bf16(g[2 * j], g[2 * j + 1]);
    store_chunk(out, tm_g, q0, m0, a.M, 0, o);
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j] = pack_bf16(up[2 * j], up[2 * j + 1]);
    store_chunk(out, tm_u, q0, m0, a.M, 0, o);
  }
  if (a.act == kGateSilu) {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      o[j] = pack_bf16(mul2(silu2(f2(g[2 * j], g[2 * j + 1])), f2(up[2 * j], up[2 * j + 1])));
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      o[j] = pack_bf16(mul2(gelu_gate2(f2(g[2 * j], g[2 * j + 1])), f2(up[2 * j], up[2 * j + 1])));
  }
  if (a.q_out) quant_out_row32(a, 0, m0 + out.row, q0, o);
  if (a.y) store_chunk(out, tm_y, q0, m0, a.M, 0, o);
}

// The same from fp32 sums (their bits).
__device__ __forceinline__ void gated_chunk(const FfnArgs &a, const OutSlot &out,
                                            const CUtensorMap *tm_y, const CUtensorMap *tm_g,
                                            const CUtensorMap *tm_u, const uint32_t (&vg)[32],
                                            const uint32_t (&vu)[32], int q0, int m0) {
  float g[32], up[32];
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    g[j] = a.alpha * __uint_as_float(vg[j]);
    up[j] = a.alpha * __uint_as_float(vu[j]);
  }
  gated_out(a, out, tm_y, tm_g, tm_u, g, up, q0, m0);
}

template <bool GATED, bool RES>
__global__ void __launch_bounds__(kLinPairThreads, 1)
    lin_pair_kernel(const __grid_constant__ CUtensorMap tm_a,
                    const __grid_constant__ CUtensorMap tm_w0,
                    const __grid_constant__ CUtensorMap tm_w1,
                    const __grid_constant__ CUtensorMap tm_y,
                    const __grid_constant__ CUtensorMap tm_g,   // RES: the residual
                    const __grid_constant__ CUtensorMap tm_u, const FfnArgs a) {
  static_assert(!(GATED && RES), "the gated block has no residual");
  using L = LinPairSmem<RES>;
  constexpr int kStages = L::kStages, kAcc = 2;
  constexpr int kTileN = GATED ? 128 : 256;  // outputs of a tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::kOffBar);
  uint64_t *empty = full + kStages;
  uint64_t *tfull = empty + kStages;
  uint64_t *tempty = tfull + kAcc;
  uint64_t *drain = tempty + kAcc;
  uint64_t *rbar = drain + 1;  // RES: a residual chunk has landed in its staging tile
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kOffMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kOffMisc + 4);

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x / 2, num_pairs = gridDim.x / 2;
  const int total_units = a.batch * a.tiles_p * a.tiles_q;

  if (threadIdx.x == 0) {
    for (int st = 0; st < kStages; ++st) {
      mbar_init(&full[st], 2);   // the leader's copy threads (bytes of both CTAs)
      mbar_init(&empty[st], 1);  // the leader's commit
    }
    for (int i = 0; i < kAcc; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 8 * kPairGroups);  // every epilogue warp of both CTAs
    }
    mbar_init(drain, 1);
    if (RES)
      for (int i = 0; i < kPairGroups * L::kSlots; ++i) mbar_init(&rbar[i], 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(rank == 1 && GATED ? &tm_w1 : &tm_w0);
  }
  if (warp == 1) tmem_alloc2(tmem_slot, L::kTmemCols);
  tc_fence_before();
  __syncthreads();
  // Copies of both CTAs complete on the leader's barriers and its commits arrive
  // on both: everything is set up before anything crosses.
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0 || warp == 2) {
    // -------------------------------------------------------- tile copies --
    if (lane == 0) {
      griddep_wait();  // both operands may come from the kernel before
      if (warp == 0) griddep_launch_dependents();
      const uint32_t tx = warp == 0 ? 2 * L::kBytesA : 2 * a.w_tile_bytes;
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int unit = pair; unit < total_units && ok; unit += num_pairs) {
        const UnitPos u = unit_pos(a, unit);
        const int row = warp == 0 ? (2 * u.tp + static_cast<int>(rank)) * 128
                        : GATED   ? u.tq * 128
                                  : u.tq * 256 + static_cast<int>(rank) * 128;
        const int bt = warp == 0 ? (a.q_batched ? u.b : 0) : (a.p_batched ? u.b : 0);
        const CUtensorMap *map = warp == 0 ? &tm_a : GATED && rank == 1 ? &tm_w1 : &tm_w0;
        for (int kt = 0; kt < a.kt_total; ++kt) {
          if (!mbar_wait(&empty[stage], phase ^ 1, a.err, abort_flag, kWaitProdEmpty)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], tx);
          tma2_load_3d(smem + stage * L::kStageTiles + (warp == 0 ? 0 : L::kBytesA), map,
                       mapa_shared(smem_u32(&full[stage]), 0), kt * kBlockK, row, bt);
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
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int unit = pair; unit < total_units && ok; unit += num_pairs) {
        if (!mbar_wait(&tempty[acc], acc_phase ^ 1, a.err, abort_flag, kWaitMmaTmemEmpty))
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
#pragma unroll
          for (int ks = 0; ks < kBlockK / kMmaK; ++ks)
            tc_mma2_i8(d, desc_kmajor_sw128(ta + ks * kMmaK), desc_kmajor_sw128(tb + ks * kMmaK),
                       idesc_i8(256, 256), (kt > 0 || ks > 0) ? 1u : 0u);
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
    const OutSlot out{smem + L::kOffY + group * L::kSlots * kYChunkBytes, row, group,
                      static_cast<int>(threadIdx.x % 128)};
    const uint32_t lead_tempty = mapa_shared(smem_u32(tempty), 0);
    int acc = 0;
    uint32_t acc_phase = 0;
    uint32_t rphase = 0;  // bit i: parity of staging tile i's residual barrier
    griddep_wait();  // scales, bias and residual may come from the kernel before
    for (int unit = pair; unit < total_units; unit += num_pairs) {
      const UnitPos u = unit_pos(a, unit);
      const int m0 = (2 * u.tp + static_cast<int>(rank)) * 128, m = m0 + row;
      const int n0 = u.tq * kTileN;
      const int nch = min(kTileN / 32, (a.N - n0 + 31) / 32);
      // what the outputs need besides the sums, fetched while the sums are formed
      const float sa = m < a.M ? __ldg(a.sa + u.b * a.sa_bstride + m) : 0.0f;
      float sw[2], bias[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // gated: the group's one chunk of both weights; plain: its two chunks
        const int n = n0 + (GATED ? group : group + kPairGroups * i) * 32 + lane;
        sw[i] = n < a.N ? a.alpha * __ldg(a.sw[GATED ? i : 0] + u.b * a.sw_bstride + n) : 0.0f;
        bias[i] = !GATED && a.bias && n < a.N ? __bfloat162float(a.bias[n]) : 0.0f;
      }
      if (RES && out.tid == 0) {
        bulk_wait_group_read<0>();  // earlier stores have read the staging tiles
        // Only chunks that exist: the group meets (group_sync) behind each wait for a
        // chunk, so no thread arms a barrier again that another has yet to wait on.
#pragma unroll
        for (int i = 0; i < L::kSlots; ++i) {
          if (group + kPairGroups * i >= nch) break;
          uint64_t *bar = &rbar[group * L::kSlots + i];
          mbar_arrive_expect_tx(bar, static_cast<uint32_t>(kYChunkBytes));
          tma_load_3d(out.slot + i * kYChunkBytes, &tm_g, bar,
                      n0 + (group + kPairGroups * i) * 32, m0, a.res_bstride ? u.b : 0);
        }
      }
      __syncwarp();
      if (!mbar_wait(&tfull[acc], acc_phase, a.err, abort_flag, kWaitEpiFull)) break;
      __syncwarp();
      tc_fence_after();
      const uint32_t t_row = tmem_base + acc * 256 + (static_cast<uint32_t>(quad * 32) << 16);
      if constexpr (GATED) {
        // This group's 32 outputs: all sums into registers, then their TMEM goes
        // back to the MMAs.
        const int q0 = n0 + group * 32;
        uint32_t vg[32], vu[32];
        tmem_ld_32x32b_x32(t_row + group * 32, vg);
        tmem_ld_32x32b_x32(t_row + 128 + group * 32, vu);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_pair(lead_tempty + acc * 8);
        if (group < nch) {  // uniform
          float g[32], up[32];
          scaled32(vg, sa, sw[0], g);
          scaled32(vu, sa, sw[1], up);
          gated_out(a, out, &tm_y, &tm_g, &tm_u, g, up, q0, m0);
        }
      } else {
        bool ok = true;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int c = group + kPairGroups * i;
          if (c >= nch) break;  // uniform
          if constexpr (RES) {
            if (!mbar_wait(&rbar[group * L::kSlots + i], rphase >> i & 1u, a.err, abort_flag,
                           kWaitEpiFull)) {
              ok = false;
              break;
            }
            rphase ^= 1u << i;
          }
          __syncwarp();
          const int q0 = n0 + c * 32;
          uint32_t v[32];
          tmem_ld_32x32b_x32(t_row + c * 32, v);
          tmem_ld_wait();
          float f[32];
          scaled32(v, sa, sw[i], f);
          if (a.bias) {
#pragma unroll
            for (int j = 0; j < 32; ++j) f[j] += __shfl_sync(0xFFFFFFFFu, bias[i], j);
          }
          if (a.act == 1) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              f2_get(gelu_gate2(f2(f[2 * j], f[2 * j + 1])), f[2 * j], f[2 * j + 1]);
          }
          uint32_t o[16];
          if constexpr (RES) {
            // the row's residual, and its outputs in the same place
            uint8_t *slot = out.slot + i * kYChunkBytes;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint4 *at = reinterpret_cast<uint4 *>(slot + row * 64 + ((j ^ ((row >> 1) & 3)) << 4));
              const uint4 rv = *at;
              const uint32_t w[4] = {rv.x, rv.y, rv.z, rv.w};
#pragma unroll
              for (int k = 0; k < 4; ++k)
                o[k] = pack_bf16(f[8 * j + 2 * k] + bf16_bits_to_f32(w[k] & 0xFFFFu),
                                 f[8 * j + 2 * k + 1] + bf16_bits_to_f32(w[k] >> 16));
              *at = make_uint4(o[0], o[1], o[2], o[3]);
            }
            fence_proxy_async_smem();
            group_sync(group);
            if (out.tid == 0 && m0 < a.M) {
              tma_store_3d(&tm_y, slot, q0, m0, u.b);
              bulk_commit_group();
            }
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = pack_bf16(f[2 * j], f[2 * j + 1]);
            store_chunk(out, &tm_y, q0, m0, a.M, u.b, o);
          }
        }
        if (!ok) break;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_pair(lead_tempty + acc * 8);
      }
      if (++acc == kAcc) {
        acc = 0;
        acc_phase ^= 1;
      }
    }
  }

  // The last stores are done, and neither CTA's barriers, shared memory or TMEM
  // are in use, when the pair leaves.
  if (threadIdx.x >= 128 && threadIdx.x % 128 == 0) bulk_wait_group_all();
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
