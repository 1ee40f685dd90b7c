// lin_swap.cuh -- int8 products and gated feed-forward blocks with few rows:
// the weights on the 128-row side of the MMA, up to BN activation rows on its
// other side, K dealt out over the CTAs of a cluster.
//
// One cluster of S CTAs computes one tile of 128 outputs x BN rows: the CTA of
// rank s multiplies K blocks [s KT / S, (s + 1) KT / S).  A gated tile keeps two
// accumulators, one per weight, over the same activation tile.  When its sums
// stand, each CTA copies them from TMEM into its shared memory (over the
// operand stages, which are done with), [weight][row m][128 outputs n], and
// after a cluster barrier all warps of the S CTAs share out the rows: a warp
// takes a row, a lane four outputs, sums the S slices in a fixed order through
// distributed shared memory, and finishes the outputs (scales, bias,
// activation, product, residual, quantization), so the arithmetic after the
// sum is spread over the cluster and every store is a row's contiguous 256
// bytes.  The order of the sum is fixed, and of int8 sums exact in any order.
//
// MX tiles of 32 or 64 rows cover all rows of A (the schedule sees to it): the
// scales of the rows from m0 on are then the first of their atom.  A tile that
// began at row 32 of an atom would have to name its scales by an odd TMEM
// column, which the MMA does not take.
//
// MX weights are read ahead of the kernel before, which by the library's rule has not
// written them.  Int8 weights are not: the quantizer of activations is theirs too, and
// may well come last before the product.  (Reading them ahead took 0.1 us off a chain of
// one-token products of 4.35, nothing off 41 x 4608 x 1536, 1.2 off 16 x 16384 x 8192 of
// 26.2.)
//
// What bounds it: the weights are read once per BN rows, so HBM for large
// weights, and for small ones the chain launch - first copies - MMAs - exchange.
// Measured: gated FP8 16 x 16384 x 8192 (277 MB) 46 us, 6.0 TB/s, 94 % of the copy
// rate; gated MXFP4 41 x 6144 x 1536 8.5 us (unsplit 10.4); int8 with a bias
// 1 x 4608 x 1536 4.35 us (unsplit 5.4).
#pragma once

#include "ffn_args.cuh"

namespace bq {

// Warps: 0 weight tile copies, 1 TMEM and MMA issue, 6 activation tile copies, 7
// weight scale copies, 8 activation scale copies, 9 the second weight's tile copies;
// 2-9 then take the sums to shared memory.
constexpr int kSwapThreads = 320;
constexpr int kSwapWarps = kSwapThreads / 32;

// OCC: CTAs an SM holds.  One with all the shared memory streams large weights;
// two with half each leave more places for the clusters of a split (an SM of
// its own for each CTA of a cluster is hard to find: of 48 clusters of three
// only some fit at once) and let a kernel's start overlap the one before.
template <int BN, bool I8, bool GATED, int OCC>
struct SwapSmem {
  static constexpr int kWeights = GATED ? 2 : 1;
  static constexpr int kBytesW = kBlockP * kBlockK;  // one weight's 128 x 128 tile
  static constexpr int kBytesA = BN * kBlockK;
  static constexpr int kBytesSf = I8 ? 0 : (kWeights + 1) * kSfAtom;
  static constexpr int kStageTiles = kWeights * kBytesW + kBytesA;  // 1024-byte multiple
  static constexpr int kFit = (OCC == 2 ? 108 * 1024 : 200 * 1024) / (kStageTiles + kBytesSf);
  static constexpr int kStages = kFit > 8 ? 8 : kFit;
  static constexpr int kOffSf = kStages * kStageTiles;
  static constexpr int kOffBar = kOffSf + kStages * kBytesSf;
  static constexpr int kNumBars = 2 * kStages + 2;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kBytes = kOffMisc + 64 + 1024;  // + alignment slack
  static constexpr int kSfCols = I8 ? 0 : 4 * (kWeights + 1);  // TMEM scale columns a stage
  static constexpr int kTmemUsed = kWeights * BN + kStages * kSfCols;
  static constexpr int kTmemCols = kTmemUsed <= 32    ? 32
                                   : kTmemUsed <= 64  ? 64
                                   : kTmemUsed <= 128 ? 128
                                   : kTmemUsed <= 256 ? 256
                                                      : 512;
  static constexpr int kPart = BN * kBlockP * 4;  // one weight's sums, over the stages
  static_assert(kTmemUsed <= 512, "TMEM budget");
  static_assert(kWeights * kPart <= kOffSf, "the sums overlay the operand stages");
  static_assert(kBytes <= (OCC == 2 ? 115712 : 232448), "shared memory budget");
  static_assert(OCC * kTmemCols <= 512, "TMEM of co-resident CTAs");
};

// Cluster barrier for leaving: orders nothing, so it does not wait for the outputs'
// stores.  Each thread has used what it read of its peers' shared memory by then.
__device__ __forceinline__ void cluster_leave() {
  asm volatile("barrier.cluster.arrive.relaxed;\n\tbarrier.cluster.wait;" ::: "memory");
}

// Four consecutive sums of one row and weight, at this shared-memory address in
// each CTA of the cluster, all slices in rank order.
template <bool I8>
__device__ __forceinline__ void sum_slices(uint32_t local, int S, float (&v)[4]) {
  if constexpr (I8) {
    int t[4] = {0, 0, 0, 0};
#pragma unroll 4
    for (int s = 0; s < S; ++s) {
      const float4 p = ld_dsmem_f4(mapa_shared(local, static_cast<uint32_t>(s)));
      t[0] += __float_as_int(p.x);
      t[1] += __float_as_int(p.y);
      t[2] += __float_as_int(p.z);
      t[3] += __float_as_int(p.w);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __int2float_rn(t[j]);
  } else {
    v[0] = v[1] = v[2] = v[3] = 0.0f;
#pragma unroll 4
    for (int s = 0; s < S; ++s) {
      const float4 p = ld_dsmem_f4(mapa_shared(local, static_cast<uint32_t>(s)));
      v[0] += p.x;
      v[1] += p.y;
      v[2] += p.z;
      v[3] += p.w;
    }
  }
}

template <int BN, bool I8, bool GATED, int OCC>
__global__ void __launch_bounds__(kSwapThreads, OCC)
    lin_swap_kernel(const __grid_constant__ CUtensorMap tm_w0,
                    const __grid_constant__ CUtensorMap tm_w1,
                    const __grid_constant__ CUtensorMap tm_a, const FfnArgs a) {
  using L = SwapSmem<BN, I8, GATED, OCC>;
  constexpr int kStages = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::kOffBar);
  uint64_t *empty = full + kStages;
  uint64_t *tfull = empty + kStages;
  uint64_t *drain = tfull + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kOffMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kOffMisc + 4);

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const int S = a.splits;
  const int rank = static_cast<int>(blockIdx.x) % S;  // the cluster's x extent is S
  int tile = static_cast<int>(blockIdx.x) / S;
  const int tq = tile % a.tiles_q;  // tiles that share weights run next to each other
  tile /= a.tiles_q;
  const int tp = tile % a.tiles_p;
  const int b = tile / a.tiles_p;
  const int kt0 = rank * a.kt_total / S, kt1 = (rank + 1) * a.kt_total / S;
  const int n0 = tp * kBlockP, m0 = tq * BN;

  if (threadIdx.x == 0) {
    for (int st = 0; st < kStages; ++st) {
      // one arrival per copy thread of a stage
      mbar_init(&full[st], (GATED ? 3 : 2) + (I8 ? 0 : 2));
      mbar_init(&empty[st], 1);
    }
    mbar_init(tfull, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_w0);
    tma_prefetch_desc(&tm_a);
    if (GATED) tma_prefetch_desc(&tm_w1);
    // The first MX weight tiles do not wait for the kernel before, nor for the
    // set-up that follows.
    for (int st = 0; !I8 && st < kStages && kt0 + st < kt1; ++st) {
      mbar_arrive_expect_tx(&full[st], a.w_tile_bytes);
      tma_load_3d(smem + st * L::kStageTiles, &tm_w0, &full[st], (kt0 + st) * kBlockK, n0,
                  a.p_batched ? b : 0);
    }
  }
  if (warp == 1) tmem_alloc(tmem_slot, L::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  const bool copier = warp == 0 || warp == 6 || (!I8 && (warp == 7 || warp == 8)) ||
                      (GATED && warp == 9);
  if (copier) {
    if (lane == 0) {
      // int8 weights may come from the kernel before as well as the activations
      if (I8 || warp == 6 || warp == 8) griddep_wait();
      if (warp == 6) griddep_launch_dependents();
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      int kt = kt0;
      if (!I8 && warp == 0) {  // the tiles issued above
        kt = min(kt0 + kStages, kt1);
        phase = 1;
      }
      for (; kt < kt1; ++kt) {
        if (!mbar_wait(&empty[stage], phase ^ 1, a.err, abort_flag, kWaitProdEmpty)) {
          ok = false;
          break;
        }
        uint8_t *st = smem + stage * L::kStageTiles;
        uint8_t *sf = smem + L::kOffSf + stage * L::kBytesSf;
        if (warp == 6) {
          mbar_arrive_expect_tx(&full[stage], static_cast<uint32_t>(a.q_box_rows * kBlockK));
          tma_load_3d(st + L::kWeights * L::kBytesW, &tm_a, &full[stage], kt * kBlockK, m0,
                      a.q_batched ? b : 0);
        } else if (warp == 0 || warp == 9) {
          mbar_arrive_expect_tx(&full[stage], a.w_tile_bytes);
          tma_load_3d(st + (warp == 9 ? L::kBytesW : 0), warp == 9 ? &tm_w1 : &tm_w0,
                      &full[stage], kt * kBlockK, n0, a.p_batched ? b : 0);
        } else if (warp == 7) {
          mbar_arrive_expect_tx(&full[stage], L::kWeights * kSfAtom);
          const int64_t at = (static_cast<int64_t>(tp) * a.sf_katoms + kt) * kSfAtom;
#pragma unroll
          for (int w = 0; w < L::kWeights; ++w)
            bulk_load(sf + w * kSfAtom, a.sf_w[w] + at, kSfAtom, &full[stage]);
        } else {
          mbar_arrive_expect_tx(&full[stage], kSfAtom);
          bulk_load(sf + L::kWeights * kSfAtom,
                    a.sf_a + (static_cast<int64_t>(m0 / 128) * a.sf_katoms + kt) * kSfAtom, kSfAtom,
                    &full[stage]);
        }
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (!ok) sleep_ns(200000);  // copies already issued land before the CTA goes away
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int kt = kt0; kt < kt1; ++kt) {
        if (!mbar_wait(&full[stage], phase, a.err, abort_flag, kWaitMmaFull)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t wa = smem_u32(smem + stage * L::kStageTiles);
        const uint32_t aa = wa + L::kWeights * L::kBytesW;
        const uint32_t sf_t = tmem_base + L::kWeights * BN + stage * L::kSfCols;
        if constexpr (!I8) {
          const uint32_t sf = smem_u32(smem + L::kOffSf + stage * L::kBytesSf);
#pragma unroll
          for (int j = 0; j <= L::kWeights; ++j)
            tc_cp_sf(sf_t + 4 * j, desc_sf_32x128b(sf + j * kSfAtom));
        }
#pragma unroll
        for (int w = 0; w < L::kWeights; ++w) {
#pragma unroll
          for (int ks = 0; ks < kBlockK / kMmaK; ++ks) {
            const uint32_t acc_in = (kt > kt0 || ks > 0) ? 1u : 0u;
            const uint64_t dw = desc_kmajor_sw128(wa + w * L::kBytesW + ks * kMmaK);
            const uint64_t da = desc_kmajor_sw128(aa + ks * kMmaK);
            if constexpr (I8)
              tc_mma_i8(tmem_base + w * BN, dw, da, idesc_i8(kBlockP, BN), acc_in);
            else
              tc_mma_mxf8f6f4(tmem_base + w * BN, dw, da, make_idesc(a.fmt_w, a.fmt_a, BN, ks),
                              sf_t + 4 * w, sf_t + 4 * L::kWeights, acc_in);
          }
        }
        tc_commit(&empty[stage]);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (ok) tc_commit(tfull);
      tc_commit(drain);
      if (!mbar_wait_timed(drain, 0, a.err, kWaitDrain)) sleep_ns(200000);
    }
  }
  __syncwarp();
  // The scales, bias and residual may come from the preceding kernel, which
  // may also still read or write the outputs.
  griddep_wait();
  // What the outputs need besides the sums, fetched while those are formed (0.4 us of int8
  // 41 x 1536 x 6144, whose scales came behind the exchange before).
  const int mt = min(BN, a.M - m0);
  const int n = n0 + 4 * lane;
  const bool nok = n < a.N;
  float sw[2][4];
#pragma unroll
  for (int w = 0; w < L::kWeights; ++w) {
    float4 s = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    if (I8 && nok) s = __ldg(reinterpret_cast<const float4 *>(a.sw[w] + b * a.sw_bstride + n));
    sw[w][0] = a.alpha * s.x;
    sw[w][1] = a.alpha * s.y;
    sw[w][2] = a.alpha * s.z;
    sw[w][3] = a.alpha * s.w;
  }
  uint2 bias = make_uint2(0u, 0u);
  if (!GATED && a.bias && nok) bias = __ldg(reinterpret_cast<const uint2 *>(a.bias + n));
  const int first = rank * kSwapWarps + warp;  // this warp's first row
  float sa = I8 && first < mt ? __ldg(a.sa + b * a.sa_bstride + m0 + first) : 1.0f;
  if (warp >= 2 && mbar_wait(tfull, 0, a.err, abort_flag, kWaitEpiFull)) {
    // Sums to shared memory: a lane holds one output n, a warp store is 32
    // consecutive n of one row m.  Every MMA that read the stages is complete.  Two
    // warps to a quadrant of the TMEM lanes, 32 rows (of one weight) a turn.
    const int quad = warp % 4;
    __syncwarp();
    tc_fence_after();
    const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
    uint32_t *dst = reinterpret_cast<uint32_t *>(smem) + quad * 32 + lane;
    const int chunks = (mt + 31) / 32;
#pragma unroll 1
    for (int i = (warp - 2) / 4; i < L::kWeights * chunks; i += 2) {
      const int w = GATED && i >= chunks ? 1 : 0, c = i - w * chunks;
      uint32_t v[32];
      __syncwarp();
      tmem_ld_32x32b_x32(t_row + w * BN + c * 32, v);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 32; ++j) dst[w * (L::kPart / 4) + (c * 32 + j) * kBlockP] = v[j];
    }
  }
  __syncwarp();
  tc_fence_before();
  if (S > 1)
    cluster_sync_all();
  else
    __syncthreads();

  // ------------------------------------------------------------- outputs --
  {
    const int64_t groups = a.N >> 5, katoms = (groups + 3) >> 2;
    // One row a warp and round, in code that is short: it runs once, from a cold
    // instruction cache (four rows a round, fetched together, took 0.5 to 2 us
    // longer on 41 x 1536 x 6144 split eight ways and gained nothing elsewhere; four
    // slices' loads under way at once 0.1 to 0.4 us longer with 41 rows).
#pragma unroll 1
    for (int r = first; r < mt; r += S * kSwapWarps) {
      const int m = m0 + r;
      if (I8 && r != first) sa = __ldg(a.sa + b * a.sa_bstride + m);
      float v[2][4];
#pragma unroll
      for (int w = 0; w < L::kWeights; ++w) {
        const uint32_t at = static_cast<uint32_t>(w * L::kPart + r * kBlockP * 4 + 16 * lane);
        if (S == 1) {
          const uint4 p = *reinterpret_cast<const uint4 *>(smem + at);
          const uint32_t t[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            v[w][j] = I8 ? __int2float_rn(static_cast<int>(t[j])) : __uint_as_float(t[j]);
        } else {
          sum_slices<I8>(smem_u32(smem) + at, S, v[w]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) v[w][j] *= I8 ? sa * sw[w][j] : sw[w][j];
      }
      float t[4];
      if constexpr (GATED) {
        if (a.gu && nok) {
          __nv_bfloat16 *g = a.gu + static_cast<int64_t>(m) * (2 * static_cast<int64_t>(a.N)) + n;
          *reinterpret_cast<uint2 *>(g) =
              make_uint2(pack_bf16(v[0][0], v[0][1]), pack_bf16(v[0][2], v[0][3]));
          *reinterpret_cast<uint2 *>(g + a.N) =
              make_uint2(pack_bf16(v[1][0], v[1][1]), pack_bf16(v[1][2], v[1][3]));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) t[j] = gate_act(v[0][j], a.act) * v[1][j];
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          t[j] = v[0][j] + bf16_bits_to_f32((j < 2 ? bias.x : bias.y) >> (16 * (j & 1)) & 0xFFFFu);
        if (a.act == 1) {
#pragma unroll
          for (int j = 0; j < 4; ++j) t[j] = gelu_erf(t[j]);
        }
        if (a.res && nok) {
          const uint2 rv = *reinterpret_cast<const uint2 *>(
              a.res + b * a.res_bstride + static_cast<int64_t>(m) * a.ldres + n);
          t[0] += bf16_bits_to_f32(rv.x & 0xFFFFu);
          t[1] += bf16_bits_to_f32(rv.x >> 16);
          t[2] += bf16_bits_to_f32(rv.y & 0xFFFFu);
          t[3] += bf16_bits_to_f32(rv.y >> 16);
        }
      }
      const uint32_t o[2] = {pack_bf16(t[0], t[1]), pack_bf16(t[2], t[3])};
      const int64_t at = b * a.y_bstride + static_cast<int64_t>(m) * a.ldy + n;
      if (a.y && nok) *reinterpret_cast<uint2 *>(a.y + at) = make_uint2(o[0], o[1]);
      if (GATED && a.q_out) {  // a group of 32 outputs is 8 lanes
        uint32_t bad = 0;
        uint32_t mx = nok ? bf16_amax_bits(o, bad) : 0u;
#pragma unroll
        for (int k = 1; k < 8; k <<= 1) mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, k));
        if (nok) {
          const int e = mx_exponent(mx);
          uint32_t codes[1];
          mx_encode(o, e, codes);
          *reinterpret_cast<uint32_t *>(a.q_out + at) = codes[0];
          if ((lane & 7) == 0)
            a.sf_out[sf_mma_offset(m, n >> 5, katoms)] = static_cast<uint8_t>(e + 127);
          if (bad) atomicOr(a.err, BQ_DEV_ERR_NONFINITE);
        }
      }
    }
    if (GATED && a.q_out && rank == 0) {
      // padding scale bytes: this tile's columns of the rows behind the last
      // one, and the columns behind the last group in this tile's rows
      const int64_t rows_pad = (static_cast<int64_t>(a.M) + 127) / 128 * 128;
      const int64_t g0 = n0 >> 5, g1 = min(g0 + 4, groups);
      const int64_t gend = g1 == groups ? katoms * 4 : g1;
      if (tq == a.tiles_q - 1) {
        const int64_t nc = gend - g0;
        for (int64_t i = threadIdx.x; i < (rows_pad - a.M) * nc; i += kSwapThreads)
          a.sf_out[sf_mma_offset(a.M + i / nc, g0 + i % nc, katoms)] = 127;
      }
      if (gend > g1) {
        const int64_t nc = gend - g1;
        for (int64_t i = threadIdx.x; i < mt * nc; i += kSwapThreads)
          a.sf_out[sf_mma_offset(m0 + i / nc, g1 + i % nc, katoms)] = 127;
      }
    }
  }
  // No CTA leaves while a peer still reads its sums.
  if (S > 1)
    cluster_leave();
  else
    __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, L::kTmemCols);
  }
}

}  // namespace bq
