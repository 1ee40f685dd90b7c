// bq_ffn.cu -- host side of the int8 and gated feed-forward entry points of
// include/bq.h: argument checks, tensor maps, schedules and launches.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>

#include "bq.h"
#include "bq_host.cuh"
#include "gated_grad.cuh"
#include "gated_mx.cuh"
#include "lin_pair.cuh"
#include "lin_swap.cuh"
#include "quant_i8.cuh"

namespace {

using bqh::aligned;
using bqh::Device;

// Weight kinds of these entry points (the GEMMs' numbers, and 6 for int8).
enum Kind { kMxfp4 = 0, kFp8Blk32 = 1, kMxfp8 = 2, kInt8 = 6 };

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int launch_status() { return cudaGetLastError() == cudaSuccess ? BQ_OK : BQ_ERR_CUDA; }

// Launch with programmatic dependence on the kernel before, in clusters of
// `cluster` blocks.
template <class... P, class... A>
int launch(void (*kern)(P...), dim3 grid, int threads, size_t smem, int cluster,
           bq_stream_t stream, A... args) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = dim3(static_cast<unsigned>(threads));
  lc.dynamicSmemBytes = smem;
  lc.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&lc, kern, args...) != cudaSuccess) {
    cudaGetLastError();
    return BQ_ERR_CUDA;
  }
  return launch_status();
}

// A K-major operand of one byte (E2M1: half a byte) per code as (K, rows,
// batch): boxes of 128 codes x box_rows rows, 128-byte swizzle, zeros outside.
int operand_map(CUtensorMap* m, const void* base, bool fp4, int64_t K, int64_t rows, int64_t batch,
                int64_t batch_bytes, int64_t box_rows) {
  auto encode = bqh::tensor_map_encoder();
  if (!encode) return BQ_ERR_CUDA;
  const int64_t row_bytes = fp4 ? K / 2 : K;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(batch)};
  const cuuint64_t strides[2] = {
      static_cast<cuuint64_t>(row_bytes),
      static_cast<cuuint64_t>(batch > 1 ? batch_bytes : row_bytes * rows)};
  const cuuint32_t box[3] = {128u, static_cast<cuuint32_t>(box_rows), 1u};
  const cuuint32_t step[3] = {1u, 1u, 1u};
  const CUresult r = encode(
      m, fp4 ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3,
      const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? BQ_OK : BQ_ERR_ALIGN;
}

// An MX scale buffer as (128 words, K atoms, 128-row bands), boxes of kMxSfChunks
// atoms of a band.
int scale_map(CUtensorMap* m, const void* base, int64_t rows, int64_t K) {
  auto encode = bqh::tensor_map_encoder();
  if (!encode) return BQ_ERR_CUDA;
  const int64_t katoms = ceil_div(K, 128), bands = ceil_div(rows, 128);
  const cuuint64_t dims[3] = {128u, static_cast<cuuint64_t>(katoms),
                              static_cast<cuuint64_t>(bands)};
  const cuuint64_t strides[2] = {512u, static_cast<cuuint64_t>(katoms * 512)};
  const cuuint32_t box[3] = {128u, bq::kMxSfChunks, 1u};
  const cuuint32_t step[3] = {1u, 1u, 1u};
  const CUresult r = encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void*>(base), dims,
                            strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? BQ_OK : BQ_ERR_ALIGN;
}

// A bf16 output [batch][M][ld] of N columns: boxes of 32 columns x 128 rows with
// the 64-byte swizzle of the epilogue's staging tile.
int output_map(CUtensorMap* m, const void* y, int64_t M, int64_t N, int64_t ld, int64_t batch,
               int64_t batch_bytes) {
  auto encode = bqh::tensor_map_encoder();
  if (!encode) return BQ_ERR_CUDA;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(M),
                              static_cast<cuuint64_t>(batch)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(2 * ld),
                                 static_cast<cuuint64_t>(batch > 1 ? batch_bytes : 2 * ld * M)};
  const cuuint32_t box[3] = {32u, 128u, 1u};
  const cuuint32_t step[3] = {1u, 1u, 1u};
  const CUresult r = encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(y), dims,
                            strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? BQ_OK : BQ_ERR_ALIGN;
}

// A bf16 matrix [rows][ld] of `cols` columns: boxes of 128 x 128, no swizzle.
int matrix_map(CUtensorMap* m, const void* x, int64_t rows, int64_t cols, int64_t ld) {
  auto encode = bqh::tensor_map_encoder();
  if (!encode) return BQ_ERR_CUDA;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(2 * ld)};
  const cuuint32_t box[2] = {128u, 128u};
  const cuuint32_t step[2] = {1u, 1u};
  const CUresult r = encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(x), dims,
                            strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? BQ_OK : BQ_ERR_ALIGN;
}

// ---------------------------------------------------------------- schedule --

struct Plan {
  bool pair = false;  // 256-row tiles on pairs of SMs (lin_pair.cuh), else lin_swap.cuh
  int bn = 0;         // swap: activation rows of a tile; pair: weight rows (256)
  int splits = 1;     // swap: K slices (CTAs of a cluster)
  int occ = 1;        // swap: CTAs an SM holds
  int64_t tiles_p = 0, tiles_q = 0, tiles = 0;
  int kt = 0;
};

constexpr int kMaxSplit = 8;  // portable cluster size

int check_config(const bq_gemm_config* cfg) {
  if (!cfg) return BQ_OK;
  const bq_gemm_config& c = *cfg;
  if (c.block_n != 0 && c.block_n != 32 && c.block_n != 64 && c.block_n != 128 &&
      c.block_n != 256)
    return BQ_ERR_INVALID;
  if (c.split_k < 0 || c.split_k > kMaxSplit || c.swap_ab < -1 ||
      c.swap_ab > 1 || (c.split_mode != BQ_SPLIT_AUTO && c.split_mode != BQ_SPLIT_CLUSTER) ||
      c.k_chunks < 0 || c.k_chunks > 1 || c.cta_pair < 0 || c.cta_pair > 2)
    return BQ_ERR_INVALID;
  // pairs: 256-row tiles, no split; everything else: tiles of one SM
  const bool pair = c.swap_ab == 0 || c.cta_pair == 2 || c.block_n == 256;
  const bool swap = c.swap_ab == 1 || c.cta_pair == 1 || c.split_k > 1 ||
                    (c.block_n != 0 && c.block_n != 256);
  if (pair && swap) return BQ_ERR_INVALID;
  return BQ_OK;
}

// Estimated microseconds of the two schedules, fitted to 260 random problems of 1 to
// 1500 rows, 256 to 16384 outputs and K of 256 to 8192, each measured in every
// schedule (a mean of 10 % off; the schedules picked take 0.9 % more than the best, 34 % at
// worst).
//   swap: launch, first copies and outputs 3 us (MX 4.1), longer by the tile's rows.  A
//         CTA fills its shared memory at 105 KB/us (packed weights at their unpacked
//         size), all of them at 8.3 GB/ms from L2.  A split adds the exchange (int8 41
//         x 4608 x 1536: 6.4 us unsplit, 5.5 in 2 slices; 41 x 1536 x 6144: 14.8 and 5.5
//         in 8; gated MXFP4 41 x 6144 x 1536: 10.4 and 8.5 in 2 or 4), more CTAs than SMs
//         their start.
//   pair: 5.1 us and 0.26 us (MX 0.33) a K block of 256 x 256 (int8 256 x 4096 x 4096:
//         15.6 us, 12.0 as 64-row tiles; 1024 x 4096 x 4096: 17.8, 28 as 128-row tiles).
double swap_us(Kind kind, bool gated, int bn, int64_t M, int64_t tiles, int splits, int kt,
               int num_sms) {
  const double ctas = static_cast<double>(tiles * splits), weights = gated ? 2 : 1;
  const double rows = static_cast<double>(std::min<int64_t>(M, bn)) / 128;
  const double blocks = static_cast<double>(kt) / splits;  // a CTA's
  const double kb = blocks * (16 * weights + bn / 8.0);
  const double l2 = blocks * ((kind == kMxfp4 ? 8 : 16) * weights + bn / 8.0);
  const double starts =
      ctas <= num_sms ? 0.0 : 0.4 + 3.5 * static_cast<double>((tiles * splits - 1) / (2 * num_sms));
  return (kind == kInt8 ? 3.0 : 4.1) + 2.2 * rows * weights + starts +
         std::max(kb / 105, ctas * l2 / 8.3e3) +
         (splits > 1 ? 0.26 + 0.26 * rows * weights / splits + 0.1 * splits : 0.0);
}

double pair_us(Kind kind, bool gated, int64_t tiles, int kt, int num_sms) {
  const int64_t waves = ceil_div(tiles, num_sms / 2);
  return 5.1 + static_cast<double>(waves) *
                   (kt * (kind == kInt8 ? 0.264 : 0.33) + (gated ? 1.4 : 0.3));
}

int make_plan(Kind kind, bool gated, int64_t M, int64_t N, int64_t K, int64_t batch,
              const bq_gemm_config* cfg, int num_sms, Plan* p) {
  const bq_gemm_config c = cfg ? *cfg : bq_gemm_config{0, 0, -1, BQ_SPLIT_AUTO, 0, 0};
  // MX tiles start at the first row of a scale atom (lin_swap.cuh)
  if (kind != kInt8 && c.block_n != 0 && c.block_n < 128 && M > c.block_n) return BQ_ERR_INVALID;
  p->kt = static_cast<int>(ceil_div(K, 128));
  const bool pair_asked = c.swap_ab == 0 || c.cta_pair == 2 || c.block_n == 256;
  const bool swap_asked = !pair_asked && (c.swap_ab == 1 || c.cta_pair == 1 || c.split_k > 0 ||
                                          c.block_n != 0);
  // outputs of a pair's tile (lin_pair.cuh, gated_mx.cuh)
  const int pair_n = gated ? 128 : 256;
  const int64_t pair_p = ceil_div(M, 256), pair_q = ceil_div(N, pair_n);
  const int64_t tiles_p = ceil_div(N, 128);
  double best = 1e30;
  for (int bn = 32; bn <= 128 && !pair_asked; bn *= 2) {
    if (c.block_n ? bn != c.block_n
                  : (bn < 128 && M > (kind == kInt8 ? bn == 32 ? 256 : M : bn)) ||
                        (bn > 32 && M <= bn / 2))
      continue;
    const int64_t tiles_q = ceil_div(M, bn), tiles = tiles_p * tiles_q * batch;
    for (int s = c.split_k ? c.split_k : 1; s <= (c.split_k ? c.split_k : kMaxSplit); s *= 2) {
      // a split's clusters find a place at once up to about nine tenths of the places,
      // two an SM (gated 128-row tiles: eight tenths of one)
      if (!c.split_k && s > 1 &&
          (p->kt / s < 2 || tiles * s * 10 > num_sms * (gated && bn == 128 ? 8 : 18)))
        break;
      const double us = swap_us(kind, gated, bn, M, tiles, s, p->kt, num_sms);
      if (us >= best) continue;
      best = us;
      p->bn = bn;
      p->splits = std::min(s, p->kt);
      p->tiles_p = tiles_p;
      p->tiles_q = tiles_q;
    }
  }
  p->pair = pair_asked ||
            (!swap_asked && M > 64 &&
             pair_us(kind, gated, pair_p * pair_q * batch, p->kt, num_sms) < best);
  if (p->pair) {
    p->bn = 256;
    p->splits = 1;
    p->tiles_p = pair_p;
    p->tiles_q = pair_q;
  }
  p->tiles = p->tiles_p * p->tiles_q * batch;
  // One CTA to an SM has twice the stages: it streams faster where there are no
  // more tiles than SMs (int8 512 x 4096 x 4096 in 128-row tiles: 14.0 us, 16.1
  // with two); two take the tiles beyond that (1024 x 4096 x 4096: 28.1 and 21.5).
  // In clusters of two as well (gated MXFP8 41 x 8192 x 2048: 10.9 and 13.0, int8 41 x
  // 8192 x 4096: 9.9 and 10.4), but for packed weights, half the bytes (gated MXFP4 16
  // x 9216 x 2048: 8.6 and 8.2); longer clusters find too few places.
  p->occ = p->splits <= (kind == kMxfp4 ? 1 : 2) && p->tiles * p->splits <= num_sms ? 1 : 2;
  return p->tiles * p->splits > 0x7FFFFFFF ? BQ_ERR_SHAPE : BQ_OK;
}

// ---------------------------------------------------------------- launches --

template <int BN, bool I8, bool GATED, int OCC>
int launch_swap(const Plan& pl, const CUtensorMap& w0, const CUtensorMap& w1,
                const CUtensorMap& ta, const bq::FfnArgs& a, int dev, bq_stream_t stream) {
  using L = bq::SwapSmem<BN, I8, GATED, OCC>;
  auto kern = bq::lin_swap_kernel<BN, I8, GATED, OCC>;
  static bool ready[bqh::kMaxDevices] = {};
  if (!ready[dev]) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes) !=
        cudaSuccess)
      return BQ_ERR_CUDA;
    ready[dev] = true;
  }
  return launch(kern, dim3(static_cast<unsigned>(pl.tiles * pl.splits)), bq::kSwapThreads,
                L::kBytes, pl.splits, stream, w0, w1, ta, a);
}

// A kernel on pairs of SMs: persistent, one pair to every two SMs.
template <class... P, class... A>
int launch_pairs(void (*kern)(P...), bool* ready, int threads, int smem, const Plan& pl,
                 const Device& dev, bq_stream_t stream, const A&... args) {
  if (!ready[dev.index]) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
        cudaSuccess)
      return BQ_ERR_CUDA;
    ready[dev.index] = true;
  }
  const int64_t pairs = std::max<int64_t>(1, std::min<int64_t>(dev.num_sms / 2, pl.tiles));
  return launch(kern, dim3(static_cast<unsigned>(2 * pairs)), threads, smem, 2, stream, args...);
}

template <bool I8, bool GATED>
int run_swap(const Plan& pl, const CUtensorMap& w0, const CUtensorMap& w1, const CUtensorMap& ta,
             const bq::FfnArgs& a, int dev, bq_stream_t stream) {
  if (pl.occ == 2) {
    switch (pl.bn) {
      case 32: return launch_swap<32, I8, GATED, 2>(pl, w0, w1, ta, a, dev, stream);
      case 64: return launch_swap<64, I8, GATED, 2>(pl, w0, w1, ta, a, dev, stream);
      default:
        if constexpr (!GATED) return launch_swap<128, I8, GATED, 2>(pl, w0, w1, ta, a, dev, stream);
    }
  }
  switch (pl.bn) {
    case 32: return launch_swap<32, I8, GATED, 1>(pl, w0, w1, ta, a, dev, stream);
    case 64: return launch_swap<64, I8, GATED, 1>(pl, w0, w1, ta, a, dev, stream);
    default: return launch_swap<128, I8, GATED, 1>(pl, w0, w1, ta, a, dev, stream);
  }
}

// What a call of either operator brings.  w[1] is NULL for the plain product.
struct Call {
  Kind kind;
  const void *a, *a_sf;
  const void *w[2], *w_sf[2];
  int64_t M, N, K;
  bq_batch batch{1, 0, 0, 0, 0, 0, 0};
};

// Sums of int8 products stay below 2^31: K 128 128 < 2^31.
constexpr int64_t kMaxInt8K = (int64_t{1} << 17) - 1;
// Row numbers of the tile behind the last one still fit 32 bits.
constexpr int64_t kMaxRows = 0x7FFFFE00;

// Checks of the operands and of the sizes.
int check_operands(const Call& c) {
  const bool i8 = c.kind == kInt8;
  if (c.M < 0 || c.N < 0 || c.K <= 0 || c.K % (i8 ? 16 : 32) != 0 || c.N % 8 != 0 ||
      c.M > kMaxRows || c.N > kMaxRows || c.K > 0x7FFFFFFF || (i8 && c.K > kMaxInt8K) ||
      (c.kind == kMxfp4 && c.K % 128 != 0) || c.batch.count < 0 || c.batch.count > 65535)
    return BQ_ERR_SHAPE;
  return BQ_OK;
}

int check_pointers(const Call& c, bool gated) {
  const bool i8 = c.kind == kInt8;
  if (!c.a || !c.a_sf) return BQ_ERR_NULL;
  for (int w = 0; w < (gated ? 2 : 1); ++w)
    if (!c.w[w] || !c.w_sf[w]) return BQ_ERR_NULL;
  if (!aligned(c.a, 16) || !aligned(c.a_sf, i8 ? 4 : 16)) return BQ_ERR_ALIGN;
  for (int w = 0; w < (gated ? 2 : 1); ++w)
    if (!aligned(c.w[w], c.kind == kMxfp4 ? 32 : 16) || !aligned(c.w_sf[w], 16))
      return BQ_ERR_ALIGN;
  return BQ_OK;
}

void operand_args(const Call& c, bq::FfnArgs* g) {
  const bool i8 = c.kind == kInt8;
  g->M = static_cast<int>(c.M);
  g->N = static_cast<int>(c.N);
  g->K = static_cast<int>(c.K);
  g->batch = static_cast<int>(c.batch.count);
  g->sf_katoms = static_cast<int>(ceil_div(c.K, 128));
  g->w_tile_bytes = 128 * 128 / (c.kind == kMxfp4 ? 2 : 1);
  g->fmt_a = bq::kFmtE4M3;
  g->fmt_w = c.kind == kMxfp4 ? bq::kFmtE2M1 : bq::kFmtE4M3;
  if (i8) {
    g->sa = static_cast<const float*>(c.a_sf);
    g->sa_bstride = c.batch.stride_a_sf / 4;
    g->sw_bstride = c.batch.stride_b_sf / 4;
  } else {
    g->sf_a = static_cast<const uint8_t*>(c.a_sf);
  }
  for (int w = 0; w < 2; ++w) {
    if (i8)
      g->sw[w] = static_cast<const float*>(c.w_sf[w]);
    else
      g->sf_w[w] = static_cast<const uint8_t*>(c.w_sf[w]);
  }
  g->ldy = c.N;
  g->y_bstride = c.batch.stride_y / 2;
  g->res_bstride = c.batch.stride_res / 2;
  g->p_batched = c.batch.count > 1 && c.batch.stride_b != 0;
  g->q_batched = c.batch.count > 1 && c.batch.stride_a != 0;
}

// The call after its argument checks.
int run(const Call& c, bool gated, bool empty, const bq_gemm_config* cfg, bq::FfnArgs* g,
        bq_stream_t stream) {
  int st = check_config(cfg);
  if (st != BQ_OK) return st;
  Device dev;
  st = bqh::current_device(&dev);
  if (st != BQ_OK || empty) return st;
  Plan pl;
  st = make_plan(c.kind, gated, c.M, c.N, c.K, c.batch.count, cfg, dev.num_sms, &pl);
  if (st != BQ_OK) return st;
  const bool i8 = c.kind == kInt8, fp4 = c.kind == kMxfp4;
  operand_args(c, g);
  g->err = dev.err;
  g->kt_total = pl.kt;
  g->splits = pl.splits;
  g->tiles_p = static_cast<int>(pl.tiles_p);
  g->tiles_q = static_cast<int>(pl.tiles_q);
  CUtensorMap ta, tw[2];
  if (pl.pair) {
    g->raster_group = 4;
    g->splits = 1;
    const bool mx = !i8;
    st = operand_map(&ta, c.a, false, c.K, c.M, g->q_batched ? c.batch.count : 1,
                     c.batch.stride_a, 128);
    for (int w = 0; st == BQ_OK && w < (gated ? 2 : 1); ++w)
      st = operand_map(&tw[w], c.w[w], fp4, c.K, c.N, g->p_batched ? c.batch.count : 1,
                       c.batch.stride_b, 128);
    if (st != BQ_OK) return st;
    CUtensorMap ty = ta, tg = ta, tu = ta;  // unused ones: placeholders
    if (g->y) st = output_map(&ty, g->y, c.M, c.N, c.N, c.batch.count, c.batch.stride_y);
    if (st == BQ_OK && g->gu) st = output_map(&tg, g->gu, c.M, c.N, 2 * c.N, 1, 0);
    if (st == BQ_OK && g->gu) st = output_map(&tu, g->gu + c.N, c.M, c.N, 2 * c.N, 1, 0);
    if (st != BQ_OK) return st;
    static bool ready[4][bqh::kMaxDevices] = {};
    if (mx) {
      CUtensorMap sfa, sf[2];
      st = scale_map(&sfa, c.a_sf, c.M, c.K);
      for (int w = 0; st == BQ_OK && w < 2; ++w) st = scale_map(&sf[w], c.w_sf[w], c.N, c.K);
      if (st != BQ_OK) return st;
      return launch_pairs(bq::gated_mx_kernel, ready[0], bq::kMxThreads, bq::GatedMxSmem::kBytes,
                          pl, dev, stream, ta, tw[0], tw[1], sfa, sf[0], sf[1], ty, tg, tu, *g);
    }
    constexpr int kT = bq::kLinPairThreads;
    if (gated)
      return launch_pairs(bq::lin_pair_kernel<true, false>, ready[1], kT,
                          bq::LinPairSmem<false>::kBytes, pl, dev, stream, ta, tw[0], tw[1], ty, tg,
                          tu, *g);
    if (!g->res)
      return launch_pairs(bq::lin_pair_kernel<false, false>, ready[2], kT,
                          bq::LinPairSmem<false>::kBytes, pl, dev, stream, ta, tw[0], tw[0], ty, tg,
                          tu, *g);
    CUtensorMap tr;  // one residual for every problem: no batch dimension
    if (c.batch.count <= 1) g->res_bstride = 0;
    st = output_map(&tr, g->res, c.M, c.N, g->ldres, g->res_bstride ? c.batch.count : 1,
                    c.batch.stride_res);
    if (st != BQ_OK) return st;
    return launch_pairs(bq::lin_pair_kernel<false, true>, ready[3], kT,
                        bq::LinPairSmem<true>::kBytes, pl, dev, stream, ta, tw[0], tw[0], ty, tr,
                        tu, *g);
  }
  // One tile over all rows: its box ends at the last row (a box whose trailing
  // rows all lie outside the tensor copies slower).
  g->q_box_rows =
      pl.tiles_q == 1 ? static_cast<int>(std::min<int64_t>(pl.bn, (c.M + 7) / 8 * 8)) : pl.bn;
  st = operand_map(&ta, c.a, false, c.K, c.M, g->q_batched ? c.batch.count : 1, c.batch.stride_a,
                   g->q_box_rows);
  for (int w = 0; st == BQ_OK && w < (gated ? 2 : 1); ++w)
    st = operand_map(&tw[w], c.w[w], fp4, c.K, c.N, g->p_batched ? c.batch.count : 1,
                     c.batch.stride_b, 128);
  if (st != BQ_OK) return st;
  if (!gated) return run_swap<true, false>(pl, tw[0], tw[0], ta, *g, dev.index, stream);
  return i8 ? run_swap<true, true>(pl, tw[0], tw[1], ta, *g, dev.index, stream)
            : run_swap<false, true>(pl, tw[0], tw[1], ta, *g, dev.index, stream);
}

}  // namespace

extern "C" {

int bq_act_quant_int8(const void* x_bf16, int64_t M, int64_t K, int64_t ldx, void* q_s8,
                      float* scale, int* d_status, bq_stream_t stream) {
  if (M < 0 || M > 0x7FFFFFFF || K <= 0 || K % 16 != 0 || ldx < K) return BQ_ERR_SHAPE;
  if (!aligned(d_status, 4)) return BQ_ERR_ALIGN;
  if (M > 0) {
    if (!x_bf16 || !q_s8 || !scale) return BQ_ERR_NULL;
    if (!aligned(x_bf16, 16) || ldx % 8 != 0 || !aligned(q_s8, 16) || !aligned(scale, 4))
      return BQ_ERR_ALIGN;
  }
  Device dev;
  const int st = bqh::current_device(&dev);
  if (st != BQ_OK || M == 0) return st;
  // Many short rows get a warp each (quant_i8.cuh): 200 x 2048 takes 1.6 us with blocks and
  // 1.9 with warps, 600 x 2048 2.4 and 2.0; of longer rows it takes more: 1200 x 3584 3.7
  // and 4.0, 2048 x 4096 5.9 and 4.5.
  const bool warps = M >= (K <= 2048 ? 4 : 10) * dev.num_sms && K <= 4096;
  const bool small = !warps && K <= 6144 && M >= 3 * dev.num_sms;  // blocks of 128
  return launch(warps   ? K <= 2048 ? bq::i8_quant_warp_kernel<8> : bq::i8_quant_warp_kernel<16>
                : small ? bq::i8_quant_kernel<128, 8>
                        : bq::i8_quant_kernel<256, 4>,
                dim3(static_cast<unsigned>(warps ? ceil_div(M, 8) : M)), small ? 128 : 256, 0, 1,
                stream,
                static_cast<const __nv_bfloat16*>(x_bf16), M, K, ldx,
                static_cast<uint8_t*>(q_s8), scale, d_status);
}

int bq_gemm_int8_int8_epilogue(const void* a_s8, const float* a_scale, const void* b_s8,
                               const float* b_scale, int64_t M, int64_t N, int64_t K, void* y_bf16,
                               const bq_epilogue* epi, const bq_batch* batch,
                               const bq_gemm_config* cfg, bq_stream_t stream) {
  Call c{kInt8, a_s8, a_scale, {b_s8, nullptr}, {b_scale, nullptr}, M, N, K};
  if (batch) c.batch = *batch;
  int st = check_operands(c);
  if (st != BQ_OK) return st;
  const bool empty = M == 0 || N == 0 || c.batch.count == 0;
  if (!empty) {
    if ((st = check_pointers(c, false)) != BQ_OK) return st;
    if (!y_bf16) return BQ_ERR_NULL;
    if (!aligned(y_bf16, 16)) return BQ_ERR_ALIGN;
  }
  bq::FfnArgs g;
  memset(&g, 0, sizeof(g));
  g.alpha = 1.0f;
  if (epi) {
    if (epi->act != BQ_ACT_NONE && epi->act != BQ_ACT_GELU) return BQ_ERR_INVALID;
    if (epi->q_out || epi->sf_out) return BQ_ERR_INVALID;
    if (epi->bias && !aligned(epi->bias, 16)) return BQ_ERR_ALIGN;
    if (epi->residual && (!aligned(epi->residual, 16) || epi->ld_residual % 8 != 0 ||
                          epi->ld_residual < N))
      return BQ_ERR_ALIGN;
    g.alpha = epi->alpha;
    g.act = epi->act;
    g.bias = static_cast<const __nv_bfloat16*>(epi->bias);
    g.res = static_cast<const __nv_bfloat16*>(epi->residual);
    g.ldres = epi->ld_residual;
  }
  if (c.batch.count > 1) {
    const bq_batch& b = c.batch;
    // outputs of two problems do not share memory: a problem's are 2 M N bytes
    if (b.stride_a < 0 || b.stride_a_sf < 0 || b.stride_b < 0 || b.stride_b_sf < 0 ||
        b.stride_y <= 0 || b.stride_y / 2 < M * N || b.stride_res < 0)
      return BQ_ERR_SHAPE;
    if (b.stride_a % 16 || b.stride_b % 16 || b.stride_a_sf % 4 || b.stride_b_sf % 16 ||
        b.stride_y % 16 || b.stride_res % 16)
      return BQ_ERR_ALIGN;
  }
  g.y = static_cast<__nv_bfloat16*>(y_bf16);
  return run(c, false, empty, cfg, &g, stream);
}

int bq_gemm_int8_int8(const void* a_s8, const float* a_scale, const void* b_s8,
                      const float* b_scale, int64_t M, int64_t N, int64_t K, void* y_bf16,
                      bq_stream_t stream) {
  return bq_gemm_int8_int8_epilogue(a_s8, a_scale, b_s8, b_scale, M, N, K, y_bf16, nullptr,
                                    nullptr, nullptr, stream);
}

int bq_gemm_gated(int weight_kind, const void* a_q, const void* a_sf, const void* b_gate,
                  const void* gate_sf, const void* b_up, const void* up_sf, int64_t M, int64_t N,
                  int64_t K, void* h_bf16, const bq_gated_epilogue* epi,
                  const bq_gemm_config* cfg, bq_stream_t stream) {
  if (weight_kind != kMxfp4 && weight_kind != kFp8Blk32 && weight_kind != kMxfp8 &&
      weight_kind != kInt8)
    return BQ_ERR_INVALID;
  const Call c{static_cast<Kind>(weight_kind), a_q, a_sf, {b_gate, b_up}, {gate_sf, up_sf},
               M, N, K};
  int st = check_operands(c);
  if (st != BQ_OK) return st;
  const bq_gated_epilogue e = epi ? *epi : bq_gated_epilogue{1.0f, BQ_GATE_SILU, nullptr, nullptr,
                                                             nullptr};
  if (e.act != BQ_GATE_SILU && e.act != BQ_GATE_GELU) return BQ_ERR_INVALID;
  if ((e.q_out || e.sf_out) && N % 32 != 0) return BQ_ERR_SHAPE;
  if ((e.q_out != nullptr) != (e.sf_out != nullptr)) return BQ_ERR_NULL;
  const bool empty = M == 0 || N == 0;
  if (!empty) {
    if ((st = check_pointers(c, true)) != BQ_OK) return st;
    if (!h_bf16 && !e.q_out) return BQ_ERR_NULL;
    if (!aligned(h_bf16, 16) || !aligned(e.gu_out, 16) || !aligned(e.q_out, 16) ||
        !aligned(e.sf_out, 4))
      return BQ_ERR_ALIGN;
  }
  bq::FfnArgs g;
  memset(&g, 0, sizeof(g));
  g.alpha = e.alpha;
  g.act = e.act;
  g.y = static_cast<__nv_bfloat16*>(h_bf16);
  g.gu = static_cast<__nv_bfloat16*>(e.gu_out);
  g.q_out = static_cast<uint8_t*>(e.q_out);
  g.sf_out = static_cast<uint8_t*>(e.sf_out);
  return run(c, true, empty, cfg, &g, stream);
}

int bq_gated_grad_quant(const void* dh_bf16, int64_t ld_dh, const void* gu_bf16, int64_t ld_gu,
                        int64_t M, int64_t N, int act, int rounding, uint64_t seed, void* q_row,
                        void* sf_row, void* q_t, void* sf_t, void* d_bf16, int* d_status,
                        bq_stream_t stream) {
  if (act != BQ_GATE_SILU && act != BQ_GATE_GELU) return BQ_ERR_INVALID;
  if (rounding != BQ_ROUND_NEAREST && rounding != BQ_ROUND_STOCHASTIC) return BQ_ERR_INVALID;
  if (M < 0 || M > kMaxRows || M % 32 != 0 || N <= 0 || N % 32 != 0 || ld_dh < N ||
      ld_gu < 2 * N)
    return BQ_ERR_SHAPE;
  const int64_t groups = ceil_div(M, 128) * 4, tiles = ceil_div(N, 64);
  if (groups > 0x7FFFFFFF || ceil_div(tiles, 2) > 65535) return BQ_ERR_SHAPE;
  if (!aligned(d_status, 4)) return BQ_ERR_ALIGN;
  if (M > 0) {
    if (!dh_bf16 || !gu_bf16 || !q_row || !sf_row || !q_t || !sf_t) return BQ_ERR_NULL;
    if (!aligned(dh_bf16, 16) || !aligned(gu_bf16, 16) || ld_dh % 8 != 0 || ld_gu % 8 != 0 ||
        !aligned(q_row, 16) || !aligned(q_t, 16) || !aligned(sf_row, 4) || !aligned(sf_t, 4) ||
        !aligned(d_bf16, 16))
      return BQ_ERR_ALIGN;
  }
  Device dev;
  const int st = bqh::current_device(&dev);
  if (st != BQ_OK || M == 0) return st;
  const auto* dh = static_cast<const __nv_bfloat16*>(dh_bf16);
  const auto* gu = static_cast<const __nv_bfloat16*>(gu_bf16);
  auto *qr = static_cast<uint8_t*>(q_row), *sr = static_cast<uint8_t*>(sf_row);
  auto *qt = static_cast<uint8_t*>(q_t), *st8 = static_cast<uint8_t*>(sf_t);
  auto* d = static_cast<__nv_bfloat16*>(d_bf16);
  if (rounding == BQ_ROUND_NEAREST) {
    auto kern = act == BQ_GATE_SILU ? bq::gated_grad_rne_kernel<bq::kGateSilu>
                                    : bq::gated_grad_rne_kernel<bq::kGateGelu>;
    static bool ready[bqh::kMaxDevices][2] = {};
    if (!ready[dev.index][act]) {
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               bq::GradSmem::kBytes) != cudaSuccess)
        return BQ_ERR_CUDA;
      ready[dev.index][act] = true;
    }
    CUtensorMap th, tg, tu;
    int mst = matrix_map(&th, dh, M, N, ld_dh);
    if (mst == BQ_OK) mst = matrix_map(&tg, gu, M, N, ld_gu);
    if (mst == BQ_OK) mst = matrix_map(&tu, gu + N, M, N, ld_gu);
    if (mst != BQ_OK) return mst;
    return launch(kern,
                  dim3(static_cast<unsigned>(ceil_div(M, 128)),
                       static_cast<unsigned>(ceil_div(N, 128))),
                  bq::kGradThreads, bq::GradSmem::kBytes, 1, stream, th, tg, tu, M, N, qr, sr, qt,
                  st8, d, d_status, dev.err);
  }
  auto kern = act == BQ_GATE_SILU ? bq::gated_grad_sr_kernel<bq::kGateSilu>
                                  : bq::gated_grad_sr_kernel<bq::kGateGelu>;
  return launch(kern, dim3(static_cast<unsigned>(groups), static_cast<unsigned>(ceil_div(tiles, 8))),
                256, 0, 1, stream, dh, ld_dh, gu, ld_gu, M, N, tiles, qr, sr, qt, st8, d, d_status,
                seed);
}

int bq_ffn_plan(int weight_kind, int gated, int64_t M, int64_t N, int64_t K, int64_t batch,
                const bq_gemm_config* cfg, int num_sms, bq_gemm_config* out) {
  if (!out) return BQ_ERR_NULL;
  if (weight_kind != kInt8 && (!gated || weight_kind < kMxfp4 || weight_kind > kMxfp8))
    return BQ_ERR_INVALID;
  Call c{static_cast<Kind>(weight_kind), nullptr, nullptr, {nullptr, nullptr}, {nullptr, nullptr},
         M, N, K};
  c.batch.count = batch;
  if (M <= 0 || N <= 0 || batch <= 0 || num_sms < 1) return BQ_ERR_SHAPE;
  int st = check_operands(c);
  if (st == BQ_OK) st = check_config(cfg);
  Plan pl;
  if (st == BQ_OK) st = make_plan(c.kind, gated != 0, M, N, K, batch, cfg, num_sms, &pl);
  if (st != BQ_OK) return st;
  out->block_n = pl.bn;
  out->split_k = pl.splits;
  out->swap_ab = pl.pair ? 0 : 1;
  out->split_mode = pl.splits > 1 ? BQ_SPLIT_CLUSTER : BQ_SPLIT_AUTO;
  out->k_chunks = 1;
  out->cta_pair = pl.pair ? 2 : 1;
  return BQ_OK;
}

}  // extern "C"
