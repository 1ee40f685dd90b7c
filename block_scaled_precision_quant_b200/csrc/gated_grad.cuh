// gated_grad.cuh -- backward pass of the gated product h = act(g) u: the
// gradients of both projections from the hidden row's gradient, quantized to
// E5M2 along both of their dimensions in the same pass.
//
//   dG = dH u act'(g),  dU = dH act(g)
//   SiLU:  s = 1 / (1 + e^-g),  act = g s,  act' = s (1 + g (1 - s))
//   GELU:  P = (1 + erf(g / sqrt 2)) / 2,  act = g P,
//          act' = P + g e^(-g^2 / 2) / sqrt(2 pi)
//
// d = [dG | dU] is the [M, 2 F] operand of both products that follow:
// dX = d [Wg; Wu] contracts over its columns, d^T X over its rows.  As all
// quantizers here read bf16, d is rounded to bf16 first, so the codes are those
// of bq_grad_quant_dual on the bf16 gradient (E5M2 keeps 3 of its 8 bits).
#pragma once

#include "grad_quant.cuh"
#include "ffn_args.cuh"

namespace bq {

template <int ACT>
__device__ __forceinline__ void gate_grad(float dh, float g, float u, float &dg, float &du) {
  if constexpr (ACT == kGateSilu) {
    const float s = rcp_fast(1.0f + exp2_fast(-kLog2e * g)), t = g * s;
    du = dh * t;
    dg = dh * u * fmaf(t, 1.0f - s, s);  // act' = s (1 + g (1 - s))
  } else {
    float e;
    const float p = gelu_cdf(g, e);
    du = dh * (g * p);
    dg = dh * u * fmaf(0.39894228040143268f * g, e, p);
  }
}

// The same for two elements.
template <int ACT>
__device__ __forceinline__ void gate_grad2(F2 dh, F2 g, F2 u, F2 &dg, F2 &du) {
  if constexpr (ACT == kGateSilu) {
    float a, b;
    f2_get(mul2(g, f2(-kLog2e, -kLog2e)), a, b);
    f2_get(add2(f2(exp2_fast(a), exp2_fast(b)), f2(1.0f, 1.0f)), a, b);
    const F2 s = f2(rcp_fast(a), rcp_fast(b)), t = mul2(g, s);
    du = mul2(dh, t);
    dg = mul2(mul2(dh, u), fma2(t, fma2(s, f2(-1.0f, -1.0f), f2(1.0f, 1.0f)), s));
  } else {
    F2 e;
    const F2 p = gelu_cdf2(g, e);
    du = mul2(dh, mul2(g, p));
    constexpr float kDensity = 0.39894228040143268f;  // 1 / sqrt(2 pi)
    dg = mul2(mul2(dh, u), fma2(mul2(g, f2(kDensity, kDensity)), e, p));
  }
}

// Both quantizations of one warp tile: 32 rows x 64 columns of d, lane l holding
// row r0 + l in w (column 2 i in the low half of word i), zeros where there is
// nothing.  c0: the tile's first column in d (C = 2 F columns), ncols = 32 or 64
// of them exist.  rows_ok: the 32 rows exist.
__device__ __forceinline__ void dual_quant_tile(const uint32_t (&w)[32], int64_t R, int64_t C,
                                                int64_t r0, int64_t c0, int ncols, bool rows_ok,
                                                int lane, uint8_t *st, uint8_t *q_row,
                                                uint8_t *sf_row, uint8_t *q_t, uint8_t *sf_t,
                                                int *status, uint64_t seed) {
  const int64_t g = r0 >> 5;
  const int64_t katoms_t = ((R >> 5) + 3) >> 2, katoms_r = ((C >> 5) + 3) >> 2;
  const int64_t row = r0 + lane;
  uint32_t m[32];
  uint32_t rmax[2] = {0u, 0u};  // this row's two 32-column groups
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    m[i] = w[i] & 0x7FFF7FFFu;
    rmax[i / 16] = max_u16x2(rmax[i / 16], m[i]);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) rmax[h] = max(rmax[h] & 0xFFFFu, rmax[h] >> 16);
  if (status && rows_ok && max(rmax[0], rmax[1]) >= 0x7F80u) atomicOr(status, 1);
  // Column maxima by recursive halving: lane l is left with columns 2l, 2l + 1.
#pragma unroll
  for (int k = 16; k >= 1; k >>= 1) {
    const bool up = (lane & k) != 0;
#pragma unroll
    for (int i = 0; i < k; ++i) {
      const uint32_t send = up ? m[i] : m[i + k];
      const uint32_t keep = up ? m[i + k] : m[i];
      m[i] = max_u16x2(keep, __shfl_xor_sync(0xFFFFFFFFu, send, k));
    }
  }
  const uint32_t pe = static_cast<uint32_t>(mx_exponent_e5m2(m[0] & 0xFFFFu) + 127) |
                      (static_cast<uint32_t>(mx_exponent_e5m2(m[0] >> 16) + 127) << 8);
  if (2 * lane < ncols) {
    sf_t[sf_mma_offset(c0 + 2 * lane, g, katoms_t)] =
        static_cast<uint8_t>(rows_ok ? pe & 0xFFu : 127u);
    sf_t[sf_mma_offset(c0 + 2 * lane + 1, g, katoms_t)] =
        static_cast<uint8_t>(rows_ok ? pe >> 8 : 127u);
  }
  const int er[2] = {mx_exponent_e5m2(rmax[0]), mx_exponent_e5m2(rmax[1])};
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (32 * h < ncols)
      sf_row[sf_mma_offset(row, (c0 >> 5) + h, katoms_r)] =
          static_cast<uint8_t>(rows_ok ? er[h] + 127 : 127);
  if (!rows_ok) return;  // warp-uniform
  const float rinv0 = __uint_as_float(static_cast<uint32_t>(127 - er[0]) << 23);
  const float rinv1 = __uint_as_float(static_cast<uint32_t>(127 - er[1]) << 23);
  Philox4 rnd;
  uint32_t rowc[16];  // this row's 64 codes, four per word
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const uint32_t p = __shfl_sync(0xFFFFFFFFu, pe, i);
    const float inv0 = __uint_as_float((254u - (p & 0xFFu)) << 23);
    const float inv1 = __uint_as_float((254u - (p >> 8)) << 23);
    const float rinv = i < 16 ? rinv0 : rinv1;
    const float x0 = __uint_as_float(w[i] << 16), x1 = __uint_as_float(w[i] & 0xFFFF0000u);
    const float t0 = __fmul_rn(x0, inv0), t1 = __fmul_rn(x1, inv1);    // along the rows
    const float r0f = __fmul_rn(x0, rinv), r1f = __fmul_rn(x1, rinv);  // along the columns
    if (i % 4 == 0)  // one Philox block serves 8 consecutive elements of a row
      rnd = philox4x64_10(static_cast<uint64_t>(row * C + c0 + 2 * i) >> 3, seed);
    const uint32_t u0 = philox_draw(rnd, (2 * i) & 7), u1 = philox_draw(rnd, ((2 * i) & 7) + 1);
    auto sr = [](float v, uint32_t u) {
      return e5m2_sr(fminf(fmaxf(v, -57344.0f), 57344.0f), u);
    };
    const uint32_t pt = sr(t0, u0) | (sr(t1, u1) << 8);
    const uint32_t pr = sr(r0f, u0) | (sr(r1f, u1) << 8);
    st[(2 * i) * 32 + lane] = static_cast<uint8_t>(pt);
    st[(2 * i + 1) * 32 + lane] = static_cast<uint8_t>(pt >> 8);
    if (i % 2 == 0)
      rowc[i / 2] = pr & 0xFFFFu;
    else
      rowc[i / 2] |= pr << 16;
  }
#pragma unroll
  for (int v = 0; v < 4; ++v)
    if (16 * v < ncols)
      *reinterpret_cast<uint4 *>(q_row + row * C + c0 + 16 * v) =
          make_uint4(rowc[4 * v], rowc[4 * v + 1], rowc[4 * v + 2], rowc[4 * v + 3]);
  __syncwarp();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = 2 * lane + h;
    if (j < ncols) {
      const uint4 *src = reinterpret_cast<const uint4 *>(st + j * 32);
      uint4 *dst = reinterpret_cast<uint4 *>(q_t + (c0 + j) * R + r0);
      dst[0] = src[0];
      dst[1] = src[1];
    }
  }
  __syncwarp();  // the staging tile is free again
}

// dh [R, ld_dh], gu [R, ld_gu] (g in columns 0 .. F - 1, u in F .. 2 F - 1); the
// outputs are those of bq_grad_quant_dual for d [R, 2 F].  d_out: d itself in
// bf16, row pitch 2 F (optional).  R % 32 == 0, F % 32 == 0.
// grid.x = 32-row group (up to the scale padding), grid.y * 8 + warp = tile of 64
// columns of F; a warp forms and quantizes its tile of dG, then that of dU.
// 4096 x 6144 300 us (bq_grad_quant_dual of a ready [4096, 12288] gradient 190): far from
// memory's 36, and from the 113 that its instructions (79 an element of d, most of them the
// random words' and both roundings') would take if one issued every cycle.  One issues in
// 35 % of them: 16 warps an SM, at 128 registers a thread, run through two unrolled copies
// of the tile's quantizer and wait for instructions most often, then for their own results.
template <int ACT>
__global__ void __launch_bounds__(256, 2) gated_grad_sr_kernel(
    const __nv_bfloat16 *__restrict__ dh, int64_t ld_dh, const __nv_bfloat16 *__restrict__ gu,
    int64_t ld_gu, int64_t R, int64_t F, int64_t col_tiles, uint8_t *__restrict__ q_row,
    uint8_t *__restrict__ sf_row, uint8_t *__restrict__ q_t, uint8_t *__restrict__ sf_t,
    __nv_bfloat16 *__restrict__ d_out, int *__restrict__ status, uint64_t seed) {
  __shared__ __align__(16) uint8_t stage[8][64 * 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t ct = static_cast<int64_t>(blockIdx.y) * 8 + warp;
  if (ct >= col_tiles) return;  // whole warps leave; only warp-level sync below
  const int64_t C = 2 * F, c0 = ct * 64, r0 = static_cast<int64_t>(blockIdx.x) * 32;
  const int64_t row = r0 + lane;
  const bool rows_ok = r0 < R;
  const int ncols = F - c0 < 64 ? 32 : 64;
  griddep_wait();
  griddep_launch_dependents();

  uint32_t wg[32], wu[32];
#pragma unroll
  for (int v = 0; v < 8; ++v) {
    uint4 th = make_uint4(0u, 0u, 0u, 0u), tg = th, tu = th;
    if (rows_ok && 8 * v < ncols) {
      const int64_t c = c0 + 8 * v;
      th = __ldg(reinterpret_cast<const uint4 *>(dh + row * ld_dh + c));
      tg = __ldg(reinterpret_cast<const uint4 *>(gu + row * ld_gu + c));
      tu = __ldg(reinterpret_cast<const uint4 *>(gu + row * ld_gu + F + c));
    }
    const uint32_t h4[4] = {th.x, th.y, th.z, th.w}, g4[4] = {tg.x, tg.y, tg.z, tg.w},
                   u4[4] = {tu.x, tu.y, tu.z, tu.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float dg[2], du[2];
      gate_grad<ACT>(bf16_bits_to_f32(h4[j] & 0xFFFFu), bf16_bits_to_f32(g4[j] & 0xFFFFu),
                     bf16_bits_to_f32(u4[j] & 0xFFFFu), dg[0], du[0]);
      gate_grad<ACT>(bf16_bits_to_f32(h4[j] >> 16), bf16_bits_to_f32(g4[j] >> 16),
                     bf16_bits_to_f32(u4[j] >> 16), dg[1], du[1]);
      wg[4 * v + j] = pack_bf16(dg[0], dg[1]);
      wu[4 * v + j] = pack_bf16(du[0], du[1]);
    }
    if (d_out && rows_ok && 8 * v < ncols) {
      __nv_bfloat16 *d = d_out + row * C + c0 + 8 * v;
      *reinterpret_cast<uint4 *>(d) =
          make_uint4(wg[4 * v], wg[4 * v + 1], wg[4 * v + 2], wg[4 * v + 3]);
      *reinterpret_cast<uint4 *>(d + F) =
          make_uint4(wu[4 * v], wu[4 * v + 1], wu[4 * v + 2], wu[4 * v + 3]);
    }
  }
  dual_quant_tile(wg, R, C, r0, c0, ncols, rows_ok, lane, stage[warp], q_row, sf_row, q_t,
                      sf_t, status, seed);
  dual_quant_tile(wu, R, C, r0, F + c0, ncols, rows_ok, lane, stage[warp], q_row, sf_row, q_t,
                      sf_t, status, seed);
  if (ct == col_tiles - 1) {  // scale padding behind the last column
    const int64_t katoms_t = ((R >> 5) + 3) >> 2, katoms_r = ((C >> 5) + 3) >> 2;
    for (int64_t g = C >> 5; g < katoms_r * 4; ++g) sf_row[sf_mma_offset(row, g, katoms_r)] = 127;
    for (int64_t c = C + lane; c < (C + 127) / 128 * 128; c += 32)
      sf_t[sf_mma_offset(c, r0 >> 5, katoms_t)] = 127;
  }
}

// ---- round to nearest ------------------------------------------------------
//
// A block owns 128 rows x 128 columns of F: three TMA loads bring dH, g and u into
// shared memory (zeros outside), and it works on them three times, each time with
// the ownership that needs no exchange between threads:
//   1. eight columns of a row a thread: dG and dU as bf16 in the places of g and u;
//   2. 16 columns of a row a thread, two threads a group (one shuffle for its
//      maximum): the row-wise codes, a row's 128 bytes by eight threads;
//   3. two columns x 32 rows a thread, whole groups: the transposed codes, which
//      turn around through the tiles' memory and leave as 128-byte lines.
// Floor: 6 bytes read and 4.1 written for each element of F.  Bound by the
// instructions it issues (41 an element, in 60 % of the cycles; 46 before pairs of values
// took one, 63 in a version that kept one ownership and met by shuffles) and the wait for
// a block's tiles: 4096 x 6144 53 us, 4.8 TB/s (GELU 59 to 66; bq_grad_quant_dual of a
// ready [4096, 12288] gradient 88).
struct GradSmem {
  static constexpr int kTile = 128 * 256;         // [128 rows][128 bf16]: g, u, dH
  static constexpr int kOffSfr = 3 * kTile;       // [2][128 rows][4 groups]
  static constexpr int kOffSft = kOffSfr + 1024;  // [2][128 columns][4 groups]
  static constexpr int kOffBar = kOffSft + 1024;
  static constexpr int kBytes = kOffBar + 16;
};

// Four E5M2 codes (round to nearest even, saturating) in one word, a in the low byte:
// packed by the conversions themselves.
__device__ __forceinline__ uint32_t e5m2x4(float a, float b, float c, float d) {
  uint32_t w;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e5m2x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e5m2x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(w)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return w;
}

// The larger magnitudes of two bf16 pairs (their signs are of no use; NaN wins).
__device__ __forceinline__ uint32_t absmax_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Byte offset of 16-byte piece q (8 columns) of row r of a tile: the pieces of a
// row's second half are swapped in pairs, so eight threads that read every second
// piece of a row meet no bank twice.
__device__ __forceinline__ uint32_t grad_at(int r, int q) {
  return static_cast<uint32_t>(r * 256 + ((q ^ (q >> 3)) << 4));
}

// Byte offset of 16-byte piece q of row r of a [128][128]-byte tile, permuted so
// that stores to every second row and loads of whole rows meet no bank twice.
__device__ __forceinline__ uint32_t code_at(int r, int q) {
  return static_cast<uint32_t>(r * 128 + ((q ^ ((r >> 1) & 7)) << 4));
}

constexpr int kGradThreads = 512;

template <int ACT>
__global__ void __launch_bounds__(kGradThreads, 2) gated_grad_rne_kernel(
    const __grid_constant__ CUtensorMap tm_dh, const __grid_constant__ CUtensorMap tm_g,
    const __grid_constant__ CUtensorMap tm_u, int64_t R, int64_t F, uint8_t *__restrict__ q_row,
    uint8_t *__restrict__ sf_row, uint8_t *__restrict__ q_t, uint8_t *__restrict__ sf_t,
    __nv_bfloat16 *__restrict__ d_out, int *__restrict__ status, int *__restrict__ err) {
  extern __shared__ __align__(128) uint8_t grad_smem[];
  __shared__ int abort_flag;
  uint8_t *sm = grad_smem;
  uint64_t *bar = reinterpret_cast<uint64_t *>(sm + GradSmem::kOffBar);
  const int tid = threadIdx.x;
  const int64_t C = 2 * F, b0 = static_cast<int64_t>(blockIdx.x) * 128;  // rows
  const int64_t c0 = static_cast<int64_t>(blockIdx.y) * 128;             // columns of F
  const int ncols = static_cast<int>(F - c0 < 128 ? F - c0 : 128);       // multiples of 32
  const int nrows = static_cast<int>(R - b0 < 128 ? R - b0 : 128);
  if (tid == 0) {
    mbar_init(bar, 1);
    abort_flag = 0;
    fence_mbar_init();
    griddep_wait();
    mbar_arrive_expect_tx(bar, 3 * GradSmem::kTile);
    const int x = static_cast<int>(c0), y = static_cast<int>(b0);
    tma_load_2d(sm, &tm_g, bar, x, y);
    tma_load_2d(sm + GradSmem::kTile, &tm_u, bar, x, y);
    tma_load_2d(sm + 2 * GradSmem::kTile, &tm_dh, bar, x, y);
  }
  __syncthreads();
  griddep_wait();  // the kernel before may still read what this one writes
  griddep_launch_dependents();
  if (!mbar_wait(bar, 0, err, &abort_flag, kWaitLanding)) return;

  {
    const int q = tid & 15, r1 = tid >> 4;  // rows r1, r1 + 32, ...: a warp holds whole rows
    const uint8_t *src = sm + r1 * 256 + q * 16;
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
      const uint4 tg = *reinterpret_cast<const uint4 *>(src + k * 32 * 256);
      const uint4 tu = *reinterpret_cast<const uint4 *>(src + GradSmem::kTile + k * 32 * 256);
      const uint4 th = *reinterpret_cast<const uint4 *>(src + 2 * GradSmem::kTile + k * 32 * 256);
      const uint32_t h4[4] = {th.x, th.y, th.z, th.w}, g4[4] = {tg.x, tg.y, tg.z, tg.w},
                     u4[4] = {tu.x, tu.y, tu.z, tu.w};
      uint32_t og[4], ou[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        F2 dg, du;
        gate_grad2<ACT>(f2_bf16(h4[j]), f2_bf16(g4[j]), f2_bf16(u4[j]), dg, du);
        og[j] = pack_bf16(dg);
        ou[j] = pack_bf16(du);
      }
      const int r = r1 + 32 * k;
      __syncwarp();  // the row has been read
      *reinterpret_cast<uint4 *>(sm + grad_at(r, q)) = make_uint4(og[0], og[1], og[2], og[3]);
      *reinterpret_cast<uint4 *>(sm + GradSmem::kTile + grad_at(r, q)) =
          make_uint4(ou[0], ou[1], ou[2], ou[3]);
      if (d_out && 8 * q < ncols && r < nrows) {
        __nv_bfloat16 *d = d_out + (b0 + r) * C + c0 + 8 * q;
        *reinterpret_cast<uint4 *>(d) = make_uint4(og[0], og[1], og[2], og[3]);
        *reinterpret_cast<uint4 *>(d + F) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
      }
    }
  }
  __syncthreads();

  {  // along the columns of d: 16 columns of rows r1, r1 + 64 of both halves
    const int j = tid & 7, r1 = tid >> 3;
    uint32_t bad = 0;
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
      const int half = k >> 1, r = r1 + 64 * (k & 1);
      const uint8_t *tile = sm + half * GradSmem::kTile;
      const uint4 a = *reinterpret_cast<const uint4 *>(tile + grad_at(r, 2 * j));
      const uint4 b = *reinterpret_cast<const uint4 *>(tile + grad_at(r, 2 * j + 1));
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      const uint32_t m2 =
          absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(w[0], w[1]), absmax_bf16x2(w[2], w[3])),
                        absmax_bf16x2(absmax_bf16x2(w[4], w[5]), absmax_bf16x2(w[6], w[7]))) &
          0x7FFF7FFFu;
      uint32_t mx = max(m2 & 0xFFFFu, m2 >> 16);
      bad |= mx >= 0x7F80u ? 1u : 0u;
      mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
      const int e = mx_exponent_e5m2(mx);
      const float inv1 = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      const F2 inv = f2(inv1, inv1);
      uint32_t codes[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float c[4];
        f2_get(mul2(f2_bf16(w[2 * i]), inv), c[0], c[1]);
        f2_get(mul2(f2_bf16(w[2 * i + 1]), inv), c[2], c[3]);
        codes[i] = e5m2x4(c[0], c[1], c[2], c[3]);
      }
      if (r < nrows && 16 * j < ncols)
        *reinterpret_cast<uint4 *>(q_row + (b0 + r) * C + half * F + c0 + 16 * j) =
            make_uint4(codes[0], codes[1], codes[2], codes[3]);
      if ((j & 1) == 0)
        sm[GradSmem::kOffSfr + (half * 128 + r) * 4 + (j >> 1)] =
            static_cast<uint8_t>(r < nrows ? e + 127 : 127);
    }
    if (bad && status) atomicOr(status, 1);
  }
  // along the rows: columns 2 p, 2 p + 1 of the 32-row group rg of one half
  const int p = tid & 63, rg = (tid >> 6) & 3, half = tid >> 8;
  uint32_t out[2][8];
  {
    const uint8_t *tile = sm + half * GradSmem::kTile + 4 * (p & 3);
    uint32_t w[32];
#pragma unroll
    for (int r = 0; r < 32; ++r)
      w[r] = *reinterpret_cast<const uint32_t *>(tile + grad_at(rg * 32 + r, p >> 2));
    uint32_t m = w[0];
#pragma unroll
    for (int r = 1; r < 32; ++r) m = absmax_bf16x2(m, w[r]);
    m &= 0x7FFF7FFFu;
    const int e0 = mx_exponent_e5m2(m & 0xFFFFu), e1 = mx_exponent_e5m2(m >> 16);
    const bool ok = rg * 32 < nrows;
    uint8_t *sft = sm + GradSmem::kOffSft + (half * 128 + 2 * p) * 4 + rg;
    sft[0] = static_cast<uint8_t>(ok ? e0 + 127 : 127);
    sft[4] = static_cast<uint8_t>(ok ? e1 + 127 : 127);
    const F2 inv = f2(__uint_as_float(static_cast<uint32_t>(127 - e0) << 23),
                      __uint_as_float(static_cast<uint32_t>(127 - e1) << 23));
#pragma unroll
    for (int j = 0; j < 8; ++j) {  // rows 4 j .. 4 j + 3
      float lo[4], hi[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) f2_get(mul2(f2_bf16(w[4 * j + t]), inv), lo[t], hi[t]);
      out[0][j] = e5m2x4(lo[0], lo[1], lo[2], lo[3]);
      out[1][j] = e5m2x4(hi[0], hi[1], hi[2], hi[3]);
    }
  }
  __syncthreads();  // the tiles have been read
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int q = 0; q < 2; ++q)
      *reinterpret_cast<uint4 *>(sm + half * 16384 + code_at(2 * p + h, 2 * rg + q)) = make_uint4(
          out[h][4 * q], out[h][4 * q + 1], out[h][4 * q + 2], out[h][4 * q + 3]);
  __syncthreads();
#pragma unroll
  for (int i = tid; i < 2048; i += kGradThreads) {
    const int hf = i >> 10, c = (i >> 3) & 127, q = i & 7;
    if (c < ncols && 16 * q < nrows)
      *reinterpret_cast<uint4 *>(q_t + (hf * F + c0 + c) * R + b0 + 16 * q) =
          *reinterpret_cast<const uint4 *>(sm + hf * 16384 + code_at(c, q));
  }
  const int64_t katoms_t = ((R >> 5) + 3) >> 2, katoms_r = ((C >> 5) + 3) >> 2;
  if (tid < 256) {
    const int t = tid & 127;
    const int64_t cd = (tid >> 7) * F + c0, g = cd >> 5;  // first column and group in d
    const uint8_t *sfr = sm + GradSmem::kOffSfr + tid * 4;
    const int ng = ncols >> 5;
    if (ng == 4 && (g & 3) == 0) {  // a word of a scale atom
      *reinterpret_cast<uint32_t *>(sf_row + sf_mma_offset(b0 + t, g, katoms_r)) =
          *reinterpret_cast<const uint32_t *>(sfr);
    } else {
      for (int i = 0; i < ng; ++i) sf_row[sf_mma_offset(b0 + t, g + i, katoms_r)] = sfr[i];
    }
    if (t < ncols)
      *reinterpret_cast<uint32_t *>(sf_t + sf_mma_offset(cd + t, b0 >> 5, katoms_t)) =
          *reinterpret_cast<const uint32_t *>(sm + GradSmem::kOffSft + tid * 4);
  }
  if (blockIdx.y == gridDim.y - 1 && tid < 128) {  // padding behind the last column
    for (int64_t g = C >> 5; g < katoms_r * 4; ++g)
      sf_row[sf_mma_offset(b0 + tid, g, katoms_r)] = 127;
    const int64_t c = C + tid;
    if (c < (C + 127) / 128 * 128)
      *reinterpret_cast<uint32_t *>(sf_t + sf_mma_offset(c, b0 >> 5, katoms_t)) = 0x7F7F7F7Fu;
  }
}

}  // namespace bq
