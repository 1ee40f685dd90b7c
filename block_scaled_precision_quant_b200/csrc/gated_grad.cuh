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
    const float s = __fdividef(1.0f, 1.0f + __expf(-g));
    du = dh * (g * s);
    dg = dh * u * (s * fmaf(g, 1.0f - s, 1.0f));
  } else {
    const float x = fabsf(g) * 0.70710678118654752f;
    const float k = __fdividef(1.0f, fmaf(0.3275911f, x, 1.0f));
    float poly = fmaf(k, 1.061405429f, -1.453152027f);
    poly = fmaf(k, poly, 1.421413741f);
    poly = fmaf(k, poly, -0.284496736f);
    poly = fmaf(k, poly, 0.254829592f);
    const float e = __expf(-x * x);  // e^(-g^2 / 2)
    const float erfc_x = k * poly * e;
    const float p = 0.5f * (g >= 0.0f ? 2.0f - erfc_x : erfc_x);
    du = dh * (g * p);
    dg = dh * u * fmaf(0.39894228040143268f * g, e, p);
  }
}

// Both quantizations of one warp tile: 32 rows x 64 columns of d, lane l holding
// row r0 + l in w (column 2 i in the low half of word i), zeros where there is
// nothing.  c0: the tile's first column in d (C = 2 F columns), ncols = 32 or 64
// of them exist.  rows_ok: the 32 rows exist.
template <bool SR>
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
    uint32_t pt, pr;
    if constexpr (SR) {
      if (i % 4 == 0)
        rnd = philox4x64_10(static_cast<uint64_t>(row * C + c0 + 2 * i) >> 3, seed);
      const uint32_t u0 = philox_draw(rnd, (2 * i) & 7), u1 = philox_draw(rnd, ((2 * i) & 7) + 1);
      auto sr = [](float v, uint32_t u) {
        return e5m2_sr(fminf(fmaxf(v, -57344.0f), 57344.0f), u);
      };
      pt = sr(t0, u0) | (sr(t1, u1) << 8);
      pr = sr(r0f, u0) | (sr(r1f, u1) << 8);
    } else {
      pt = e5m2x2(t0, t1);
      pr = e5m2x2(r0f, r1f);
    }
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
template <int ACT, bool SR>
__global__ void __launch_bounds__(256, 2) gated_grad_kernel(
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
  dual_quant_tile<SR>(wg, R, C, r0, c0, ncols, rows_ok, lane, stage[warp], q_row, sf_row, q_t,
                      sf_t, status, seed);
  dual_quant_tile<SR>(wu, R, C, r0, F + c0, ncols, rows_ok, lane, stage[warp], q_row, sf_row, q_t,
                      sf_t, status, seed);
  if (ct == col_tiles - 1) {  // scale padding behind the last column
    const int64_t katoms_t = ((R >> 5) + 3) >> 2, katoms_r = ((C >> 5) + 3) >> 2;
    for (int64_t g = C >> 5; g < katoms_r * 4; ++g) sf_row[sf_mma_offset(row, g, katoms_r)] = 127;
    for (int64_t c = C + lane; c < (C + 127) / 128 * 128; c += 32)
      sf_t[sf_mma_offset(c, r0 >> 5, katoms_t)] = 127;
  }
}

}  // namespace bq
