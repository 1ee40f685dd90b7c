// ffn_args.cuh -- arguments and arithmetic that the int8 product and the
// gated feed-forward kernels share (lin_swap.cuh, lin_pair.cuh, gated_mx.cuh,
// gated_grad.cuh).
//
// Both compute products A B^T of K-major operands of one byte per code:
//   int8   s8 codes, exact s32 sums (tcgen05.mma kind::i8); a token's scale
//          sa[m] and a channel's sb[n] multiply the sum:
//            y = bf16(act(alpha sa[m] sb[n] acc + bias[n]) + residual)
//   MX     E4M3 activations and E4M3 or E2M1 weights with E8M0 scales per 32
//          inputs, applied by the MMA (kind::mxf8f6f4, fp32 sums).
// The gated form multiplies A with two weights of the same shape and leaves
//   h = bf16(act(g) u),  g = alpha A Wg^T,  u = alpha A Wu^T
// (int8: g and u with their scales), act SiLU or the erf GELU, g and u in
// fp32 up to the one rounding of h.
#pragma once

#include "f32x2.cuh"
#include "gemm_bs.cuh"

namespace bq {

enum GateAct : int { kGateSilu = 0, kGateGelu = 1 };

// GemmArgs names the P side the 128-row side of an MMA; here its sf_p / sf_q
// pairs are unused and the operands' scales are named by operand.
struct FfnArgs : GemmArgs {
  uint32_t w_tile_bytes;   // transaction bytes of a 128 x 128 weight tile (E2M1: half)
  uint32_t fmt_w, fmt_a;   // kind::mxf8f6f4 operand formats
  const uint8_t *sf_a;     // MX: scale atoms of A and of the weights
  const uint8_t *sf_w[2];
  const float *sa;         // int8: token scales [M] and channel scales [N]
  const float *sw[2];
  int64_t sa_bstride, sw_bstride;  // elements
  __nv_bfloat16 *gu;       // optional [M, 2 N]: g, then u, each rounded to bf16
};

__device__ __forceinline__ void tc_mma_i8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t"
      "}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor of kind::i8 with signed 8-bit operands and s32 sums.
__host__ __device__ constexpr uint32_t idesc_i8(int m, int n) {
  return (2u << 4)                                // D: s32
         | (1u << 7) | (1u << 10)                 // A, B: signed 8-bit
         | (static_cast<uint32_t>(n >> 3) << 17)  // N / 8
         | (static_cast<uint32_t>(m >> 4) << 24); // M / 16
}

__device__ __forceinline__ float rcp_fast(float x) {  // relative error 2^-23
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {  // relative error 2^-22
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float kLog2e = 1.4426950408889634f;

// g / (1 + e^-g).  Relative error at most |g| 2^-23.7 for g < 0 (the exponent's argument
// rounds: 2^-21 at -6, 2^-19 at -30, 2^-17.3 at -87) and 2^-21 of the two fast operations,
// for any g above -87; half a bf16 step is 2^-8.  Below that the quotient, under 2^-118,
// comes out as -0.
__device__ __forceinline__ float silu(float g) {
  return g * rcp_fast(1.0f + exp2_fast(-kLog2e * g));
}

// e^(-g^2 / 2), and P(g) = (1 + erf(g / sqrt 2)) / 2 by the formula of gelu_erf
// (Abramowitz and Stegun 7.1.26, absolute error 0.8e-7).
__device__ __forceinline__ float gelu_cdf(float g, float &e) {
  const float x = fabsf(g) * 0.70710678118654752f;
  const float k = rcp_fast(fmaf(0.3275911f, x, 1.0f));
  float poly = fmaf(k, 1.061405429f, -1.453152027f);
  poly = fmaf(k, poly, 1.421413741f);
  poly = fmaf(k, poly, -0.284496736f);
  poly = fmaf(k, poly, 0.254829592f);
  e = exp2_fast(-kLog2e * x * x);
  const float half_erfc = 0.5f * k * poly * e;  // of |g| / sqrt 2
  return g >= 0.0f ? 1.0f - half_erfc : half_erfc;
}

__device__ __forceinline__ float gelu_gate(float g) {
  float e;
  return g * gelu_cdf(g, e);
}

__device__ __forceinline__ float gate_act(float g, int act) {
  return act == kGateSilu ? silu(g) : gelu_gate(g);
}

// gelu_cdf of two values.
__device__ __forceinline__ F2 gelu_cdf2(F2 g, F2 &e) {
  constexpr float kSlope = 0.3275911f * 0.70710678118654752f;
  float g0, g1, e0, e1, h0, h1;
  f2_get(g, g0, g1);
  const F2 k = f2(rcp_fast(fmaf(kSlope, fabsf(g0), 1.0f)), rcp_fast(fmaf(kSlope, fabsf(g1), 1.0f)));
  F2 poly = fma2(k, f2(0.5307027145f, 0.5307027145f), f2(-0.7265760135f, -0.7265760135f));
  poly = fma2(k, poly, f2(0.7107068705f, 0.7107068705f));
  poly = fma2(k, poly, f2(-0.142248368f, -0.142248368f));
  poly = fma2(k, poly, f2(0.127414796f, 0.127414796f));  // the polynomial's half
  f2_get(mul2(mul2(g, f2(-0.5f * kLog2e, -0.5f * kLog2e)), g), e0, e1);
  e = f2(exp2_fast(e0), exp2_fast(e1));
  f2_get(mul2(mul2(k, poly), e), h0, h1);
  return f2(g0 >= 0.0f ? 1.0f - h0 : h0, g1 >= 0.0f ? 1.0f - h1 : h1);
}

__device__ __forceinline__ F2 gelu_gate2(F2 g) {
  F2 e;
  return mul2(g, gelu_cdf2(g, e));
}
__device__ __forceinline__ F2 silu2(F2 g) {
  float a, b;
  f2_get(mul2(g, f2(-kLog2e, -kLog2e)), a, b);
  f2_get(add2(f2(exp2_fast(a), exp2_fast(b)), f2(1.0f, 1.0f)), a, b);
  return mul2(g, f2(rcp_fast(a), rcp_fast(b)));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&p);
}
__device__ __forceinline__ uint32_t pack_bf16(F2 v) {
  float lo, hi;
  f2_get(v, lo, hi);
  return pack_bf16(lo, hi);
}

}  // namespace bq
