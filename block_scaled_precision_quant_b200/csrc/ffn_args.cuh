// ffn_args.cuh -- arguments and arithmetic that the int8 product and the
// gated feed-forward kernels share (lin_swap.cuh, lin_pair.cuh).
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
  int sf_a_bands;          // 128-row bands of A's scale buffer
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

// g / (1 + e^-g) with the fast exponential and division (relative errors near
// 2^-21, half a bf16 step is 2^-9).  e^-g overflows to +inf for g < -88, where
// the quotient's -0 is the value's own rounding.
__device__ __forceinline__ float silu(float g) {
  return __fdividef(g, 1.0f + __expf(-g));
}

__device__ __forceinline__ float gate_act(float g, int act) {
  return act == kGateSilu ? silu(g) : gelu_erf(g);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&p);
}

}  // namespace bq
