// quant_i8.cuh -- per-token int8 quantization of bf16 rows.
//
//   amax = max(max_k |x[m, k]|, 2^-64);  scale[m] = fp32(amax / 127)
//   q = the integer nearest 127 x / amax, ties to even (in -127 .. 127)
//
// The quotient's rounding is exact.  Let c = fp32(127 / amax) and y = fp32(x c):
// two roundings, so y is within 2^-23 (relative) of n = 127 x / amax.  A tie
// (n = k + 1/2, k < 127) has at most 8 significant bits.  With x = X 2^i and
// amax = A 2^j, X and A below 2^8, any other n is at least 1 / (2 A) of a unit
// of 2^(i - j) away from a tie, that is 2^-17 relative.  Rounding y to 18
// bits moves it by at most 2^-18 relative: ties land on themselves, nothing
// else does.  Then an addition's own round to nearest even decides.  The
// floor of amax is a power of two so that A stays short.
//
// Reads 2 bytes and writes 1 an element; HBM bounds it: 8192 x 8192 30.5 us, 6.6 TB/s,
// the copy rate.
//
// The next kernel may start early: int8 products, whose weight these codes may be, wait
// for this one's end before they read either operand.  A product behind it gains 0.3 to 1
// us (both kernels: 41 x 4608 x 1536 7.6 to 7.2 us, 512 x 4096 x 4096 18.1 to 17.2), a chain
// of long quantizers as well (4096 x 4096 10.3 to 10.1 us, 8192 x 8192 31.1 to 30.5); alone
// and tiny it takes 0.1 longer (41 x 1536: 1.4 and 1.5 us).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "bq_ptx.cuh"
#include "f32x2.cuh"
#include "mx_quant.cuh"

namespace bq {

// Codes of two bf16 values in the low bytes of lo and hi: y rounded to 18 bits (the
// product with 2^6 + 1 carries the rest of y beyond the 24), then to an integer by
// adding 1.5 2^23, whose low byte is the code.
__device__ __forceinline__ void i8_codes2(uint32_t w, F2 c, uint32_t &lo, uint32_t &hi) {
  const F2 y = mul2(f2_bf16(w), c), p = mul2(y, f2(65.0f, 65.0f)), minus = f2(-1.0f, -1.0f);
  const F2 s = fma2(fma2(y, minus, p), minus, p);
  float a, b;
  f2_get(add2(s, f2(12582912.0f, 12582912.0f)), a, b);
  lo = __float_as_uint(a);
  hi = __float_as_uint(b);
}

// Four codes of two words of bf16 pairs.
__device__ __forceinline__ uint32_t i8_codes4(uint32_t w0, uint32_t w1, F2 c) {
  uint32_t a, b, d, e;
  i8_codes2(w0, c, a, b);
  i8_codes2(w1, c, d, e);
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(d, e, 0x0040), 0x5410);
}

// One warp per row of up to 256 VECS values, which stay in its registers (VECS
// 16-byte pieces a lane).  Many short rows want it: a block to a row leaves most
// of its threads idle (8192 x 256: 13.5 us, 3.6 with a warp each; 8192 x 2048: 18.7
// and 9.5; but 41 x 1536: 1.26 and 1.73, so few rows keep their blocks).
template <int kI8WarpVecs>
__global__ void __launch_bounds__(256) i8_quant_warp_kernel(const __nv_bfloat16 *__restrict__ x,
                                                            int64_t M, int64_t K, int64_t ldx,
                                                            uint8_t *__restrict__ q,
                                                            float *__restrict__ scale,
                                                            int *__restrict__ status) {
  const int lane = threadIdx.x & 31;
  const int64_t m = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  griddep_wait();
  griddep_launch_dependents();
  if (m >= M) return;  // whole warps leave
  const uint4 *src = reinterpret_cast<const uint4 *>(x + m * ldx);
  const int nv = static_cast<int>(K / 8);
  uint4 t[kI8WarpVecs];
  uint32_t mx = 0, bad = 0;
#pragma unroll
  for (int i = 0; i < kI8WarpVecs; ++i) {
    t[i] = make_uint4(0u, 0u, 0u, 0u);
    if (lane + 32 * i < nv) t[i] = __ldg(src + lane + 32 * i);
  }
#pragma unroll
  for (int i = 0; i < kI8WarpVecs; ++i) {
    const uint32_t w[4] = {t[i].x, t[i].y, t[i].z, t[i].w};
    mx = max(mx, bf16_amax_bits(w, bad));
  }
  mx = __reduce_max_sync(0xFFFFFFFFu, mx);
  const float amax = fmaxf(__uint_as_float(mx << 16), 0x1p-64f);
  const float c1 = __fdiv_rn(127.0f, amax);
  const F2 c = f2(c1, c1);
  if (lane == 0) {
    scale[m] = __fdiv_rn(amax, 127.0f);
    if (mx >= 0x7F80u && status) atomicOr(status, 1);
  }
  uint2 *dst = reinterpret_cast<uint2 *>(q + m * K);
#pragma unroll
  for (int i = 0; i < kI8WarpVecs; ++i)
    if (lane + 32 * i < nv)
      dst[lane + 32 * i] = make_uint2(i8_codes4(t[i].x, t[i].y, c), i8_codes4(t[i].z, t[i].w, c));
}

// One block of THREADS per row.  Each thread keeps its first VECS 16-byte pieces; the
// rest of a longer row is read twice, the second time from the caches.  (With 8 pieces the
// compiler spills 16 bytes of a thread's.)  256 threads
// of 4 pieces suit long rows, 128 of 8 many middling ones (8192 x 4112: 23.7 and
// 19.0 us, 600 x 4096: 2.6 and 2.45; 200 x 2048: 1.67 and 1.71, 8192 x 8192: 31.1
// and 31.9).
template <int THREADS, int VECS>
__global__ void __launch_bounds__(THREADS) i8_quant_kernel(const __nv_bfloat16 *__restrict__ x,
                                                           int64_t M, int64_t K, int64_t ldx,
                                                           uint8_t *__restrict__ q,
                                                           float *__restrict__ scale,
                                                           int *__restrict__ status) {
  __shared__ uint32_t part[THREADS / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int64_t m = blockIdx.x;
  const uint4 *src = reinterpret_cast<const uint4 *>(x + m * ldx);
  const int64_t nv = K / 8;
  uint4 t[VECS];
  uint32_t mx = 0, bad = 0;
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    t[i] = make_uint4(0u, 0u, 0u, 0u);
    if (threadIdx.x + THREADS * i < nv) t[i] = __ldg(src + threadIdx.x + THREADS * i);
  }
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    const uint32_t w[4] = {t[i].x, t[i].y, t[i].z, t[i].w};
    mx = max(mx, bf16_amax_bits(w, bad));
  }
  for (int64_t i = threadIdx.x + THREADS * VECS; i < nv; i += THREADS) {
    const uint4 v = __ldg(src + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    mx = max(mx, bf16_amax_bits(w, bad));
  }
  mx = __reduce_max_sync(0xFFFFFFFFu, mx);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = mx;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) mx = max(mx, part[i]);
  const float amax = fmaxf(__uint_as_float(mx << 16), 0x1p-64f);
  const float c1 = __fdiv_rn(127.0f, amax);
  const F2 c = f2(c1, c1);
  if (threadIdx.x == 0) {
    scale[m] = __fdiv_rn(amax, 127.0f);
    if (mx >= 0x7F80u && status) atomicOr(status, 1);
  }
  uint2 *dst = reinterpret_cast<uint2 *>(q + m * K);
#pragma unroll
  for (int i = 0; i < VECS; ++i)
    if (threadIdx.x + THREADS * i < nv)
      dst[threadIdx.x + THREADS * i] =
          make_uint2(i8_codes4(t[i].x, t[i].y, c), i8_codes4(t[i].z, t[i].w, c));
  for (int64_t i = threadIdx.x + THREADS * VECS; i < nv; i += THREADS) {
    const uint4 v = __ldg(src + i);
    dst[i] = make_uint2(i8_codes4(v.x, v.y, c), i8_codes4(v.z, v.w, c));
  }
}

}  // namespace bq
