// What the two attention kernels over the 8-bit paged cache share.
//
// Scores are log2-scaled: t = scale log2(e) 2^Ek (q . k codes), the K scale of a block of 16
// keys applied to its scores.  The V scale goes into the exponent: weights 2^(t + Ev - m),
// m near the running maximum of t + Ev, multiply the V codes as they are, and the sum of the
// weights takes 2^-Ev back out block by block.  So both matrix products have the 8-bit codes
// as operands, which fp16 holds exactly (so does the fp16 instruction's product); q is scaled
// by a power of two per row and rounded to fp16's 11 bits (exact for bf16 values unless the
// rotation went over them), the weights to 11 bits.  Exponents of scales lie within +-40, so
// that neither a weight nor a sum leaves fp32's range.
#pragma once

#include <cuda_fp16.h>

#include "kv_cache.cuh"
#include "quad_block.cuh"

namespace w4a4 {

// Weights are 2^(t + Ev - m) with m kShift below the maximum that was last looked for, which may
// lag the true one: by kLag at most with few rows (2^(kShift + kLag), well below fp16's 65504), by
// as much as the weights' sums allow with many.  What lies 2^-28 below the largest still has a bit
// in fp16's subnormals.
constexpr float kShift = 4.0f, kLag = 10.0f;
constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}
// Two bytes (signed codes + 128, at the places that `sel` picks) to fp16: the byte below
// 0x64 is 1024 + byte, and one exact subtraction of 1152 leaves the code.
__device__ __forceinline__ uint32_t codes_half2(uint32_t biased, uint32_t sel) {
  const uint32_t u = prmt(biased, 0x64646464u, sel);
  uint32_t r;
  asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(u), "r"(0x64806480u));
  return r;
}

// The row's power-of-two scale: the largest magnitude goes to 2^7 .. 2^8.
__device__ __forceinline__ int row_exponent(float amax) {
  return max(static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 7, -107);
}

// Keys that the query at position pos sees: lo .. hi - 1.
__device__ __forceinline__ void seen(const KvAttn& a, int pos, int len, int& lo, int& hi) {
  hi = a.causal ? min(len, pos + 1) : len;
  lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
}

}  // namespace w4a4
