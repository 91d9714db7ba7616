// Int8 pools: a code c of a (block, KV head) stands for c * 2^e, e the block's
// exponent for K or V, |c| <= 127 and -126 <= e <= kMaxExp.  Every such value is
// a normal bf16 value (or zero): a code has seven bits, and 127 * 2^121 is below
// the largest bf16.  So widening is exact, and a product with 2^e in bf16 is too.
#pragma once
#include <cuda_runtime.h>

#include "internal.h"

namespace pkv {

constexpr int kMinExp = -126, kMaxExp = 121;

// The exponent of a block as read (a page never written may hold anything).
__device__ __forceinline__ int safe_exp(int e) { return min(max(e, kMinExp), kMaxExp); }
__device__ __forceinline__ float exp_f32(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
// 2^e twice, as bf16.
__device__ __forceinline__ uint32_t exp_bf16x2(int e) { return static_cast<uint32_t>(e + 127) * 0x00800080u; }

// Four codes c (lowest first) to bf16 values c * 2^-kWidenShift, codes 0-1 in `lo`, 2-3
// in `hi`.  A bf16 below 2^-125 is a fixed-point number: the bits 0x00uu are uu *
// 2^-133 for all eight bits (subnormal to 127, then the first binade, whose step is
// the same).  With uu = c + 128 the fused uu * 2^-133 * 2^127 - 128 * 2^-6 is exact.
// Three integer instructions a word; taking 128 + (low bits) and the sign apart, as
// exponents in place, takes six: 10 requests of 1 to 733 new tokens over int8, 64 / 8 heads,
// on tiles 294 us against 280 (both before the widening's later steps); decoding took the same time.
constexpr int kWidenShift = 6;
__device__ __forceinline__ void int8x4_to_bf16x4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  const uint32_t x = codes ^ 0x80808080u;
  const uint32_t x0 = __byte_perm(x, 0u, 0x4140), x1 = __byte_perm(x, 0u, 0x4342);
  constexpr uint32_t kUp = 0x7f007f00u, kOff = 0xc000c000u;   // 2^127, -2
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(lo) : "r"(x0), "r"(kUp), "r"(kOff));
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(hi) : "r"(x1), "r"(kUp), "r"(kOff));
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace pkv
