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

// Four codes (lowest first) to bf16, codes 0-1 in `lo`, 2-3 in `hi`.  With u the
// low seven bits of a code and s its sign, c = u - 128 s = (128 + u) - 128 (1 + s):
// both terms are the bits of a bf16 with 0x43 above the code's byte, the first
// with the sign bit cleared (128 + u has a step of one), the second with that bit
// alone (0x4300 = 128, 0x4380 = 256); their difference is exact.
__device__ __forceinline__ void int8x4_to_bf16x4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  const uint32_t x = codes & 0x7f7f7f7fu, y = codes & 0x80808080u;
  const uint32_t x0 = __byte_perm(x, 0x43434343u, 0x4140), x1 = __byte_perm(x, 0x43434343u, 0x4342);
  const uint32_t y0 = __byte_perm(y, 0x43434343u, 0x4140), y1 = __byte_perm(y, 0x43434343u, 0x4342);
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(x0), "r"(y0));
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(x1), "r"(y1));
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace pkv
