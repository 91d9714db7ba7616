// What the tensor-core attention kernels share: the shared-memory layout of
// query tiles and K/V stages, paired fp32 arithmetic, and the widening of FP8
// stages.
#pragma once
#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"

namespace pkv {

constexpr int kNK = kTcKeys;            // keys per tile (128)
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;
constexpr float kRescaleLog2 = 8.f;     // lazy O rescale threshold (log2 units)

template <int D>
struct TcSmem {
  static constexpr int kHalves = D / 64;                 // 128-byte-wide column slabs
  static constexpr int kKSt = D == 128 ? 2 : 4;          // K stages
  static constexpr int kVSt = D == 128 ? 3 : 4;          // V stages (the PV copies bound the pair period)
  static constexpr int kQ = kTcRows * D * 2;             // one query tile: [halves][128 rows][64]
  // One stage of K (or V), 128 keys: [8-key group][half][8 keys][64 columns],
  // each [8][64] piece a 1024-byte swizzle atom; one TMA box fills the two
  // groups of a block.  kGS: bytes between 8-key groups; kHS: between halves.
  static constexpr int kKV = kNK * D * 2;
  static constexpr int kGS = kHalves * 1024;
  static constexpr int kHS = 1024;
  static constexpr int kBlkBytes = 2 * kGS;              // one block (16 keys) of a stage
  static constexpr int kOffQ = 0;                        // tile A, then tile B
  static constexpr int kOffK = 2 * kQ;
  static constexpr int kOffV = kOffK + kKSt * kKV;
  static constexpr int kOffBar = kOffV + kVSt * kKV;
  static constexpr int kNumBars = 3 * kKSt + 3 * kVSt + 17;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kTotal = kOffMisc + 64;
};
static_assert(TcSmem<128>::kTotal <= 232448, "shared memory of the D=128 kernel");

__device__ __forceinline__ float max3f(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// (x0, x1) * s + (c, c) with one paired fp32 FMA.
__device__ __forceinline__ void fma2(float& x0, float& x1, float s, float c) {
  asm("{\n\t.reg .b64 p, q, r;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %2};\n\tmov.b64 r, {%3, %3};\n\t"
      "fma.rn.f32x2 p, p, q, r;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(x0), "+f"(x1) : "f"(s), "f"(c));
}

// (a0, a1) += (b0, b1) with one paired fp32 add.
__device__ __forceinline__ void add2(float& a0, float& a1, float b0, float b1) {
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\t"
      "add.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(a0), "+f"(a1) : "f"(b0), "f"(b1));
}

// FP8 pools: a stage holds the tile's e4m3 codes, [128 keys][D] bytes, in its
// upper half (as the TMA landed them); widen them in place to the f16 operand
// layout of the whole stage: [8-key group][64-column half][8 keys][128 bytes],
// 16-byte chunk c of a key's 128-byte line at c ^ (key % 8).  One warp.
//
// Each lane converts 8 codes into one 16-byte chunk per step, so the 8 lanes
// of a store phase fill the 8 chunks of one line (distinct banks after the
// swizzle) and read one key's contiguous codes.  Keys go in increasing order,
// 16 steps' codes loaded before any of their stores (the loads would
// otherwise wait behind the previous step's store).  The f16 line of key r
// (for r >= 64, in the upper half) covers the codes of a key no later than r:
// a batch overwrites only codes it or an earlier batch has already read.
template <int D>
__device__ __forceinline__ void widen_stage(uint8_t* stage, int lane) {
  using S = TcSmem<D>;
  constexpr int kGroups = D / 8;              // 8-code groups per key
  constexpr int kKeysPerStep = 32 / kGroups;  // keys converted per warp step
  constexpr int kBatch = 16;                  // steps whose codes are loaded together
  const uint8_t* codes = stage + S::kKV / 2;
  const int kk = lane / kGroups, g8 = lane % kGroups;
  const int hf = (g8 * 8) / 64, cw = g8 % 8;
#pragma unroll 1
  for (int b = 0; b < kNK / kKeysPerStep; b += kBatch) {
    uint2 v[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      v[u] = *reinterpret_cast<const uint2*>(codes + ((b + u) * kKeysPerStep + kk) * D + g8 * 8);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int r = (b + u) * kKeysPerStep + kk, r8 = r % 8;
      uint4 h;
      e4m3x4_to_f16x4(v[u].x, h.x, h.y);
      e4m3x4_to_f16x4(v[u].y, h.z, h.w);
      *reinterpret_cast<uint4*>(stage + (r / 8) * S::kGS + hf * S::kHS + r8 * 128 + ((cw ^ r8) * 16)) = h;
    }
  }
}

}  // namespace pkv
