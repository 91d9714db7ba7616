// Attention of up to 16 query rows on the warp-level MMA (mma.sync m16n8k16,
// fp32 accumulation), one 16-key block of the pool at a time: the core that
// the tree and the block-selected attention share.
//
// One warp holds its rows' queries as A fragments in registers, streams
// (block, KV head) chunks of K and V through a shared-memory ring that it fills
// with asynchronous copies, and keeps the rows' online softmax (running max m, sum l, fp32 accumulator
// o).  Thread t = 4g + c (g = t / 4, c = t % 4) owns rows g and g + 8.
//
//   S = Q K^T     16 rows x 16 keys: two n-tiles of 8 keys, D / 16 k-steps
//   O += P V      D / 8 n-tiles of 8 dims, one k-step of 16 keys
//
// bf16 pools: the chunk lies in 128-byte lines, 16-byte piece x of line r at
// x ^ (r % 8), and ldmatrix reads the fragments
// without bank conflicts; P is rounded to bf16, each p by at most 2^-8 of itself, as
// much as O's own rounding: for a row that one or a few keys dominate the two add up,
// over many keys the roundings of P average out.
//
// FP8 pools: operands are f16 (every e4m3 value is an f16 value).  The dims of
// S's k-steps and of O's n-tiles are permuted so that a thread reads whole
// 16-byte pieces of codes: k-step s holds dims (D/4) c + 4 s .. + 3, n-tile j's
// column x is dim (D/8) x + j.  P is rounded to f16.
//
// Rows see a 16-bit mask of each block's keys; a block that every row sees
// whole skips the masks.  A masked key must not reach a row as 0 * inf: where
// all rows see the same keys (kMaskKeys) the other keys' V rows are read as
// zero; where rows differ (kMaskRows) V elements that are not finite are read
// as zero, and the caller adds them to the rows that do see them (see `odd`).
#pragma once
#include <cuda_runtime.h>
#include <math_constants.h>

#include "internal.h"
#include "ptx.cuh"

namespace pkv {

constexpr int kRowTile = 16;    // query rows of a warp's tile
constexpr int kRowWarps = 4;    // warps of a CTA, each with its own blocks and state (whole groups: up to 12)
constexpr int kMaskNone = 0, kMaskRows = 1, kMaskKeys = 2;

template <int D, bool F8, int W = kRowWarps>
struct RowsSmem {
  static constexpr int kStages = F8 ? 4 : 2;                     // per-warp ring depth
  static constexpr int kChunk = kBlockSize * D * (F8 ? 1 : 2);   // one (block, head) of K or V
  static constexpr int kStage = 2 * kChunk;
  static constexpr int kRing = W * kStages * kStage;
  // The warps' states are merged in the ring once it has drained.
  static constexpr int kMergeRow = D + 4;                        // o, m, l, pad (floats)
  static constexpr int kMerge = W * kRowTile * kMergeRow * 4;
  static constexpr int kBuf = kRing > kMerge ? kRing : kMerge;
  static constexpr int kTotal = kBuf + 1024;                     // + alignment
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3) : "r"(addr) : "memory");
}
// d += A B, 16 x 8 x 16, fp32 accumulation.
template <bool F16>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The pair with elements that are not finite replaced by zero; `odd` is set if there was one.
template <bool F16>
__device__ __forceinline__ uint32_t finite_pair(uint32_t w, bool& odd) {
  constexpr uint32_t kExp = F16 ? 0x7c00u : 0x7f80u;
  if ((w & kExp) == kExp) { w &= 0xffff0000u; odd = true; }
  if ((w & (kExp << 16)) == (kExp << 16)) { w &= 0x0000ffffu; odd = true; }
  return w;
}

template <int D, bool F8>
struct RowTile {
  static constexpr int kSteps = D / 16;    // k-steps of S
  static constexpr int kTiles = D / 8;     // n-tiles of O
  uint32_t q[kSteps][4];
  float o[kTiles][4];
  float m[2], l[2];    // rows g and g + 8; l is this thread's share of the sum
  bool odd;            // kMaskRows: a V element that is not finite was left out

  // q0, q1: rows g and g + 8 of the tile ([D] bf16), nullptr for a row that is not there.  (Plain loads: the queries may
  // be what the kernel ahead wrote.)
  __device__ __forceinline__ void load(const uint16_t* q0, const uint16_t* q1, int lane) {
    const int c = lane & 3;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      // Element pairs of the k-step that this thread holds (see the layouts above).
      const int d0 = F8 ? (D / 4) * c + 4 * s : 16 * s + 2 * c;
      const int d1 = F8 ? d0 + 2 : d0 + 8;
      q[s][0] = q0 ? *reinterpret_cast<const uint32_t*>(q0 + d0) : 0u;
      q[s][1] = q1 ? *reinterpret_cast<const uint32_t*>(q1 + d0) : 0u;
      q[s][2] = q0 ? *reinterpret_cast<const uint32_t*>(q0 + d1) : 0u;
      q[s][3] = q1 ? *reinterpret_cast<const uint32_t*>(q1 + d1) : 0u;
    }
  }
  // The loaded queries as operands, and an empty state.
  __device__ __forceinline__ void start() {
    if constexpr (F8) {
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) q[s][i] = pack_f16x2(bf16lo_to_f32(q[s][i]), bf16hi_to_f32(q[s][i]));
    }
#pragma unroll
    for (int j = 0; j < kTiles; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    m[0] = m[1] = -CUDART_INF_F;
    l[0] = l[1] = 0.f;
    odd = false;
  }

  // NB blocks: the first one's K and V chunks at shared addresses kb and vb, the
  // second one's at kb1 and vb1.  sl2: score scale times log2(e).  Masked (one
  // block): vis0 / vis1 hold the keys that rows g and g + 8 see.
  template <int MASK, int NB = 1>
  __device__ __forceinline__ void block(uint32_t kb, uint32_t vb, float sl2, uint32_t vis0, uint32_t vis1, int lane,
                                        uint32_t kb1 = 0, uint32_t vb1 = 0) {
    static_assert(NB == 1 || MASK == kMaskNone, "masks are those of one block");
    const int g = lane >> 2, c = lane & 3;
    float s[NB][2][4];
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int t = 0; t < 2; ++t) s[n][t][0] = s[n][t][1] = s[n][t][2] = s[n][t][3] = 0.f;
    if constexpr (!F8) {
      // Lane l addresses line (l / 16) * 8 + l % 8, 16-byte chunk 2 s + (l / 8) % 2.
      const int r8 = lane & 7, key8 = lane >> 4, cx = (lane >> 3) & 1;
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const uint32_t base = (n ? kb1 : kb) + key8 * (D / 64) * 1024 + r8 * 128;
#pragma unroll
        for (int st = 0; st < kSteps; ++st) {
          const int ch = 2 * st + cx;
          uint32_t b0, b1, b2, b3;
          ldsm4(base + (ch >> 3) * 1024 + (((ch & 7) ^ r8) << 4), b0, b1, b2, b3);
          mma16<false>(s[n][0], q[st], b0, b1);
          mma16<false>(s[n][1], q[st], b2, b3);
        }
      }
    } else {
      // Keys g and g + 8: D / 4 codes from dim (D / 4) c.
#pragma unroll
      for (int u = 0; u < D / 64; ++u) {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            uint4 x;
            ld_codes(n ? kb1 : kb, g + 8 * t, (D / 64) * c + u, x);
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t b0, b1;
              e4m3x4_to_f16x4(w[i], b0, b1);
              mma16<true>(s[n][t], q[4 * u + i], b0, b1);
            }
          }
      }
    }
    if constexpr (MASK != kMaskNone) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t v = e < 2 ? vis0 : vis1;
          if (!((v >> (8 * t + 2 * c + (e & 1))) & 1u)) s[0][t][e] = -CUDART_INF_F;
        }
    }
    float mx0 = -CUDART_INF_F, mx1 = -CUDART_INF_F;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      mx0 = fmaxf(mx0, fmaxf(fmaxf(s[n][0][0], s[n][0][1]), fmaxf(s[n][1][0], s[n][1][1])));
      mx1 = fmaxf(mx1, fmaxf(fmaxf(s[n][0][2], s[n][0][3]), fmaxf(s[n][1][2], s[n][1][3])));
    }
#pragma unroll
    for (int x = 1; x < 4; x <<= 1) {
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, x));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, x));
    }
    const float n0 = fmaxf(m[0], mx0 * sl2), n1 = fmaxf(m[1], mx1 * sl2);   // sl2 > 0
    if (__any_sync(0xffffffffu, n0 > m[0] || n1 > m[1])) {
      // A row's max grew: rescale (rows without a visible key so far keep m = -inf and o = 0).
      const float a0 = n0 == -CUDART_INF_F ? 1.f : fast_exp2(m[0] - n0);
      const float a1 = n1 == -CUDART_INF_F ? 1.f : fast_exp2(m[1] - n1);
      l[0] *= a0;
      l[1] *= a1;
#pragma unroll
      for (int j = 0; j < kTiles; ++j) {
        o[j][0] *= a0; o[j][1] *= a0;
        o[j][2] *= a1; o[j][3] *= a1;
      }
      m[0] = n0;
      m[1] = n1;
    }
    const float u0 = m[0] == -CUDART_INF_F ? 0.f : -m[0], u1 = m[1] == -CUDART_INF_F ? 0.f : -m[1];
    uint32_t p[NB][4];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        s[n][t][0] = fast_exp2(fmaf(s[n][t][0], sl2, u0));
        s[n][t][1] = fast_exp2(fmaf(s[n][t][1], sl2, u0));
        s[n][t][2] = fast_exp2(fmaf(s[n][t][2], sl2, u1));
        s[n][t][3] = fast_exp2(fmaf(s[n][t][3], sl2, u1));
        if constexpr (F8) {
          p[n][2 * t] = pack_f16x2(s[n][t][0], s[n][t][1]);
          p[n][2 * t + 1] = pack_f16x2(s[n][t][2], s[n][t][3]);
        } else {
          p[n][2 * t] = pack_bf16x2(s[n][t][0], s[n][t][1]);
          p[n][2 * t + 1] = pack_bf16x2(s[n][t][2], s[n][t][3]);
        }
      }
      l[0] += (s[n][0][0] + s[n][0][1]) + (s[n][1][0] + s[n][1][1]);
      l[1] += (s[n][0][2] + s[n][0][3]) + (s[n][1][2] + s[n][1][3]);
    }
    // kMaskKeys: the halves of b0 / b1 that hold seen keys (2c, 2c + 1 and 2c + 8, 2c + 9).
    uint32_t k01 = 0xffffffffu, k89 = 0xffffffffu;
    if constexpr (MASK == kMaskKeys) {
      const uint32_t v = vis0 >> (2 * c);
      k01 = ((v & 1u) ? 0xffffu : 0u) | ((v & 2u) ? 0xffff0000u : 0u);
      k89 = ((v & 0x100u) ? 0xffffu : 0u) | ((v & 0x200u) ? 0xffff0000u : 0u);
    }
    if constexpr (!F8) {
      // Lane l addresses line ((l / 8) % 2) * 8 + l % 8, chunk j + l / 16; transposed on the way.
      const int r8 = lane & 7, key8 = (lane >> 3) & 1, cx = lane >> 4;
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const uint32_t base = (n ? vb1 : vb) + key8 * (D / 64) * 1024 + r8 * 128;
#pragma unroll
        for (int j = 0; j < kTiles; j += 2) {
          const int ch = j + cx;
          uint32_t b0, b1, b2, b3;
          ldsm4_t(base + (ch >> 3) * 1024 + (((ch & 7) ^ r8) << 4), b0, b1, b2, b3);
          if constexpr (MASK == kMaskRows) {
            b0 = finite_pair<false>(b0, odd); b1 = finite_pair<false>(b1, odd);
            b2 = finite_pair<false>(b2, odd); b3 = finite_pair<false>(b3, odd);
          } else if constexpr (MASK == kMaskKeys) {
            b0 &= k01; b1 &= k89;
            b2 &= k01; b3 &= k89;
          }
          mma16<false>(o[j], p[n], b0, b1);
          mma16<false>(o[j + 1], p[n], b2, b3);
        }
      }
    } else {
      // Keys 2c, 2c + 1, 2c + 8, 2c + 9: D / 8 codes from dim (D / 8) g; a byte
      // permute pairs two keys' codes of one dim before the conversion.
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        uint32_t v[4][D / 32];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int key = 2 * c + (k & 1) + 8 * (k >> 1);
          if constexpr (D == 128) {
            uint4 x;
            ld_codes(n ? vb1 : vb, key, g, x);
            v[k][0] = x.x; v[k][1] = x.y; v[k][2] = x.z; v[k][3] = x.w;
          } else {
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[k][0]), "=r"(v[k][1])
                         : "r"((n ? vb1 : vb) + key * D + 8 * g) : "memory");
          }
        }
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {   // word i: n-tiles 4 i .. 4 i + 3
          const uint32_t x01 = __byte_perm(v[0][i], v[1][i], 0x5140), y01 = __byte_perm(v[0][i], v[1][i], 0x7362);
          const uint32_t x89 = __byte_perm(v[2][i], v[3][i], 0x5140), y89 = __byte_perm(v[2][i], v[3][i], 0x7362);
          uint32_t b[8];
          e4m3x4_to_f16x4(x01, b[0], b[2]);
          e4m3x4_to_f16x4(x89, b[1], b[3]);
          e4m3x4_to_f16x4(y01, b[4], b[6]);
          e4m3x4_to_f16x4(y89, b[5], b[7]);
          if constexpr (MASK == kMaskRows) {
#pragma unroll
            for (int e = 0; e < 8; ++e) b[e] = finite_pair<true>(b[e], odd);
          } else if constexpr (MASK == kMaskKeys) {
#pragma unroll
            for (int e = 0; e < 8; ++e) b[e] &= (e & 1) ? k89 : k01;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) mma16<true>(o[4 * i + e], p[n], b[2 * e], b[2 * e + 1]);
        }
      }
    }
  }

  // 16 codes of key `key` from 16-byte chunk x (D = 128: swizzled lines; D = 64: plain rows).
  __device__ __forceinline__ static void ld_codes(uint32_t base, int key, int x, uint4& v) {
    const uint32_t a = D == 128 ? base + key * 128 + ((x ^ (key & 7)) << 4) : base + key * D + x * 16;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a) : "memory");
  }

  // Sums l over the threads that share a row.
  __device__ __forceinline__ void total_l(float& l0, float& l1) const {
    l0 = l[0];
    l1 = l[1];
#pragma unroll
    for (int x = 1; x < 4; x <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, x);
      l1 += __shfl_xor_sync(0xffffffffu, l1, x);
    }
  }

  // Stores row g (i = 0) or g + 8 (i = 1), scaled, as bf16 or as floats.
  __device__ __forceinline__ void put_bf16(uint16_t* row, int i, float f, int lane) const {
    const int c = lane & 3;
    if constexpr (F8) {   // dims (D/4) c .. (D/4)(c + 1) - 1, in two runs of D / 8
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int j = 0; j < kTiles; j += 8) {
          uint4 w;
          w.x = pack_bf16x2(o[j][2 * i + e] * f, o[j + 1][2 * i + e] * f);
          w.y = pack_bf16x2(o[j + 2][2 * i + e] * f, o[j + 3][2 * i + e] * f);
          w.z = pack_bf16x2(o[j + 4][2 * i + e] * f, o[j + 5][2 * i + e] * f);
          w.w = pack_bf16x2(o[j + 6][2 * i + e] * f, o[j + 7][2 * i + e] * f);
          *reinterpret_cast<uint4*>(row + (D / 4) * c + (D / 8) * e + j) = w;
        }
    } else {
#pragma unroll
      for (int j = 0; j < kTiles; ++j)
        *reinterpret_cast<uint32_t*>(row + 8 * j + 2 * c) = pack_bf16x2(o[j][2 * i] * f, o[j][2 * i + 1] * f);
    }
  }
  __device__ __forceinline__ void put_f32(float* row, int i, float f, int lane) const {
    const int c = lane & 3;
    if constexpr (F8) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int j = 0; j < kTiles; j += 4)
          *reinterpret_cast<float4*>(row + (D / 4) * c + (D / 8) * e + j) =
              make_float4(o[j][2 * i + e] * f, o[j + 1][2 * i + e] * f, o[j + 2][2 * i + e] * f, o[j + 3][2 * i + e] * f);
    } else {
#pragma unroll
      for (int j = 0; j < kTiles; ++j)
        *reinterpret_cast<float2*>(row + 8 * j + 2 * c) = make_float2(o[j][2 * i] * f, o[j][2 * i + 1] * f);
    }
  }

  // Writes the warp's state to `buf` ([16][D + 4] floats: o unnormalised, m in log2 units, l).
  __device__ __forceinline__ void store(float* buf, int lane) {
    const int g = lane >> 2, c = lane & 3;
    float l0, l1;
    total_l(l0, l1);
    float* r0 = buf + g * (D + 4);
    float* r1 = r0 + 8 * (D + 4);
    if (c == 0) {
      r0[D] = m[0]; r0[D + 1] = l0;
      r1[D] = m[1]; r1[D + 1] = l1;
    }
#pragma unroll
    for (int j = 0; j < kTiles; ++j) {
      if constexpr (F8) {   // columns 2c and 2c + 1 of n-tile j: dims (D/8) 2c + j and (D/8)(2c + 1) + j
        const int d = (D / 4) * c + j;
        r0[d] = o[j][0]; r0[d + D / 8] = o[j][1];
        r1[d] = o[j][2]; r1[d + D / 8] = o[j][3];
      } else {
        const int d = 8 * j + 2 * c;
        *reinterpret_cast<float2*>(r0 + d) = make_float2(o[j][0], o[j][1]);
        *reinterpret_cast<float2*>(r1 + d) = make_float2(o[j][2], o[j][3]);
      }
    }
  }
};

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Copies chunk `chunk` (block * kv heads + head) of K and V into the stage at shared
// address dst; a whole warp, 512 bytes an instruction.  (One lane's tensor copies,
// with the barriers around them, took 1200 of a warp's 3900 cycles for two FP8
// blocks, and boxes of 2 KB arrive at 26 bytes a clock and SM at most.)
template <int D, bool F8>
__device__ __forceinline__ void rows_copy(const PoolView& pool, uint32_t dst, int chunk, int lane) {
  constexpr int kBytes = RowsSmem<D, F8>::kChunk;
  constexpr int kRow = D * (F8 ? 1 : 2);   // bytes of a key's row
  const int64_t at = static_cast<int64_t>(chunk) * kBytes + lane * 16;
  const uint8_t* k = static_cast<const uint8_t*>(pool.k) + at;
  const uint8_t* v = static_cast<const uint8_t*>(pool.v) + at;
  // Where the lane's 16 bytes go: rows of 64 bytes as they are; of 128, chunk c of row r at c ^ (r % 8); of 256 in
  // two halves of that kind, eight rows of each together.
  uint32_t to;
  if constexpr (kRow == 64) to = lane * 16;
  else if constexpr (kRow == 128) to = (lane >> 3) * 128 + (((lane & 7) ^ (lane >> 3)) << 4);
  else to = ((lane & 15) >> 3) * 1024 + (lane >> 4) * 128 + (((lane & 7) ^ (lane >> 4)) << 4);
#pragma unroll
  for (int i = 0; i < kBytes / 512; ++i) {
    uint32_t off;
    if constexpr (kRow == 64) off = to + i * 512;
    else if constexpr (kRow == 128) off = (to ^ ((i & 1) * 64)) + i * 512;
    else off = (to ^ (((2 * i) & 7) << 4)) + (i >> 2) * 2048 + ((2 * i) & 7) * 128;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + off), "l"(k + i * 512) : "memory");
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + kBytes + off), "l"(v + i * 512) : "memory");
  }
}

// Element d of key slot `slot` (block-relative) of chunk `chunk` of V, in the pool's units (codes unscaled).
template <int D, bool F8>
__device__ __forceinline__ float pool_v(const PoolView& pool, int64_t chunk, int slot, int d) {
  const int64_t at = (chunk * kBlockSize + slot) * D + d;
  if constexpr (F8) {
    const uint32_t c = static_cast<const uint8_t*>(pool.v)[at];
    uint32_t h = e4m3x2_lo_to_f16x2(c) & 0xffffu;
    // f16 -> f32 (NaN stays NaN)
    float f;
    asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %1;\n\tcvt.f32.f16 %0, x;\n\t}" : "=f"(f) : "r"(h));
    return f;
  } else {
    return bf16lo_to_f32(static_cast<const uint16_t*>(pool.v)[at]);
  }
}

}  // namespace pkv
