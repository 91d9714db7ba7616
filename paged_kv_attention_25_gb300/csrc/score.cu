// Attention with modified scores and masks over a pool of any type
// (pkv_score_attn), the form for few query rows: 16 query rows a warp on the
// warp-level MMA, one 16-key block at a time, as the tree attention's rows form
// (rows.cuh), with the keys that a token does not see left out of the copies.
//
//   x_j = scale q . K_j (capped, less slope_h |p - j|),   m = max_j x_j
//   O = sum_j exp(x_j - m) V_j / sum_j exp(x_j - m),   LSE = m + ln sum_j exp(x_j - m)
//
// over the keys that the token sees; none: O = 0, LSE = -inf.
//
// Int8 pools: codes are widened to bf16 (exact, seven bits), and the block's
// powers of two go to the scores and to P: 2^e_K on 16 x 16 scores and 2^e_V on
// as many p are a sixteenth of the products that scaling the operands would take,
// and neither rounds while p 2^(e_V + 6) is a normal bf16 number (below, values of V
// under 2^-100 or so, a key's share of O is off by 2^-133 at most).  P is rounded to
// bf16 (8 bits, as for bf16 pools).
#include <cuda_runtime.h>
#include <math_constants.h>

#include <cstdint>

#include "internal.h"
#include "ops.h"
#include "ptx.cuh"
#include "rows.cuh"
#include "sched.cuh"
#include "score.cuh"

namespace pkv {
namespace {

constexpr int kGroupUnits = 2;
constexpr int kManyTokens = 64;   // a request of more tokens is planned as if they saw its whole context
using RowsShare = Share<4 * kRowWarps>;   // few groups: four blocks a warp at least
using WarpShare = Share<4>;

// Factors of one block: of its scores (raw products to log2 units, or to the cap's argument; int8: the block's power of
// two alone, which with Modify::base in one factor could leave fp32's range), of P.
struct BlockFactor {
  float score, value;
};
// What becomes of the scores of rows g and g + 8 of a thread.
struct Modify {
  float base;          // int8: what products are multiplied with, beside the block's power
  bool on;             // cap or slopes
  float cap_out;       // 0: no cap
  bool slopes;
  float slope0, slope1;   // log2 units
  int p0, p1;          // positions
};
template <int KIND>
__device__ __forceinline__ float raw_score(float s, const BlockFactor& f, const Modify& mod) {
  return (KIND == kPoolInt8 ? s * mod.base : s) * f.score;
}

template <int D, int KIND>
struct ScoreTile : RowTile<D, KIND != kPoolBf16> {
  using Base = RowTile<D, KIND != kPoolBf16>;
  static constexpr int kRows = kRowTile;
  // The rows whose queries, and whose state, a thread holds.
  __device__ __forceinline__ static int row_a(int lane) { return lane >> 2; }
  __device__ __forceinline__ static int row_b(int lane) { return (lane >> 2) + 8; }
  template <class Q>
  __device__ __forceinline__ void ask(Q&& q_row, int lane) { Base::load(q_row(row_a(lane)), q_row(row_b(lane)), lane); }
  // The rows times f0 (f1), to where o_row says (nullptr: nowhere).
  template <class R>
  __device__ __forceinline__ void put_bf16(R&& o_row, float f0, float f1, int lane) const {
    if (uint16_t* p = o_row(row_a(lane))) Base::put_bf16(p, 0, f0, lane);
    if (uint16_t* p = o_row(row_b(lane))) Base::put_bf16(p, 1, f1, lane);
  }
  template <class R>
  __device__ __forceinline__ void put_f32(R&& o_row, float f0, float f1, int lane) const {
    if (float* p = o_row(row_a(lane))) Base::put_f32(p, 0, f0, lane);
    if (float* p = o_row(row_b(lane))) Base::put_f32(p, 1, f1, lane);
  }
  __device__ __forceinline__ static bool first_of_row(int lane) { return (lane & 3) == 0; }
  static constexpr bool kCodes = KIND != kPoolBf16;
  using Base::kSteps, Base::kTiles, Base::q, Base::o, Base::m, Base::l, Base::odd, Base::ld_codes;

  // The loaded queries as operands (int8: bf16 as they are), and an empty state.
  __device__ __forceinline__ void begin() {
    if constexpr (KIND == kPoolInt8) {
#pragma unroll
      for (int j = 0; j < kTiles; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
      m[0] = m[1] = -CUDART_INF_F;
      l[0] = l[1] = 0.f;
      odd = false;
    } else {
      Base::start();
    }
  }
  __device__ __forceinline__ static void widen(uint32_t codes, uint32_t& lo, uint32_t& hi) {
    if constexpr (KIND == kPoolInt8) int8x4_to_bf16x4(codes, lo, hi);
    else e4m3x4_to_f16x4(codes, lo, hi);
  }

  // Raw products to scores in log2 units.  Thread t = 4g + c holds keys 8t + 2c + (e & 1) of rows g (e < 2) and g + 8.
  template <int NB>
  __device__ __forceinline__ static void modify(float (&s)[NB][2][4], const BlockFactor (&f)[NB], const Modify& mod,
                                                const int (&key0)[NB], int c) {
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][t][e] = raw_score<KIND>(s[n][t][e], f[n], mod);
    if (!mod.on) return;
    if (mod.cap_out != 0.f) {
      float top = 0.f;
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(s[n][t][e]));
      const bool small = !__any_sync(0xffffffffu, top >= 0.5f);
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float y = s[n][t][e];
            float r = tanh_small(y);
            if (!small && !(fabsf(y) < 0.5f)) r = tanh_large(y);
            s[n][t][e] = mod.cap_out * r;
          }
    }
    if (mod.slopes) {
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const float d0 = static_cast<float>(mod.p0 - key0[n] - 2 * c), d1 = static_cast<float>(mod.p1 - key0[n] - 2 * c);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float dist = fabsf((e < 2 ? d0 : d1) - static_cast<float>(8 * t + (e & 1)));
            s[n][t][e] = fmaf(-(e < 2 ? mod.slope0 : mod.slope1), dist, s[n][t][e]);
          }
      }
    }
  }

  // NB blocks: K and V chunks at shared addresses kb, vb (kb1, vb1), first keys key0, factors f.  Masked (one block):
  // vis0 / vis1 hold the keys that rows g and g + 8 see.
  template <int MASK, int NB>
  __device__ __forceinline__ void block(uint32_t kb, uint32_t vb, const BlockFactor (&f)[NB], const int (&key0)[NB],
                                        const Modify& mod, uint32_t vis0, uint32_t vis1, int lane, uint32_t kb1 = 0,
                                        uint32_t vb1 = 0) {
    static_assert(NB == 1 || MASK == kMaskNone, "masks are those of one block");
    const int g = lane >> 2, c = lane & 3;
    float s[NB][2][4];
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int t = 0; t < 2; ++t) s[n][t][0] = s[n][t][1] = s[n][t][2] = s[n][t][3] = 0.f;
    if constexpr (!kCodes) {
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
              widen(w[i], b0, b1);
              mma16<KIND == kPoolFp8>(s[n][t], q[4 * u + i], b0, b1);
            }
          }
      }
    }
    float sl = f[0].score;   // what is left to multiply the scores with
    if (KIND == kPoolInt8 || mod.on) {
      modify<NB>(s, f, mod, key0, c);
      sl = 1.f;
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
    const float n0 = fmaxf(m[0], mx0 * sl), n1 = fmaxf(m[1], mx1 * sl);   // sl > 0
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
        s[n][t][0] = fast_exp2(fmaf(s[n][t][0], sl, u0));
        s[n][t][1] = fast_exp2(fmaf(s[n][t][1], sl, u0));
        s[n][t][2] = fast_exp2(fmaf(s[n][t][2], sl, u1));
        s[n][t][3] = fast_exp2(fmaf(s[n][t][3], sl, u1));
        if constexpr (KIND == kPoolFp8) {
          p[n][2 * t] = pack_f16x2(s[n][t][0], s[n][t][1]);
          p[n][2 * t + 1] = pack_f16x2(s[n][t][2], s[n][t][3]);
        } else if constexpr (KIND == kPoolInt8) {   // (a power of two: P is rounded as without it, see above)
          p[n][2 * t] = pack_bf16x2(s[n][t][0] * f[n].value, s[n][t][1] * f[n].value);
          p[n][2 * t + 1] = pack_bf16x2(s[n][t][2] * f[n].value, s[n][t][3] * f[n].value);
        } else {
          p[n][2 * t] = pack_bf16x2(s[n][t][0], s[n][t][1]);
          p[n][2 * t + 1] = pack_bf16x2(s[n][t][2], s[n][t][3]);
        }
      }
      l[0] += (s[n][0][0] + s[n][0][1]) + (s[n][1][0] + s[n][1][1]);
      l[1] += (s[n][0][2] + s[n][0][3]) + (s[n][1][2] + s[n][1][3]);
    }
    if constexpr (!kCodes) {
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
          widen(x01, b[0], b[2]);
          widen(x89, b[1], b[3]);
          widen(y01, b[4], b[6]);
          widen(y89, b[5], b[7]);
          if constexpr (MASK == kMaskRows && KIND == kPoolFp8) {
#pragma unroll
            for (int e = 0; e < 8; ++e) b[e] = finite_pair<true>(b[e], odd);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) mma16<KIND == kPoolFp8>(o[4 * i + e], p[n], b[2 * e], b[2 * e + 1]);
        }
      }
    }
  }
};

__device__ __forceinline__ uint32_t movm_t(uint32_t a) {   // an 8 x 8 matrix of 16 bits, transposed
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// The same for up to 8 rows, keys and dims as the MMA's rows instead:
//   S^T = K Q^T    16 keys x 8 rows, D / 16 k-steps
//   O^T += V^T P^T   D / 16 m-tiles of 16 dims x 8 rows, one k-step of 16 keys
// half the products, scores and registers of a tile of 16 rows of which half are
// not there.  Thread t = 4g + c holds the state of rows 2c and 2c + 1, the scores of
// keys g and g + 8.  Codes: k-step s holds dims (D/4) c + 4 s .. + 3, m-tile j's rows
// g and g + 8 are dims (D/8) g + 2 j and + 1: a thread reads whole 16-byte pieces.
template <int D, int KIND>
struct ScoreCol {
  static constexpr bool kCodes = KIND != kPoolBf16, kF16 = KIND == kPoolFp8;
  static constexpr int kRows = 8, kSteps = D / 16, kTiles = D / 16;
  using Row = ScoreTile<D, KIND>;
  uint32_t q[kSteps][2];
  float o[kTiles][4];   // (dim, row 2c), (dim, row 2c + 1), (dim', row 2c), (dim', row 2c + 1)
  float m[2], l[2];     // rows 2c and 2c + 1; l is this thread's share of the sum
  bool odd;

  __device__ __forceinline__ static int row_a(int lane) { return 2 * (lane & 3); }
  __device__ __forceinline__ static int row_b(int lane) { return 2 * (lane & 3) + 1; }
  __device__ __forceinline__ static bool first_of_row(int lane) { return lane < 4; }
  template <class Q>
  __device__ __forceinline__ void ask(Q&& q_row, int lane) {
    const int c = lane & 3;
    const uint16_t* p = q_row(lane >> 2);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int d0 = kCodes ? (D / 4) * c + 4 * s : 16 * s + 2 * c;
      q[s][0] = p ? *reinterpret_cast<const uint32_t*>(p + d0) : 0u;
      q[s][1] = p ? *reinterpret_cast<const uint32_t*>(p + d0 + (kCodes ? 2 : 8)) : 0u;
    }
  }
  __device__ __forceinline__ void begin() {
    if constexpr (kF16) {
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) q[s][i] = pack_f16x2(bf16lo_to_f32(q[s][i]), bf16hi_to_f32(q[s][i]));
    }
#pragma unroll
    for (int j = 0; j < kTiles; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    m[0] = m[1] = -CUDART_INF_F;
    l[0] = l[1] = 0.f;
    odd = false;
  }

  // As ScoreTile::block; vis0 / vis1: the keys that rows 2c and 2c + 1 see.
  template <int MASK, int NB>
  __device__ __forceinline__ void block(uint32_t kb, uint32_t vb, const BlockFactor (&f)[NB], const int (&key0)[NB],
                                        const Modify& mod, uint32_t vis0, uint32_t vis1, int lane, uint32_t kb1 = 0,
                                        uint32_t vb1 = 0) {
    static_assert(NB == 1 || MASK == kMaskNone, "masks are those of one block");
    const int g = lane >> 2, c = lane & 3;
    float s[NB][4];
#pragma unroll
    for (int n = 0; n < NB; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
    if constexpr (!kCodes) {
      // Lane l addresses line ((l / 8) % 2) * 8 + l % 8, 16-byte chunk 2 s + l / 16.
      const int r8 = lane & 7, key8 = (lane >> 3) & 1, cx = lane >> 4;
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const uint32_t base = (n ? kb1 : kb) + key8 * (D / 64) * 1024 + r8 * 128;
#pragma unroll
        for (int st = 0; st < kSteps; ++st) {
          const int ch = 2 * st + cx;
          uint32_t a[4];
          ldsm4(base + (ch >> 3) * 1024 + (((ch & 7) ^ r8) << 4), a[0], a[1], a[2], a[3]);
          mma16<false>(s[n], a, q[st][0], q[st][1]);
        }
      }
    } else {
#pragma unroll
      for (int u = 0; u < D / 64; ++u) {
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          uint4 x, y;
          Row::ld_codes(n ? kb1 : kb, g, (D / 64) * c + u, x);
          Row::ld_codes(n ? kb1 : kb, g + 8, (D / 64) * c + u, y);
          const uint32_t wx[4] = {x.x, x.y, x.z, x.w}, wy[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t a[4];
            Row::widen(wx[i], a[0], a[2]);
            Row::widen(wy[i], a[1], a[3]);
            mma16<kF16>(s[n], a, q[4 * u + i][0], q[4 * u + i][1]);
          }
        }
      }
    }
    float sl = f[0].score;   // what is left to multiply the scores with
    if (KIND == kPoolInt8 || mod.on) {
      modify<NB>(s, f, mod, key0, g);
      sl = 1.f;
    }
    if constexpr (MASK != kMaskNone) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (!(((e & 1 ? vis1 : vis0) >> (g + 8 * (e >> 1))) & 1u)) s[0][e] = -CUDART_INF_F;
    }
    float mx0 = -CUDART_INF_F, mx1 = -CUDART_INF_F;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      mx0 = fmaxf(mx0, fmaxf(s[n][0], s[n][2]));
      mx1 = fmaxf(mx1, fmaxf(s[n][1], s[n][3]));
    }
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, x));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, x));
    }
    const float n0 = fmaxf(m[0], mx0 * sl), n1 = fmaxf(m[1], mx1 * sl);   // sl > 0
    if (__any_sync(0xffffffffu, n0 > m[0] || n1 > m[1])) {
      const float a0 = n0 == -CUDART_INF_F ? 1.f : fast_exp2(m[0] - n0);
      const float a1 = n1 == -CUDART_INF_F ? 1.f : fast_exp2(m[1] - n1);
      l[0] *= a0;
      l[1] *= a1;
#pragma unroll
      for (int j = 0; j < kTiles; ++j) {
        o[j][0] *= a0; o[j][1] *= a1;
        o[j][2] *= a0; o[j][3] *= a1;
      }
      m[0] = n0;
      m[1] = n1;
    }
    const float u0 = m[0] == -CUDART_INF_F ? 0.f : -m[0], u1 = m[1] == -CUDART_INF_F ? 0.f : -m[1];
    uint32_t p[NB][2];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = fast_exp2(fmaf(s[n][e], sl, e & 1 ? u1 : u0));
      l[0] += s[n][0] + s[n][2];
      l[1] += s[n][1] + s[n][3];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float p0 = s[n][2 * h], p1 = s[n][2 * h + 1];
        if constexpr (kF16) p[n][h] = movm_t(pack_f16x2(p0, p1));
        else if constexpr (KIND == kPoolInt8) p[n][h] = movm_t(pack_bf16x2(p0 * f[n].value, p1 * f[n].value));
        else p[n][h] = movm_t(pack_bf16x2(p0, p1));
      }
    }
    if constexpr (!kCodes) {
      // Lane l addresses line (l / 16) * 8 + l % 8, chunk 2 j + (l / 8) % 2; transposed on the way.
      const int r8 = lane & 7, key8 = lane >> 4, cx = (lane >> 3) & 1;
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const uint32_t base = (n ? vb1 : vb) + key8 * (D / 64) * 1024 + r8 * 128;
#pragma unroll
        for (int j = 0; j < kTiles; ++j) {
          const int ch = 2 * j + cx;
          uint32_t a[4];
          ldsm4_t(base + (ch >> 3) * 1024 + (((ch & 7) ^ r8) << 4), a[0], a[1], a[2], a[3]);
          if constexpr (MASK == kMaskRows) {
#pragma unroll
            for (int e = 0; e < 4; ++e) a[e] = finite_pair<false>(a[e], odd);
          }
          mma16<false>(o[j], a, p[n][0], p[n][1]);
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
            Row::ld_codes(n ? vb1 : vb, key, g, x);
            v[k][0] = x.x; v[k][1] = x.y; v[k][2] = x.z; v[k][3] = x.w;
          } else {
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[k][0]), "=r"(v[k][1])
                         : "r"((n ? vb1 : vb) + key * D + 8 * g) : "memory");
          }
        }
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {   // word i: m-tiles 2 i and 2 i + 1
          uint32_t a[2][4];
          Row::widen(__byte_perm(v[0][i], v[1][i], 0x5140), a[0][0], a[0][1]);
          Row::widen(__byte_perm(v[2][i], v[3][i], 0x5140), a[0][2], a[0][3]);
          Row::widen(__byte_perm(v[0][i], v[1][i], 0x7362), a[1][0], a[1][1]);
          Row::widen(__byte_perm(v[2][i], v[3][i], 0x7362), a[1][2], a[1][3]);
          if constexpr (MASK == kMaskRows && KIND == kPoolFp8) {
#pragma unroll
            for (int e = 0; e < 8; ++e) a[e >> 2][e & 3] = finite_pair<true>(a[e >> 2][e & 3], odd);
          }
          mma16<kF16>(o[2 * i], a[0], p[n][0], p[n][1]);
          mma16<kF16>(o[2 * i + 1], a[1], p[n][0], p[n][1]);
        }
      }
    }
  }

  // Raw products to scores in log2 units.
  template <int NB>
  __device__ __forceinline__ static void modify(float (&s)[NB][4], const BlockFactor (&f)[NB], const Modify& mod,
                                                const int (&key0)[NB], int g) {
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = raw_score<KIND>(s[n][e], f[n], mod);
    if (!mod.on) return;
    if (mod.cap_out != 0.f) {
      float top = 0.f;
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(s[n][e]));
      const bool small = !__any_sync(0xffffffffu, top >= 0.5f);
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float y = s[n][e];
          float r = tanh_small(y);
          if (!small && !(fabsf(y) < 0.5f)) r = tanh_large(y);
          s[n][e] = mod.cap_out * r;
        }
    }
    if (mod.slopes) {
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const float d0 = static_cast<float>(mod.p0 - key0[n] - g), d1 = static_cast<float>(mod.p1 - key0[n] - g);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          s[n][e] = fmaf(-(e & 1 ? mod.slope1 : mod.slope0), fabsf((e & 1 ? d1 : d0) - (e < 2 ? 0.f : 8.f)), s[n][e]);
      }
    }
  }

  __device__ __forceinline__ void total_l(float& l0, float& l1) const {
    l0 = l[0];
    l1 = l[1];
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, x);
      l1 += __shfl_xor_sync(0xffffffffu, l1, x);
    }
  }
  // The rows times f0 (rows 2c), f1 (2c + 1), to where o_row says (nullptr: nowhere).
  template <class R>
  __device__ __forceinline__ void put_bf16(R&& o_row, float f0, float f1, int lane) const {
    const int g = lane >> 2, c = lane & 3;
    if constexpr (kCodes) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint16_t* row = o_row(2 * c + i);
        if (!row) continue;
        const float f = i ? f1 : f0;
        uint32_t w[kTiles];
#pragma unroll
        for (int j = 0; j < kTiles; ++j) w[j] = pack_bf16x2(o[j][i] * f, o[j][2 + i] * f);
#pragma unroll
        for (int j = 0; j < kTiles; j += 4)
          *reinterpret_cast<uint4*>(row + (D / 8) * g + 2 * j) = make_uint4(w[j], w[j + 1], w[j + 2], w[j + 3]);
      }
    } else {
      uint16_t* row = o_row(g);
#pragma unroll
      for (int j = 0; j < kTiles; ++j) {
        const uint32_t lo = movm_t(pack_bf16x2(o[j][0] * f0, o[j][1] * f1));
        const uint32_t hi = movm_t(pack_bf16x2(o[j][2] * f0, o[j][3] * f1));
        if (row) {
          *reinterpret_cast<uint32_t*>(row + 16 * j + 2 * c) = lo;
          *reinterpret_cast<uint32_t*>(row + 16 * j + 8 + 2 * c) = hi;
        }
      }
    }
  }
  // Dim of o[j][0] (o[j][1]); o[j][2] (o[j][3]) is dim_step further on.
  __device__ __forceinline__ static int dim(int j, int lane) {
    return kCodes ? (D / 8) * (lane >> 2) + 2 * j : 16 * j + (lane >> 2);
  }
  static constexpr int kDimStep = kCodes ? 1 : 8;
  template <class R>
  __device__ __forceinline__ void put_f32(R&& o_row, float f0, float f1, int lane) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float* row = o_row(2 * (lane & 3) + i);
      if (!row) continue;
#pragma unroll
      for (int j = 0; j < kTiles; ++j) {
        row[dim(j, lane)] = o[j][i] * (i ? f1 : f0);
        row[dim(j, lane) + kDimStep] = o[j][2 + i] * (i ? f1 : f0);
      }
    }
  }
  // Writes the warp's state to `buf` ([8][D + 4] floats: o unnormalised, m in log2 units, l).
  __device__ __forceinline__ void store(float* buf, int lane) const {
    float l0, l1;
    total_l(l0, l1);
    float* r0 = buf + 2 * (lane & 3) * (D + 4);
    float* r1 = r0 + (D + 4);
    if (lane < 4) {
      r0[D] = m[0]; r0[D + 1] = l0;
      r1[D] = m[1]; r1[D + 1] = l1;
    }
#pragma unroll
    for (int j = 0; j < kTiles; ++j) {
      const int d = dim(j, lane);
      r0[d] = o[j][0]; r0[d + kDimStep] = o[j][2];
      r1[d] = o[j][1]; r1[d + kDimStep] = o[j][3];
    }
  }
};

// A request as the rows form plans it: the blocks that hold its prefix, then
// those from `gap` blocks further on up to the last that a token sees.
struct RowsReq : ScoreReq {
  int pblk, gap, blocks;
};
__device__ __forceinline__ void plan_blocks(RowsReq& q, int lo, int hi) {
  q.pblk = (q.prefix + kBlockSize - 1) / kBlockSize;
  const int b0 = max(q.pblk, lo / kBlockSize);
  q.gap = b0 - q.pblk;
  q.blocks = max(1, q.pblk + max(0, (hi + kBlockSize) / kBlockSize - b0));   // (one at least: its rows are written too)
}
// By one thread (the scan), and by a warp (a segment): the same plan.
__device__ __forceinline__ RowsReq rows_req(const ScoreArgs& a, int r) {
  RowsReq q;
  static_cast<ScoreReq&>(q) = score_req(a, r);
  int lo = 0, hi = q.ctx - 1;
  if (q.n >= 1 && q.n <= kManyTokens) {
    lo = q.ctx;
    hi = -1;
    for (int t = q.t0; t < q.t0 + q.n; ++t) {
      const KeySpan s = key_span(a, t, q.prefix, q.ctx);
      lo = min(lo, s.lo);
      hi = max(hi, s.hi);
    }
  }
  plan_blocks(q, lo, hi);
  return q;
}
__device__ __forceinline__ RowsReq rows_req_warp(const ScoreArgs& a, int r, int lane) {
  RowsReq q;
  static_cast<ScoreReq&>(q) = score_req(a, r);
  int lo = 0, hi = q.ctx - 1;
  if (q.n >= 1 && q.n <= kManyTokens) {
    lo = q.ctx;
    hi = -1;
    for (int t = lane; t < q.n; t += 32) {
      const KeySpan s = key_span(a, q.t0 + t, q.prefix, q.ctx);
      lo = min(lo, s.lo);
      hi = max(hi, s.hi);
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
  }
  plan_blocks(q, lo, hi);
  return q;
}
template <int RT>
__device__ __forceinline__ int rows_tiles(const ScoreReq& q, int group) {
  return static_cast<int>((static_cast<int64_t>(q.n) * group + RT - 1) / RT);
}

// V elements that are not finite, added to a stored row that sees them (they
// were left out of the products of blocks that not every row sees whole: `all` is
// what they all see); D / 32 dims a lane.  Blocks i of [i0, i1).
template <int D, bool F8>
__device__ __noinline__ void score_add_odd(const ScoreArgs& a, const RowsReq& q, const int32_t* bt_row, int g,
                                           KeySpan s, KeySpan all, int i0, int i1, uint16_t* o, float* part, int lane) {
  const int64_t Hkv = a.t.pool.num_kv_heads;
  for (int i = i0; i < i1; i += 32) {
    const int b1 = i + lane < q.pblk ? i + lane : i + lane + q.gap, key = b1 * kBlockSize;
    const bool odd = i + lane < i1 && b1 < a.t.max_blocks && key + kBlockSize > q.prefix &&
                     !(key >= all.lo && key + kBlockSize - 1 <= all.hi) && (span_bits(q.prefix, s, key) & 0xffffu);
    for (uint32_t left = __ballot_sync(0xffffffffu, odd); left; left &= left - 1) {
      const int b = __shfl_sync(0xffffffffu, b1, __ffs(left) - 1);
      const uint32_t vis = span_bits(q.prefix, s, b * kBlockSize);
      const int pb = __ldg(bt_row + b);
      if (pb < 0 || pb >= a.t.pool.num_blocks) continue;
      for (int d = lane; d < D; d += 32) {
        float v[kBlockSize], sum = 0.f;   // loads under way together: row by row a block took 10 us
#pragma unroll
        for (int k = 0; k < kBlockSize; ++k) v[k] = pool_v<D, F8>(a.t.pool, pb * Hkv + g, k, d);
#pragma unroll
        for (int k = 0; k < kBlockSize; ++k)
          if (((vis >> k) & 1u) && !(fabsf(v[k]) < CUDART_INF_F)) sum += v[k];
        if (sum == 0.f) continue;
        if (part) part[d] += sum;
        else o[d] = static_cast<uint16_t>(pack_bf16x2(bf16lo_to_f32(o[d]) + sum, 0.f) & 0xffffu);
      }
    }
  }
}

// A worker walks its share of the line of all groups' blocks, segment by
// segment (blocks [b0, b1) of one group: a tile of 16 or 8 query rows, one KV head), as in the
// tree attention: shares of single warps where there are many groups, of CTAs of
// four warps where there are few, whole groups where they are short.
//
// Bound by HBM for bf16 (64 conversations of 0.6 to 30 thousand tokens, 64 / 8 heads,
// D = 128: 6.1 TB/s), by a warp's chain of copies, conversions and products for codes
// (the same in int8: 5.6 TB/s, issue slots 46 % busy, 167 us with the merge;
// e4m3 162).  12 warps an SM: with 16, and rings of three or two blocks, it took 169 to
// 179 us.  On tiles of 16 rows, half of them empty, the int8 case took 187.
template <int D, int KIND, int W, class Tile>
__global__ void __launch_bounds__(32 * W, 12 / W)
score_rows_kernel(const ScoreArgs a) {
  constexpr bool kCodes = KIND != kPoolBf16;
  constexpr int kRT = Tile::kRows;
  using S = RowsSmem<D, kCodes, W>;
  constexpr bool kAlways = W != kRowWarps;   // always whole groups
  extern __shared__ uint8_t raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  __shared__ int64_t scratch[2 * W];
  __shared__ int s_odd;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const TreeArgs& t = a.t;
  const int G = t.group, Hkv = t.pool.num_kv_heads;
  griddep_wait();
  griddep_launch();   // the merge may take its place and wait
  if (!kAlways && tid < W) t.cuts[cut_record(blockIdx.x, W, true, tid)].count = 0;
  if (tid == 0) s_odd = 0;
  auto groups = [&](const ScoreReq& q) { return static_cast<int64_t>(rows_tiles<kRT>(q, G)) * Hkv; };
  auto flag = [&](const ScoreReq& q) {
    if (q.bad && blockIdx.x == 0) atomicOr(t.pool.err, PKV_DEVERR_POSITION);
  };
  // The shares: of this warp if there are many groups, of the CTA otherwise.
  const int warp_id = static_cast<int>(blockIdx.x) * W + warp, many_from = t.form.many_groups;
  TreeShare sh{0, 0, 0, 0, 1, 0};
  bool solo = false;
  int64_t left = 0;   // whole groups: how many the CTA still has to do
  const bool all_whole = kAlways || t.form.whole;
  if (all_whole) {
    int64_t n[1], off[1], first = 0;
    int reqs[1];
    line_scan<32 * W, 1, 1>(
        t.num_reqs, scratch, n, reqs, off,
        [&](int r, int64_t (&len)[1]) {
          const ScoreReq q = score_req(a, r);
          len[0] = groups(q);
          flag(q);
        },
        [&](const int64_t (&len)[1], int, int& line, int64_t& unit) {
          const int C = static_cast<int>(min(len[0], static_cast<int64_t>(t.ctas)));
          const bool has = static_cast<int>(blockIdx.x) < C;
          first = has ? RowsShare::begin(len[0], C, blockIdx.x) : 0;
          left = has ? RowsShare::begin(len[0], C, blockIdx.x + 1) - first : 0;
          line = 0;
          unit = left > 0 ? first : -1;
        });
    sh.req = reqs[0];
    if (left > 0) sh.off = off[0];   // (in groups: units follow below)
    sh.end = left > 0 ? INT64_MAX : 0;
  } else if constexpr (!kAlways) {
    // Line 0: units; line 1: groups (for their number alone).  Probe p: where warp p's share begins.
    int64_t U[2], off[W];
    int reqs[W];
    auto share = [&](const int64_t (&len)[2], int p, TreeShare& x) {
      const bool alone = len[1] >= many_from;
      x.U = len[0];
      x.workers = alone ? WarpShare::workers(len[0], t.ctas * W) : RowsShare::workers(len[0], t.ctas);
      const int w = alone ? static_cast<int>(blockIdx.x) * W + p : static_cast<int>(blockIdx.x);
      x.u = x.end = 0;
      if (len[0] > 0 && w < x.workers) {
        x.u = RowsShare::begin(len[0], x.workers, w);
        x.end = RowsShare::begin(len[0], x.workers, w + 1);
      }
    };
    line_scan<32 * W, 2, W>(
        t.num_reqs, scratch, U, reqs, off,
        [&](int r, int64_t (&len)[2]) {
          const RowsReq q = rows_req(a, r);
          len[1] = groups(q);
          len[0] = len[1] * (q.blocks + kGroupUnits);
          flag(q);
        },
        [&](const int64_t (&len)[2], int p, int& line, int64_t& unit) {
          TreeShare x;
          share(len, p, x);
          line = 0;
          unit = x.u < x.end ? x.u : -1;
        });
    solo = U[1] >= many_from;
    share(U, warp, sh);
#pragma unroll
    for (int p = 0; p < W; ++p)
      if (warp == p) {
        sh.req = reqs[p];
        sh.off = off[p];
      }
  }
  __syncthreads();   // s_odd, and scratch is free
  if (sh.u >= sh.end) return;   // a warp's (solo) or the CTA's

  const int worker = solo ? warp_id : static_cast<int>(blockIdx.x);
  const int wi = solo ? 0 : warp, wn = solo ? 1 : W;   // this warp's place among those of the segment
  const uint32_t my_ring = smem_u32(ring) + warp * S::kStages * S::kStage;
  const bool cap = a.cap_out != 0.f;
  int req = sh.req;
  RowsReq rq = rows_req_warp(a, req, lane);
  if (all_whole) sh.off *= rq.blocks + kGroupUnits;
  for (; sh.u < sh.end; ) {
    if (all_whole && left-- <= 0) return;
    for (;;) {   // the next request with work (there is one)
      const int64_t n = groups(rq) * (rq.blocks + kGroupUnits);
      if (sh.off < n) break;
      sh.off -= n;
      if (++req >= t.num_reqs) return;
      rq = rows_req_warp(a, req, lane);
    }
    const int kblk = rq.blocks, glen = kblk + kGroupUnits;
    const int grp = static_cast<int>(sh.off / glen);
    const int x = static_cast<int>(sh.off - static_cast<int64_t>(grp) * glen);
    const int ntile = rows_tiles<kRT>(rq, G);
    const int g = grp / ntile;
    const int row0 = (grp - g * ntile) * kRT;
    const int nrows = static_cast<int>(min(static_cast<int64_t>(kRT), static_cast<int64_t>(rq.n) * G - row0));
    const int len = static_cast<int>(min(static_cast<int64_t>(glen - x), sh.end - sh.u));
    const int64_t gbegin = sh.u - x;
    sh.u += len;
    sh.off += len;
    const int b0 = x, b1 = min(x + len, kblk);
    if (b0 >= b1) continue;   // the group's fixed units only
    // The rows whose state this thread holds.
    const int ra = Tile::row_a(lane), rb = Tile::row_b(lane);
    auto tok_of = [&](int rr) { return rq.t0 + (row0 + min(rr, nrows - 1)) / G; };
    auto q_row = [&](int rr) -> const uint16_t* {
      if (rr >= nrows) return nullptr;
      const int f = row0 + rr;
      return static_cast<const uint16_t*>(t.q) +
             (static_cast<int64_t>(rq.t0 + f / G) * t.num_q_heads + g * G + f % G) * D;
    };
    const int ta = tok_of(ra), tb = tok_of(rb);
    const KeySpan sa = key_span(a, ta, rq.prefix, rq.ctx), sb = key_span(a, tb, rq.prefix, rq.ctx);
    Modify mod{a.base, cap || a.slopes != nullptr, a.cap_out, a.slopes != nullptr, 0.f, 0.f,
               max(__ldg(t.positions + ta), -1), max(__ldg(t.positions + tb), -1)};
    if (mod.slopes) {
      mod.slope0 = a.slopes[g * G + (row0 + min(ra, nrows - 1)) % G] * 1.4426950408889634f;
      mod.slope1 = a.slopes[g * G + (row0 + min(rb, nrows - 1)) % G] * 1.4426950408889634f;
    }
    if (b0 == 0 && wi == 0 && Tile::first_of_row(lane)) {
      const int most = t.max_blocks * kBlockSize;
      if (mod.p0 < 0 || mod.p0 >= most || mod.p1 < 0 || mod.p1 >= most) atomicOr(t.pool.err, PKV_DEVERR_POSITION);
    }
    // What the tile's rows see in common, and what any of them sees.
    const int lo_all = __reduce_max_sync(0xffffffffu, max(sa.lo, sb.lo));
    const int hi_all = __reduce_min_sync(0xffffffffu, min(sa.hi, sb.hi));
    const int lo_any = __reduce_min_sync(0xffffffffu, min(sa.lo, sb.lo));
    const int hi_any = __reduce_max_sync(0xffffffffu, max(sa.hi, sb.hi));
    const int live = b1 - b0;
    const int nb_w = live > wi ? (live - wi + wn - 1) / wn : 0;
    const int32_t* bt_row = t.block_tables + static_cast<int64_t>(req) * t.max_blocks;
    // Windows of 32 iterations: lane l holds the chunk of iteration base + l (-1: no such block, or none of its keys is
    // seen), its exponents, and the block's first key; `there` and `plain` are the window's iterations that have a block,
    // and those whose block every row sees whole, as bits.
    auto block_of = [&](int i) {
      const int at = b0 + wi + wn * i;
      return at < rq.pblk ? at : at + rq.gap;
    };
    auto load_ids = [&](int from, int& exps) -> int {
      const int i = from + lane;
      exps = 0;
      if (i >= nb_w) return -1;
      const int blk = block_of(i), key0 = blk * kBlockSize;
      if (blk >= t.max_blocks || !(key0 < rq.prefix || (key0 <= hi_any && key0 + kBlockSize > lo_any))) return -1;
      const int pb = __ldg(bt_row + blk);
      if (pb < 0 || pb >= t.pool.num_blocks) {
        atomicOr(t.pool.err, PKV_DEVERR_BLOCK_ID);
        return -1;
      }
      const int chunk = pb * Hkv + g;
      if constexpr (KIND == kPoolInt8)   // (the kernel ahead may have written them)
        exps = (safe_exp(t.pool.k_exps[chunk]) & 0xffff) | (safe_exp(t.pool.v_exps[chunk]) << 16);
      return chunk;
    };
    int exps_cur, exps_next, win = 0;
    int chunk_cur = load_ids(0, exps_cur), chunk_next = load_ids(32, exps_next);
    uint32_t there, plain;
    auto look = [&] {
      const bool has = chunk_cur >= 0;
      there = __ballot_sync(0xffffffffu, has);
      const int key0 = block_of(32 * win + lane) * kBlockSize;
      plain = __ballot_sync(0xffffffffu, has && (key0 + kBlockSize <= rq.prefix ||
                                                  (key0 >= lo_all && key0 + kBlockSize - 1 <= hi_all)));
    };
    look();
    Tile rt;
    rt.ask(q_row, lane);   // asked for before the first blocks
    // One group of copies an iteration (an empty one for a block that is not there, and behind the last).
    auto copy = [&](int j) {
      const int chunk = __shfl_sync(0xffffffffu, (j >> 5) == win ? chunk_cur : chunk_next, j & 31);
      if (j < nb_w && chunk >= 0)
        rows_copy<D, kCodes>(t.pool, my_ring + static_cast<uint32_t>(j) % S::kStages * S::kStage, chunk, lane);
      cp_commit();
    };
    for (int j = 0; j < S::kStages; ++j) copy(j);
    rt.begin();
    auto factor = [&](int i) {
      BlockFactor f{a.base, 1.f};
      if constexpr (KIND == kPoolInt8) {
        const int e = __shfl_sync(0xffffffffu, exps_cur, i & 31);
        f.score = exp_f32(static_cast<int16_t>(e & 0xffff) + kWidenShift);
        f.value = exp_f32((e >> 16) + kWidenShift);
      }
      return f;
    };
    for (int i = 0; i < nb_w; ++i) {
      if ((i & 31) == 0 && i > 0) {
        chunk_cur = chunk_next;
        exps_cur = exps_next;
        win = i >> 5;
        look();
        chunk_next = load_ids(i + 32, exps_next);
      }
      const uint32_t bit = 1u << (i & 31);
      const uint32_t kb = my_ring + static_cast<uint32_t>(i) % S::kStages * S::kStage;
      // Codes: two blocks at once where both are seen whole (half the shuffles and votes, two chains to interleave).
      if (kCodes && (plain & bit) && (plain & (bit << 1)) && i + 1 < nb_w) {
        cp_wait<S::kStages - 2>();
        __syncwarp();
        const uint32_t kb1 = my_ring + static_cast<uint32_t>(i + 1) % S::kStages * S::kStage;
        const BlockFactor f[2] = {factor(i), factor(i + 1)};
        const int key0[2] = {block_of(i) * kBlockSize, block_of(i + 1) * kBlockSize};
        rt.template block<kMaskNone, 2>(kb, kb + S::kChunk, f, key0, mod, 0u, 0u, lane, kb1, kb1 + S::kChunk);
        __syncwarp();   // the stages have been read
        copy(i + S::kStages);
        ++i;
      } else {
        cp_wait<S::kStages - 1>();
        __syncwarp();
        const BlockFactor f[1] = {factor(i)};
        const int key0[1] = {block_of(i) * kBlockSize};
        if (plain & bit)
          rt.template block<kMaskNone, 1>(kb, kb + S::kChunk, f, key0, mod, 0u, 0u, lane);
        else if (there & bit)
          rt.template block<kMaskRows, 1>(kb, kb + S::kChunk, f, key0, mod, span_bits(rq.prefix, sa, key0[0]),
                                          span_bits(rq.prefix, sb, key0[0]), lane);
        __syncwarp();
      }
      copy(i + S::kStages);
    }
    const bool whole = b0 == 0 && b1 == kblk;
    const int64_t slot = (2 * static_cast<int64_t>(worker) + (b0 == 0 ? 1 : 0)) * kRowTile;
    const float v_scale = KIND == kPoolFp8 ? t.pool.v_scale : 1.f;
    auto out_row = [&](int rr) {   // row index of O and LSE
      const int f = row0 + rr;
      return static_cast<int64_t>(rq.t0 + f / G) * t.num_q_heads + g * G + f % G;
    };
    auto add_odd = [&](int rr) {
      score_add_odd<D, KIND == kPoolFp8>(a, rq, bt_row, g, key_span(a, tok_of(rr), rq.prefix, rq.ctx), KeySpan{lo_all, hi_all}, b0, b1,
                                         static_cast<uint16_t*>(t.o) + out_row(rr) * D,
                                         whole ? nullptr : t.part_o + (slot + rr) * D, lane);
    };
    if (solo) {
      float l0, l1;
      rt.total_l(l0, l1);
      const float f0 = l0 == 0.f ? 0.f : v_scale / l0, f1 = l1 == 0.f ? 0.f : v_scale / l1;
      if (whole)
        rt.put_bf16([&](int rr) { return rr < nrows ? static_cast<uint16_t*>(t.o) + out_row(rr) * D : nullptr; }, f0, f1, lane);
      else
        rt.put_f32([&](int rr) { return rr < nrows ? t.part_o + (slot + rr) * D : nullptr; }, f0, f1, lane);
      if (Tile::first_of_row(lane)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int rr = i ? rb : ra;
          const float L = i ? l1 : l0;
          const float lse2 = L == 0.f ? -CUDART_INF_F : rt.m[i] + fast_log2(L);
          if (rr >= nrows) continue;
          if (!whole) t.part_lse[slot + rr] = lse2;
          else if (t.lse) t.lse[out_row(rr)] = lse2 * 0.69314718055994530942f;
        }
      }
      if (KIND != kPoolInt8 && __any_sync(0xffffffffu, rt.odd)) {
        __syncwarp();
        for (int rr = 0; rr < nrows; ++rr) add_odd(rr);
      }
    } else {
      if (KIND != kPoolInt8 && rt.odd) s_odd = 1;
      __syncthreads();   // every warp's ring has drained
      // Merge the warps' states: [warp][16][D + 4] floats over the ring.
      float* mbuf = reinterpret_cast<float*>(ring);
      rt.store(mbuf + warp * kRT * S::kMergeRow, lane);
      __syncthreads();
      constexpr int kDims = D / 8;   // dims of a thread's part of a row
      const int rr = tid >> 3, d0 = (tid & 7) * kDims;
      if (rr < nrows) {
        float M = -CUDART_INF_F, L = 0.f, acc[kDims];
#pragma unroll
        for (int d = 0; d < kDims; ++d) acc[d] = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) M = fmaxf(M, mbuf[(w * kRT + rr) * S::kMergeRow + D]);
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float* src = mbuf + (w * kRT + rr) * S::kMergeRow;
          if (src[D + 1] == 0.f) continue;   // the warp saw no key of this row (a NaN score leaves m, not l, as it was)
          const float f = fast_exp2(src[D] - M);
          L = fmaf(f, src[D + 1], L);
#pragma unroll
          for (int d = 0; d < kDims; ++d) acc[d] = fmaf(f, src[d0 + d], acc[d]);
        }
        const float inv = L == 0.f ? 0.f : v_scale / L;
#pragma unroll
        for (int d = 0; d < kDims; ++d) acc[d] *= inv;
        const float lse2 = L == 0.f ? -CUDART_INF_F : M + fast_log2(L);
        if (whole) {
          const int64_t at = out_row(rr);
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(t.o) + at * D + d0);
#pragma unroll
          for (int d = 0; d < kDims; d += 8)
            dst[d / 8] = make_uint4(pack_bf16x2(acc[d], acc[d + 1]), pack_bf16x2(acc[d + 2], acc[d + 3]),
                                    pack_bf16x2(acc[d + 4], acc[d + 5]), pack_bf16x2(acc[d + 6], acc[d + 7]));
          if (d0 == 0 && t.lse) t.lse[at] = lse2 * 0.69314718055994530942f;
        } else {
          float4* dst = reinterpret_cast<float4*>(t.part_o + (slot + rr) * D + d0);
#pragma unroll
          for (int d = 0; d < kDims; d += 4) dst[d / 4] = make_float4(acc[d], acc[d + 1], acc[d + 2], acc[d + 3]);
          if (d0 == 0) t.part_lse[slot + rr] = lse2;
        }
      }
      __syncthreads();   // the ring and the flags are free again, the rows stored
      if (KIND != kPoolInt8) {
        if (s_odd) {
          for (int r2 = warp; r2 < nrows; r2 += W) add_odd(r2);
          __syncthreads();
          if (tid == 0) s_odd = 0;
        }
        __syncthreads();
      }
    }
    if (b0 == 0 && b1 < kblk && lane == 0 && (solo || warp == 0)) {   // the group's first part: its other owners follow
      // (the last block names the last owner; those between each have a block, a share being longer than the fixed units)
      const int c1 = RowsShare::owner(sh.U, sh.workers, gbegin + kblk - 1);
      TreeCut& cut = t.cuts[cut_record(blockIdx.x, W, solo, warp)];
      cut.first = 2 * worker + 1;
      cut.next = 2 * (worker + 1);
      cut.stride = 2;
      cut.tok_a = rq.t0;
      cut.rows_a = nrows;
      cut.tok_b = cut.rows_b = 0;
      cut.f0 = row0;
      cut.g = g;
      cut.count = c1 - worker + 1;
    }
  }
}

template <int D, int KIND, int W, class Tile>
int launch_w(const ScoreArgs& a, cudaStream_t s) {
  constexpr int smem = RowsSmem<D, KIND != kPoolBf16, W>::kTotal;
  static_assert(smem <= 232448, "shared memory of a CTA");
  const cudaError_t e = smem_attr_once<score_rows_kernel<D, KIND, W, Tile>>(smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(score_rows_kernel<D, KIND, W, Tile>, dim3(a.t.ctas), 32 * W, smem, s, a);
}
template <int D, int KIND, class Tile>
int launch_r(const ScoreArgs& a, cudaStream_t s) {
  return a.t.form.warps == 12 ? launch_w<D, KIND, 12, Tile>(a, s) : launch_w<D, KIND, kRowWarps, Tile>(a, s);
}
template <int D, int KIND>
int launch_k(const ScoreArgs& a, cudaStream_t s) {
  return a.row_tile == 8 ? launch_r<D, KIND, ScoreCol<D, KIND>>(a, s) : launch_r<D, KIND, ScoreTile<D, KIND>>(a, s);
}

}  // namespace

int launch_score_rows(const ScoreArgs& a, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const PoolView& p = a.t.pool;
  const int kind = p.k_exps ? kPoolInt8 : p.elem_bytes == 1 ? kPoolFp8 : kPoolBf16;
  if (p.head_dim == 128)
    return kind == kPoolInt8 ? launch_k<128, kPoolInt8>(a, s) : kind == kPoolFp8 ? launch_k<128, kPoolFp8>(a, s)
                                                                                 : launch_k<128, kPoolBf16>(a, s);
  return kind == kPoolInt8 ? launch_k<64, kPoolInt8>(a, s) : kind == kPoolFp8 ? launch_k<64, kPoolFp8>(a, s)
                                                                              : launch_k<64, kPoolBf16>(a, s);
}

}  // namespace pkv
