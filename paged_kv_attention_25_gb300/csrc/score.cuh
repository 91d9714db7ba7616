// What the two forms of the attention with modified scores (pkv_score_attn)
// share: which keys a token sees, and what becomes of a score.
//
// Token t at position p of request r sees key j < ctx_r if
//   j < prefix_r,  or  first_t <= j <= p and (window = 0 or j > p - window),
// and its score is
//   x = scale q . K_j,   x = cap tanh(x / cap) if cap > 0,   x -= slope_h |p - j| if there are slopes.
#pragma once
#include <cuda_runtime.h>

#include "int8.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "sched.cuh"

namespace pkv {

constexpr int kPoolBf16 = 0, kPoolFp8 = 1, kPoolInt8 = 2;

// Two neighbouring query tiles of a request (rows1 = 0: one), of the tiles form's
// plan: key tiles 0 .. ktiles - 1, of which those below pre_tiles hold the prefix
// and the others lie `gap` tiles further on.  Every row sees the prefix and the keys
// [all_lo, all_hi], none sees others than these of [any_lo, any_hi].
struct alignas(16) ScoreItem {
  int req, tok0, rows0, rows1;
  int pre_tiles, gap, ktiles, prefix;
  int all_lo, all_hi, any_lo, any_hi;
  int ctx, pad[3];
};
static_assert(sizeof(ScoreItem) == 64, "ScoreItem layout: four 16-byte loads");
// The plan in the workspace, for `most` items at most.
struct ScorePlan {
  ScoreItem* items;   // [most]
  int64_t* cum;       // [most + 2]: units of a head's line before each item; total; number of items
  int* first;         // [num_reqs]: items before each request's
  int most;
};

// One call.  t.prefix_lens may be nullptr; t.positions holds the queries' positions; t.mask, t.sel are not used.
struct ScoreArgs {
  TreeArgs t;
  float base;                 // raw products to log2 units, or to the cap's argument (FP8: with k_scale)
  float cap_out;              // cap * log2 e (0: no cap)
  float cap_small, cap_q[4];  // products below cap_small: x (q0 + q1 x^2 + ...) is the capped score in log2 units
  const float* slopes;        // [num_q_heads], or nullptr
  int window;                 // 0: none
  const int32_t* first_keys;  // [num_tokens], or nullptr
  int row_tile;               // rows form: 16 or 8 rows a tile
  ScorePlan plan;             // tiles form
};

// The keys [lo, hi] that a token sees beside the prefix (they may begin inside it).  None behind it: [ctx, -1], so that a
// token without such keys (a document that begins behind it, a position in the prefix or in front of the sequence) does
// not widen what the others of its tile see.
struct KeySpan {
  int lo, hi;
};
__device__ __forceinline__ KeySpan key_span(const ScoreArgs& a, int pos, int first, int prefix, int ctx) {
  const int p = max(pos, -1);
  KeySpan s{max(first, 0), min(p, ctx - 1)};
  if (a.window > 0) s.lo = max(s.lo, p - a.window + 1);
  return s.hi < max(s.lo, prefix) ? KeySpan{ctx, -1} : s;
}
__device__ __forceinline__ KeySpan key_span(const ScoreArgs& a, int t, int prefix, int ctx) {
  return key_span(a, __ldg(a.t.positions + t), a.first_keys ? __ldg(a.first_keys + t) : 0, prefix, ctx);
}
// Keys [key0, key0 + 32) that a token sees, as bits.
__device__ __forceinline__ uint32_t span_bits(int prefix, KeySpan s, int key0) {
  return low_bits(prefix - key0) | (low_bits(s.hi + 1 - key0) & ~low_bits(s.lo - key0));
}

// A request's lengths, made safe.
struct ScoreReq {
  int t0, n, ctx, prefix;
  bool bad;
};
__device__ __forceinline__ ScoreReq score_req(const ScoreArgs& a, int r) {
  ScoreReq q;
  const int c0 = __ldg(a.t.cu_q_lens + r), c1 = __ldg(a.t.cu_q_lens + r + 1);
  const int ctx = __ldg(a.t.ctx_lens + r), pre = a.t.prefix_lens ? __ldg(a.t.prefix_lens + r) : 0;
  q.t0 = min(max(c0, 0), a.t.num_tokens);
  q.n = min(max(c1, q.t0), a.t.num_tokens) - q.t0;
  q.ctx = min(max(ctx, 0), a.t.max_blocks * kBlockSize);
  q.prefix = min(max(pre, 0), q.ctx);
  q.bad = c0 < 0 || c1 < c0 || c1 > a.t.num_tokens || q.ctx != ctx || q.prefix != pre;
  return q;
}

// tanh(y), off by 2^-23 of it for |y| < 1/2 and by about 2^-22 above.  Below 1/2
// an odd polynomial of degree 9, interpolated at Chebyshev nodes of y^2 in [0, 1/4];
// above, (1 - e) / (1 + e) with e = exp(-2 |y|).
constexpr float kTanh0 = 0.99999999f, kTanh1 = -0.33333068f, kTanh2 = 0.13324751f, kTanh3 = -0.052984238f,
                kTanh4 = 0.017131345f;
__device__ __forceinline__ float tanh_small(float y) {
  const float z = y * y;
  float r = fmaf(z, kTanh4, kTanh3);
  r = fmaf(r, z, kTanh2);
  r = fmaf(r, z, kTanh1);
  r = fmaf(r, z, kTanh0);
  return r * y;
}
__device__ __forceinline__ float tanh_large(float y) {
  const float e = fast_exp2(fabsf(y) * -2.8853900817779268f);
  return copysignf(__fdividef(1.f - e, 1.f + e), y);
}

__device__ __forceinline__ float tanh_any(float y) { return fabsf(y) < 0.5f ? tanh_small(y) : tanh_large(y); }

}  // namespace pkv
