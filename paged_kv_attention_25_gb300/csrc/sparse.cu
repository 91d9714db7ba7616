// Attention over blocks that a cheap score selects for each query token.
//
// Bounds (pkv_summarize).  For each (block, KV head), over the block's written
// keys: the largest and the smallest value of every channel, rounded outwards
// to 8-bit codes of one power-of-two unit,
//   up_d = ceil(max_j K_j[d] / 2^e),  lo_d = floor(min_j K_j[d] / 2^e),
// e the smallest exponent >= -126 with max|K| <= 127 2^e.
//
// Score (pkv_select_blocks).  q_g . K_j <= sum_d max(q_d, 0) up_d + min(q_d, 0) lo_d
// (times 2^e) for every key j of the block.  Summed over the G heads of a
// group this needs the sums P_d = sum_g max(q_gd, 0) and N_d = sum_g min(q_gd, 0)
// alone: one product of length 2 D per block whatever the group.  q is taken as
// whole numbers of a power-of-two unit with G |q| < 2^15, so that the score is
// an exact 32-bit integer (P - N <= 32767 in
// each of at most 128 channels, codes of at most 127: below 2^30), rounded to fp32 once and scaled by
// 2^e exactly: the order of the blocks, ties included, does not depend on the
// order of any sum.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <algorithm>

#include "internal.h"
#include "ops.h"
#include "ptx.cuh"
#include "sched.cuh"

namespace pkv {
namespace {

__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }   // -126 <= e <= 127

// x = m 2^e with m in [0.5, 1), for a normal x > 0.
__device__ __forceinline__ int exp_of(float x) { return static_cast<int>(__float_as_uint(x) >> 23) - 126; }
__device__ __forceinline__ float mant_of(float x) {
  return __uint_as_float((__float_as_uint(x) & 0x7fffffu) | 0x3f000000u);
}

// ---------------------------------------------------------------- bounds
// One warp per TOK consecutive tokens and KV head: it handles the blocks that
// these tokens open (the first of the request's consecutive tokens in a
// block).  Lane l holds channels [l D/32, (l + 1) D/32).  Bound by the latency of a
// chain of reads (request and position, table, keys): 96 single tokens 6.2 us, 25
// thousand tokens of prompts, 8 heads, 12.4 us warm (51 MB of keys, 4.1 TB/s) and 20
// from HBM.  (32 tokens a warp: the same; four heads a warp: 16 us.)
template <int D, bool F8, int TOK>
__global__ void __launch_bounds__(256) summarize_kernel(const SparseArgs a) {
  constexpr int kDPL = D / 32;
  const int lane = threadIdx.x & 31;
  const int Hkv = a.pool.num_kv_heads;
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int groups = (a.num_tokens + TOK - 1) / TOK;
  if (blockIdx.x == 0 && threadIdx.x == 0) check_cu(a.cu_q_lens, a.num_reqs, a.num_tokens, a.pool.err);
  if (w >= static_cast<int64_t>(groups) * Hkv) return;
  const int g = static_cast<int>(w % Hkv), t0 = static_cast<int>(w / Hkv) * TOK;
  // Lane i: token t0 + i's request, and whether it opens a block.
  const int mine = t0 + lane;
  int my_req = -1;
  bool opens = false;
  if (lane < TOK && mine < a.num_tokens) {
    my_req = req_of(a.cu_q_lens, a.num_reqs, mine);
    // (no token lies before the first, wherever its request begins)
    opens = my_req >= 0 && (mine == 0 || mine == __ldg(a.cu_q_lens + my_req) ||
                            (__ldg(a.positions + mine) >> 4) != (__ldg(a.positions + mine - 1) >> 4));
  }
  uint32_t todo = __ballot_sync(0xffffffffu, opens);
  while (todo) {
    const int i = __ffs(todo) - 1;
    todo &= todo - 1;
    const int t = t0 + i;
    const int r = __shfl_sync(0xffffffffu, my_req, i);
    const int p = __ldg(a.positions + t);
    const int ctx = min(__ldg(a.ctx_lens + r), a.max_blocks * kBlockSize);
    if (p < 0 || p >= ctx) {
      if (lane == 0) atomicOr(a.pool.err, PKV_DEVERR_POSITION);
      continue;
    }
    const int b = p >> 4;
    const int pb = __ldg(a.block_tables + static_cast<int64_t>(r) * a.max_blocks + b);
    if (pb < 0 || pb >= a.pool.num_blocks) {
      if (lane == 0) atomicOr(a.pool.err, PKV_DEVERR_BLOCK_ID);
      continue;
    }
    const int n = min(kBlockSize, ctx - b * kBlockSize);
    const int64_t chunk = static_cast<int64_t>(pb) * Hkv + g;
    const uint8_t* src = static_cast<const uint8_t*>(a.pool.k) + chunk * kBlockSize * D * (F8 ? 1 : 2) +
                         lane * kDPL * (F8 ? 1 : 2);
    // All rows' loads first (past the written keys: the last one again), so that they are in flight together.
    uint32_t raw[kBlockSize][F8 ? 1 : kDPL / 2];
#pragma unroll
    for (int j = 0; j < kBlockSize; ++j) {
      const uint8_t* row = src + min(j, n - 1) * D * (F8 ? 1 : 2);
      if constexpr (F8) {
        if constexpr (kDPL == 4) raw[j][0] = __ldg(reinterpret_cast<const uint32_t*>(row));
        else raw[j][0] = __ldg(reinterpret_cast<const uint16_t*>(row));
      } else if constexpr (kDPL == 4) {
        const uint2 y = __ldg(reinterpret_cast<const uint2*>(row));
        raw[j][0] = y.x;
        raw[j][1] = y.y;
      } else {
        raw[j][0] = __ldg(reinterpret_cast<const uint32_t*>(row));
      }
    }
    float hi[kDPL], lo[kDPL];
#pragma unroll
    for (int d = 0; d < kDPL; ++d) { hi[d] = -CUDART_INF_F; lo[d] = CUDART_INF_F; }
#pragma unroll
    for (int j = 0; j < kBlockSize; ++j) {
      float x[kDPL];
      if constexpr (F8) {
        uint32_t h[2];
        if constexpr (kDPL == 4) e4m3x4_to_f16x4(raw[j][0], h[0], h[1]);
        else h[0] = e4m3x2_lo_to_f16x2(raw[j][0]);
#pragma unroll
        for (int d = 0; d < kDPL; d += 2)
          asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.f32.f16 %0, x;\n\tcvt.f32.f16 %1, y;\n\t}"
              : "=f"(x[d]), "=f"(x[d + 1]) : "r"(h[d / 2]));
      } else {
#pragma unroll
        for (int d = 0; d < kDPL; d += 2) { x[d] = bf16lo_to_f32(raw[j][d / 2]); x[d + 1] = bf16hi_to_f32(raw[j][d / 2]); }
      }
#pragma unroll
      for (int d = 0; d < kDPL; ++d) {   // NaN: no change (fmaxf and fminf return the other operand)
        hi[d] = fmaxf(hi[d], x[d]);
        lo[d] = fminf(lo[d], x[d]);
      }
    }
    constexpr float kMost = 3.38953138925e38f;   // the largest finite bf16; infinities count as it
    float amax = 0.f;
#pragma unroll
    for (int d = 0; d < kDPL; ++d) {
      if (hi[d] < lo[d]) hi[d] = lo[d] = 0.f;   // NaN in every key
      hi[d] = fminf(fmaxf(hi[d], -kMost), kMost);
      lo[d] = fminf(fmaxf(lo[d], -kMost), kMost);
      amax = fmaxf(amax, fmaxf(fabsf(hi[d]), fabsf(lo[d])));
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, x));
    int e = -126;
    if (amax >= 1.17549435e-38f) e = max(e, exp_of(amax) - (mant_of(amax) <= 0.9921875f ? 7 : 6));
    const float inv = pow2f(-e);
    uint32_t up = 0, dn = 0;
#pragma unroll
    for (int d = 0; d < kDPL; ++d) {
      // Products below fp32's range round to 0, but outwards they are one unit.
      const int u = hi[d] > 0.f ? max(1, static_cast<int>(ceilf(hi[d] * inv))) : static_cast<int>(ceilf(hi[d] * inv));
      const int v = lo[d] < 0.f ? min(-1, static_cast<int>(floorf(lo[d] * inv))) : static_cast<int>(floorf(lo[d] * inv));
      up |= static_cast<uint32_t>(u & 0xff) << (8 * d);
      dn |= static_cast<uint32_t>(v & 0xff) << (8 * d);
    }
    int8_t* dst = a.codes + chunk * 2 * D + lane * kDPL;
    if constexpr (kDPL == 4) {
      *reinterpret_cast<uint32_t*>(dst) = up;
      *reinterpret_cast<uint32_t*>(dst + D) = dn;
    } else {
      *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(up);
      *reinterpret_cast<uint16_t*>(dst + D) = static_cast<uint16_t>(dn);
    }
    if (lane == 0) a.exps[chunk] = static_cast<int8_t>(e);
  }
}

// ---------------------------------------------------------------- selection
// Two kernels.  score_kernel reads the bounds once, eight heads of a block
// together, in equal shares of the line (token, heads, block), and leaves a 32-bit
// key for every (token, block, head); pick_kernel finds each (token, head)'s
// threshold and writes its list.  (One kernel a (token, head), clusters or not,
// left the memory idle while it looked for thresholds and took as long as the
// longest context on the fullest SM: 35 us against 30 for 32 requests of 9 to 32
// thousand tokens; now 18 + 8.)
constexpr int kScoreThreads = 256;
constexpr int kScoreWarps = kScoreThreads / 32;
// Heads go in octets (all heads if there are no more than eight): an item of the line is a token's octet.
__host__ __device__ inline int octets_of(int num_kv_heads) { return num_kv_heads > 8 ? (num_kv_heads + 7) / 8 : 1; }
// Blocks that an item's start costs (about 40 KB of bounds and a bit).
__host__ __device__ inline int start_units(int num_kv_heads) { return 4 + 160 / (num_kv_heads < 8 ? num_kv_heads : 8); }
using ScoreShare = Share<16>;

// Order-preserving key of a score: larger score, larger key.  0 (no block) is
// below every score, 0xffffffff (taken in any case) above.
__device__ __forceinline__ uint32_t key_of(float f) {
  f += 0.f;   // -0 counts as 0
  const uint32_t u = __float_as_uint(f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// P and N of a group's queries ([G][D]) as whole numbers: unit 2^f, the smallest
// with |q| <= most 2^f, most = floor(32767 / G).  One warp, D / 32 channels a lane.
template <int D>
__device__ __forceinline__ void whole_queries(const uint16_t* q, int G, int16_t* dst, int lane) {
  constexpr int kDPL = D / 32;
  const float mostq = static_cast<float>(32767 / G);
  auto channels = [&](int r, float (&v)[kDPL]) {   // row r of the group; values that are not finite count as 0
    uint32_t w[2];
    if constexpr (kDPL == 4) {
      const uint2 y = *reinterpret_cast<const uint2*>(q + r * D + lane * kDPL);
      w[0] = y.x; w[1] = y.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(q + r * D + lane * kDPL);
    }
#pragma unroll
    for (int d = 0; d < kDPL; ++d) {
      const float f = (d & 1) ? bf16hi_to_f32(w[d >> 1]) : bf16lo_to_f32(w[d >> 1]);
      v[d] = fabsf(f) < CUDART_INF_F ? f : 0.f;
    }
  };
  float amax = 0.f;
#pragma unroll 8
  for (int r = 0; r < G; ++r) {
    float v[kDPL];
    channels(r, v);
#pragma unroll
    for (int d = 0; d < kDPL; ++d) amax = fmaxf(amax, fabsf(v[d]));
  }
#pragma unroll
  for (int y = 16; y > 0; y >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, y));
  // Tiny queries (below 2^-100) count as 0: the unit stays a normal number.
  const bool none = !(amax >= 7.8886090522101181e-31f);
  const int f = none ? 0 : exp_of(amax) - exp_of(mostq) + (mant_of(amax) <= mant_of(mostq) ? 0 : 1);
  // x 2^-f in two exact steps (2^-f alone may exceed the normal range)
  const float f1 = none ? 0.f : pow2f(-f / 2), f2 = pow2f(-(f - f / 2));
  int P[kDPL], N[kDPL];
#pragma unroll
  for (int d = 0; d < kDPL; ++d) P[d] = N[d] = 0;
#pragma unroll 8
  for (int r = 0; r < G; ++r) {
    float v[kDPL];
    channels(r, v);
#pragma unroll
    for (int d = 0; d < kDPL; ++d) {
      const int w = static_cast<int>(rintf(v[d] * f1 * f2));
      P[d] += max(w, 0);
      N[d] += min(w, 0);
    }
  }
#pragma unroll
  for (int d = 0; d < kDPL; ++d) {
    dst[lane * kDPL + d] = static_cast<int16_t>(P[d]);
    dst[D + lane * kDPL + d] = static_cast<int16_t>(N[d]);
  }
}

// A warp's view of one iteration: eight groups of four lanes; group i takes head i
// of the octet of one block, or head i % Hkv of block i / Hkv (fewer than 8 heads:
// 8 / Hkv blocks an iteration).  Lane s of a group takes the
// 16-byte pieces s, s + 4, ... of the head's 2 D codes, and copies them itself
// into its own places of the ring, so that it waits for nothing but its copies.
// Bound by HBM: 105 MB of bounds (32 contexts of 9 to 40 thousand tokens, 8 heads)
// in 18 us, of which 5 are the start (positions, block ids, queries).  All heads of a
// token as one item, their queries made at its start by every CTA, took 99 us instead
// of 93 for the 7 tokens below.
//
// NT = 2: the tokens of a request go in pairs, which read its bounds once.  A
// pair is an item of the line at its first token, its second token has no units.
// Taken where there are more tokens than requests (selection and attention, us,
// single / pairs; 40 heads, 5 contexts of 60 to 131 thousand tokens: 7 tokens in all
// 100 / 93, 4 each 197 / 162; 8 heads, 32 contexts of 9 to 40 thousand: 2 each 138 /
// 135, 4 each 237 / 232; 2 x 256 tokens of 8 thousand: 167 / 156).
template <int D, int NT>
struct ScoreShape {
  static constexpr int kStages = NT == 1 ? 3 : 4;   // warp iterations of bounds in flight
  static constexpr int kCtas = NT == 1 ? 3 : 2;     // CTAs an SM
  static constexpr int kPieces = 2 * D / 64;
  static constexpr int kStage = kScoreThreads * (kPieces * 16 + 4);   // codes, exponents
  static constexpr int kRing = kStages * kStage;
  static constexpr int kRawStages = NT;             // stages that first take queries as they are
  static constexpr int kRawRows = 64;               // rows of each token that fit
  static_assert(kRawStages * kPieces * 16 * kScoreThreads >= NT * kRawRows * D * 2, "query rows fit their stages");
  static constexpr int kQuery = NT * 4 * D + 16;    // bytes a KV head (heads 16 bytes apart in the banks)
  static constexpr int kRingAt = 8 * kQuery;
  static constexpr int kTotal = kRingAt + kRing;
};
template <int D, int NT>
__global__ void __launch_bounds__(kScoreThreads, ScoreShape<D, NT>::kCtas) score_kernel(const SparseArgs a) {
  using S = ScoreShape<D, NT>;
  constexpr int kPieces = S::kPieces, kScoreStages = S::kStages;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int64_t scratch[kScoreWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int Hkv = a.pool.num_kv_heads, G = a.group;
  // smem: [8 heads][NT][P: D, N: D] 16-bit whole-number queries; ring: [stage][piece][thread] 16 bytes, [stage][thread] 4
  const uint32_t slot = smem_u32(smem) + S::kRingAt + tid * 16;
  const uint32_t slot_e = smem_u32(smem) + S::kRingAt + kScoreStages * kScoreThreads * kPieces * 16 + tid * 4;
  griddep_wait();
  griddep_launch();
  if (blockIdx.x == 0 && tid == 0) check_cu(a.cu_q_lens, a.num_reqs, a.num_tokens, a.pool.err);

  // The share: each octet of token t (of this launch's) has a unit for each block up to its position, and some for
  // its start.
  const int end_tok = min(max(__ldg(a.cu_q_lens + a.num_reqs), 0), a.num_tokens);
  const int tokens = max(0, min(a.tok_count, end_tok - a.tok_first));
  const int most = a.max_blocks * kBlockSize;
  auto token_blocks = [&](int t) -> int {   // 0 for a position outside the table
    const int p = __ldg(a.positions + t);
    return p >= 0 && p < most ? (p >> 4) + 1 : 0;
  };
  // Pairs: the blocks of the pair's two tokens; false for a token that opens none (r < 0, or a pair's second).
  auto pair_blocks = [&](int t, int r, int& n0, int& n1) -> bool {
    if (r < 0) return false;
    const int first = max(__ldg(a.cu_q_lens + r), a.tok_first);
    if ((t - first) & 1) return false;
    n0 = token_blocks(t);
    n1 = t + 1 < min(__ldg(a.cu_q_lens + r + 1), a.tok_first + tokens) ? token_blocks(t + 1) : 0;
    return true;
  };
  const int start = start_units(Hkv), octets = octets_of(Hkv);
  int64_t U[1], off[1];
  int at[1];
  int64_t u = 0, end = 0;
  line_scan<kScoreThreads, 1, 1>(
      tokens, scratch, U, at, off,
      [&](int i, int64_t (&n)[1]) {
        const int t = a.tok_first + i, b = token_blocks(t);
        if constexpr (NT == 1) {
          n[0] = static_cast<int64_t>(octets) * (b + start);
        } else {
          int n0, n1;
          n[0] = pair_blocks(t, req_of(a.cu_q_lens, a.num_reqs, t), n0, n1)
                     ? static_cast<int64_t>(octets) * (max(n0, n1) + start)
                     : 0;
        }
        if (b == 0 && blockIdx.x == 0) atomicOr(a.pool.err, PKV_DEVERR_POSITION);
      },
      [&](const int64_t (&len)[1], int, int& line, int64_t& unit) {
        const int C = ScoreShare::workers(len[0], gridDim.x);
        if (len[0] > 0 && static_cast<int>(blockIdx.x) < C) {
          u = ScoreShare::begin(len[0], C, blockIdx.x);
          end = ScoreShare::begin(len[0], C, blockIdx.x + 1);
        }
        line = 0;
        unit = u < end ? u : -1;
      });
  if (u >= end) return;

  const int grp = lane >> 2, sub = lane & 3;
  const int bpw = Hkv >= 8 ? 1 : 8 / Hkv;               // blocks of a warp iteration
  const int my_blk = Hkv >= 8 ? 0 : grp / Hkv;
  const bool lane_on = Hkv >= 8 || grp < bpw * Hkv;
  int tok = a.tok_first + at[0];
  int64_t x = off[0];   // unit within the token
  while (u < end) {
    int nt[NT], r = -1;   // blocks of each token
    bool opens = true;
    if constexpr (NT == 1) {
      nt[0] = token_blocks(tok);
    } else {
      r = req_of_warp(a.cu_q_lens, a.num_reqs, tok, lane);
      opens = pair_blocks(tok, r, nt[0], nt[1]);   // (otherwise it has no units)
    }
    const int n = opens ? max(nt[0], nt[NT - 1]) : 0, span = n + start;
    const int octet = static_cast<int>(x / span);
    if (!opens || octet >= octets) {
      ++tok;
      x = 0;
      continue;
    }
    const int b0 = static_cast<int>(x - static_cast<int64_t>(octet) * span);
    const int len = static_cast<int>(min(static_cast<int64_t>(span - b0), end - u));
    const int b1 = min(b0 + len, n);
    u += len;
    x += len;
    if (b0 >= b1) continue;   // block-uniform
    if constexpr (NT == 1) {
      r = req_of_warp(a.cu_q_lens, a.num_reqs, tok, lane);
      if (r < 0) continue;
    }
    const int head0 = octet * 8, heads = min(8, Hkv - head0);
    const int32_t* bt_row = a.block_tables + static_cast<int64_t>(r) * a.max_blocks;
    // Iterations of this warp: blocks first, first + step, ... (`per` of them).  Everything that is read comes
    // through copies in flight, but for the block ids: lane l holds the id of the warp's block base + l, and the next
    // 32 are on their way.  (A load into a register, consumed iterations later, waits for the newest such load:
    // exponents read so made every iteration as long as a read of DRAM.)
    const int step = kScoreWarps * bpw, first = b0 + warp * bpw + my_blk;
    const int per = (b1 - b0 + step - 1) / step;
    const int h = head0 + (Hkv >= 8 ? grp : grp % Hkv);   // this lane's
    const bool on = lane_on && h < Hkv;
    const int own = per * bpw;   // the warp's blocks
    auto load_ids = [&](int base) -> int {
      const int i = base + lane, b = b0 + (i / bpw * kScoreWarps + warp) * bpw + i % bpw;
      return i < own && b < b1 ? __ldg(bt_row + b) : -1;
    };
    int id_cur = load_ids(0), id_next = load_ids(32);
    int id_at = 0;   // the copies' cursor
    int ids[kScoreStages];
    auto copy = [&](int st) {   // the next iteration's
      int pb = __shfl_sync(0xffffffffu, id_cur, (id_at & 31) + my_blk);
      if (id_at >= own || !on) pb = -1;
      ids[st] = pb;
      if (static_cast<unsigned>(pb) < static_cast<unsigned>(a.pool.num_blocks)) {
        const int64_t chunk = static_cast<int64_t>(pb) * Hkv + h;
        const int8_t* src = a.codes + chunk * 2 * D + sub * 16;
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                       ::"r"(slot + (st * kPieces + i) * (kScoreThreads * 16)), "l"(src + i * 64) : "memory");
        if (sub < NT)   // the aligned word that holds the exponent
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;"
                       ::"r"(slot_e + st * (kScoreThreads * 4)),
                       "l"(reinterpret_cast<uintptr_t>(a.exps + chunk) & ~uintptr_t(3)) : "memory");
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      id_at += bpw;
      if ((id_at & 31) == 0) {
        id_cur = id_next;
        id_next = load_ids(id_at + 32);
      }
    };
    // The queries of the first heads (of up to kRawRows rows) are asked for before the first bounds, into the ring's
    // last stages: behind three stages of bounds they took 4 us to come.
    const int raw_heads = min(heads, S::kRawRows / G);
    const int raw_at = S::kRingAt + (kScoreStages - S::kRawStages) * kPieces * kScoreThreads * 16;
    __syncthreads();   // the previous token's queries and bounds are no longer read
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int chunks = nt[j] == 0 ? 0 : raw_heads * G * (D / 8);
      const uint8_t* src = static_cast<const uint8_t*>(a.q) +
                           (static_cast<int64_t>(tok + j) * a.num_q_heads + head0 * G) * D * 2;
      const uint32_t dst = smem_u32(smem) + raw_at + j * (S::kRawRows * D * 2);
      for (int i = tid; i < chunks; i += kScoreThreads)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + i * 16), "l"(src + i * 16) : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll
    for (int v = 0; v < kScoreStages - S::kRawStages; ++v) copy(v);
    asm volatile("cp.async.wait_group %0;" ::"n"(kScoreStages - S::kRawStages) : "memory");
    __syncthreads();

    // Whole-number queries of the heads, while the first copies are under way: a warp a (head, token).
    for (int i = warp; i < heads * NT; i += kScoreWarps) {
      const int hh = i / NT, j = i % NT;
      if (nt[j] == 0) continue;   // no second token (its sums are not used)
      const uint16_t* q = hh < raw_heads
          ? reinterpret_cast<const uint16_t*>(smem + raw_at) + (j * S::kRawRows + hh * G) * D
          : static_cast<const uint16_t*>(a.q) + (static_cast<int64_t>(tok + j) * a.num_q_heads + (head0 + hh) * G) * D;
      whole_queries<D>(q, G, reinterpret_cast<int16_t*>(smem + hh * S::kQuery) + j * 2 * D, lane);
    }
    __syncthreads();
#pragma unroll
    for (int v = kScoreStages - S::kRawStages; v < kScoreStages; ++v) copy(v);

    int qq[NT][kPieces][8];
    {
      const int* src = reinterpret_cast<const int*>(smem + min(h - head0, heads - 1) * S::kQuery);
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
#pragma unroll
          for (int w = 0; w < 8; ++w) qq[j][i][w] = src[j * D + (i * 4 + sub) * 8 + w];
    }
    // This lane's head and token.
    uint32_t* row = a.keys + (static_cast<int64_t>(tok - a.tok_first + sub) * Hkv + h) * a.max_blocks;
    const int n_tok = NT == 1 || sub == 0 ? nt[0] : nt[NT - 1];
    const int most_b = on && sub < NT ? min(b1, n_tok) : 0;   // blocks whose keys this lane writes
    int b = first;
    for (int k0 = 0; k0 < per; k0 += kScoreStages) {
#pragma unroll
      for (int v = 0; v < kScoreStages; ++v) {
        if (k0 + v < per) {
          asm volatile("cp.async.wait_group %0;" ::"n"(kScoreStages - 1) : "memory");
          int part[NT][kPieces] = {};   // (short chains: a warp waits for fixed latencies otherwise)
#pragma unroll
          for (int i = 0; i < kPieces; ++i) {
            uint32_t w[4];
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(slot + (v * kPieces + i) * (kScoreThreads * 16)) : "memory");
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                part[j][i] = __dp2a_lo(qq[j][i][2 * y], static_cast<int>(w[y]), part[j][i]);
                part[j][i] = __dp2a_hi(qq[j][i][2 * y + 1], static_cast<int>(w[y]), part[j][i]);
              }
          }
          int sum[NT];
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            sum[j] = part[j][0] + part[j][1];
            if constexpr (kPieces == 4) sum[j] += part[j][2] + part[j][3];
          }
          // Lane j of a group ends up with token j's sum.
          int s = sum[0];
          if constexpr (NT == 2) {
            const int give = (sub & 1) ? sum[0] : sum[1];
            s = ((sub & 1) ? sum[1] : sum[0]) + __shfl_xor_sync(0xffffffffu, give, 1);
          } else {
            s += __shfl_xor_sync(0xffffffffu, s, 1);
          }
          s += __shfl_xor_sync(0xffffffffu, s, 2);
          if (b < most_b) {
            uint32_t key = 0u;
            if (static_cast<unsigned>(ids[v]) >= static_cast<unsigned>(a.pool.num_blocks))
              atomicOr(a.pool.err, PKV_DEVERR_BLOCK_ID);
            else if (b < a.sinks || b >= n_tok - a.recent) key = 0xffffffffu;
            else {
              uint32_t w;
              asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(slot_e + v * (kScoreThreads * 4)) : "memory");
              const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(a.exps)) + ids[v] * Hkv + h;
              const int e = static_cast<int8_t>(w >> (8 * (at & 3u)));
              key = key_of(__int2float_rn(s) * pow2f(max(-126, e)));
            }
            row[b] = key;
          }
          b += step;
          copy(v);
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
}

constexpr int kPickThreads = 512;
// Few short lists: a CTA of pick_kernel scores its (token, head)'s blocks itself,
// which saves a launch and the way through the workspace.  Four lanes a block,
// 16-byte pieces as above; the first blocks' codes are on their way while a warp
// makes the whole-number query.  (Bounds are read from L2: the kernel ahead may be a
// copy of pages that has read and written them.)
template <int D>
__device__ __forceinline__ void alone_keys(const SparseArgs& a, int t, int g, int req, int n, uint32_t* s_keys) {
  constexpr int kPieces = 2 * D / 64, kRound = kPickThreads / 4;
  __shared__ __align__(16) int16_t s_q[2 * D];
  const int tid = threadIdx.x, sub = tid & 3;
  const int32_t* bt_row = a.block_tables + static_cast<int64_t>(req) * a.max_blocks;
  int qq[kPieces][8];
  for (int base = 0; base < n; base += kRound) {
    const int b = base + (tid >> 2), pb = b < n ? __ldg(bt_row + b) : 0;
    const bool there = b < n && static_cast<unsigned>(pb) < static_cast<unsigned>(a.pool.num_blocks);
    const int64_t chunk = static_cast<int64_t>(pb) * a.pool.num_kv_heads + g;
    uint4 w[kPieces];
    int e = 0;
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      w[i] = there ? __ldcg(reinterpret_cast<const uint4*>(a.codes + chunk * 2 * D + sub * 16 + i * 64)) : make_uint4(0, 0, 0, 0);
    if (there) e = __ldcg(reinterpret_cast<const signed char*>(a.exps) + chunk);
    if (base == 0) {
      if (tid < 32)
        whole_queries<D>(static_cast<const uint16_t*>(a.q) + (static_cast<int64_t>(t) * a.num_q_heads + g * a.group) * D,
                         a.group, s_q, tid);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
#pragma unroll
        for (int y = 0; y < 8; ++y) qq[i][y] = reinterpret_cast<const int*>(s_q)[(i * 4 + sub) * 8 + y];
    }
    int s = 0;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        s = __dp2a_lo(qq[i][2 * y], static_cast<int>(x[y]), s);
        s = __dp2a_hi(qq[i][2 * y + 1], static_cast<int>(x[y]), s);
      }
    }
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    if (sub == 0 && b < n) {
      uint32_t key = 0u;
      if (!there) atomicOr(a.pool.err, PKV_DEVERR_BLOCK_ID);
      else if (b < a.sinks || b >= n - a.recent) key = 0xffffffffu;
      else key = key_of(__int2float_rn(s) * pow2f(max(-126, e)));
      s_keys[b] = key;
    }
  }
}

// One CTA per (token, KV head).  Keys of up to kPickKeys blocks stay in shared
// memory, more are read again from L2.  The radix passes run on key - lo, shifted
// until the largest uses all 32 bits, so that the first 8-bit pass spreads the
// keys over its bins (as they are they share their top byte, and hundreds of
// additions to one counter take a microsecond), and stop as soon as the
// threshold's bin is taken whole, or holds so few keys that ranking them against
// each other is shorter than another pass (for 190 blocks 18.4 -> 16.6 us of a
// selection and attention).  Bound by the latency of these steps: 8 us for 256 lists
// of 1500 blocks.
constexpr int kPickWarps = kPickThreads / 32;
constexpr int kPickKeys = 8192;
constexpr int kPickRank = 64;
// pick_kernel alone up to kAloneBlocks blocks a list and kAloneLists lists an SM
// (selection and attention, us, both kernels / alone; 190 blocks: 2 lists 16.5 / 14.5,
// 64 lists 20.6 / 16.5, 256 lists 26.7 / 22.1, 1024 lists 65.7 / 74.1; 500 blocks: 64
// lists 20.6 / 18.6, 512 lists 49.9 / 50.7; 8 lists of 940 blocks 19.4 / 20.6, of 1900
// 20.6 / 27.0).
constexpr int kAloneBlocks = 512, kAloneLists = 3;
template <int D, bool ALONE>
__global__ void __launch_bounds__(kPickThreads) pick_kernel(const SparseArgs a) {
  __shared__ uint32_t s_keys[kPickKeys];
  __shared__ uint32_t s_hist[4][256];
  __shared__ uint32_t s_lohi[2];
  __shared__ int s_count[2];           // forced, ordinary
  __shared__ int s_scan[2][kPickWarps];
  __shared__ int s_pick[3];            // radix pass: bin, keys above it, keys in it
  __shared__ uint32_t s_cand[kPickRank];
  __shared__ int s_cands;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int Hkv = a.pool.num_kv_heads;
  const int g = static_cast<int>(blockIdx.x % Hkv), i_tok = static_cast<int>(blockIdx.x / Hkv);
  const int t = a.tok_first + i_tok;
  for (int i = tid; i < 4 * 256; i += kPickThreads) (&s_hist[0][0])[i] = 0;
  if (tid == 0) {
    s_lohi[0] = 0xffffffffu;
    s_lohi[1] = 0u;
    s_count[0] = s_count[1] = s_cands = 0;
  }
  // (After the scores' kernel the caller's arrays are complete already: every CTA of it waited before it let this one start.)
  if constexpr (ALONE) griddep_wait();
  const int req = req_of_warp(a.cu_q_lens, a.num_reqs, t, lane);
  const int p = __ldg(a.positions + t);
  if constexpr (!ALONE) griddep_wait();
  griddep_launch();
  if (ALONE && blockIdx.x == 0 && tid == 0) check_cu(a.cu_q_lens, a.num_reqs, a.num_tokens, a.pool.err);
  if (ALONE && g == 0 && tid == 0 && t < __ldg(a.cu_q_lens + a.num_reqs) && (p < 0 || p >= a.max_blocks * kBlockSize))
    atomicOr(a.pool.err, PKV_DEVERR_POSITION);
  if (req < 0) return;   // block-uniform
  int32_t* out = a.sel + (static_cast<int64_t>(t) * Hkv + g) * a.top_k;
  const int n = p >= 0 && p < a.max_blocks * kBlockSize ? (p >> 4) + 1 : 0;
  const uint32_t* src = a.keys + (static_cast<int64_t>(i_tok) * Hkv + g) * a.max_blocks;
  const bool kept = ALONE || n <= kPickKeys;
  if constexpr (ALONE) alone_keys<D>(a, t, g, req, n, s_keys);
  __syncthreads();
  uint32_t lo = 0xffffffffu, hi = 0u;
  int forced = 0, ordinary = 0;
#pragma unroll 4
  for (int i = tid; i < n; i += kPickThreads) {
    const uint32_t k = ALONE ? s_keys[i] : __ldcg(src + i);
    if (!ALONE && kept) s_keys[i] = k;
    if (k == 0xffffffffu) {
      ++forced;
    } else if (k != 0u) {
      lo = min(lo, k);
      hi = max(hi, k);
      ++ordinary;
    }
  }
  auto key = [&](int i) { return kept ? s_keys[i] : __ldcg(src + i); };
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  forced = __reduce_add_sync(0xffffffffu, forced);
  ordinary = __reduce_add_sync(0xffffffffu, ordinary);
  if (lane == 0) {
    atomicMin(&s_lohi[0], lo);
    atomicMax(&s_lohi[1], hi);
    atomicAdd(&s_count[0], forced);
    atomicAdd(&s_count[1], ordinary);
  }
  __syncthreads();
  lo = s_lohi[0];
  hi = s_lohi[1];
  forced = s_count[0];
  ordinary = s_count[1];
  // Ordinary keys in the passes' form: key - lo, shifted up.  Taken are the forced keys, the ordinary ones above
  // `thr`, and the first `need` equal to it.
  const int shift0 = hi > lo ? __clz(hi - lo) : 0;
  auto form = [&](uint32_t k) { return (k - lo) << shift0; };
  const bool forced_only = forced >= a.top_k;   // the first top_k of the forced ones
  bool all = false;                             // every ordinary key
  uint32_t thr = 0;
  int need = forced_only ? a.top_k : min(a.top_k - forced, ordinary);
  if (!forced_only && need == ordinary) {
    all = true;
  } else if (!forced_only && hi > lo) {
    for (int pass = 0; pass < 4; ++pass) {
      const int shift = 24 - 8 * pass;
      for (int i = tid; i < n; i += kPickThreads) {
        const uint32_t k = key(i), v = form(k);
        if (k != 0u && k != 0xffffffffu && (pass == 0 || (v >> (shift + 8)) == (thr >> (shift + 8))))
          atomicAdd(&s_hist[pass][(v >> shift) & 255u], 1u);
      }
      __syncthreads();
      // Thread i < 256: bin 255 - i, then an inclusive scan from the top bin.
      const int c = tid < 256 ? static_cast<int>(s_hist[pass][255 - tid]) : 0;
      int inc = c;
#pragma unroll
      for (int y = 1; y < 32; y <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, inc, y);
        if (lane >= y) inc += z;
      }
      if (lane == 31) s_scan[0][warp] = inc;
      __syncthreads();
      for (int w = 0; w < warp; ++w) inc += s_scan[0][w];
      if (inc >= need && inc - c < need) {
        s_pick[0] = 255 - tid;
        s_pick[1] = inc - c;
        s_pick[2] = c;
      }
      __syncthreads();
      thr |= static_cast<uint32_t>(s_pick[0]) << shift;
      need -= s_pick[1];
      if (need == s_pick[2]) {   // everything from the bin on: thr > 0, or every ordinary key would be taken
        thr -= 1u;
        need = 0;
        break;
      }
      const int c_bin = s_pick[2];
      if (pass < 3 && c_bin <= kPickRank) {
        // Few keys left in the bin: each is compared with all of them.
        for (int i = tid; i < n; i += kPickThreads) {
          const uint32_t k = key(i), v = form(k);
          if (k != 0u && k != 0xffffffffu && (v >> shift) == (thr >> shift)) s_cand[atomicAdd(&s_cands, 1)] = v;
        }
        __syncthreads();
        if (tid < c_bin) {
          const uint32_t v = s_cand[tid];
          int above = 0, same = 0;
          for (int i = 0; i < c_bin; ++i) {
            above += s_cand[i] > v;
            same += s_cand[i] == v;
          }
          if (above < need && need <= above + same) {   // the threshold (every key equal to it says the same)
            s_pick[0] = static_cast<int>(v);
            s_pick[1] = above;
          }
        }
        __syncthreads();
        thr = static_cast<uint32_t>(s_pick[0]);
        need -= s_pick[1];
        break;
      }
      __syncthreads();
    }
  }
  // 2: taken, 1: equal to the threshold, 0: not taken.
  auto kind = [&](uint32_t k) -> int {
    if (k == 0u) return 0;
    if (k == 0xffffffffu) return forced_only ? 1 : 2;
    if (forced_only) return 0;
    if (all) return 2;
    const uint32_t v = form(k);
    return v > thr ? 2 : v == thr && need > 0 ? 1 : 0;
  };
  // Each warp writes the entries of its own stretch of the blocks, in order: first every warp counts.
  const int per = ((n + kPickWarps - 1) / kPickWarps + 31) / 32 * 32;
  const int w0 = min(n, warp * per), w1 = min(n, w0 + per);
  int gt = 0, eq = 0;
  for (int i = w0 + lane; i < w1; i += 32) {
    const int x = kind(key(i));
    gt += x == 2;
    eq += x == 1;
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  __syncthreads();   // s_scan is free
  if (lane == 0) {
    s_scan[0][warp] = eq;
    s_scan[1][warp] = gt;
  }
  __syncthreads();
  int at = 0, left = need, total = 0;   // where the warp writes, equal keys that it and later ones may take
  for (int w = 0, l = need; w < kPickWarps; ++w) {
    const int take = min(l, s_scan[0][w]);
    if (w < warp) {
      at += s_scan[1][w] + take;
      left -= take;
    }
    l -= take;
    total += s_scan[1][w] + take;
  }
  for (int base = w0; base < w1; base += 32) {
    const int i = base + lane;
    const int x = i < w1 ? kind(key(i)) : 0;
    const uint32_t beq = __ballot_sync(0xffffffffu, x == 1), bgt = __ballot_sync(0xffffffffu, x == 2);
    const uint32_t below = (1u << lane) - 1u;
    const int peq = __popc(beq & below), pgt = __popc(bgt & below);
    if (x == 2 || (x == 1 && peq < left)) out[at + pgt + min(peq, left)] = i;
    const int teq = min(left, __popc(beq));
    at += __popc(bgt) + teq;
    left -= teq;
  }
  for (int i = total + tid; i < a.top_k; i += kPickThreads) out[i] = -1;
}

template <int D, int NT>
int launch_select_d(SparseArgs a, cudaStream_t s) {
  using S = ScoreShape<D, NT>;
  cudaError_t e = smem_attr_once<score_kernel<D, NT>>(S::kTotal);
  if (e != cudaSuccess) return e;
  // Tokens in parts whose keys fit the workspace.
  for (int t = 0; t < a.num_tokens; t += a.tok_most) {
    a.tok_first = t;
    a.tok_count = std::min(a.tok_most, a.num_tokens - t);
    // No more CTAs than there can be shares of 16 units.
    const int64_t units = static_cast<int64_t>(a.tok_count) * octets_of(a.pool.num_kv_heads) *
                          (a.max_blocks + start_units(a.pool.num_kv_heads));
    const unsigned ctas = static_cast<unsigned>(std::min<int64_t>(S::kCtas * a.num_sms, (units + 15) / 16));
    e = launch_dependent(score_kernel<D, NT>, dim3(ctas), kScoreThreads, S::kTotal, s, a);
    if (e == cudaSuccess)
      e = launch_dependent(pick_kernel<0, false>, dim3(static_cast<unsigned>(a.tok_count) * a.pool.num_kv_heads), kPickThreads, 0, s, a);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int D>
int launch_alone_d(SparseArgs a, cudaStream_t s) {
  a.tok_first = 0;
  a.tok_count = a.num_tokens;
  return launch_dependent(pick_kernel<D, true>, dim3(static_cast<unsigned>(a.num_tokens) * a.pool.num_kv_heads), kPickThreads,
                          0, s, a);
}

template <int D, bool F8>
int launch_summarize_d(const SparseArgs& a, cudaStream_t s) {
  // A warp of 16 tokens finds about one new block in a prompt; a batch of
  // single tokens opens one block a token and takes a warp for each.
  const int64_t one = static_cast<int64_t>(a.num_tokens) * a.pool.num_kv_heads;
  if (one <= 64ll * a.num_sms) {
    summarize_kernel<D, F8, 1><<<static_cast<unsigned>((one + 7) / 8), 256, 0, s>>>(a);
  } else {
    const int64_t w = static_cast<int64_t>((a.num_tokens + 15) / 16) * a.pool.num_kv_heads;
    summarize_kernel<D, F8, 16><<<static_cast<unsigned>((w + 7) / 8), 256, 0, s>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace

int launch_summarize(const SparseArgs& a, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool f8 = a.pool.elem_bytes == 1;
  if (a.pool.head_dim == 128) return f8 ? launch_summarize_d<128, true>(a, s) : launch_summarize_d<128, false>(a, s);
  return f8 ? launch_summarize_d<64, true>(a, s) : launch_summarize_d<64, false>(a, s);
}

// Keys of as many tokens as fit 64 MB, of one at least.
int select_part(int num_tokens, int max_blocks, int num_kv_heads) {
  const int64_t one = static_cast<int64_t>(max_blocks) * num_kv_heads * 4;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(num_tokens, (64ll << 20) / one)));
}

int launch_select(const SparseArgs& a, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.max_blocks <= kAloneBlocks && static_cast<int64_t>(a.num_tokens) * a.pool.num_kv_heads <= kAloneLists * static_cast<int64_t>(a.num_sms))
    return a.pool.head_dim == 128 ? launch_alone_d<128>(a, s) : launch_alone_d<64>(a, s);
  const bool pairs = a.num_tokens > a.num_reqs;
  if (a.pool.head_dim == 128) return pairs ? launch_select_d<128, 2>(a, s) : launch_select_d<128, 1>(a, s);
  return pairs ? launch_select_d<64, 2>(a, s) : launch_select_d<64, 1>(a, s);
}

}  // namespace pkv
