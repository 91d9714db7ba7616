// Attention with modified scores and masks (pkv_score_attn), the form on the
// tcgen05 tensor cores for batches that bring many query rows per KV head.
//
// The warp roles are those of the tree attention on tiles (K and V producers that
// gather blocks by TMA, one MMA issuer, two softmax warpgroups A and B, scores, P
// and O in TMEM, a scheduler that hands out segments ahead of their use).  What
// differs is the work: a tile of 128 query rows sees keys from the first that its
// window or document leaves up to its last position, so that tiles of one request
// differ in length.  A plan kernel of one CTA lists them first:
//   item    two neighbouring tiles of a request (A and B share every K/V tile), or
//           its odd last one (A takes the even key tiles, B the odd ones, and A
//           joins B's state at the end); the key tiles that hold the prefix, then
//           those from the first key that any row sees to the last;
//   line    the items of one KV head after another's, a key tile of a pair three
//           units, of a single tile two (codes: three), and kGroupUnits for start
//           and epilogue.
// A CTA takes an equal share of the line; a group that several share is merged by
// log-sum-exp.
//
// Masks: in key tiles that some row does not see whole each row's thread forms its
// 128 visibility bits from its span of keys.  The V producer reads those tiles once
// in shared memory and clears elements that are not finite (a masked key must not
// reach a row as 0 * inf) and the rows past the context; rows that do see such an
// element get it added after their result is stored.  Int8 values are finite.
//
// Scores: tanh on the FMA pipe, as a polynomial with the scales in its coefficients,
// five paired operations for two scores, while every score of the warp's rows stays
// below half the cap; otherwise by tanh_small and tanh_large.  It is monotonic:
// without a bias the raw products' maximum gives the scores', and the last operation
// subtracts it (4 prompts of 1.8 to 5 thousand tokens, 64 / 8 heads, D = 128: 769 us;
// 912 with scores written back to TMEM first, as masked or biased ones still are; scores on
// both sides of half the cap 1,700).
//
// Pools of codes: they land in the upper half of each block's lines, and four more warps widen
// them in place, two for K and two for V (int8: to bf16 times the block's power of
// two, exactly, so that the MMAs are those of bf16 pools; FP8: to f16).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <climits>
#include <type_traits>

#include "internal.h"
#include "ops.h"
#include "ptx.cuh"
#include "rows.cuh"
#include "sched.cuh"
#include "score.cuh"
#include "tc.cuh"

namespace pkv {
namespace {

// What becomes of scores: a kernel for each, as code that does not run takes room in the instruction cache, too (the
// capped prompts of the header 791 us with the code for a bias beside theirs, biased ones 900 us, 823 by itself).
enum { kPlain, kCapped, kBiased };   // kBiased: capped or not
constexpr int kTeam = 2;   // codes: warps that widen K, and V
// Registers of a CTA for codes, of 128 each at the launch.  Widening wants more (104: 5 % slower, 88: 20 %), and four
// warps a team would leave it 48 (80 % slower).
constexpr int kRegsWiden = 120, kRegsCodes = 56, kRegsSoft = 168;
static_assert(kRegsCodes <= 128 && kRegsWiden <= 128 && kRegsSoft >= 128 && 2 * kRegsSoft + kRegsWiden + kRegsCodes <= 4 * 128,
              "setmaxnreg.dec goes down, .inc up, within the launch's registers");
// Warps 0 .. 7 softmax, 8 Q and K producer, 9 MMA issuer, 10 V producer, 11 scheduler; codes: 12 .. 15 widen.
template <int KIND>
constexpr int kThreads = KIND == kPoolBf16 ? 384 : 384 + 64 * kTeam;
constexpr int kBlkPerTile = kNK / kBlockSize;   // 8
constexpr int kSegSlots = 4;                    // segments handed out ahead
constexpr int kSegRing = 8;                     // V producer's reports (it is at most kSegSlots + 1 ahead)
template <int KIND>
constexpr int kSegReaders = KIND == kPoolBf16 ? 11 : 11 + 2 * kTeam;   // warps that read a segment
// (Codes: a single tile waits for the widening as a pair does; as two units it made 10 requests of 1 to 733 new tokens
// 10 % slower.)
constexpr int kPairUnits = 3, kSingleUnits = 2, kCodeSingleUnits = 3, kGroupUnits = 6;
__device__ __forceinline__ int tile_cost(const PoolView& pool, bool single) {
  return !single ? kPairUnits : pool.elem_bytes == 1 ? kCodeSingleUnits : kSingleUnits;
}
using TcShare = Share<kPairUnits + kGroupUnits>;

template <int KS, int VS>
struct ScoreBars {
  static constexpr int kKFull = 0, kKEmpty = KS, kKLanded = 2 * KS;
  static constexpr int kVFull = 3 * KS, kVEmpty = 3 * KS + VS, kVLanded = 3 * KS + 2 * VS;
  static constexpr int kT = 3 * KS + 3 * VS;
  static constexpr int kS = kT;             // + group: S of its next key tile in TMEM
  static constexpr int kP = kT + 2;         // + group: P written, O rescaled (128 arrivals)
  static constexpr int kPv = kT + 4;        // + group: its last PV of the segment done
  static constexpr int kQFull = kT + 6;     // + tile
  static constexpr int kQEmpty = kT + 8;    // + tile
  static constexpr int kQc = kT + 10;       // + tile: FP8: Q rows converted to f16 (128 arrivals)
  static constexpr int kMl = kT + 12;       // single: B's state is final (128 arrivals)
  static constexpr int kJoined = kT + 13;   // single: A has read it (128 arrivals)
  static constexpr int kDrain = kT + 14;
  static constexpr int kVDone = kT + 15;    // + segment % kSegRing: its V tiles are all handed over
  static constexpr int kSegFull = kT + 15 + kSegRing;               // + segment % kSegSlots: published
  static constexpr int kSegEmpty = kSegFull + kSegSlots;            // + segment % kSegSlots: read by every role
  static constexpr int kCount = kSegEmpty + kSegSlots;
};

// What one CTA does with one group: key tiles [kt0, kt1) of an item, numbered from
// 0: those below pre_tiles lie at their number, the others `gap` further on.
struct alignas(16) Seg {
  int req, g, prefix, ctx;
  int tok0, tok1, rows0, rows1;   // query tiles (rows1 = 0: single)
  int kt0, kt1, slot, flags;
  int pre_tiles, gap, all_lo, all_hi;   // every row sees the keys [all_lo, all_hi],
  int any_lo, any_hi, pad0, pad1;       // none sees others than these (and the prefix)
};
static_assert(sizeof(Seg) == 80, "Seg layout: five 16-byte loads");
constexpr int kSegSingle = 1, kSegWhole = 2, kSegMissing = 4, kSegEnd = 8;

// A V element that is not finite and was left out of the products of a segment.
constexpr int kOddMost = 8;   // noted of a segment; all are counted
struct Odd {
  int key;
  uint16_t dim, bits;   // value: bf16, or the f16 of an FP8 code
};

template <int D>
struct ScoreSmem {
  using S = TcSmem<D>;
  using B = ScoreBars<S::kKSt, S::kVSt>;
  static constexpr int kOffBar = S::kOffBar;
  static constexpr int kOffMl = kOffBar + ((B::kCount * 8 + 15) / 16) * 16;   // float2 [128]: B's m, l
  static constexpr int kOffSeg = kOffMl + kTcRows * 8;
  static constexpr int kOffOdd = kOffSeg + kSegSlots * static_cast<int>(sizeof(Seg));   // Odd [kSegRing][kOddMost]
  static constexpr int kOffMisc = kOffOdd + kSegRing * kOddMost * 8;
  static constexpr int kTotal = kOffMisc + 64;
};
static_assert(ScoreSmem<128>::kTotal <= 232448, "shared memory of the D = 128 kernel");

// Key tile j of a segment's (or an item's) numbering, as a tile of the context.
__device__ __forceinline__ int tile_at(int j, int pre_tiles, int gap) { return j < pre_tiles ? j : j + gap; }

// Whether every row of the segment sees the whole key tile that begins at key0.
__device__ __forceinline__ bool seen_whole(const Seg& s, int key0) {
  return key0 + kNK <= s.prefix || (key0 >= s.all_lo && key0 + kNK - 1 <= s.all_hi);
}

// The blocks of the key tile at key0 that some row sees a key of, as bits; those that every row sees whole.
__device__ __forceinline__ uint32_t blocks_below(int keys) { return low_bits(min(max(keys, 0) / kBlockSize, kBlkPerTile)); }
__device__ __forceinline__ uint32_t blocks_needed(const Seg& s, int key0) {
  const uint32_t span = s.any_hi < s.any_lo ? 0u : blocks_below(s.any_hi - key0 + kBlockSize) & ~blocks_below(s.any_lo - key0);
  return blocks_below(s.prefix - key0 + kBlockSize - 1) | span;
}
__device__ __forceinline__ uint32_t blocks_whole(const Seg& s, int key0) {
  return blocks_below(s.prefix - key0) |
         (blocks_below(s.all_hi - key0 + 1) & ~blocks_below(s.all_lo - key0 + kBlockSize - 1));
}

// Walks a CTA's share of the line.  Key tile k of a group that begins at unit 0
// belongs to the worker that holds unit k * cost; the group's fixed units follow
// its last tile.
struct Walk {
  int64_t U, total, u, end;   // all heads' units, one head's, the share
  int workers, n_items, g, idx;
  bool fresh;                 // `it` is not item idx yet
  ScoreItem it;
  int64_t at;                 // units of the head's line before it
  int glen;

  // Every thread; false: the CTA has no share.
  __device__ __forceinline__ bool begin(const ScoreArgs& a) {
    total = __ldcg(a.plan.cum + a.plan.most);
    n_items = static_cast<int>(__ldcg(a.plan.cum + a.plan.most + 1));
    U = total * a.t.pool.num_kv_heads;
    workers = TcShare::workers(U, a.t.ctas);
    if (U == 0 || static_cast<int>(blockIdx.x) >= workers) return false;
    u = TcShare::begin(U, workers, blockIdx.x);
    end = TcShare::begin(U, workers, blockIdx.x + 1);
    return true;
  }
  // The warp that walks: the item that holds the share's first unit.
  __device__ __forceinline__ void find(const ScoreArgs& a, int lane) {
    g = static_cast<int>(u / total);
    const int64_t rem = u - g * total;
    int lo = 0, n = n_items;
    while (n > 1) {
      const int step = (n + 31) / 32;
      const uint32_t le = __ballot_sync(0xffffffffu, lane * step < n && __ldcg(a.plan.cum + lo + min(lane * step, n - 1)) <= rem);
      const int k = max(0, __popc(le) - 1);
      n = min(step, n - k * step);
      lo += k * step;
    }
    idx = lo;
    fresh = true;
  }
  // The next segment with key tiles.  cut: the record of a group that this CTA begins and others go on with.
  __device__ __forceinline__ bool next(const ScoreArgs& a, Seg& s, TreeCut& cut) {
    for (;;) {
      if (u >= end) return false;
      if (fresh) {
        const int4* p = reinterpret_cast<const int4*>(a.plan.items + idx);
        const int4 x = __ldcg(p), y = __ldcg(p + 1), z = __ldcg(p + 2);
        it = ScoreItem{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w, z.x, z.y, z.z, z.w, __ldcg(&a.plan.items[idx].ctx), {0, 0, 0}};
        at = __ldcg(a.plan.cum + idx);
        fresh = false;
      }
      const bool single = it.rows1 == 0;
      const int cost = tile_cost(a.t.pool, single);
      glen = cost * it.ktiles + kGroupUnits;
      const int x = static_cast<int>(u - g * total - at);
      const int len = static_cast<int>(min(static_cast<int64_t>(glen - x), end - u));
      const int kt = it.ktiles, kt0 = min(kt, (x + cost - 1) / cost), kt1 = min(kt, (x + len + cost - 1) / cost);
      const int64_t gbegin = u - x;
      s.g = g;
      u += len;
      if (x + len == glen) {
        if (++idx == n_items) {
          idx = 0;
          ++g;
        }
        fresh = true;
      }
      if (kt0 >= kt1) continue;   // the group's fixed units only
      s.req = it.req;
      s.prefix = it.prefix;
      s.ctx = it.ctx;
      s.tok0 = it.tok0;
      s.tok1 = it.tok0 + a.t.tile_tokens;
      s.rows0 = it.rows0;
      s.rows1 = it.rows1;
      s.kt0 = kt0;
      s.kt1 = kt1;
      s.slot = static_cast<int>(blockIdx.x) * 2 + (kt0 == 0 ? 1 : 0);
      s.flags = (single ? kSegSingle : 0) | (kt0 == 0 && kt1 == kt ? kSegWhole : 0);
      s.pre_tiles = it.pre_tiles;
      s.gap = it.gap;
      s.all_lo = it.all_lo;
      s.all_hi = it.all_hi;
      s.any_lo = it.any_lo;
      s.any_hi = it.any_hi;
      cut.count = 0;
      if (kt0 == 0 && kt1 < kt) {
        // The last tile's first unit names the last worker; the workers between each have a tile (a share is
        // longer than a tile).
        cut.count = TcShare::owner(U, workers, gbegin + static_cast<int64_t>(kt - 1) * cost) - static_cast<int>(blockIdx.x) + 1;
        cut.first = s.slot;
        cut.next = (static_cast<int>(blockIdx.x) + 1) * 2;
        cut.stride = 2;
        cut.tok_a = s.tok0;
        cut.rows_a = s.rows0;
        cut.tok_b = s.tok1;
        cut.rows_b = s.rows1;
        cut.f0 = 0;
        cut.g = s.g;
      }
      return true;
    }
  }
};

// The plan: items and their units before them, by one CTA (a warp an item, whose
// tokens' spans it reads; their number and total at the end of `cum`).
constexpr int kPlanThreads = 1024;
__device__ __forceinline__ int pairs_of(const ScoreReq& q, int tile_tokens) {
  return (q.n + 2 * tile_tokens - 1) / (2 * tile_tokens);
}
// Exclusive scan of x over the block's threads; `carry` is added and becomes the total.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t& carry, int64_t* scratch) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t inc = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += y;
  }
  if (lane == 31) scratch[warp] = inc;
  __syncthreads();
  int64_t w = scratch[lane];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += y;
  }
  const int64_t all = __shfl_sync(0xffffffffu, w, 31), before = warp ? __shfl_sync(0xffffffffu, w, (warp - 1) & 31) : 0;
  __syncthreads();
  const int64_t r = carry + before + inc - x;
  carry += all;
  return r;
}

// Requests' lengths and items' costs are kept in shared memory where they fit (kept
// requests, kept items).  Eight lanes take an item, and the code is short: it runs
// once, and much of its time is its first reading (382 items of 32 tokens: 17 us with
// a warp an item, four unrolled).
constexpr int kPlanReqs = 1024, kPlanItems = 2048, kPlanLanes = 8;
struct PlanReq {
  int t0, n, ctx, prefix, first;
};
__global__ void __launch_bounds__(kPlanThreads) score_plan_kernel(const ScoreArgs a) {
  __shared__ int64_t scratch[32];
  __shared__ PlanReq s_req[kPlanReqs];
  __shared__ int s_cost[kPlanItems];
  const int tid = threadIdx.x, sub = tid % kPlanLanes;
  const int tt = a.t.tile_tokens, R = a.t.num_reqs;
  griddep_wait();
  griddep_launch();
  const bool kept = R <= kPlanReqs;
  int* const first = a.plan.first;   // items before each request's
  // (Counted in 64 bits and cut: ranges of tokens that overlap could make more items than there is room for, or than 32
  // bits hold.  An item looked for below lies before the cut, where the sums are whole.)
  const int64_t most = a.plan.most;
  int64_t count = 0;
#pragma unroll 1
  for (int base = 0; base < R; base += kPlanThreads) {
    ScoreReq q{0, 0, 0, 0, false};
    int n = 0;
    if (base + tid < R) {
      q = score_req(a, base + tid);
      n = pairs_of(q, tt);
      if (q.bad) atomicOr(a.t.pool.err, PKV_DEVERR_POSITION);
    }
    const int f = static_cast<int>(min(block_scan(static_cast<int64_t>(n), count, scratch), most));
    if (kept) s_req[tid] = PlanReq{q.t0, q.n, q.ctx, q.prefix, f};
    else if (base + tid < R) first[base + tid] = f;
  }
  __syncthreads();
  const int n_items = static_cast<int>(min(count, most));
  const bool costs = n_items <= kPlanItems;
  const int rounds = (n_items + kPlanThreads / kPlanLanes - 1) / (kPlanThreads / kPlanLanes);
#pragma unroll 1
  for (int round = 0; round < rounds; ++round) {
    const int i = round * (kPlanThreads / kPlanLanes) + tid / kPlanLanes;
    const bool live = i < n_items;
    PlanReq q{0, 0, 0, 0, 0};
    int lo = 0;
    if (live) {
      int hi = R - 1;   // the last request with first <= i (those without items share their successor's)
#pragma unroll 1
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((kept ? s_req[mid].first : first[mid]) <= i) lo = mid; else hi = mid - 1;
      }
      if (kept) {
        q = s_req[lo];
      } else {
        const ScoreReq r = score_req(a, lo);
        q = PlanReq{r.t0, r.n, r.ctx, r.prefix, first[lo]};
      }
    }
    ScoreItem it;
    it.tok0 = q.t0 + (i - q.first) * 2 * tt;
    const int nt = live ? min(2 * tt, q.t0 + q.n - it.tok0) : 0;
    it.any_lo = INT_MAX;
    it.all_lo = 0;
    it.any_hi = -1;
    it.all_hi = INT_MAX;
    bool bad = false;
#pragma unroll 4
    for (int x = sub; x < nt; x += kPlanLanes) {
      const int p = __ldg(a.t.positions + it.tok0 + x);
      const KeySpan s = key_span(a, p, a.first_keys ? __ldg(a.first_keys + it.tok0 + x) : 0, q.prefix, q.ctx);
      it.any_lo = min(it.any_lo, s.lo);
      it.all_lo = max(it.all_lo, s.lo);
      it.any_hi = max(it.any_hi, s.hi);
      it.all_hi = min(it.all_hi, s.hi);
      bad |= p < 0 || p >= a.t.max_blocks * kBlockSize;
    }
    if (bad) atomicOr(a.t.pool.err, PKV_DEVERR_POSITION);
#pragma unroll
    for (int d = 1; d < kPlanLanes; d <<= 1) {
      it.any_lo = min(it.any_lo, __shfl_xor_sync(0xffffffffu, it.any_lo, d));
      it.all_lo = max(it.all_lo, __shfl_xor_sync(0xffffffffu, it.all_lo, d));
      it.any_hi = max(it.any_hi, __shfl_xor_sync(0xffffffffu, it.any_hi, d));
      it.all_hi = min(it.all_hi, __shfl_xor_sync(0xffffffffu, it.all_hi, d));
    }
    if (live && sub == 0) {
      it.req = lo;
      it.rows0 = min(tt, nt) * a.t.group;
      it.rows1 = max(0, nt - tt) * a.t.group;
      it.prefix = q.prefix;
      it.ctx = q.ctx;
      it.pre_tiles = (it.prefix + kNK - 1) / kNK;
      const int k0 = max(it.pre_tiles, it.any_lo / kNK);
      it.gap = k0 - it.pre_tiles;
      it.ktiles = max(1, it.pre_tiles + max(0, (it.any_hi + kNK) / kNK - k0));   // (one at least: its rows are written too)
      it.pad[0] = it.pad[1] = it.pad[2] = 0;
      const int cost = tile_cost(a.t.pool, it.rows1 == 0) * it.ktiles + kGroupUnits;
      a.plan.items[i] = it;
      if (costs) s_cost[i] = cost;
      else a.plan.cum[i] = cost;
    }
  }
  __syncthreads();
  int64_t total = 0;
  for (int base = 0; base < n_items; base += kPlanThreads) {
    const int i = base + tid;
    const int64_t x = i < n_items ? (costs ? s_cost[i] : a.plan.cum[i]) : 0;
    const int64_t c = block_scan(x, total, scratch);
    if (i < n_items) a.plan.cum[i] = c;
  }
  if (tid == 0) {
    a.plan.cum[a.plan.most] = total;
    a.plan.cum[a.plan.most + 1] = n_items;
  }
}

__device__ __forceinline__ float f16_value(uint32_t bits) {
  float f;
  asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %1;\n\tcvt.f32.f16 %0, x;\n\t}" : "=f"(f) : "r"(bits));
  return f;
}
// Adds them to the stored result of a row that sees them.
template <int D, bool F8>
__device__ __noinline__ void add_odd(const ScoreArgs& sa, const Seg& s, KeySpan span, const Odd* list, int count, uint16_t* o,
                                     float* part) {
  const TreeArgs& a = sa.t;
  auto add = [&](int d, float v) {
    if (part) part[d] += v;
    else o[d] = static_cast<uint16_t>(pack_bf16x2(bf16lo_to_f32(o[d]) + v, 0.f) & 0xffffu);
  };
  if (count <= kOddMost) {
    for (int i = 0; i < count; ++i) {
      const Odd x = list[i];
      if (x.key < s.prefix || (x.key >= span.lo && x.key <= span.hi))
        add(x.dim, F8 ? f16_value(x.bits) : bf16lo_to_f32(x.bits));
    }
    return;
  }
  // Too many to note: the blocks that were cleaned are looked at again.
  const int64_t Hkv = a.pool.num_kv_heads;
  const int32_t* bt = a.block_tables + static_cast<int64_t>(s.req) * a.max_blocks;
  for (int j = s.kt0; j < s.kt1; ++j) {
    const int tile = tile_at(j, s.pre_tiles, s.gap);
    const uint32_t dirty = blocks_needed(s, tile * kNK) & ~blocks_whole(s, tile * kNK);
    for (int x = 0; x < kBlkPerTile; ++x) {
      if (!((dirty >> x) & 1u)) continue;
      const int b = tile * kBlkPerTile + x, pb = __ldg(bt + b);
      if (pb < 0 || pb >= a.pool.num_blocks) continue;
      const uint32_t vis = span_bits(s.prefix, span, b * kBlockSize);
      for (int k = 0; k < kBlockSize; ++k) {
        if (!((vis >> k) & 1u)) continue;
        for (int d = 0; d < D; ++d) {
          const float v = pool_v<D, F8>(a.pool, pb * Hkv + s.g, k, d);
          if (!(fabsf(v) < CUDART_INF_F)) add(d, v);
        }
      }
    }
  }
}

// What the widening warps know of a tile: its first key, its blocks as bits
// (needed; to be cleaned; copied), and in lane l < 8 the exponent of block l.
struct CodeTile {
  int exp, key0, ctx, ring;
  uint32_t store, dirty, there;
  bool last;   // of the segment
};

// Widening warps, two (w = 0, 1) for K and two for V: blocks w, w + 2, ... of every
// tile, exponents asked for a tile ahead, the next block's codes while one is widened.
// A block's codes land on the second half of its own lines: the warp that has read
// them all may write.  Bound by one warp's chain of instructions; short code matters
// more than overlap (two blocks at once: 18 % slower, all four 45 %; piece by piece,
// 512 bytes each: 19 to 50 %).
template <int D, int KIND>
__device__ __forceinline__ bool widen_codes(const ScoreArgs& sa, uint8_t* smem, uint64_t* bars, const Seg* s_seg, int* s_odd,
                                            Odd* s_oddl, volatile int* s_abort, bool is_v, int w, int lane) {
  using S = TcSmem<D>;
  using B = typename ScoreSmem<D>::B;
  constexpr int kPer = D / 32;   // 16-byte pieces that a lane has of a block
  const TreeArgs& a = sa.t;
  const int Hkv = a.pool.num_kv_heads;
  Seg sg{};
  int r = -1, rel = 0, n = 0;                // segment, its next tile of n
  int ids_cur = -1, ids_next = -1, win = 0;
  const int32_t* bt_row = nullptr;
  bool ok = true;
  // Lane l holds block l of four key tiles, from tile kt0 + 4 from on.
  auto load_window = [&](int from) -> int {
    const int j = sg.kt0 + from * 4 + lane / kBlkPerTile;
    const int b = tile_at(j, sg.pre_tiles, sg.gap) * kBlkPerTile + lane % kBlkPerTile;
    return j < sg.kt1 && b < (sg.ctx + kBlockSize - 1) / kBlockSize ? __ldg(bt_row + b) : -1;
  };
  auto check_window = [&](int pb) -> int { return pb >= 0 && pb < a.pool.num_blocks ? pb : -1; };
  // The next tile; false: no more (or gave up).
  auto fetch = [&](CodeTile& t) -> bool {
    if (rel == n) {
      ++r;
      const int slot = r % kSegSlots;
      if (!(ok = mbar_wait_warp(&bars[B::kSegFull + slot], (r / kSegSlots) & 1, s_abort, a.wait_ns))) return false;
      sg = s_seg[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[B::kSegEmpty + slot]);
      if (sg.flags & kSegEnd) return false;
      rel = 0;
      n = sg.kt1 - sg.kt0;
      bt_row = a.block_tables + static_cast<int64_t>(sg.req) * a.max_blocks;
      win = 0;
      ids_cur = check_window(load_window(0));
      ids_next = load_window(1);
    }
    if ((rel >> 2) > win) {
      ++win;
      ids_cur = check_window(ids_next);
      ids_next = load_window(win + 1);
    }
    t.key0 = tile_at(sg.kt0 + rel, sg.pre_tiles, sg.gap) * kNK;
    t.ctx = sg.ctx;
    t.ring = r % kSegRing;
    t.store = blocks_needed(sg, t.key0);
    t.dirty = is_v ? t.store & ~blocks_whole(sg, t.key0) : 0u;
    const int pb = __shfl_sync(0xffffffffu, ids_cur, (rel & 3) * kBlkPerTile + (lane & 7));
    const bool has = lane < kBlkPerTile && ((t.store >> lane) & 1u) && pb >= 0;
    t.there = __ballot_sync(0xffffffffu, has);
    t.exp = 0;
    if (KIND == kPoolInt8 && has)   // (the kernel ahead may have written them)
      t.exp = (is_v ? a.pool.v_exps : a.pool.k_exps)[static_cast<int64_t>(pb) * Hkv + sg.g];
    t.last = ++rel == n;
    return true;
  };
  const int nst = is_v ? S::kVSt : S::kKSt;
  const int bar_landed = is_v ? B::kVLanded : B::kKLanded, bar_full = is_v ? B::kVFull : B::kKFull;
  CodeTile next{};
  bool more = fetch(next);
  for (int cnt = 0; more; ++cnt) {
    const CodeTile t = next;
    const int st = cnt % nst;
    uint8_t* const stage = smem + (is_v ? S::kOffV : S::kOffK) + st * S::kKV;
    if (!(ok = mbar_wait_warp(&bars[bar_landed + st], (cnt / nst) & 1, s_abort, a.wait_ns))) return false;
    auto load = [&](int b, uint4 (&v)[kPer]) {
      const bool there = (t.there >> b) & 1u;
#pragma unroll
      for (int u = 0; u < kPer; ++u)    // (a block that is not there becomes zero)
        v[u] = there ? *reinterpret_cast<const uint4*>(stage + b * S::kBlkBytes + S::kBlkBytes / 2 + (u * 32 + lane) * 16)
                     : make_uint4(0, 0, 0, 0);
    };
    uint4 v[kPer], ahead[kPer];
    load(w, v);
    more = fetch(next);
#pragma unroll 1
    for (int b = w; b < kBlkPerTile; b += kTeam) {
      if (b + kTeam < kBlkPerTile) load(b + kTeam, ahead);
      __syncwarp();   // block b's codes have been read
      if ((t.store >> b) & 1u) {
        const uint32_t f = exp_bf16x2(safe_exp(__shfl_sync(0xffffffffu, t.exp, b)) + kWidenShift);
        const bool clean = KIND == kPoolFp8 && ((t.dirty >> b) & 1u);
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
          const int at = u * 32 + lane, key = b * kBlockSize + at / (D / 16), c16 = at % (D / 16);
          const uint32_t c[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
          uint32_t o[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (KIND == kPoolInt8) {
              int8x4_to_bf16x4(c[k], o[2 * k], o[2 * k + 1]);
              o[2 * k] = mul_bf16x2(o[2 * k], f);
              o[2 * k + 1] = mul_bf16x2(o[2 * k + 1], f);
            } else {
              e4m3x4_to_f16x4(c[k], o[2 * k], o[2 * k + 1]);
            }
          }
          if (clean) {   // codes that are NaN, and what lies behind the context
            uint32_t bad = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) bad |= ((o[k] & 0x7c007c00u) + 0x04000400u) & 0x80008000u;
            if (bad) {
#pragma unroll
              for (int k = 0; k < 8; ++k) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const uint32_t h = (o[k] >> (16 * e)) & 0xffffu;
                  if ((h & 0x7c00u) != 0x7c00u) continue;
                  o[k] &= e ? 0x0000ffffu : 0xffff0000u;
                  if (t.key0 + key >= t.ctx) continue;
                  const int nth = atomicAdd(&s_odd[t.ring], 1);
                  if (nth < kOddMost)
                    s_oddl[t.ring * kOddMost + nth] =
                      Odd{t.key0 + key, static_cast<uint16_t>(c16 * 16 + 2 * k + e), static_cast<uint16_t>(h)};
                }
              }
            }
          }
          // Chunks 2 c16 and 2 c16 + 1 of the key's 128-byte lines (swizzled); lanes of the second half of a 256-byte
          // row store the odd one first, so that eight lanes meet eight banks.
          const int hf = (2 * c16) / 8, cw = (2 * c16) % 8, r8 = key % 8;
          uint8_t* line = stage + (key / 8) * S::kGS + hf * S::kHS + r8 * 128;
          const uint4 lo = make_uint4(o[0], o[1], o[2], o[3]), hi = make_uint4(o[4], o[5], o[6], o[7]);
          *reinterpret_cast<uint4*>(line + (((cw + hf) ^ r8) * 16)) = hf ? hi : lo;
          *reinterpret_cast<uint4*>(line + (((cw + 1 - hf) ^ r8) * 16)) = hf ? lo : hi;
        }
      }
#pragma unroll
      for (int u = 0; u < kPer; ++u) v[u] = ahead[u];
    }
    fence_proxy_async_smem();   // read by the tensor cores
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&bars[bar_full + st]);
      if (is_v && t.last) mbar_arrive(&bars[B::kVDone + t.ring]);
    }
    __syncwarp();
  }
  return ok;
}

__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  uint64_t p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(a), "f"(b));
  return p;
}
// (x0, x1) *= q0 + q1 x^2 + q2 x^4 + q3 x^6 element by element, in paired fp32 operations (q: each coefficient twice).
__device__ __forceinline__ void cap2(float& x0, float& x1, const uint64_t (&q)[4]) {
  asm("{\n\t.reg .b64 p, z, r;\n\tmov.b64 p, {%0, %1};\n\tmul.rn.f32x2 z, p, p;\n\tfma.rn.f32x2 r, %5, z, %4;\n\t"
      "fma.rn.f32x2 r, r, z, %3;\n\tfma.rn.f32x2 r, r, z, %2;\n\tmul.rn.f32x2 p, p, r;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(x0), "+f"(x1) : "l"(q[0]), "l"(q[1]), "l"(q[2]), "l"(q[3]));
}
// (x0, x1) = (x0, x1) * (q0 + q1 x^2 + q2 x^4 + q3 x^6) + (b, b).
__device__ __forceinline__ void cap2_add(float& x0, float& x1, const uint64_t (&q)[4], uint64_t b) {
  asm("{\n\t.reg .b64 p, z, r;\n\tmov.b64 p, {%0, %1};\n\tmul.rn.f32x2 z, p, p;\n\tfma.rn.f32x2 r, %5, z, %4;\n\t"
      "fma.rn.f32x2 r, r, z, %3;\n\tfma.rn.f32x2 r, r, z, %2;\n\tfma.rn.f32x2 p, p, r, %6;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(x0), "+f"(x1) : "l"(q[0]), "l"(q[1]), "l"(q[2]), "l"(q[3]), "l"(b));
}
__device__ __forceinline__ float min3f(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
struct CapPairs {
  uint64_t q[4];
  __device__ __forceinline__ explicit CapPairs(const ScoreArgs& a) {
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = pair_of(a.cap_q[i], a.cap_q[i]);
  }
};
// (x0, x1) = (x0, x1) * f + (b0, b1).
__device__ __forceinline__ void fma2v(float& x0, float& x1, float f, float b0, float b1) {
  asm("{\n\t.reg .b64 p, q, r;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %2};\n\tmov.b64 r, {%3, %4};\n\t"
      "fma.rn.f32x2 p, p, q, r;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(x0), "+f"(x1) : "f"(f), "f"(b0), "f"(b1));
}

// One row's scores of 32 keys in TMEM, to or from registers (tmem_wait_ld / tmem_wait_st follow).
__device__ __forceinline__ void tmem_ld32(uint32_t at, float (&v)[32]) {
  tmem_ld16(at, v);
  tmem_ld16(at + 16, v + 16);
}
__device__ __forceinline__ void tmem_st32(uint32_t at, const float (&v)[32]) {
  tmem_st16(at, v);
  tmem_st16(at + 16, v + 16);
}

// Waits for the thread's loads from TMEM; what uses v comes behind it.
__device__ __forceinline__ void tmem_wait_ld32(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                 "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                 "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
               :: "memory");
}

// A row's raw products with N keys (at `at` in TMEM; masked ones zero) to scores in log2 units; dpos: its position less
// the first of the keys; valid: the row is the segment's (others have no say in what the warp does).
template <bool BIAS, int N>
__device__ __forceinline__ void modify(float (&s)[N], uint32_t at, const ScoreArgs& a, float slope, int dpos, bool valid) {
  if (!BIAS || a.cap_out != 0.f) {
    const CapPairs k(a);
    float top[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < N; c += 2) top[(c >> 1) & 1] = max3f(top[(c >> 1) & 1], fabsf(s[c]), fabsf(s[c + 1]));
    if (__any_sync(0xffffffffu, valid && !(fmaxf(top[0], top[1]) < a.cap_small))) {
      // (rarely taken: short code, by way of TMEM)
#pragma unroll
      for (int c = 0; c < N; c += 16) tmem_st16(at + c, s + c);
      tmem_wait_st();
#pragma unroll 1
      for (int c0 = 0; c0 < N; c0 += 16) {
        float x[16];
        tmem_ld16(at + c0, x);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 16; ++c) x[c] = a.cap_out * tanh_any(x[c] * a.base);
        tmem_st16(at + c0, x);
      }
      tmem_wait_st();
#pragma unroll
      for (int c = 0; c < N; c += 16) tmem_ld16(at + c, s + c);
      tmem_wait_ld();
    } else {
#pragma unroll
      for (int c = 0; c < N; c += 2) cap2(s[c], s[c + 1], k.q);
    }
  }
  if constexpr (BIAS) {
    const float f = a.cap_out != 0.f ? 1.f : a.base;
    if (__all_sync(0xffffffffu, dpos >= N - 1)) {   // every key at or before the position: - slope (dpos - c)
      const float b = -slope * static_cast<float>(dpos);
#pragma unroll
      for (int c = 0; c < N; c += 2)
        fma2v(s[c], s[c + 1], f, fmaf(slope, static_cast<float>(c), b), fmaf(slope, static_cast<float>(c + 1), b));
    } else {
      const float d = static_cast<float>(dpos);
#pragma unroll
      for (int c = 0; c < N; ++c) s[c] = fmaf(-slope, fabsf(d - static_cast<float>(c)), s[c] * f);
    }
  }
}

// A row's masked scores, 32 keys at a time from TMEM and back; vis(c): the keys c .. c + 31 that it sees.  (Modified
// scores: masked ones become zero.)
template <bool MOD, class V>
__device__ __forceinline__ void mask_scores(uint32_t at_s, V&& vis) {
#pragma unroll 1
  for (int c0 = 0; c0 < kNK; c0 += 32) {
    float s[32];
    tmem_ld32(at_s + c0, s);
    tmem_wait_ld32(s);
    const uint32_t v = vis(c0);
#pragma unroll
    for (int c = 0; c < 32; ++c) s[c] = (v >> c) & 1u ? s[c] : MOD ? 0.f : -CUDART_INF_F;
    tmem_st32(at_s + c0, s);
  }
  tmem_wait_st();
}

template <int D, int KIND, int HOW>
__global__ void __launch_bounds__(kThreads<KIND>, 1)
score_tc_kernel(const ScoreArgs sa, const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
               const __grid_constant__ CUtensorMap tmap_q) {
  constexpr bool F8 = KIND == kPoolFp8;            // f16 operands
  constexpr bool MOD = HOW != kPlain, BIAS = HOW == kBiased;
  constexpr bool kCodes = KIND != kPoolBf16;       // stages are widened
  const TreeArgs& a = sa.t;
  using S = TcSmem<D>;
  using M = ScoreSmem<D>;
  using B = typename M::B;
  constexpr int kKSt = S::kKSt, kVSt = S::kVSt;
  extern __shared__ __align__(1024) uint8_t smem[];
  griddep_wait();
  griddep_launch();   // the merge may take its place and wait
  if (threadIdx.x == 0) a.cuts[blockIdx.x].count = 0;
  if ((smem_u32(smem) & 1023u) != 0) {   // swizzle atoms need 1024-byte alignment
    if (threadIdx.x == 0) atomicOr(a.pool.err, PKV_DEVERR_INTERNAL);
    return;
  }
  const unsigned err0 = *reinterpret_cast<volatile unsigned*>(a.pool.err);
  if (__syncthreads_or((err0 & PKV_DEVERR_TIMEOUT) != 0)) return;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + M::kOffBar);
  float2* s_ml = reinterpret_cast<float2*>(smem + M::kOffMl);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + M::kOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + M::kOffMisc + 8);
  int* s_odd = reinterpret_cast<int*>(smem + M::kOffMisc + 16);   // [kSegRing]: how many of a segment
  Odd* s_oddl = reinterpret_cast<Odd*>(smem + M::kOffOdd);
  Seg* s_seg = reinterpret_cast<Seg*>(smem + M::kOffSeg);   // [kSegSlots]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.group, Hkv = a.pool.num_kv_heads;
  Walk walk;
  if (!walk.begin(sa)) return;   // block-uniform
  if (threadIdx.x == 0) {
    for (int i = 0; i < kKSt; ++i) {
      mbar_init(&bars[B::kKFull + i], kCodes ? kTeam : 1);
      mbar_init(&bars[B::kKEmpty + i], 1);
      mbar_init(&bars[B::kKLanded + i], 1);
    }
    for (int i = 0; i < kVSt; ++i) {
      mbar_init(&bars[B::kVFull + i], kCodes ? kTeam : 1);
      mbar_init(&bars[B::kVEmpty + i], 1);
      mbar_init(&bars[B::kVLanded + i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars[B::kS + t], 1);
      mbar_init(&bars[B::kP + t], 128);
      mbar_init(&bars[B::kPv + t], 1);
      mbar_init(&bars[B::kQFull + t], 1);
      mbar_init(&bars[B::kQEmpty + t], 1);
      mbar_init(&bars[B::kQc + t], 128);
    }
    mbar_init(&bars[B::kMl], 128);
    mbar_init(&bars[B::kJoined], 128);
    mbar_init(&bars[B::kDrain], 1);
    for (int i = 0; i < kSegRing; ++i) mbar_init(&bars[B::kVDone + i], kCodes ? kTeam : 1);
    for (int i = 0; i < kSegSlots; ++i) {
      mbar_init(&bars[B::kSegFull + i], 1);
      mbar_init(&bars[B::kSegEmpty + i], kSegReaders<KIND>);
    }
    *s_abort = 0;
    fence_mbar_init();
  }
  if (warp == 8 && lane == 0) {
    prefetch_tmap(&tmap_q);
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
  }
  if (warp == 9) {
    tmem_alloc(s_tmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const uint32_t sQ = smem_u32(smem + S::kOffQ);
  const uint32_t sK = smem_u32(smem + S::kOffK);
  const uint32_t sV = smem_u32(smem + S::kOffV);
  // The CTA's r-th segment: waits until it is published, reads it and frees its slot.  false: gave up, or no more (`ok`
  // tells which).
  Seg sg;
  bool ok = true;
  auto take = [&](int r) -> bool {
    const int slot = r % kSegSlots;
    if (!(ok = mbar_wait_warp(&bars[B::kSegFull + slot], (r / kSegSlots) & 1, s_abort, a.wait_ns))) return false;
    sg = s_seg[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[B::kSegEmpty + slot]);
    return (sg.flags & kSegEnd) == 0;
  };

  // Registers: 384 x 168 (codes: 512 x 128) at the launch; the softmax warps' come from the others.
  if (warp >= 12) {
    // ------------------------------------------------------------ widening of codes
    if constexpr (kCodes) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsWiden));
      ok = widen_codes<D, KIND>(sa, smem, bars, s_seg, s_odd, s_oddl, s_abort, warp >= 12 + kTeam, warp % kTeam, lane);
      if (!ok) {
        if (lane == 0) atomicOr(a.pool.err, PKV_DEVERR_TIMEOUT);
        *s_abort = 1;
      }
    }
  } else if (warp >= 8) {
    if constexpr (kCodes) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsCodes));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == 8 || warp == 10) {
      // ------------------------------------------------------------ producers: warp 8 Q (and K), warp 10 V
      const bool is_k = warp == 8;
      const int nst = is_k ? kKSt : kVSt;
      uint8_t* const stages = smem + (is_k ? S::kOffK : S::kOffV);
      const int bar_full = is_k ? B::kKFull : B::kVFull, bar_empty = is_k ? B::kKEmpty : B::kVEmpty;
      const int bar_landed = is_k ? B::kKLanded : B::kVLanded;
      const CUtensorMap* const tm = is_k ? &tmap_k : &tmap_v;
      int cnt = 0;      // tiles issued in the launch
      int nq = 0;       // segments whose query tiles have been issued
      uint32_t landed_par = 0;
      for (int r = 0; ok && take(r); ++r) {
        if (is_k) {
          for (int t = 0; t < 2 && ok; ++t) {
            if (!(ok = mbar_wait_warp(&bars[B::kQEmpty + t], (r & 1) ^ 1, s_abort, a.wait_ns))) break;
            if (lane == 0) {
              if ((t ? sg.rows1 : sg.rows0) > 0) {
                mbar_arrive_expect_tx(&bars[B::kQFull + t], static_cast<uint32_t>(D * 2 * G * a.q_box_tokens));
                uint8_t* qt = smem + S::kOffQ + t * S::kQ;
#pragma unroll
                for (int hf = 0; hf < S::kHalves; ++hf)
                  tma_load_3d(qt + hf * (kTcRows * 128), &tmap_q, hf * 64, sg.g * G, t ? sg.tok1 : sg.tok0,
                              &bars[B::kQFull + t]);
              } else {
                mbar_arrive(&bars[B::kQFull + t]);
              }
            }
            __syncwarp();
          }
          if (!ok) break;
          nq = r + 1;
        }
        const int32_t* bt_row = a.block_tables + static_cast<int64_t>(sg.req) * a.max_blocks;
        const int nblk = (sg.ctx + kBlockSize - 1) / kBlockSize;
        // Lane l holds block 32 w + l of the segment (window w: four key tiles), the next window in flight.
        auto load_window = [&](int w) -> int {
          const int j = sg.kt0 + w * 4 + lane / kBlkPerTile;
          const int b = tile_at(j, sg.pre_tiles, sg.gap) * kBlkPerTile + lane % kBlkPerTile;
          return j < sg.kt1 && b < nblk ? __ldg(bt_row + b) : -1;
        };
        auto check_window = [&](int pb) -> int { return pb >= 0 && pb < a.pool.num_blocks ? pb : -1; };
        int win = 0;
        int ids_cur = check_window(load_window(0)), ids_next = load_window(1);
        // Lane l < 8: chunk index of key tile j's block l, or -1.
        auto block_chunk = [&](int j) -> int {
          const int rel = j - sg.kt0;
          if ((rel >> 2) != win) {
            win = rel >> 2;
            ids_cur = check_window(ids_next);
            ids_next = load_window(win + 1);
          }
          const int pb = __shfl_sync(0xffffffffu, ids_cur, (rel & 3) * kBlkPerTile + (lane & 7));
          const uint32_t need = blocks_needed(sg, tile_at(j, sg.pre_tiles, sg.gap) * kNK);
          return lane < kBlkPerTile && ((need >> lane) & 1u) && pb >= 0 ? pb * Hkv + sg.g : -1;
        };
        // bf16 V blocks that some row does not see whole: cleared of what they hold behind
        // the context, and of elements that are not finite, which are noted; blocks that
        // are not there (copied: have) become zero.  A lane has the 16-byte pieces
        // lane, lane + 32, ... of a block's rows, eight (four) loads under way.
        auto dirty_blocks = [&](int j, uint32_t have) -> uint32_t {
          const int key0 = tile_at(j, sg.pre_tiles, sg.gap) * kNK;
          return blocks_needed(sg, key0) & ~(blocks_whole(sg, key0) & have);
        };
        auto clean_v = [&](uint8_t* stage, int j, uint32_t have) {
          constexpr int kCh = S::kHalves * 8;   // 16-byte pieces of a key's row
          constexpr int kIt = kBlockSize * kCh / 32;
          const int key0 = tile_at(j, sg.pre_tiles, sg.gap) * kNK;
          const int ch = lane % kCh;
          for (uint32_t left = dirty_blocks(j, have); left; left &= left - 1) {
            const int b = __ffs(left) - 1;
            const bool there = (have >> b) & 1u;
            uint4* p[kIt];
            uint4 v[kIt];
#pragma unroll
            for (int i = 0; i < kIt; ++i) {
              const int key = b * kBlockSize + (lane + 32 * i) / kCh;
              p[i] = reinterpret_cast<uint4*>(stage + (key / 8) * S::kGS + (ch / 8) * S::kHS + (key % 8) * 128 +
                                              (((ch % 8) ^ (key % 8)) * 16));
              v[i] = there ? *p[i] : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < kIt; ++i) {
              const int key = key0 + b * kBlockSize + (lane + 32 * i) / kCh;
              if (!there || key >= sg.ctx) {
                *p[i] = make_uint4(0, 0, 0, 0);
                continue;
              }
              // An exponent of ones carries into the sign's place.
              constexpr uint32_t kExp = 0x7f807f80u, kOne = 0x00800080u;
              const uint32_t bad = (((v[i].x & kExp) + kOne) | ((v[i].y & kExp) + kOne) | ((v[i].z & kExp) + kOne) |
                                    ((v[i].w & kExp) + kOne)) & 0x80008000u;
              if (!bad) continue;
              uint16_t h[8];
              *reinterpret_cast<uint4*>(h) = v[i];
              for (int e = 0; e < 8; ++e) {
                if ((h[e] & (kExp & 0xffffu)) != (kExp & 0xffffu)) continue;
                const int n = atomicAdd(&s_odd[r % kSegRing], 1);
                if (n < kOddMost) s_oddl[(r % kSegRing) * kOddMost + n] = Odd{key, static_cast<uint16_t>(ch * 8 + e), h[e]};
                h[e] = 0;
              }
              *p[i] = *reinterpret_cast<uint4*>(h);
            }
          }
        };
        for (int j = sg.kt0; j < sg.kt1; ++j, ++cnt) {
          const int y = block_chunk(j);
          const int st = cnt % nst;
          const uint32_t have = __ballot_sync(0xffffffffu, y >= 0);
          if (!(ok = mbar_wait_warp(&bars[bar_empty + st], ((cnt / nst) & 1) ^ 1, s_abort, a.wait_ns))) break;
          // Test hook: CTA 0 never issues its first K tile, so that the issuer's bounded wait for it runs out.
          if (a.withhold == 2 && is_k && cnt == 0 && blockIdx.x == 0) continue;
          const bool clean = !kCodes && !is_k && dirty_blocks(j, have) != 0;
          uint64_t* bar = &bars[(clean || kCodes ? bar_landed : bar_full) + st];
          if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(__popc(have)) * (kBlockSize * D * (kCodes ? 1 : 2)));
          __syncwarp();
          uint8_t* stage = stages + st * S::kKV;
          if (y >= 0) {
            if constexpr (kCodes) tma_load_2d(stage + lane * S::kBlkBytes + S::kBlkBytes / 2, tm, 0, y * kBlockSize, bar);
            else if constexpr (D == 128) tma_load_4d(stage + lane * S::kBlkBytes, tm, 0, 0, 0, 2 * y, bar);
            else tma_load_2d(stage + lane * S::kBlkBytes, tm, 0, y * kBlockSize, bar);
          }
          if (clean) {
            const uint32_t par = (landed_par >> st) & 1u;
            landed_par ^= 1u << st;
            if (!mbar_wait_warp(bar, par, s_abort, a.wait_ns)) {
              (void)mbar_wait(bar, par, nullptr, a.wait_ns);   // let this tile's copies land
              ok = false;
              break;
            }
            clean_v(stage, j, have);
            fence_proxy_async_smem();   // read by the tensor cores
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[bar_full + st]);
          }
        }
        if (!ok) break;
        if constexpr (!kCodes) {
          __syncwarp();   // the notes are written
          if (!is_k && lane == 0) mbar_arrive(&bars[B::kVDone + r % kSegRing]);
          __syncwarp();
        }
      }
      if (!ok) {   // gave up: flag it and let copies already issued land
        if (lane == 0) atomicOr(a.pool.err, PKV_DEVERR_TIMEOUT);
        *s_abort = 1;
        for (int i = max(0, cnt - nst); i < cnt; ++i)
          (void)mbar_wait(&bars[(kCodes ? bar_landed : bar_full) + i % nst], (i / nst) & 1, nullptr, a.wait_ns);
        if (is_k && nq > 0) {
          for (int t = 0; t < 2; ++t) (void)mbar_wait(&bars[B::kQFull + t], (nq - 1) & 1, nullptr, a.wait_ns);
        }
      }
    } else if (warp == 9) {
      // ------------------------------------------------------------ MMA issuer
      constexpr uint32_t idesc_s = F8 ? make_idesc_f16(128, kNK, false) : make_idesc_bf16(128, kNK, false);
      constexpr uint32_t idesc_o = F8 ? make_idesc_f16(128, D, true) : make_idesc_bf16(128, D, true);
      const uint64_t dk = make_sdesc_sw128(sK, 16, S::kGS);
      const uint64_t dv = make_sdesc_sw128(sV, S::kHS, S::kGS);
      const uint64_t dqA = make_sdesc_sw128(sQ, 16, 1024), dqB = make_sdesc_sw128(sQ + S::kQ, 16, 1024);
      auto k_desc = [&](int gk) { return dk + static_cast<uint64_t>(((gk % kKSt) * S::kKV) >> 4); };
      auto v_desc = [&](int gv) { return dv + static_cast<uint64_t>(((gv % kVSt) * S::kKV) >> 4); };
      const uint32_t lead = elect_one();   // every lane runs the issue code, the elected one issues
      auto release = [&](int bar) { tc_commit_lead(lead, &bars[bar]); };
      // S of group t = (query tile) K^T
      auto issue_s = [&](int t, uint64_t dq, uint64_t kd) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const int hf = ks / 4, kk = ks % 4;
          tc_mma_lead(lead, tmem + t * kNK, dq + static_cast<uint64_t>((hf * (kTcRows * 128) + kk * 32) >> 4),
                      kd + static_cast<uint64_t>((hf * S::kHS + kk * 32) >> 4), idesc_s, ks > 0 ? 1u : 0u);
        }
        release(B::kS + t);
      };
      // O of group t (+)= P V
      // (of the tile's blocks that some row sees; acc: O has products of the segment)
      bool acc0 = false, acc1 = false;
      auto issue_pv = [&](int t, int j, uint64_t vd) {
        const uint32_t need = blocks_needed(sg, tile_at(sg.kt0 + j, sg.pre_tiles, sg.gap) * kNK);
        bool acc = t ? acc1 : acc0;
        if (need == 0xffu) {
#pragma unroll
          for (int ks = 0; ks < kNK / 16; ++ks)
            tc_mma_ts_lead(lead, tmem + kColO + t * 128, tmem + t * kNK + ks * 8,
                           vd + static_cast<uint64_t>((ks * 2 * S::kGS) >> 4), idesc_o, (acc || ks > 0) ? 1u : 0u);
          acc = true;
        } else {
          for (int ks = 0; ks < kNK / 16; ++ks) {
            if (!((need >> ks) & 1u)) continue;
            tc_mma_ts_lead(lead, tmem + kColO + t * 128, tmem + t * kNK + ks * 8,
                           vd + static_cast<uint64_t>((ks * 2 * S::kGS) >> 4), idesc_o, acc ? 1u : 0u);
            acc = true;
          }
        }
        if (t) acc1 = acc; else acc0 = acc;
      };
      constexpr int kQReady = F8 ? B::kQc : B::kQFull;
      int kc = 0, vc = 0;          // K / V tiles consumed
      uint32_t pc0 = 0, pc1 = 0;   // P phases of group A / B waited so far
      auto wait_k = [&] { return mbar_wait_warp(&bars[B::kKFull + kc % kKSt], (kc / kKSt) & 1, s_abort, a.wait_ns); };
      auto wait_v = [&] { return mbar_wait_warp(&bars[B::kVFull + vc % kVSt], (vc / kVSt) & 1, s_abort, a.wait_ns); };
      auto wait_p = [&](int t) {
        const bool o = mbar_wait_warp(&bars[B::kP + t], (t ? pc1 : pc0) & 1, s_abort, a.wait_ns);
        if (t) ++pc1; else ++pc0;
        return o;
      };
      for (int r = 0; ok && take(r); ++r) {
        const int n = sg.kt1 - sg.kt0;   // >= 1
        acc0 = acc1 = false;
        if (!(ok = mbar_wait_warp(&bars[kQReady], r & 1, s_abort, a.wait_ns) &&
                   mbar_wait_warp(&bars[kQReady + 1], r & 1, s_abort, a.wait_ns)))
          break;
        if (!(sg.flags & kSegSingle)) {
          // Both groups use every key tile: PV_A(j) S_A(j+1) PV_B(j) S_B(j+1).
          if (!(ok = wait_k())) break;
          tc_fence_after();
          issue_s(0, dqA, k_desc(kc));
          issue_s(1, dqB, k_desc(kc));
          if (n == 1) {
            release(B::kQEmpty);
            release(B::kQEmpty + 1);
          }
          release(B::kKEmpty + kc % kKSt);
          ++kc;
          for (int j = 0; ok && j < n; ++j) {
            if (!(ok = wait_v())) break;
            const uint64_t vd = v_desc(vc), kd = k_desc(kc);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (!(ok = wait_p(t))) break;
              tc_fence_after();
              issue_pv(t, j, vd);
              if (j == n - 1) release(B::kPv + t);
              if (j + 1 < n) {
                if (t == 0 && !(ok = wait_k())) break;
                issue_s(t, t ? dqB : dqA, kd);
                if (j + 1 == n - 1) release(B::kQEmpty + t);
              }
            }
            if (!ok) break;
            if (j + 1 < n) {
              release(B::kKEmpty + kc % kKSt);
              ++kc;
            }
            release(B::kVEmpty + vc % kVSt);
            ++vc;
          }
        } else {
          // Group j % 2 uses key tile j: S_A(0) S_B(1), then PV(j) S(j+2).
          release(B::kQEmpty + 1);   // no second query tile
          for (int j = 0; ok && j < 2 && j < n; ++j) {
            if (!(ok = wait_k())) break;
            tc_fence_after();
            issue_s(j, dqA, k_desc(kc));
            if (j == n - 1) release(B::kQEmpty);
            release(B::kKEmpty + kc % kKSt);
            ++kc;
          }
          for (int j = 0; ok && j < n; ++j) {
            const int t = j & 1;
            if (!(ok = wait_v() && wait_p(t))) break;
            tc_fence_after();
            if (t) issue_pv(1, j, v_desc(vc)); else issue_pv(0, j, v_desc(vc));
            if (j + 2 >= n) release(B::kPv + t);
            release(B::kVEmpty + vc % kVSt);
            ++vc;
            if (j + 2 < n) {
              if (!(ok = wait_k())) break;
              if (t) issue_s(1, dqA, k_desc(kc)); else issue_s(0, dqA, k_desc(kc));
              if (j + 2 == n - 1) release(B::kQEmpty);
              release(B::kKEmpty + kc % kKSt);
              ++kc;
            }
          }
        }
      }
      if (!ok) {
        if (lane == 0) atomicOr(a.pool.err, PKV_DEVERR_TIMEOUT);
        *s_abort = 1;
      }
      // Drain: every MMA issued has completed before TMEM is released.
      release(B::kDrain);
      (void)mbar_wait_warp(&bars[B::kDrain], 0, nullptr, a.wait_ns);
    } else if (warp == 11) {
      // ------------------------------------------------------------ scheduler
      walk.find(sa, lane);
      for (int r = 0;; ++r) {
        Seg s;
        TreeCut cut;
        const bool more = walk.next(sa, s, cut);
        if (more) {
          if (cut.count > 0 && lane == 0) a.cuts[blockIdx.x] = cut;
          // Blocks that some row sees and that are not there: flagged here, and only then looked for by the softmax warps.
          // The segment's blocks of the prefix, and those behind it between the first and the last key seen: the table may
          // hold anything for the others, pages freed behind a window for instance.  (No branch on what a load brings, so
          // that several are under way: with one the int8 new turns took 221 us, not 212.)
          const int32_t* bt_row = a.block_tables + static_cast<int64_t>(s.req) * a.max_blocks;
          bool gone = false;
          auto look = [&](int b0, int b1) {
            for (int b = b0 + lane; b < b1; b += 32) {
              const int pb = __ldg(bt_row + b);
              gone |= pb < 0 || pb >= a.pool.num_blocks;
            }
          };
          const int pblk = (s.prefix + kBlockSize - 1) / kBlockSize, t0 = s.kt0 * kBlkPerTile, t1 = s.kt1 * kBlkPerTile;
          const int skip = s.gap * kBlkPerTile;   // (0 if the prefix's last tile holds keys seen behind it)
          look(t0, min(t1, pblk));
          look(max(max(t0 + skip, pblk), s.any_lo / kBlockSize), min(t1 + skip, (s.any_hi + kBlockSize) / kBlockSize));
          if (__any_sync(0xffffffffu, gone)) {
            s.flags |= kSegMissing;
            if (lane == 0) atomicOr(a.pool.err, PKV_DEVERR_BLOCK_ID);
          }
        } else {
          s.flags = kSegEnd;
        }
        const int slot = r % kSegSlots;
        if (!(ok = mbar_wait_warp(&bars[B::kSegEmpty + slot], ((r / kSegSlots) & 1) ^ 1, s_abort, a.wait_ns))) break;
        if (lane == 0) {
          s_odd[r % kSegRing] = 0;   // (segment r - kSegRing is long done)
          s_seg[slot] = s;
          mbar_arrive(&bars[B::kSegFull + slot]);
        }
        __syncwarp();
        if (!more) break;
      }
      if (!ok) {
        if (lane == 0) atomicOr(a.pool.err, PKV_DEVERR_TIMEOUT);
        *s_abort = 1;
      }
    }
  } else {
    // ------------------------------------------------------------ softmax / epilogue of group X
    if constexpr (kCodes) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    const int X = (warp >> 2) & 1;
    const int row = threadIdx.x & 127;        // row within the tile (TMEM lane)
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t colS = X * kNK, colO = kColO + X * 128;
    const float sl2 = MOD ? 1.f : sa.base;   // what is left to multiply the scores with
    uint32_t sc = 0, pvc = 0, joins = 0;      // phases waited so far
    for (int r = 0; ok && take(r); ++r) {
      const int g = sg.g;
      const bool single = (sg.flags & kSegSingle) != 0, whole = (sg.flags & kSegWhole) != 0;
      const bool mine = X == 0 || !single;               // stores its rows
      const int nrows = X && !single ? sg.rows1 : sg.rows0;
      const int tok = X && !single ? sg.tok1 : sg.tok0;
      const bool valid = row < nrows;
      const int t_row = tok + (valid ? row / G : 0);
      // (asked for here, waited for where a tile is not seen whole)
      const int raw_pos = __ldg(a.positions + t_row), raw_first = sa.first_keys ? __ldg(sa.first_keys + t_row) : 0;
      const int pos = max(raw_pos, -1);
      float slope = 0.f;   // log2 units
      if (BIAS) slope = sa.slopes[g * G + row % G] * 1.4426950408889634f;
      const int step = single ? 2 : 1;
      const int n = sg.kt1 - sg.kt0;
      const int nt = single ? (n + 1 - X) / 2 : n;    // key tiles of this group
      if constexpr (F8) {
        // Operands of one MMA share a type: this thread's Q row to f16, in place (exact within f16's range).
        ok = mbar_wait_warp(&bars[B::kQFull + X], r & 1, s_abort, a.wait_ns);
        if (ok && mine) {
          uint8_t* qrow = smem + S::kOffQ + X * S::kQ + row * 128;
#pragma unroll
          for (int hf = 0; hf < S::kHalves; ++hf) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              uint4* q16 = reinterpret_cast<uint4*>(qrow + hf * (kTcRows * 128) + c * 16);
              uint4 v = *q16;
              v.x = pack_f16x2(bf16lo_to_f32(v.x), bf16hi_to_f32(v.x));
              v.y = pack_f16x2(bf16lo_to_f32(v.y), bf16hi_to_f32(v.y));
              v.z = pack_f16x2(bf16lo_to_f32(v.z), bf16hi_to_f32(v.z));
              v.w = pack_f16x2(bf16lo_to_f32(v.w), bf16hi_to_f32(v.w));
              *q16 = v;
            }
          }
          fence_proxy_async_smem();   // read by the tensor cores
        }
        mbar_arrive(&bars[B::kQc + X]);
      }
      // Blocks that are not there, as bits: window of 32 blocks (four key tiles) at a time.  (Where no row sees such a
      // block its keys are masked anyway.)
      const int32_t* bt_row = a.block_tables + static_cast<int64_t>(sg.req) * a.max_blocks;
      const int nblk = (sg.ctx + kBlockSize - 1) / kBlockSize;
      auto missing_of = [&](int w) -> uint32_t {
        const int j = sg.kt0 + w * 4 + lane / kBlkPerTile;
        const int b = tile_at(j, sg.pre_tiles, sg.gap) * kBlkPerTile + lane % kBlkPerTile;
        bool gone = false;
        if (b < nblk && j < sg.kt1) {
          const int pb = __ldg(bt_row + b);
          gone = pb < 0 || pb >= a.pool.num_blocks;
        }
        return __ballot_sync(0xffffffffu, gone);
      };
      const bool any_missing = (sg.flags & kSegMissing) != 0;
      uint32_t missing = any_missing ? missing_of(0) : 0u;
      float m = -CUDART_INF_F, l = 0.f;
      for (int i = 0; ok && i < nt; ++i) {
        const int rel = single ? 2 * i + X : i;
        const int key0 = tile_at(sg.kt0 + rel, sg.pre_tiles, sg.gap) * kNK;
        if (any_missing && rel > 0 && (rel & 3) < step) missing = missing_of(rel >> 2);
        const uint32_t gone = (missing >> ((rel & 3) * kBlkPerTile)) & 0xffu;
        const bool masked = gone != 0 || !seen_whole(sg, key0);
        const KeySpan span = masked ? key_span(sa, raw_pos, raw_first, sg.prefix, sg.ctx) : KeySpan{0, -1};
        if (!(ok = mbar_wait_warp(&bars[B::kS + X], sc & 1, s_abort, a.wait_ns))) break;
        ++sc;
        tc_fence_after();
        // The code is kept short: what is unrolled for 128 keys and more drives the rest out of the instruction cache
        // (the neighbouring SM's, too: its warps then waited two steps' time at each masked tile).  Masked scores are
        // rewritten in TMEM by a loop; modified ones are so 64 keys at a time, and P is made from there.
        const uint32_t at_s = tmem + lane_base + colS;
        auto vis = [&](int c0) {
          uint32_t v = span_bits(sg.prefix, span, key0 + c0);
          const uint32_t lost = gone >> (c0 / kBlockSize);
          if (lost & 1u) v &= 0xffff0000u;
          if (lost & 2u) v &= 0x0000ffffu;
          return v;
        };
        if (masked) mask_scores<MOD>(at_s, vis);
        constexpr int kAtOnce = MOD ? 64 : kNK;
        float s[kAtOnce], mx = -CUDART_INF_F;
        auto load = [&](int c0) {
#pragma unroll
          for (int c = 0; c < kAtOnce; c += 16) tmem_ld16(at_s + c0 + c, s + c);
          tmem_wait_ld();
        };
        // Small capped scores (no bias, seen whole): the cap is monotonic, so that the largest raw product names the
        // largest score, and the raw products become P in one go.
        bool straight = false;
        if constexpr (MOD && !BIAS) {
          if (!masked) {
            float hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              hi[k] = -CUDART_INF_F;
              lo[k] = CUDART_INF_F;
            }
#pragma unroll 1
            for (int c0 = 0; c0 < kNK; c0 += kAtOnce) {
              load(c0);
#pragma unroll
              for (int c = 0; c < kAtOnce; c += 2) {
                hi[(c >> 1) & 3] = max3f(hi[(c >> 1) & 3], s[c], s[c + 1]);
                lo[(c >> 1) & 3] = min3f(lo[(c >> 1) & 3], s[c], s[c + 1]);
              }
            }
            mx = fmaxf(fmaxf(hi[0], hi[1]), fmaxf(hi[2], hi[3]));
            const float mn = fminf(fminf(lo[0], lo[1]), fminf(lo[2], lo[3]));
            straight = !__any_sync(0xffffffffu, valid && !(fmaxf(mx, -mn) < sa.cap_small));
            if (straight) {
              float other = 0.f;
              cap2(mx, other, CapPairs(sa).q);
            } else {
              mx = -CUDART_INF_F;
            }
          }
        }
        if (!straight) {
          // (Short code again: 32 keys at a time where it is a detour.)
          constexpr int kStep = MOD && !BIAS ? 32 : kAtOnce;
#pragma unroll 1
          for (int c0 = 0; c0 < kNK; c0 += kStep) {
            float (&y)[kStep] = reinterpret_cast<float (&)[kStep]>(s);
#pragma unroll
            for (int c = 0; c < kStep; c += 16) tmem_ld16(at_s + c0 + c, y + c);
            tmem_wait_ld();
            if constexpr (MOD) {
              modify<BIAS, kStep>(y, at_s + c0, sa, slope, pos - key0 - c0, valid);
              if (masked) {   // (in words of 32)
#pragma unroll
                for (int w = 0; w < kStep; w += 32) {
                  const uint32_t v = vis(c0 + w);
#pragma unroll
                  for (int c = 0; c < 32; ++c) y[w + c] = (v >> c) & 1u ? y[w + c] : -CUDART_INF_F;
                }
              }
#pragma unroll
              for (int c = 0; c < kStep; c += 16) tmem_st16(at_s + c0 + c, y + c);
            }
            float mx8[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) mx8[k] = fmaxf(y[2 * k], y[2 * k + 1]);
#pragma unroll
            for (int c = 16; c < kStep; c += 2) mx8[(c >> 1) & 7] = max3f(mx8[(c >> 1) & 7], y[c], y[c + 1]);
            mx = max3f(mx, max3f(max3f(mx8[0], mx8[1], mx8[2]), max3f(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])), mx);
          }
        }
        if constexpr (MOD) tmem_wait_st();
        // Lazy rescaling: a row keeps its reference while the tile's maximum
        // stays within 2^kRescaleLog2 of it.  (Rows of the tile that are not the
        // segment's, other requests' or whatever the buffer held, have no say:
        // they would move the warp's references, and with them roundings.)
        const float m_tile = valid ? mx * sl2 : -CUDART_INF_F;
        const bool grow = __any_sync(0xffffffffu, m_tile > m + kRescaleLog2);
        const float m_new = grow ? fmaxf(m, m_tile) : m;
        const float neg_m = m_new == -CUDART_INF_F ? 0.f : -m_new;
        float rs0[4] = {0.f, 0.f, 0.f, 0.f}, rs1[4] = {0.f, 0.f, 0.f, 0.f};
        auto to_p = [&](auto capped) {
          const CapPairs k(sa);
          const uint64_t b2 = pair_of(neg_m, neg_m);
#pragma unroll 1
          for (int c0 = 0; c0 < kNK; c0 += kAtOnce) {
            if constexpr (MOD) load(c0);
#pragma unroll
            for (int cc = 0; cc < kAtOnce; cc += 32) {
              uint32_t pk[16];
#pragma unroll
              for (int c = cc; c < cc + 32; c += 2) {
                float x0 = s[c], x1 = s[c + 1];
                if constexpr (decltype(capped)::value) cap2_add(x0, x1, k.q, b2);
                else fma2(x0, x1, sl2, neg_m);
                const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
                add2(rs0[(c >> 1) & 3], rs1[(c >> 1) & 3], p0, p1);
                pk[(c - cc) / 2] = F8 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
              }
              tmem_st16(at_s + (c0 + cc) / 2, reinterpret_cast<const float*>(pk));
            }
          }
        };
        if constexpr (MOD && !BIAS) {
          if (straight) to_p(std::true_type{});
          else to_p(std::false_type{});
        } else {
          to_p(std::false_type{});
        }
        const float rsum = ((rs0[0] + rs1[0]) + (rs0[1] + rs1[1])) + ((rs0[2] + rs1[2]) + (rs0[3] + rs1[3]));
        const float alpha = grow && m != -CUDART_INF_F ? fast_exp2(m + neg_m) : 1.f;
        if (grow && i > 0) {   // O is complete: S was issued after the group's previous PV
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float o[32];
            tmem_ld32(tmem + lane_base + colO + c, o);
            tmem_wait_ld32(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= alpha;
            tmem_st32(tmem + lane_base + colO + c, o);
          }
        }
        l = l * alpha + rsum;
        m = m_new;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bars[B::kP + X]);
      }
      if (!ok) break;
      if (nt > 0) {
        if (!(ok = mbar_wait_warp(&bars[B::kPv + X], pvc & 1, s_abort, a.wait_ns))) break;
        ++pvc;
        tc_fence_after();
      }
      float wa = 1.f, wb = 0.f;   // weights of A's and B's accumulators
      bool join = false;
      if (single) {
        if (X == 1) {
          s_ml[row] = make_float2(m, l);
          tc_fence_before();
          mbar_arrive(&bars[B::kMl]);
          ok = mbar_wait_warp(&bars[B::kJoined], joins & 1, s_abort, a.wait_ns);
          ++joins;
          tc_fence_after();
          // Its rows are A's to store; the segment's flag is still to be passed.
          if (ok) ok = mbar_wait_warp(&bars[B::kVDone + r % kSegRing], (r / kSegRing) & 1, s_abort, a.wait_ns);
          continue;
        }
        if (!(ok = mbar_wait_warp(&bars[B::kMl], joins & 1, s_abort, a.wait_ns))) break;
        ++joins;
        tc_fence_after();
        join = n > 1;
        const float2 b = s_ml[row];
        if (join && b.y != 0.f) {   // l = 0: B saw no key of this row
          if (l == 0.f) {
            wa = 0.f;
            wb = 1.f;
            m = b.x;
            l = b.y;
          } else {
            const float mm = fmaxf(m, b.x);
            wa = fast_exp2(m - mm);
            wb = fast_exp2(b.x - mm);
            l = l * wa + b.y * wb;
            m = mm;
          }
        }
      }
      const float inv = l == 0.f ? 0.f : (F8 ? a.pool.v_scale : 1.f) / l;
      const float lse2 = l == 0.f ? -CUDART_INF_F : m + fast_log2(l);
      const int h = g * G + row % G;
      const int64_t prow = static_cast<int64_t>(sg.slot) * 256 + X * 128 + row;
      const int64_t orow = static_cast<int64_t>(t_row) * a.num_q_heads + h;
      uint4* dst_o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + orow * D);
      float4* dst_p = reinterpret_cast<float4*>(a.part_o + prow * D);
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32) {
        float ob[32];
        tmem_ld32(tmem + lane_base + colO + c0, ob);
        if (join) {   // warp-uniform
          float oc[32];
          tmem_ld16(tmem + lane_base + kColO + 128 + c0, oc);
          tmem_ld16(tmem + lane_base + kColO + 128 + c0 + 16, oc + 16);
          tmem_wait_ld();
          // (a weight of 0 stands for a state without keys: its columns may hold anything)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            ob[e] = (wa == 0.f ? 0.f : ob[e] * wa) + (wb == 0.f ? 0.f : oc[e] * wb);
        } else {
          tmem_wait_ld();
        }
        if (valid && l != 0.f) {
#pragma unroll
          for (int e = 0; e < 32; ++e) ob[e] *= inv;
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) ob[e] = 0.f;
        }
        if (valid) {
          if (whole) {
#pragma unroll
            for (int e = 0; e < 32; e += 16) {
              uint4 w0, w1;
              w0.x = pack_bf16x2(ob[e], ob[e + 1]);       w0.y = pack_bf16x2(ob[e + 2], ob[e + 3]);
              w0.z = pack_bf16x2(ob[e + 4], ob[e + 5]);   w0.w = pack_bf16x2(ob[e + 6], ob[e + 7]);
              w1.x = pack_bf16x2(ob[e + 8], ob[e + 9]);   w1.y = pack_bf16x2(ob[e + 10], ob[e + 11]);
              w1.z = pack_bf16x2(ob[e + 12], ob[e + 13]); w1.w = pack_bf16x2(ob[e + 14], ob[e + 15]);
              // A thread writes its own row: 32 bytes a store, a whole sector, where o allows it.
              if (a.o_align32) {
                st_global_v8(dst_o + (c0 + e) / 8, w0, w1);
              } else {
                dst_o[(c0 + e) / 8] = w0;
                dst_o[(c0 + e) / 8 + 1] = w1;
              }
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              const uint32_t* w = reinterpret_cast<const uint32_t*>(ob + e);
              st_global_v8(dst_p + (c0 + e) / 4, make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7]));
            }
          }
        }
      }
      if (single) {
        tc_fence_before();
        mbar_arrive(&bars[B::kJoined]);   // B's columns have been read
      }
      if (valid) {
        if (whole) {
          if (a.lse) a.lse[orow] = lse2 * 0.69314718055994530942f;
        } else {
          a.part_lse[prow] = lse2;
        }
      }
      if (!(ok = mbar_wait_warp(&bars[B::kVDone + r % kSegRing], (r / kSegRing) & 1, s_abort, a.wait_ns))) break;
      const int odd = s_odd[r % kSegRing];
      if (odd && valid)
        add_odd<D, F8>(sa, sg, key_span(sa, raw_pos, raw_first, sg.prefix, sg.ctx), s_oddl + (r % kSegRing) * kOddMost, odd,
                       static_cast<uint16_t*>(a.o) + orow * D, whole ? nullptr : a.part_o + prow * D);
    }
    if (!ok) {
      if (lane == 0) atomicOr(a.pool.err, PKV_DEVERR_TIMEOUT);
      *s_abort = 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, int KIND, int HOW>
int launch_m(const ScoreArgs& a, const CUtensorMap* tk, const CUtensorMap* tv, const CUtensorMap* tq, cudaStream_t s) {
  const int smem = ScoreSmem<D>::kTotal;
  const cudaError_t e = smem_attr_once<score_tc_kernel<D, KIND, HOW>>(smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(score_tc_kernel<D, KIND, HOW>, dim3(a.t.ctas), kThreads<KIND>, smem, s, a, *tk, *tv, *tq);
}
template <int D, int KIND>
int launch_k(const ScoreArgs& a, const CUtensorMap* tk, const CUtensorMap* tv, const CUtensorMap* tq, cudaStream_t s) {
  if (a.slopes) return launch_m<D, KIND, kBiased>(a, tk, tv, tq, s);
  return a.cap_out != 0.f ? launch_m<D, KIND, kCapped>(a, tk, tv, tq, s) : launch_m<D, KIND, kPlain>(a, tk, tv, tq, s);
}

}  // namespace

template <int D>
int launch_score_tc(const ScoreArgs& a, const void* tmk, const void* tmv, const void* tmq, void* stream) {
  const CUtensorMap* k = static_cast<const CUtensorMap*>(tmk);
  const CUtensorMap* v = static_cast<const CUtensorMap*>(tmv);
  const CUtensorMap* q = static_cast<const CUtensorMap*>(tmq);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_dependent(score_plan_kernel, dim3(1), kPlanThreads, 0, s, a);
  if (e != cudaSuccess) return e;
  const PoolView& p = a.t.pool;
  if (p.k_exps) return launch_k<D, kPoolInt8>(a, k, v, q, s);
  return p.elem_bytes == 1 ? launch_k<D, kPoolFp8>(a, k, v, q, s) : launch_k<D, kPoolBf16>(a, k, v, q, s);
}

}  // namespace pkv
