// Attention of drafted tokens over a cache (pkv_tree_attn): token t of request
// r sees key slot j of its request if j < prefix_r, or if j lies in
// [prefix_r, ctx_r) and bit j - prefix_r of the token's mask is set.
// Attention of tokens over listed blocks (pkv_sparse_attn): token t at position
// p sees the keys j <= p of the blocks of its list.
//
//   s_j = scale q . K_j,   O = sum_j exp(s_j - m) V_j / sum_j exp(s_j - m),
//   LSE = m + ln sum_j exp(s_j - m)       over the slots that the token sees;
//
// a token that sees none has O = 0 and LSE = -inf.
#include <cuda_runtime.h>
#include <math_constants.h>

#include <cstdint>

#include "internal.h"
#include "ops.h"
#include "ptx.cuh"
#include "rows.cuh"
#include "sched.cuh"

namespace pkv {
namespace {

// Rows kernel: a group has 16 query rows and one KV head; a unit is one block
// (or one entry of a list), and a group has kGroupUnits besides, for its start
// and end.  A request without keys keeps one empty block: its rows are written
// too.
//
// Two ways to share the line, chosen by the number of groups:
//   many groups   a worker is one warp: it walks its share alone, nothing waits
//                 for another warp, and a group has a few owners (kManyGroups
//                 groups a CTA: eight at most);
//   few groups    a worker is a CTA, whose four warps take a segment's blocks in
//                 turn and merge their states in shared memory: a quarter of the
//                 partials of long groups.
// Where groups are short, or about as many as there are SMs, CTAs of W warps take
// whole groups and there is nothing to merge: one launch less (one request, 28 rows,
// 15 blocks: 9.8 us with W = 12, 10.2 with 4, 11.2 with shares and a merge).
constexpr int kGroupUnits = 2;
using RowsShare = Share<4 * kRowWarps>;   // few groups: four blocks a warp at least
using WarpShare = Share<4>;
__device__ __forceinline__ int rows_tiles(const TreeReq& q, int group) {
  return static_cast<int>((static_cast<int64_t>(q.n) * group + kRowTile - 1) / kRowTile);
}
__device__ __forceinline__ int rows_blocks(const TreeReq& q) { return max(1, (q.ctx + kBlockSize - 1) / kBlockSize); }

// V elements that are not finite, added to a stored row that sees them (they
// were left out of the products); D / 32 dims a lane.
template <int D, bool F8>
__device__ __noinline__ void rows_add_odd(const TreeArgs& a, const int32_t* bt_row, int g, int prefix, int ctx, int b0,
                                          int end_blk, const uint32_t* mrow, uint16_t* o, float* part, int lane) {
  const int64_t Hkv = a.pool.num_kv_heads;
  for (int b = max(b0, prefix / kBlockSize); b < end_blk; ++b) {
    const uint32_t vis = tree_sees(prefix, ctx, mrow, a.mask_words, b * kBlockSize);
    const int pb = __ldg(bt_row + b);
    if (pb < 0 || pb >= a.pool.num_blocks) continue;
    for (int k = 0; k < kBlockSize; ++k) {
      if (!((vis >> k) & 1u)) continue;
      for (int d = lane; d < D; d += 32) {
        const float v = pool_v<D, F8>(a.pool, pb * Hkv + g, k, d);
        if (fabsf(v) < CUDART_INF_F) continue;
        if (part) part[d] += v;
        else o[d] = static_cast<uint16_t>(pack_bf16x2(bf16lo_to_f32(o[d]) + v, 0.f) & 0xffffu);
      }
    }
  }
}

// A worker walks its share of the line, segment by segment: blocks (list
// entries) [b0, b1) of one group.  Every warp has its own ring of copies and its
// own state.  Bound by the reads of K and V (lists of 128 bf16 blocks of 8 KB for 256
// groups: 49 us, 5.5 TB/s), for FP8 by the fixed latencies of conversions and
// products (24 trees of 5 to 27 nodes over 300 to 4000 tokens, 40 heads: 88 us, 460 MB
// from HBM, 100 MB of them the second row tiles'); equal shares matter more than the
// work per block (lists of 128 blocks for 256 groups took 62 us in clusters of
// two CTAs: 512 CTAs leave a second, nearly empty wave; 46 us here).
template <int D, bool F8, bool LIST, int W>
__global__ void __launch_bounds__(32 * W, 12 / W)
rows_kernel(const TreeArgs a) {
  using S = RowsSmem<D, F8, W>;
  constexpr bool kAlways = W != kRowWarps;   // always whole groups
  extern __shared__ uint8_t raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  __shared__ int64_t scratch[2 * W];
  __shared__ int s_odd;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.group, Hkv = a.pool.num_kv_heads;
  griddep_wait();
  griddep_launch();   // the merge may take its place and wait
  if (!kAlways && tid < W) a.cuts[cut_record(blockIdx.x, W, true, tid)].count = 0;
  if (tid == 0) s_odd = 0;
  if (LIST && blockIdx.x == 0 && tid == 0) check_cu(a.cu_q_lens, a.num_reqs, a.num_tokens, a.pool.err);
  const int rtiles = (G + kRowTile - 1) / kRowTile;   // LIST: row tiles of a token's group
  auto groups = [&](const TreeReq& q) { return static_cast<int64_t>(rows_tiles(q, G)) * Hkv; };
  auto units = [&](const TreeReq& q) { return groups(q) * (rows_blocks(q) + kGroupUnits); };
  // The shares: of this warp if there are many groups, of the CTA otherwise.
  const int warp_id = static_cast<int>(blockIdx.x) * W + warp, many_from = a.form.many_groups;
  TreeShare sh;
  bool solo;
  int64_t left = 0;   // whole groups: how many the CTA still has to do
  const bool all_whole = kAlways || a.form.whole;
  if (all_whole) {
    int64_t n[1], off[1];
    int reqs[1];
    auto share = [&](int64_t len, int64_t& first) {
      const int C = static_cast<int>(min(len, static_cast<int64_t>(a.ctas)));
      const bool has = static_cast<int>(blockIdx.x) < C;
      first = has ? RowsShare::begin(len, C, blockIdx.x) : 0;
      left = has ? RowsShare::begin(len, C, blockIdx.x + 1) - first : 0;
    };
    sh = TreeShare{0, 0, 0, 0, 1, 0};
    solo = false;
    int64_t first;
    if constexpr (LIST) {
      const int tokens = min(max(__ldg(a.cu_q_lens + a.num_reqs), 0), a.num_tokens);
      share(static_cast<int64_t>(tokens) * Hkv * rtiles, first);
      sh.u = first * (a.top_k + kGroupUnits);
    } else {
      tree_scan<32 * W, 1, 1>(
          a, scratch, n, reqs, off, [&](const TreeReq& q, int) { return groups(q); },
          [&](const int64_t (&len)[1], int, int& line, int64_t& unit) {
            share(len[0], first);
            line = 0;
            unit = left > 0 ? first : -1;
          });
      sh.req = reqs[0];
      if (left > 0) sh.off = off[0] * (rows_blocks(tree_req(a, sh.req)) + kGroupUnits);
    }
    sh.end = left > 0 ? INT64_MAX : 0;
    if (left == 0) sh.u = 0;
  } else if constexpr (kAlways) {
  } else if constexpr (LIST) {
    // Every token of the requests has top_k units a group.
    const int tokens = min(max(__ldg(a.cu_q_lens + a.num_reqs), 0), a.num_tokens);
    const int64_t n = static_cast<int64_t>(tokens) * Hkv * rtiles;
    sh = TreeShare{n * (a.top_k + kGroupUnits), 0, 0, 0, 1, 0};
    solo = n >= many_from;
    sh.workers = solo ? WarpShare::workers(sh.U, a.ctas * W) : RowsShare::workers(sh.U, a.ctas);
    const int w = solo ? warp_id : static_cast<int>(blockIdx.x);
    if (sh.U > 0 && w < sh.workers) {
      sh.u = RowsShare::begin(sh.U, sh.workers, w);
      sh.end = RowsShare::begin(sh.U, sh.workers, w + 1);
    }
  } else {
    // Line 0: units; line 1: groups (for their number alone).  Probe p: where warp p's share begins.
    int64_t U[2], off[W];
    int reqs[W];
    auto share = [&](const int64_t (&len)[2], int p, TreeShare& t) {
      const bool alone = len[1] >= many_from;
      t.U = len[0];
      t.workers = alone ? WarpShare::workers(len[0], a.ctas * W) : RowsShare::workers(len[0], a.ctas);
      const int w = alone ? static_cast<int>(blockIdx.x) * W + p : static_cast<int>(blockIdx.x);
      t.u = t.end = 0;
      if (len[0] > 0 && w < t.workers) {
        t.u = RowsShare::begin(len[0], t.workers, w);
        t.end = RowsShare::begin(len[0], t.workers, w + 1);
      }
    };
    tree_scan<32 * W, 2, W>(
        a, scratch, U, reqs, off, [&](const TreeReq& q, int line) { return line == 0 ? units(q) : groups(q); },
        [&](const int64_t (&len)[2], int p, int& line, int64_t& unit) {
          TreeShare t;
          share(len, p, t);
          line = 0;
          unit = t.u < t.end ? t.u : -1;
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
  const float sl2 = F8 ? a.scale_log2 * a.pool.k_scale : a.scale_log2;
  int req = LIST ? 0 : sh.req;
  TreeReq rq{0, 0, 0, 0, false};
  if constexpr (!LIST) rq = tree_req(a, req);
  for (; sh.u < sh.end; ) {
    if (all_whole && left-- <= 0) return;
    int kblk, x, g, row0, nrows, pos = 0;   // blocks of the group, its first unit here, its rows
    const int32_t* list = nullptr;
    if constexpr (LIST) {
      kblk = a.top_k;
      const int64_t grp = sh.u / (kblk + kGroupUnits);
      x = static_cast<int>(sh.u - grp * (kblk + kGroupUnits));
      const int64_t th = grp / rtiles;
      row0 = static_cast<int>(grp - th * rtiles) * kRowTile;
      g = static_cast<int>(th % Hkv);
      rq.t0 = static_cast<int>(th / Hkv);
      nrows = min(kRowTile, G - row0);
      req = req_of_warp(a.cu_q_lens, a.num_reqs, rq.t0, lane);
      pos = __ldg(a.positions + rq.t0);
      if (lane == 0 && req >= 0 && (pos < 0 || pos >= a.max_blocks * kBlockSize)) atomicOr(a.pool.err, PKV_DEVERR_POSITION);
      list = a.sel + th * a.top_k;
    } else {
      for (int64_t n = units(rq); sh.off >= n; n = units(rq)) {   // the next request with work (there is one)
        sh.off -= n;
        if (++req >= a.num_reqs) return;
        rq = tree_req(a, req);
      }
      kblk = rows_blocks(rq);
      const int glen = kblk + kGroupUnits;
      const int grp = static_cast<int>(sh.off / glen);
      x = static_cast<int>(sh.off - static_cast<int64_t>(grp) * glen);
      const int ntile = rows_tiles(rq, G);
      g = grp / ntile;
      row0 = (grp - g * ntile) * kRowTile;
      nrows = min(kRowTile, rq.n * G - row0);
    }
    const int len = static_cast<int>(min(static_cast<int64_t>(kblk + kGroupUnits - x), sh.end - sh.u));
    const int64_t gbegin = sh.u - x;
    sh.u += len;
    sh.off += len;
    const int b0 = x, b1 = min(x + len, kblk);
    // The group's fixed units only, or a token that belongs to no request (its rows are left alone).
    if (b0 >= b1 || (LIST && req < 0)) continue;
    // Rows g' and g' + 8 of this thread.
    const int ra = lane >> 2, rb = ra + 8;
    auto q_row = [&](int rr) -> const uint16_t* {
      if (rr >= nrows) return nullptr;
      const int f = row0 + rr;
      return static_cast<const uint16_t*>(a.q) +
             (static_cast<int64_t>(rq.t0 + f / G) * a.num_q_heads + g * G + f % G) * D;
    };
    auto mask_row = [&](int rr) {
      return a.mask + static_cast<int64_t>(rq.t0 + (row0 + min(rr, nrows - 1)) / G) * a.mask_words;
    };
    const int end_blk = LIST ? b1 : min(b1, (rq.ctx + kBlockSize - 1) / kBlockSize);
    const int live = max(0, end_blk - b0);
    const int nb_w = live > wi ? (live - wi + wn - 1) / wn : 0;
    const int32_t* bt_row = a.block_tables + static_cast<int64_t>(req) * a.max_blocks;
    // Windows of 32 iterations: lane l holds the chunk of iteration base + l (-1: no such block) and the block's index
    // in the request; `there` and `plain` are the window's iterations that have a block, and those whose block every
    // row sees whole, as bits.  (A shuffle for each of these in every iteration took 300 of a pair's 3900 cycles.)
    auto load_ids = [&](int base, int& blk) -> int {
      const int i = base + lane;
      blk = -1;
      if (i >= nb_w) return -1;
      blk = b0 + wi + wn * i;
      if constexpr (LIST) {
        blk = __ldcg(list + blk);   // (the kernel ahead may have picked it)
        if (blk < 0 || pos < 0 || blk > (pos >> 4)) return -1;   // padding, or a block that the token does not see
        if (blk >= a.max_blocks) {
          atomicOr(a.pool.err, PKV_DEVERR_POSITION);
          return -1;
        }
      }
      const int pb = __ldg(bt_row + blk);
      if (pb < 0 || pb >= a.pool.num_blocks) {
        atomicOr(a.pool.err, PKV_DEVERR_BLOCK_ID);
        return -1;
      }
      return pb * Hkv + g;
    };
    int blk_cur, blk_next, win = 0;
    int chunk_cur = load_ids(0, blk_cur), chunk_next = load_ids(32, blk_next);
    uint32_t there, plain;
    auto look = [&] {
      const bool has = chunk_cur >= 0;
      there = __ballot_sync(0xffffffffu, has);
      const int blk = LIST ? blk_cur : b0 + wi + wn * (32 * win + lane);
      plain = __ballot_sync(0xffffffffu, has && (LIST ? pos - blk * kBlockSize >= kBlockSize - 1
                                                      : (blk + 1) * kBlockSize <= rq.prefix));
    };
    look();
    RowTile<D, F8> rt;
    rt.load(q_row(ra), q_row(rb), lane);   // asked for before the first blocks
    // One group of copies an iteration (an empty one for a block that is not there, and behind the last).
    auto copy = [&](int j) {
      const int chunk = __shfl_sync(0xffffffffu, (j >> 5) == win ? chunk_cur : chunk_next, j & 31);
      if (j < nb_w && chunk >= 0)
        rows_copy<D, F8>(a.pool, my_ring + static_cast<uint32_t>(j) % S::kStages * S::kStage, chunk, lane);
      cp_commit();
    };
    for (int j = 0; j < S::kStages; ++j) copy(j);
    rt.start();
    const uint32_t* m0 = LIST ? nullptr : mask_row(ra);
    const uint32_t* m1 = LIST ? nullptr : mask_row(rb);
    for (int i = 0; i < nb_w; ++i) {
      if ((i & 31) == 0 && i > 0) {
        chunk_cur = chunk_next;
        blk_cur = blk_next;
        win = i >> 5;
        look();
        chunk_next = load_ids(i + 32, blk_next);
      }
      const uint32_t bit = 1u << (i & 31);
      const uint32_t kb = my_ring + static_cast<uint32_t>(i) % S::kStages * S::kStage;
      // FP8: two blocks at once where both are seen whole.  Half the shuffles and votes, and two chains of products
      // and conversions to interleave (the warps wait for fixed latencies most of the time).
      if (F8 && (plain & bit) && (plain & (bit << 1)) && i + 1 < nb_w) {
        cp_wait<S::kStages - 2>();
        __syncwarp();
        const uint32_t kb1 = my_ring + static_cast<uint32_t>(i + 1) % S::kStages * S::kStage;
        rt.template block<kMaskNone, 2>(kb, kb + S::kChunk, sl2, 0u, 0u, lane, kb1, kb1 + S::kChunk);
        __syncwarp();   // the stages have been read
        copy(i + S::kStages);
        ++i;
      } else {
        cp_wait<S::kStages - 1>();
        __syncwarp();
        if (plain & bit) {
          rt.template block<kMaskNone>(kb, kb + S::kChunk, sl2, 0u, 0u, lane);
        } else if (there & bit) {
          if constexpr (LIST) {
            const int seen = pos - __shfl_sync(0xffffffffu, blk_cur, i & 31) * kBlockSize + 1;   // keys up to the position
            rt.template block<kMaskKeys>(kb, kb + S::kChunk, sl2, (1u << seen) - 1u, (1u << seen) - 1u, lane);
          } else {
            const int key0 = (b0 + wi + wn * i) * kBlockSize;
            rt.template block<kMaskRows>(kb, kb + S::kChunk, sl2, tree_sees(rq.prefix, rq.ctx, m0, a.mask_words, key0),
                                         tree_sees(rq.prefix, rq.ctx, m1, a.mask_words, key0), lane);
          }
        }
        __syncwarp();
      }
      copy(i + S::kStages);
    }
    const bool whole = b0 == 0 && b1 == kblk;
    const int64_t slot = (2 * static_cast<int64_t>(worker) + (b0 == 0 ? 1 : 0)) * kRowTile;
    auto out_row = [&](int rr) {   // row index of O and LSE
      const int f = row0 + rr;
      return static_cast<int64_t>(rq.t0 + f / G) * a.num_q_heads + g * G + f % G;
    };
    if (solo) {
      float l0, l1;
      rt.total_l(l0, l1);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int rr = i ? rb : ra;
        const float L = i ? l1 : l0;
        const float f = L == 0.f ? 0.f : (F8 ? a.pool.v_scale : 1.f) / L;
        const float lse2 = L == 0.f ? -CUDART_INF_F : rt.m[i] + fast_log2(L);
        if (rr < nrows) {
          if (whole) {
            const int64_t at = out_row(rr);
            rt.put_bf16(static_cast<uint16_t*>(a.o) + at * D, i, f, lane);
            if ((lane & 3) == 0 && a.lse) a.lse[at] = lse2 * 0.69314718055994530942f;
          } else {
            rt.put_f32(a.part_o + (slot + rr) * D, i, f, lane);
            if ((lane & 3) == 0) a.part_lse[slot + rr] = lse2;
          }
        }
      }
      if (!LIST && __any_sync(0xffffffffu, rt.odd)) {
        __syncwarp();
        for (int rr = 0; rr < nrows; ++rr)
          rows_add_odd<D, F8>(a, bt_row, g, rq.prefix, rq.ctx, b0, end_blk, mask_row(rr),
                              static_cast<uint16_t*>(a.o) + out_row(rr) * D,
                              whole ? nullptr : a.part_o + (slot + rr) * D, lane);
      }
    } else {
      if (!LIST && rt.odd) s_odd = 1;
      __syncthreads();   // every warp's ring has drained
      // Merge the warps' states: [warp][16][D + 4] floats over the ring.
      float* mbuf = reinterpret_cast<float*>(ring);
      rt.store(mbuf + warp * kRowTile * S::kMergeRow, lane);
      __syncthreads();
      constexpr int kDims = D / 8;   // dims of a thread's part of a row
      const int rr = tid >> 3, d0 = (tid & 7) * kDims;
      if (rr < nrows) {
        float M = -CUDART_INF_F, L = 0.f, acc[kDims];
#pragma unroll
        for (int d = 0; d < kDims; ++d) acc[d] = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) M = fmaxf(M, mbuf[(w * kRowTile + rr) * S::kMergeRow + D]);
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float* src = mbuf + (w * kRowTile + rr) * S::kMergeRow;
          if (src[D + 1] == 0.f) continue;   // the warp saw no key of this row (a NaN score leaves m, not l, as it was)
          const float f = fast_exp2(src[D] - M);
          L = fmaf(f, src[D + 1], L);
#pragma unroll
          for (int d = 0; d < kDims; ++d) acc[d] = fmaf(f, src[d0 + d], acc[d]);
        }
        const float inv = L == 0.f ? 0.f : (F8 ? a.pool.v_scale : 1.f) / L;
#pragma unroll
        for (int d = 0; d < kDims; ++d) acc[d] *= inv;
        const float lse2 = L == 0.f ? -CUDART_INF_F : M + fast_log2(L);
        if (whole) {
          const int64_t at = out_row(rr);
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + at * D + d0);
#pragma unroll
          for (int d = 0; d < kDims; d += 8)
            dst[d / 8] = make_uint4(pack_bf16x2(acc[d], acc[d + 1]), pack_bf16x2(acc[d + 2], acc[d + 3]),
                                    pack_bf16x2(acc[d + 4], acc[d + 5]), pack_bf16x2(acc[d + 6], acc[d + 7]));
          if (d0 == 0 && a.lse) a.lse[at] = lse2 * 0.69314718055994530942f;
        } else {
          float4* dst = reinterpret_cast<float4*>(a.part_o + (slot + rr) * D + d0);
#pragma unroll
          for (int d = 0; d < kDims; d += 4) dst[d / 4] = make_float4(acc[d], acc[d + 1], acc[d + 2], acc[d + 3]);
          if (d0 == 0) a.part_lse[slot + rr] = lse2;
        }
      }
      __syncthreads();   // the ring and the flags are free again, the rows stored
      if (!LIST && s_odd) {
        for (int r2 = warp; r2 < nrows; r2 += W)
          rows_add_odd<D, F8>(a, bt_row, g, rq.prefix, rq.ctx, b0, end_blk, mask_row(r2),
                              static_cast<uint16_t*>(a.o) + out_row(r2) * D,
                              whole ? nullptr : a.part_o + (slot + r2) * D, lane);
        __syncthreads();
        if (tid == 0) s_odd = 0;
      }
      __syncthreads();
    }
    if (b0 == 0 && b1 < kblk && lane == 0 && (solo || warp == 0)) {   // the group's first part: its other owners follow
      // (the last block names the last owner; those between each have a block, a share being longer than the fixed units)
      const int c1 = RowsShare::owner(sh.U, sh.workers, gbegin + kblk - 1);
      TreeCut& cut = a.cuts[cut_record(blockIdx.x, W, solo, warp)];
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

// One warp per kRows rows of a cut group: merges their partials in the workers'
// order with a running maximum, kBatch partials of each row in flight.
//   M = max LSE_c, LSE = M + log2 sum 2^(LSE_c - M), O = sum 2^(LSE_c - LSE) O_c
// Bound by the latency of its loads (the record, then the partials): 304 cuts of up
// to 512 rows in 19 us by itself, most of them read from L2; 1824 of 16 rows in 10.
template <int D, int SlotRows, int kRows, int kBatch>
__global__ void __launch_bounds__(256) tree_merge_kernel(const TreeArgs a) {
  constexpr int kDPL = D / 32;
  griddep_wait();   // the attention kernel's writes
  const int lane = threadIdx.x & 31;
  const int row0 = (static_cast<int>(blockIdx.y) * 8 + (threadIdx.x >> 5)) * kRows;
  const int4* rec = reinterpret_cast<const int4*>(a.cuts + blockIdx.x);
  const int4 s = __ldcg(rec);
  const int4 tk = __ldcg(rec + 1), fg = __ldcg(rec + 2);
  if (s.x < 2) return;
  if (SlotRows >= 128 && (__ldcg(a.pool.err) & PKV_DEVERR_TIMEOUT)) return;   // (partials may be incomplete)
  // The rows of a warp lie in one tile (kRows divides 128).
  const int tok = row0 < 128 ? tk.x : tk.z, rows = row0 < 128 ? tk.y : tk.w, i0 = row0 & 127;
  if (i0 >= rows) return;
  auto slot_row = [&](int c) {
    return static_cast<int64_t>(c == 0 ? s.y : s.z + (c - 1) * s.w) * SlotRows + row0;
  };
  float M[kRows], sum[kRows], acc[kRows][kDPL];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    M[k] = -CUDART_INF_F;
    sum[k] = 0.f;
#pragma unroll
    for (int d = 0; d < kDPL; ++d) acc[k][d] = 0.f;
  }
  for (int c0 = 0; c0 < s.x; c0 += kBatch) {
    float e[kBatch][kRows], v[kBatch][kRows][kDPL];
#pragma unroll
    for (int c = 0; c < kBatch; ++c) {
      const int64_t at = slot_row(c0 + c);
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        e[c][k] = -CUDART_INF_F;
        if (c0 + c >= s.x) continue;
        const int64_t r = at + (i0 + k < rows ? k : 0);
        e[c][k] = __ldcg(a.part_lse + r);
        const float* src = a.part_o + r * D + lane * kDPL;
        if constexpr (kDPL == 4) {
          const float4 x = __ldcg(reinterpret_cast<const float4*>(src));
          v[c][k][0] = x.x; v[c][k][1] = x.y; v[c][k][2] = x.z; v[c][k][3] = x.w;
        } else {
          const float2 x = __ldcg(reinterpret_cast<const float2*>(src));
          v[c][k][0] = x.x; v[c][k][1] = x.y;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      float m = M[k];
#pragma unroll
      for (int c = 0; c < kBatch; ++c) m = fmaxf(m, e[c][k]);
      if (m > M[k]) {
        const float f = M[k] == -CUDART_INF_F ? 1.f : fast_exp2(M[k] - m);   // (nothing, or NaN, summed so far)
        sum[k] *= f;
#pragma unroll
        for (int d = 0; d < kDPL; ++d) acc[k][d] *= f;
        M[k] = m;
      }
#pragma unroll
      for (int c = 0; c < kBatch; ++c) {
        if (e[c][k] == -CUDART_INF_F) continue;   // no key of this row there
        const float wgt = fast_exp2(e[c][k] - M[k]);
        sum[k] += wgt;
#pragma unroll
        for (int d = 0; d < kDPL; ++d) acc[k][d] = fmaf(wgt, v[c][k][d], acc[k][d]);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    if (i0 + k >= rows) break;
    const float inv = sum[k] == 0.f ? 0.f : 1.f / sum[k];
    const int f = fg.x + i0 + k;
    const int64_t at = static_cast<int64_t>(tok + f / a.group) * a.num_q_heads + fg.y * a.group + f % a.group;
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o) + at * D + lane * kDPL);
    if constexpr (kDPL == 4)
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc[k][0] * inv, acc[k][1] * inv),
                                                  pack_bf16x2(acc[k][2] * inv, acc[k][3] * inv));
    else
      *dst = pack_bf16x2(acc[k][0] * inv, acc[k][1] * inv);
    if (lane == 0 && a.lse)
      a.lse[at] = sum[k] == 0.f ? -CUDART_INF_F : (M[k] + fast_log2(sum[k])) * 0.69314718055994530942f;
  }
}

// Ancestor bits from parents: token i of a request sets its own bit and its
// ancestors' (parent indexes below its own, -1 for a root; others are flagged
// and end the walk).  One warp per token; lane l owns words l, l + 32, ...
// Bound by the walk's dependent reads: 64 trees of 64 nodes 6 us, chains of 64
// nodes 10.
__global__ void __launch_bounds__(256) tree_mask_kernel(const int32_t* __restrict__ parents,
                                                        const int32_t* __restrict__ cu, int num_reqs, int num_tokens,
                                                        uint32_t* __restrict__ mask, int words, unsigned* err) {
  const int lane = threadIdx.x & 31;
  const int t = static_cast<int>((static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5);
  griddep_wait();
  griddep_launch();
  if (blockIdx.x == 0 && threadIdx.x == 0) check_cu(cu, num_reqs, num_tokens, err);
  if (t >= num_tokens) return;
  const int r = req_of(cu, num_reqs, t), c0 = r >= 0 ? __ldg(cu + r) : -1;
  if (c0 < 0) return;
  for (int w0 = 0; w0 < words; w0 += 32) {
    uint32_t bits = 0;
    // Parents lie strictly before their children, so the walk ends.
    for (int i = t - c0; i >= 0;) {
      if ((i >> 5) == w0 + lane) bits |= 1u << (i & 31);
      const int p = __ldg(parents + c0 + i);
      if (p >= i || p < -1) {
        if (lane == 0) atomicOr(err, PKV_DEVERR_POSITION);
        break;
      }
      i = p;
    }
    if (w0 + lane < words) mask[static_cast<int64_t>(t) * words + w0 + lane] = bits;
  }
  if (lane == 0 && t - c0 >= words * 32) atomicOr(err, PKV_DEVERR_POSITION);   // its own bit has no word
}

template <int D, bool F8, bool LIST, int W>
int launch_rows_w(const TreeArgs& a, cudaStream_t s) {
  const int smem = RowsSmem<D, F8, W>::kTotal;
  static_assert(RowsSmem<D, F8, W>::kTotal <= 232448, "shared memory of a CTA");
  cudaError_t e = smem_attr_once<rows_kernel<D, F8, LIST, W>>(smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(rows_kernel<D, F8, LIST, W>, dim3(a.ctas), 32 * W, smem, s, a);
}

template <int D, bool F8, bool LIST>
int launch_rows_l(const TreeArgs& a, cudaStream_t s) {
  if (a.form.warps == 12) return launch_rows_w<D, F8, LIST, 12>(a, s);
  if (a.form.warps == 6) return launch_rows_w<D, F8, LIST, 6>(a, s);
  return launch_rows_w<D, F8, LIST, kRowWarps>(a, s);
}

template <int D, bool F8>
int launch_rows(const TreeArgs& a, cudaStream_t s) {
  return a.sel ? launch_rows_l<D, F8, true>(a, s) : launch_rows_l<D, F8, false>(a, s);
}

template <int D, int SlotRows, int kRows, int kBatch>
int launch_merge_t(const TreeArgs& a, int rows, cudaStream_t s) {
  return launch_dependent(tree_merge_kernel<D, SlotRows, kRows, kBatch>, dim3(a.form.cuts, rows / (8 * kRows)), 256, 0, s, a);
}

}  // namespace

TreeForm tree_form(bool tensor, int num_sms) {
  TreeForm f;
  f.tensor = tensor;
  f.ctas = tensor ? num_sms : 3 * num_sms;
  f.cuts = tensor ? 2 * f.ctas : kRowWarps * f.ctas;   // two lines of work, or a share a warp
  f.slot_rows = tensor ? 256 : kRowTile;
  f.slots = 2 * f.cuts;
  f.many_groups = f.ctas / 2;
  f.whole = 0;
  f.warps = kRowWarps;
  return f;
}

int launch_tree_rows(const TreeArgs& a, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool f8 = a.pool.elem_bytes == 1;
  if (a.pool.head_dim == 128) return f8 ? launch_rows<128, true>(a, s) : launch_rows<128, false>(a, s);
  return f8 ? launch_rows<64, true>(a, s) : launch_rows<64, false>(a, s);
}

int launch_tree_merge(const TreeArgs& a, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.form.tensor)
    return a.pool.head_dim == 128 ? launch_merge_t<128, 256, 4, 2>(a, 256, s) : launch_merge_t<64, 256, 4, 2>(a, 256, s);
  return a.pool.head_dim == 128 ? launch_merge_t<128, kRowTile, 2, 4>(a, kRowTile, s)
                                : launch_merge_t<64, kRowTile, 2, 4>(a, kRowTile, s);
}

// (The scored attention's: tiles of 8 rows leave a warp one row, and one user's long context is cut into hundreds of
// parts.  Rows, a warp a row with 32 registers of partials under way: 16 thousand tokens of 2 KV heads, D = 64, 12.6 us
// with the attention, as above 17.0.  Tiles, fewer rows and more parts a warp where a group has many parts, from eight
// CTAs a group on: 32 tokens on 100 thousand, 2 KV heads, 37 us, as above 50; 3 prompts of packed documents 43 and 40.)
template <int D>
int launch_score_merge_d(const TreeArgs& a, int row_tile, int64_t groups, cudaStream_t s) {
  if (!a.form.tensor) return launch_merge_t<D, kRowTile, 1, 1024 / D>(a, row_tile, s);
  return a.ctas >= 8 * groups ? launch_merge_t<D, 256, 2, 8>(a, 256, s) : launch_merge_t<D, 256, 4, 2>(a, 256, s);
}
int launch_score_merge(const TreeArgs& a, int row_tile, int64_t groups, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return a.pool.head_dim == 128 ? launch_score_merge_d<128>(a, row_tile, groups, s)
                                : launch_score_merge_d<64>(a, row_tile, groups, s);
}

int launch_tree_mask(const int32_t* parents, const int32_t* cu, int num_reqs, int num_tokens, uint32_t* mask, int words,
                     unsigned* err, void* stream) {
  return launch_dependent(tree_mask_kernel, dim3((num_tokens + 7) / 8), 256, 0, static_cast<cudaStream_t>(stream), parents,
                          cu, num_reqs, num_tokens, mask, words, err);
}

}  // namespace pkv
