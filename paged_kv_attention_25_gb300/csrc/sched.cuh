// Work split of an attention call whose lengths live on the device.
//
// The work of request r is groups (KV head, tile of query rows) of a number of
// key units each; all requests' units form one line of U units, and worker w
// of C takes [w U / C, (w + 1) U / C): equal shares whatever the lengths, no
// plan on the host, nothing to upload, and a captured call follows the lengths
// it finds.  A group that falls into several shares is merged by log-sum-exp
// afterwards.  Of a worker's share only the first and the last group can be
// cut, so it has two partial slots: 0 for a group that began before its share,
// 1 for one that ends after it; the worker that begins a cut group leaves a
// record of it for the merge.
#pragma once
#include <cuda_runtime.h>

#include "internal.h"
#include "ops.h"

namespace pkv {

// One call of the tree attention (pkv_tree_attn), or of the attention over
// selected blocks (pkv_sparse_attn: `sel` is not nullptr).
struct TreeArgs {
  PoolView pool;
  const void* q;
  int num_q_heads, group;
  const int32_t* block_tables;
  int max_blocks;
  const int32_t* ctx_lens;
  const int32_t* prefix_lens;
  const int32_t* cu_q_lens;
  int num_reqs, num_tokens;
  const uint32_t* mask;
  int mask_words;
  const int32_t* positions;   // selected blocks: the tokens' positions,
  const int32_t* sel;         // their lists [tokens][kv heads][top_k]
  int top_k;
  float scale_log2;
  void* o;
  float* lse;
  // Workspace: the cut groups, their partial rows.
  struct TreeCut* cuts;
  float* part_o;     // [slots][slot rows][D]
  float* part_lse;   // [slots][slot rows], log2 units
  TreeForm form;
  int ctas;          // CTAs of the attention launch
  int tile_tokens;   // tensor-core form: tokens of a tile of 128 rows
  int q_box_tokens;  // ... and of a copy of its query map
  int o_align32;     // o is 32-byte aligned
  uint64_t wait_ns;
  int withhold;      // test hook: 2 = CTA 0 of the tiles form skips its first K copy
};

// A group that several workers share: rows [0, rows_a) and [128, 128 + rows_b)
// of its slots; row i belongs to token tok + (f0 + i) / G and head
// g G + (f0 + i) % G.  Its partials are slot `first` and slots
// next, next + stride, ... (count - 1 of them).
struct alignas(16) TreeCut {
  int count, first, next, stride;
  int tok_a, rows_a, tok_b, rows_b;
  int f0, g, pad0, pad1;
};
static_assert(sizeof(TreeCut) == 48, "TreeCut layout: three 16-byte loads");

// Flags token ranges that reach outside [0, num_tokens); the kernels cut them.  One thread of a launch.
__device__ __forceinline__ void check_cu(const int32_t* cu, int num_reqs, int num_tokens, unsigned* err) {
  if (__ldg(cu) < 0 || __ldg(cu + num_reqs) > num_tokens) atomicOr(err, PKV_DEVERR_POSITION);
}

// The request of token t (the last with cu <= t), or -1 for a token that belongs to none.
__device__ __forceinline__ int req_of(const int32_t* cu, int num_reqs, int t) {
  int lo = 0, hi = num_reqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(cu + mid) <= t) lo = mid; else hi = mid - 1;
  }
  return __ldg(cu + lo) <= t && t < __ldg(cu + lo + 1) ? lo : -1;
}

// The same by a whole warp: each round narrows the range 32-fold.
__device__ __forceinline__ int req_of_warp(const int32_t* cu, int num_reqs, int t, int lane) {
  int lo = 0, n = num_reqs;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lo + lane * step;
    const uint32_t le = __ballot_sync(0xffffffffu, lane * step < n && __ldg(cu + at) <= t);
    const int k = max(0, __popc(le) - 1);
    n = min(step, n - k * step);
    lo += k * step;
  }
  return __ldg(cu + lo) <= t && t < __ldg(cu + lo + 1) ? lo : -1;
}

// A request's lengths, made safe: whatever the device arrays hold, tokens stay
// inside [0, num_tokens) and keys inside the block table's row.
struct TreeReq {
  int t0, n, ctx, prefix;
  bool bad;
};

__device__ __forceinline__ TreeReq tree_req(const TreeArgs& a, int r) {
  TreeReq q;
  const int c0 = __ldg(a.cu_q_lens + r), c1 = __ldg(a.cu_q_lens + r + 1);
  const int ctx = __ldg(a.ctx_lens + r), pre = __ldg(a.prefix_lens + r);
  q.t0 = min(max(c0, 0), a.num_tokens);
  q.n = min(max(c1, q.t0), a.num_tokens) - q.t0;
  q.ctx = min(max(ctx, 0), a.max_blocks * kBlockSize);
  q.prefix = min(max(pre, 0), q.ctx);
  q.bad = c0 < 0 || c1 < c0 || c1 > a.num_tokens || q.ctx != ctx || q.prefix != pre;
  return q;
}

// Shares of U units among `most` workers at most, kMin units each at least.
template <int kMin>
struct Share {
  __device__ static int workers(int64_t U, int most) {
    const int64_t want = (U + kMin - 1) / kMin;
    return static_cast<int>(want < 1 ? 1 : want > most ? most : want);
  }
  __device__ static int64_t begin(int64_t U, int C, int w) { return U * w / C; }
  // The worker whose share holds unit u.
  __device__ static int owner(int64_t U, int C, int64_t u) { return static_cast<int>(((u + 1) * C - 1) / U); }
};

// A worker's share of a line: units [u, end) of U, the first of them unit
// `off` of request `req`.
struct TreeShare {
  int64_t U, u, end, off;
  int workers, req;
};

// Block-wide: the lengths U[i] of NL lines in which item r of `items` has n[i]
// units, units(r, n) filling n, and for each of NP probes the item that holds a
// unit and the unit's offset in it.  probe(U, p, line, unit), called once U is
// known, names probe p's line and unit (-1: none); the answers are req[p] and
// off[p].  One pass over the items (kept in registers) when there are no more of
// them than threads, two otherwise.  scratch: max(NL * warps, 2 * NP) int64.
template <int Threads, int NL, int NP, class F, class P>
__device__ __forceinline__ void line_scan(int items, int64_t* scratch, int64_t (&U)[NL], int (&req)[NP],
                                          int64_t (&off)[NP], F&& units, P&& probe) {
  constexpr int kW = Threads / 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int64_t n[NL], excl[NL];
  auto scan = [&](int base) {   // units and exclusive offset of item base + tid; U: total so far
    const int r = base + tid;
#pragma unroll
    for (int i = 0; i < NL; ++i) n[i] = 0;
    if (r < items) units(r, n);
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      int64_t inc = n[i];
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, inc, x);
        if (lane >= x) inc += y;
      }
      if (lane == 31) scratch[i * kW + warp] = inc;
      excl[i] = inc - n[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      int64_t total = U[i];
      excl[i] += U[i];
#pragma unroll
      for (int v = 0; v < kW; ++v) {
        const int64_t x = scratch[i * kW + v];
        if (v < warp) excl[i] += x;
        total += x;
      }
      U[i] = total;
    }
    __syncthreads();
  };
#pragma unroll
  for (int i = 0; i < NL; ++i) U[i] = 0;
  for (int base = 0; base < items; base += Threads) scan(base);
  int line[NP];
  int64_t unit[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    probe(U, p, line[p], unit[p]);
    req[p] = 0;
    off[p] = 0;
  }
  const bool kept = items <= Threads;
  int64_t total[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    total[i] = U[i];
    if (!kept) U[i] = 0;
  }
  for (int base = 0; base < items; base += Threads) {
    if (!kept) scan(base);
    bool here[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      int64_t e = excl[0], m = n[0];
#pragma unroll
      for (int i = 1; i < NL; ++i)
        if (line[p] == i) { e = excl[i]; m = n[i]; }
      here[p] = unit[p] >= 0 && e <= unit[p] && unit[p] < e + m;
      if (here[p]) {
        scratch[2 * p] = base + tid;
        scratch[2 * p + 1] = unit[p] - e;
      }
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      // (the chunk that holds the probe's unit: its total has passed it)
      int64_t end = U[0];
#pragma unroll
      for (int i = 1; i < NL; ++i)
        if (line[p] == i) end = U[i];
      if (unit[p] >= 0 && unit[p] < end) {
        req[p] = static_cast<int>(scratch[2 * p]);
        off[p] = scratch[2 * p + 1];
        unit[p] = -1;
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < NL; ++i) U[i] = total[i];
}

// The lines of a tree-attention call: request r has units(tree_req(a, r), i) units in line i.
template <int Threads, int NL, int NP, class F, class P>
__device__ __forceinline__ void tree_scan(const TreeArgs& a, int64_t* scratch, int64_t (&U)[NL], int (&req)[NP],
                                          int64_t (&off)[NP], F&& units, P&& probe) {
  line_scan<Threads, NL, NP>(
      a.num_reqs, scratch, U, req, off,
      [&](int r, int64_t (&n)[NL]) {
        const TreeReq q = tree_req(a, r);
#pragma unroll
        for (int i = 0; i < NL; ++i) n[i] = units(q, i);
        if (q.bad && blockIdx.x == 0) atomicOr(a.pool.err, PKV_DEVERR_POSITION);
      },
      probe);
}

// Bits [x0, x0 + 32) of a token's tree mask (bits outside the row's words are
// 0; x0 may be negative).  Plain loads: the kernel ahead may have written the mask.
__device__ __forceinline__ uint32_t tree_bits(const uint32_t* row, int words, int x0) {
  if (x0 <= -32) return 0u;
  if (x0 < 0) return (words > 0 ? row[0] : 0u) << (-x0);
  const int w = x0 >> 5;
  const uint32_t lo = w < words ? row[w] : 0u;
  const uint32_t hi = w + 1 < words ? row[w + 1] : 0u;
  return __funnelshift_r(lo, hi, x0 & 31);
}

// The lowest n bits (n <= 0: none, n >= 32: all).
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// Keys [key0, key0 + 32) that a token of a request sees, as bits.
__device__ __forceinline__ uint32_t tree_sees(int prefix, int ctx, const uint32_t* row, int words, int key0) {
  const uint32_t tree = tree_bits(row, words, key0 - prefix) & ~low_bits(prefix - key0);
  return (low_bits(prefix - key0) | tree) & low_bits(ctx - key0);
}

}  // namespace pkv
