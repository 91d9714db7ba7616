// Work split of an attention call whose lengths live on the device.
//
// The work of request r is groups (KV head, tile of query rows) of kblk key
// units each; all requests' units form one line of U units, and CTA c of C
// takes [c U / C, (c + 1) U / C): equal shares whatever the lengths, no plan
// on the host, nothing to upload, and a captured call follows the lengths it
// finds.  A group that falls into several CTAs is merged by log-sum-exp
// afterwards: of a CTA's share only the first and the last group can be cut,
// so a CTA has two partial slots, 2 c (a group that began before its share)
// and 2 c + 1 (a group that ends after it).
#pragma once
#include <cuda_runtime.h>

#include "internal.h"

namespace pkv {

// One tree-attention call (pkv_tree_attn).
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
  float scale_log2;
  void* o;
  float* lse;
  // Workspace: unit offset of each request (num_reqs + 1), partial slots.
  int64_t* offs;
  float* part_o;     // [2 C][tile rows][D]
  float* part_lse;   // [2 C][tile rows], log2 units
  int ctas;          // C at most
  uint64_t wait_ns;
};

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

// Tiling of a kernel: TileRows query rows per group, KeyUnit keys per unit, at least MinUnits units a CTA.
template <int TileRows_, int KeyUnit_, int MinUnits_>
struct Tiling {
  static constexpr int kRows = TileRows_, kKeys = KeyUnit_, kMin = MinUnits_;
  __device__ static int tiles(const TreeReq& q, int group) {
    return static_cast<int>((static_cast<int64_t>(q.n) * group + kRows - 1) / kRows);
  }
  // A request without keys keeps one (empty) unit a group: its rows are written too.
  __device__ static int kblk(const TreeReq& q) { return max(1, (q.ctx + kKeys - 1) / kKeys); }
  __device__ static int64_t units(const TreeReq& q, int group, int hkv) {
    return static_cast<int64_t>(tiles(q, group)) * hkv * kblk(q);
  }
  // CTAs that share U units.
  __device__ static int ctas(int64_t U, int most) {
    const int64_t want = (U + kMin - 1) / kMin;
    return static_cast<int>(want < 1 ? 1 : want > most ? most : want);
  }
  __device__ static int64_t begin(int64_t U, int C, int c) { return U * c / C; }
  // The CTA whose share holds unit u.
  __device__ static int owner(int64_t U, int C, int64_t u) { return static_cast<int>(((u + 1) * C - 1) / U); }
};

// Block-wide: the total number of units, and the request that holds the first
// unit of this CTA's share with the unit's offset inside it.  CTA 0 writes the
// requests' offsets for the merge.  scratch: one int64 per warp, plus two.
template <class T, int Threads>
__device__ __forceinline__ void tree_locate(const TreeArgs& a, int64_t* scratch, int64_t& U, int& C, int64_t& u0,
                                            int64_t& u1, int& req, int64_t& off) {
  constexpr int kW = Threads / 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hkv = a.pool.num_kv_heads;
  U = 0;
  for (int pass = 0; pass < 2; ++pass) {
    int64_t run = 0;
    for (int base = 0; base < a.num_reqs; base += Threads) {
      const int r = base + tid;
      int64_t n = 0;
      if (r < a.num_reqs) {
        const TreeReq q = tree_req(a, r);
        n = T::units(q, a.group, hkv);
        if (pass == 0 && q.bad && blockIdx.x == 0) atomicOr(a.pool.err, PKV_DEVERR_POSITION);
      }
      int64_t inc = n;
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, inc, x);
        if (lane >= x) inc += y;
      }
      if (lane == 31) scratch[warp] = inc;
      __syncthreads();
      int64_t before = run, total = run;
#pragma unroll
      for (int w = 0; w < kW; ++w) {
        if (w < warp) before += scratch[w];
        total += scratch[w];
      }
      const int64_t excl = before + inc - n;
      if (pass == 0) {
        if (blockIdx.x == 0 && r < a.num_reqs) a.offs[r] = excl;
      } else if (n > 0 && excl <= u0 && u0 < excl + n) {
        scratch[kW] = r;
        scratch[kW + 1] = u0 - excl;
      }
      run = total;
      __syncthreads();
      if (pass == 1 && run > u0) break;   // block-uniform
    }
    if (pass == 0) {
      U = run;
      if (blockIdx.x == 0 && tid == 0) a.offs[a.num_reqs] = U;
      C = T::ctas(U, a.ctas);
      if (U == 0 || static_cast<int>(blockIdx.x) >= C) {
        u0 = u1 = 0;
        req = 0;
        off = 0;
        return;
      }
      u0 = T::begin(U, C, blockIdx.x);
      u1 = T::begin(U, C, blockIdx.x + 1);
    }
  }
  req = static_cast<int>(scratch[kW]);
  off = scratch[kW + 1];
  __syncthreads();
}

// Bits [x0, x0 + 32) of a token's tree mask (bits outside the row's words are
// 0; x0 may be negative).
__device__ __forceinline__ uint32_t tree_bits(const uint32_t* row, int words, int x0) {
  if (x0 <= -32) return 0u;
  if (x0 < 0) return (words > 0 ? __ldg(row) : 0u) << (-x0);
  const int w = x0 >> 5;
  const uint32_t lo = w < words ? __ldg(row + w) : 0u;
  const uint32_t hi = w + 1 < words ? __ldg(row + w + 1) : 0u;
  return __funnelshift_r(lo, hi, x0 & 31);
}

// The lowest n bits (n <= 0: none, n >= 32: all).
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// Keys [key0, key0 + 32) that a token of request q sees, as bits.
__device__ __forceinline__ uint32_t tree_sees(const TreeReq& q, const uint32_t* row, int words, int key0) {
  const uint32_t tree = tree_bits(row, words, key0 - q.prefix) & ~low_bits(q.prefix - key0);
  return (low_bits(q.prefix - key0) | tree) & low_bits(q.ctx - key0);
}

}  // namespace pkv
