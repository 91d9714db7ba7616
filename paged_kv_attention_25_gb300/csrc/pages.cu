// Pages of a cache: sharing, copying, allocating and freeing them for the next
// generation of sequences (pkv_fork), copying whole pages (pkv_copy_blocks),
// and moving kept tokens together (pkv_compact).
//
// A page's owners are counted in `refs`; a page is free when its count is 0,
// so freeing needs no list and allocation takes the lowest free pages: the
// outcome depends on the inputs alone.
#include <cuda_runtime.h>

#include <algorithm>

#include "internal.h"
#include "ops.h"

namespace pkv {
namespace {

constexpr int kPlanThreads = 1024;

// Workspace of a fork, in ints.
struct ForkWs {
  int* kids;     // [rows] children of the row
  int* first;    // [rows] its lowest child
  int* keep;     // [rows] 1: that child keeps the partly filled page
  int* start;    // [children] the child's first fresh page in `fresh`
  int* fresh;    // [num_blocks] free pages in ascending order, as many as are needed
  int* total;    // [1] fresh pages needed
};
__host__ __device__ inline ForkWs fork_ws(int* ws, int rows, int children, int num_blocks) {
  ForkWs w;
  w.kids = ws;
  w.first = w.kids + rows;
  w.keep = w.first + rows;
  w.start = w.keep + rows;
  w.fresh = w.start + children;
  w.total = w.fresh + num_blocks;
  return w;
}

// Lengths of old row r, made safe: len <= cap <= the table's row.
struct ForkRow { int len, pages, full, part; bool bad; };
__device__ __forceinline__ ForkRow fork_row(const ForkArgs& a, int r) {
  const int most = a.max_blocks * kBlockSize;
  const int len = __ldg(a.lens + r), cap = __ldg(a.caps + r);
  ForkRow x;
  const int c = min(max(cap, 0), most);
  x.len = min(max(len, 0), c);
  x.bad = c != cap || x.len != len;
  x.pages = (c + kBlockSize - 1) / kBlockSize;
  x.full = x.len / kBlockSize;
  x.part = x.len % kBlockSize;
  return x;
}
// Pages of child i, and how many of them its parent's row provides.
struct ForkChild { int parent, pages, shared; bool copies; };
__device__ __forceinline__ ForkChild fork_child(const ForkArgs& a, const ForkWs& w, int i) {
  ForkChild c;
  const int p = __ldg(a.parents + i);
  c.parent = p >= 0 && p < a.num_rows ? p : -1;
  int len = 0;
  c.shared = 0;
  c.copies = false;
  if (c.parent >= 0) {
    const ForkRow r = fork_row(a, c.parent);
    len = r.len;
    const bool keeps = r.part > 0 && w.keep[c.parent] != 0 && w.first[c.parent] == i;
    c.shared = r.full + (keeps ? 1 : 0);
    c.copies = r.part > 0 && !keeps;
  }
  const int cap = min(max(__ldg(a.new_caps + i), len), a.max_blocks * kBlockSize);
  c.pages = (cap + kBlockSize - 1) / kBlockSize;
  return c;
}

__device__ __forceinline__ int block_scan(int v, int* s_warp, int* total) {   // inclusive, kPlanThreads threads
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, x);
    if (lane >= x) v += y;
  }
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int s = s_warp[lane];
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, x);
      if (lane >= x) s += y;
    }
    s_warp[lane] = s;
  }
  __syncthreads();
  if (warp > 0) v += s_warp[warp - 1];
  *total = s_warp[31];
  __syncthreads();
  return v;
}

// Counts, allocation: one CTA.
__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const ForkArgs a) {
  __shared__ int s_warp[32];
  const int tid = threadIdx.x;
  const int nb = a.pool.num_blocks;
  const ForkWs w = fork_ws(a.ws, a.num_rows, a.num_children, nb);
  volatile int* refs = a.new_refs;
  for (int r = tid; r < a.num_rows; r += kPlanThreads) {
    w.kids[r] = 0;
    w.first[r] = 0x7fffffff;
    w.keep[r] = 0;
  }
  if (a.new_refs != a.refs)
    for (int i = tid; i < nb; i += kPlanThreads) a.new_refs[i] = __ldg(a.refs + i);
  __syncthreads();
  for (int i = tid; i < a.num_children; i += kPlanThreads) {
    const int p = __ldg(a.parents + i);
    if (p < -1 || p >= a.num_rows) atomicOr(a.pool.err, PKV_DEVERR_POSITION);
    if (p >= 0 && p < a.num_rows) {
      atomicAdd(&w.kids[p], 1);
      atomicMin(&w.first[p], i);
    }
  }
  __syncthreads();
  // Every page of a row: one owner less, and one more for each child that
  // shares it.  A row with one child keeps its full pages: nothing to count.
  const int lane = tid & 31;
  for (int r = tid >> 5; r < a.num_rows; r += kPlanThreads / 32) {
    const ForkRow x = fork_row(a, r);
    if (x.bad && lane == 0) atomicOr(a.pool.err, PKV_DEVERR_POSITION);
    const int kids = w.kids[r];
    const int32_t* row = a.tables + static_cast<int64_t>(r) * a.max_blocks;
    for (int j = (kids == 1 ? x.full : 0) + lane; j < x.pages; j += 32) {
      const int delta = j < x.full ? kids - 1 : j == x.full && x.part > 0 && kids > 0 ? 0 : -1;
      const int pb = __ldg(row + j);
      if (pb < 0 || pb >= nb) atomicOr(a.pool.err, PKV_DEVERR_BLOCK_ID);
      else if (delta != 0) atomicAdd(a.new_refs + pb, delta);
    }
  }
  __syncthreads();
  // The partly filled page of a continued row: its lowest child keeps it if the row was its only owner.
  for (int r = tid; r < a.num_rows; r += kPlanThreads) {
    const ForkRow x = fork_row(a, r);
    if (w.kids[r] > 0 && x.part > 0) {
      const int pb = __ldg(a.tables + static_cast<int64_t>(r) * a.max_blocks + x.full);
      w.keep[r] = pb >= 0 && pb < nb && refs[pb] == 1;
    }
  }
  __syncthreads();
  int run = 0;
  for (int base = 0; base < a.num_children; base += kPlanThreads) {
    const int i = base + tid;
    int need = 0;
    if (i < a.num_children) {
      const ForkChild c = fork_child(a, w, i);
      need = max(0, c.pages - c.shared);
    }
    int tot;
    const int inc = block_scan(need, s_warp, &tot);
    if (i < a.num_children) w.start[i] = run + inc - need;
    run += tot;
  }
  const int total = run;
  // The lowest free pages, in order.
  int found = 0;
  for (int base = 0; base < nb && found < total; base += kPlanThreads) {
    const int i = base + tid;
    const int is_free = i < nb && refs[i] == 0;
    int tot;
    const int k = found + block_scan(is_free, s_warp, &tot) - is_free;
    if (is_free && k < total) {
      w.fresh[k] = i;
      a.new_refs[i] = 1;
    }
    found += tot;
  }
  if (tid == 0) *w.total = min(found, total);
  if (found < total && tid == 0) atomicOr(a.pool.err, PKV_DEVERR_NO_PAGES);
  __syncthreads();
  // Partly filled pages whose children all copied them lose the row's ownership (after the allocation: they are
  // still read by the copies).
  for (int r = tid; r < a.num_rows; r += kPlanThreads) {
    const ForkRow x = fork_row(a, r);
    if (w.kids[r] > 0 && x.part > 0 && !w.keep[r]) {
      const int pb = __ldg(a.tables + static_cast<int64_t>(r) * a.max_blocks + x.full);
      if (pb >= 0 && pb < nb) atomicAdd(a.new_refs + pb, -1);
    }
  }
}

// One CTA per child: its table row, and the copy of its parent's partly filled page.
__global__ void __launch_bounds__(256) fork_fill_kernel(const ForkArgs a) {
  const int i = blockIdx.x, tid = threadIdx.x;
  const int nb = a.pool.num_blocks;
  const ForkWs w = fork_ws(a.ws, a.num_rows, a.num_children, nb);
  const ForkChild c = fork_child(a, w, i);
  const int total = *w.total, start = w.start[i];
  const int32_t* old = a.tables + static_cast<int64_t>(max(c.parent, 0)) * a.max_blocks;
  int32_t* row = a.new_tables + static_cast<int64_t>(i) * a.max_blocks;
  auto fresh = [&](int j) {
    const int k = start + j - c.shared;
    return k < total ? w.fresh[k] : -1;
  };
  for (int j = tid; j < a.max_blocks; j += 256)
    row[j] = j < c.shared ? __ldg(old + j) : j < c.pages ? fresh(j) : -1;
  if (!c.copies) return;
  const ForkRow x = fork_row(a, c.parent);
  const int src = __ldg(old + x.full), dst = x.full < c.pages ? fresh(x.full) : -1;
  if (src < 0 || src >= nb || dst < 0) return;
  // Rows [0, part) of every KV head, K and V.
  const int row_chunks = a.pool.head_dim * a.pool.elem_bytes / 16;
  const int head = kBlockSize * row_chunks, live = x.part * row_chunks;
  const int64_t page = static_cast<int64_t>(a.pool.num_kv_heads) * head;
  for (int e = tid; e < 2 * a.pool.num_kv_heads * live; e += 256) {
    const int u = e / live, ch = e % live;
    uint4* pool = static_cast<uint4*>((u & 1) ? a.vp : a.kp);
    const int64_t at = static_cast<int64_t>(u >> 1) * head + ch;
    pool[dst * page + at] = pool[src * page + at];
  }
  if (a.codes) {
    const int n = a.pool.num_kv_heads * 2 * a.pool.head_dim / 16;
    uint4* codes = reinterpret_cast<uint4*>(a.codes);
    for (int e = tid; e < n; e += 256) codes[static_cast<int64_t>(dst) * n + e] = codes[static_cast<int64_t>(src) * n + e];
    for (int e = tid; e < a.pool.num_kv_heads; e += 256)
      a.exps[static_cast<int64_t>(dst) * a.pool.num_kv_heads + e] = a.exps[static_cast<int64_t>(src) * a.pool.num_kv_heads + e];
  }
}

// One CTA per pair: the whole page.
__global__ void __launch_bounds__(256) copy_blocks_kernel(const PoolView pool, uint4* kp, uint4* vp,
                                                          const int32_t* __restrict__ src,
                                                          const int32_t* __restrict__ dst, int8_t* codes,
                                                          int8_t* exps) {
  const int tid = threadIdx.x;
  const int s = __ldg(src + blockIdx.x), d = __ldg(dst + blockIdx.x);
  if (s < 0 || s >= pool.num_blocks || d < 0 || d >= pool.num_blocks) {
    if (tid == 0) atomicOr(pool.err, PKV_DEVERR_BLOCK_ID);
    return;
  }
  if (s == d) return;
  const int64_t page = static_cast<int64_t>(pool.num_kv_heads) * kBlockSize * pool.head_dim * pool.elem_bytes / 16;
  for (int64_t e = tid; e < page; e += 256) {
    kp[d * page + e] = kp[s * page + e];
    vp[d * page + e] = vp[s * page + e];
  }
  if (codes) {
    const int64_t n = static_cast<int64_t>(pool.num_kv_heads) * 2 * pool.head_dim / 16;
    uint4* c = reinterpret_cast<uint4*>(codes);
    for (int64_t e = tid; e < n; e += 256) c[d * n + e] = c[s * n + e];
    for (int e = tid; e < pool.num_kv_heads; e += 256)
      exps[static_cast<int64_t>(d) * pool.num_kv_heads + e] = exps[static_cast<int64_t>(s) * pool.num_kv_heads + e];
  }
}

// One thread per 16-byte column of a token's K and V rows: it moves its column
// of the request's kept tokens, kMoveBatch at a time, all loads before the
// stores.  Sources ascend and lie at or behind their targets, so a store never
// reaches a row that is still to be read: no two threads touch one column.
constexpr int kMoveBatch = 8;
__global__ void __launch_bounds__(256) compact_kernel(const PoolView pool, uint4* kp, uint4* vp,
                                                      const int32_t* __restrict__ bt, int max_blocks, int num_reqs,
                                                      const int32_t* __restrict__ cu, const int32_t* __restrict__ src,
                                                      const int32_t* __restrict__ dst, int num_kept) {
  const int cpr = pool.head_dim * pool.elem_bytes / 16;   // 16-byte chunks of one head's row
  const int cols = 2 * pool.num_kv_heads * cpr;
  const int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int r = static_cast<int>(e / cols);
  if (r >= num_reqs) return;
  const int col = static_cast<int>(e % cols);
  const int ch = col % cpr, g = (col / cpr) % pool.num_kv_heads;
  uint4* p = col < cols / 2 ? kp : vp;
  const int k0 = min(max(__ldg(cu + r), 0), num_kept), k1 = min(max(__ldg(cu + r + 1), k0), num_kept);
  const int d0 = __ldg(dst + r);
  const int32_t* row = bt + static_cast<int64_t>(r) * max_blocks;
  const int most = max_blocks * kBlockSize;
  // Chunk index of position x in this column, or -1 (flagged).
  auto at = [&](int x) -> int64_t {
    if (x < 0 || x >= most) {
      atomicOr(pool.err, PKV_DEVERR_POSITION);
      return -1;
    }
    const int pb = __ldg(row + x / kBlockSize);
    if (pb < 0 || pb >= pool.num_blocks) {
      atomicOr(pool.err, PKV_DEVERR_BLOCK_ID);
      return -1;
    }
    return ((static_cast<int64_t>(pb) * pool.num_kv_heads + g) * kBlockSize + x % kBlockSize) * cpr + ch;
  };
  int prev = -1;
  for (int k = k0; k < k1; k += kMoveBatch) {
    uint4 v[kMoveBatch];
    int64_t to[kMoveBatch];
#pragma unroll
    for (int u = 0; u < kMoveBatch; ++u) {
      to[u] = -1;
      if (k + u < k1) {
        const int s = __ldg(src + k + u), d = d0 + (k + u - k0);
        if (s <= prev || s < d) {
          atomicOr(pool.err, PKV_DEVERR_POSITION);
        } else if (s != d) {
          const int64_t from = at(s);
          if (from >= 0) {
            to[u] = at(d);
            if (to[u] >= 0) v[u] = p[from];
          }
        }
        prev = max(prev, s);
      }
    }
#pragma unroll
    for (int u = 0; u < kMoveBatch; ++u)
      if (to[u] >= 0) p[to[u]] = v[u];
  }
}

}  // namespace

size_t fork_ws_ints(int num_blocks, int num_rows, int num_children) {
  return static_cast<size_t>(3) * num_rows + num_children + num_blocks + 1;
}

int launch_fork(const ForkArgs& a, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  fork_plan_kernel<<<1, kPlanThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.num_children == 0) return e;
  fork_fill_kernel<<<a.num_children, 256, 0, s>>>(a);
  return cudaGetLastError();
}

int launch_copy_blocks(const PoolView& pool, void* kp, void* vp, const int32_t* src, const int32_t* dst, int n,
                       int8_t* codes, int8_t* exps, void* stream) {
  copy_blocks_kernel<<<n, 256, 0, static_cast<cudaStream_t>(stream)>>>(pool, static_cast<uint4*>(kp),
                                                                       static_cast<uint4*>(vp), src, dst, codes, exps);
  return cudaGetLastError();
}

int launch_compact(const PoolView& pool, void* kp, void* vp, const int32_t* block_tables, int max_blocks, int num_reqs,
                   const int32_t* cu_keep, const int32_t* src, const int32_t* dst, int num_kept, void* stream) {
  const int64_t cols = static_cast<int64_t>(2) * pool.num_kv_heads * (pool.head_dim * pool.elem_bytes / 16);
  const int64_t grid = (cols * num_reqs + 255) / 256;
  compact_kernel<<<static_cast<unsigned>(grid), 256, 0, static_cast<cudaStream_t>(stream)>>>(
      pool, static_cast<uint4*>(kp), static_cast<uint4*>(vp), block_tables, max_blocks, num_reqs, cu_keep, src, dst,
      num_kept);
  return cudaGetLastError();
}

}  // namespace pkv
