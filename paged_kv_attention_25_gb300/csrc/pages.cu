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
#include "ptx.cuh"
#include "sched.cuh"

namespace pkv {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanRows = 2048;   // rows whose children are counted in shared memory
constexpr int kRowBatch = 4;      // rows a warp has under way

// Workspace of a fork, in ints.
struct ForkWs {
  int* kids;     // [rows] children of the row (more than kPlanRows rows)
  int* keeper;   // [rows] the child that keeps the partly filled page, or -1
  int* first;    // [rows] the row's lowest child (more than kPlanRows rows)
  int4* child;   // [children][2] what the child's table row is made of (ForkFill)
  int* fresh;    // [num_blocks] free pages in ascending order, as many as are needed
};
__host__ __device__ inline ForkWs fork_ws(int* ws, int rows, int children, int num_blocks) {
  ForkWs w;
  w.kids = ws;
  w.keeper = w.kids + rows;
  w.first = w.keeper + rows;
  // (16-byte aligned: the workspace is)
  w.child = reinterpret_cast<int4*>(ws + (3 * rows + 3) / 4 * 4);
  w.fresh = reinterpret_cast<int*>(w.child + 2 * children);
  return w;
}

// Child i's row: `shared` pages of row `parent`, then `pages` - shared fresh
// ones from fresh[start] on, of which there are `total`; src >= 0: page `full`
// is a copy of that page's first `part` tokens.
struct ForkFill { int parent, shared, pages, start, src, part, full, total; };
static_assert(sizeof(ForkFill) == 32, "ForkFill layout: two 16-byte loads");

// Lengths of old row r, made safe: len <= cap <= the table's row.
struct ForkRow { int len, pages, full, part; bool bad; };
__device__ __forceinline__ ForkRow fork_row_of(const ForkArgs& a, int len, int cap) {
  const int most = a.max_blocks * kBlockSize;
  ForkRow x;
  const int c = min(max(cap, 0), most);
  x.len = min(max(len, 0), c);
  x.bad = c != cap || x.len != len;
  x.pages = (c + kBlockSize - 1) / kBlockSize;
  x.full = x.len / kBlockSize;
  x.part = x.len % kBlockSize;
  return x;
}
__device__ __forceinline__ ForkRow fork_row(const ForkArgs& a, int r) {
  return fork_row_of(a, __ldg(a.lens + r), __ldg(a.caps + r));
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
    const bool keeps = r.part > 0 && w.keeper[c.parent] == i;
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

// Counts, allocation: one CTA.  Bound by the latency of a chain of dependent
// reads (children, rows, tables, counts), so that each link keeps as many reads
// under way as there are: a warp takes kRowBatch rows at a time (one row at a
// time took 12 of 19 us for 240 rows of 60 pages), and a row with one child
// skips the full pages, whose counts do not change.  (1500 rows of 16 pages: 39 us
// with the fill, 4000 rows of 8: 95.)
__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const ForkArgs a) {
  __shared__ int s_warp[32];
  __shared__ int s_kids[kPlanRows], s_first[kPlanRows];
  const int tid = threadIdx.x;
  const int nb = a.pool.num_blocks;
  const ForkWs w = fork_ws(a.ws, a.num_rows, a.num_children, nb);
  const bool small = a.num_rows <= kPlanRows;
  int* kids = small ? s_kids : w.kids;
  int* first = small ? s_first : w.first;
  volatile int* refs = a.new_refs;
  griddep_wait();
  griddep_launch();
  for (int r = tid; r < a.num_rows; r += kPlanThreads) {
    kids[r] = 0;
    first[r] = 0x7fffffff;
  }
  if (a.new_refs != a.refs)
    for (int i = tid; i < nb; i += kPlanThreads) a.new_refs[i] = __ldcg(a.refs + i);   // (a fork ahead may have written them)
  __syncthreads();
  for (int i = tid; i < a.num_children; i += kPlanThreads) {
    const int p = __ldg(a.parents + i);
    if (p < -1 || p >= a.num_rows) atomicOr(a.pool.err, PKV_DEVERR_POSITION);
    if (p >= 0 && p < a.num_rows) {
      atomicAdd(&kids[p], 1);
      atomicMin(&first[p], i);
    }
  }
  __syncthreads();
  // Every page of a row: one owner less, and one more for each child that
  // shares it.
  const int lane = tid & 31;
  for (int r0 = (tid >> 5) * kRowBatch; r0 < a.num_rows; r0 += kPlanThreads / 32 * kRowBatch) {
    ForkRow x[kRowBatch];
    int from[kRowBatch], most = 0;
#pragma unroll
    for (int u = 0; u < kRowBatch; ++u) {
      x[u] = ForkRow{0, 0, 0, 0, false};
      if (r0 + u < a.num_rows) x[u] = fork_row(a, r0 + u);
    }
#pragma unroll
    for (int u = 0; u < kRowBatch; ++u) {
      if (x[u].bad && lane == 0) atomicOr(a.pool.err, PKV_DEVERR_POSITION);
      from[u] = r0 + u < a.num_rows && kids[r0 + u] == 1 ? x[u].full : 0;
      most = max(most, x[u].pages - from[u]);
    }
    for (int j0 = lane; j0 < most; j0 += 32) {
      int pb[kRowBatch];
#pragma unroll
      for (int u = 0; u < kRowBatch; ++u) {
        const int j = from[u] + j0;
        pb[u] = j < x[u].pages ? __ldg(a.tables + static_cast<int64_t>(r0 + u) * a.max_blocks + j) : 0;
      }
#pragma unroll
      for (int u = 0; u < kRowBatch; ++u) {
        const int j = from[u] + j0;
        if (j >= x[u].pages) continue;
        const int k = kids[r0 + u];
        const int delta = j < x[u].full ? k - 1 : j == x[u].full && x[u].part > 0 && k > 0 ? 0 : -1;
        if (pb[u] < 0 || pb[u] >= nb) atomicOr(a.pool.err, PKV_DEVERR_BLOCK_ID);
        else if (delta != 0) atomicAdd(a.new_refs + pb[u], delta);
      }
    }
  }
  __syncthreads();
  // The partly filled page of a continued row: its lowest child keeps it if the row was its only owner.
  for (int r = tid; r < a.num_rows; r += kPlanThreads) {
    const ForkRow x = fork_row(a, r);
    int keeper = -1;
    if (kids[r] > 0 && x.part > 0) {
      const int pb = __ldg(a.tables + static_cast<int64_t>(r) * a.max_blocks + x.full);
      if (pb >= 0 && pb < nb && refs[pb] == 1) keeper = first[r];
    }
    w.keeper[r] = keeper;
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
    if (i < a.num_children) w.child[2 * i] = make_int4(0, 0, 0, run + inc - need);
    run += tot;
  }
  const int total = run;
  // The lowest free pages, in order.
  int found = 0;
  for (int base = 0; base < nb && found < total; base += 4 * kPlanThreads) {
    const int i = base + 4 * tid;
    int is_free[4], mine = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      is_free[u] = i + u < nb && refs[i + u] == 0;
      mine += is_free[u];
    }
    int tot;
    int k = found + block_scan(mine, s_warp, &tot) - mine;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (is_free[u]) {
        if (k < total) {
          w.fresh[k] = i + u;
          a.new_refs[i + u] = 1;
        }
        ++k;
      }
    found += tot;
  }
  if (found < total && tid == 0) atomicOr(a.pool.err, PKV_DEVERR_NO_PAGES);
  __syncthreads();
  // Partly filled pages whose children all copied them lose the row's ownership (after the allocation: they are
  // still read by the copies).
  for (int r = tid; r < a.num_rows; r += kPlanThreads) {
    const ForkRow x = fork_row(a, r);
    if (kids[r] > 0 && x.part > 0 && w.keeper[r] < 0) {
      const int pb = __ldg(a.tables + static_cast<int64_t>(r) * a.max_blocks + x.full);
      if (pb >= 0 && pb < nb) atomicAdd(a.new_refs + pb, -1);
    }
  }
  for (int i = tid; i < a.num_children; i += kPlanThreads) {
    const ForkChild c = fork_child(a, w, i);
    const int start = w.child[2 * i].w;
    int src = -1;
    ForkRow x{0, 0, 0, 0, false};
    if (c.copies) {
      x = fork_row(a, c.parent);
      src = __ldg(a.tables + static_cast<int64_t>(c.parent) * a.max_blocks + x.full);
      if (src >= nb) src = -1;
    }
    w.child[2 * i] = make_int4(c.parent, c.shared, c.pages, start);
    w.child[2 * i + 1] = make_int4(src, x.part, x.full, min(found, total));
  }
}

// The same for up to kPlanThreads rows and children: thread i has row i and
// child i in registers, so that the chain is three reads long: lengths and
// parents, tables, counts.  4 rows of 8 pages: 8.3 us with the fill (the general
// kernel: 10); 240 rows of up to 130: 14.4 (19), of which the additions to 7 thousand
// counts, from one SM, are 4 and the first read behind them 2; 1024 rows of 16: 21.
__global__ void __launch_bounds__(kPlanThreads) fork_plan_small_kernel(const ForkArgs a) {
  __shared__ int s_warp[32];
  __shared__ int s_kids[kPlanThreads], s_first[kPlanThreads], s_keeper[kPlanThreads];
  __shared__ int s_from[kPlanThreads], s_pages[kPlanThreads], s_full[kPlanThreads], s_part[kPlanThreads],
      s_last[kPlanThreads], s_len[kPlanThreads];
  const int tid = threadIdx.x, lane = tid & 31;
  const int nb = a.pool.num_blocks;
  const ForkWs w = fork_ws(a.ws, a.num_rows, a.num_children, nb);
  volatile int* refs = a.new_refs;
  s_kids[tid] = 0;
  s_first[tid] = 0x7fffffff;
  griddep_wait();
  griddep_launch();
  const bool is_row = tid < a.num_rows, is_child = tid < a.num_children;
  const int len = is_row ? __ldg(a.lens + tid) : 0, cap = is_row ? __ldg(a.caps + tid) : 0;
  int parent = is_child ? __ldg(a.parents + tid) : -1;
  const int new_cap = is_child ? __ldg(a.new_caps + tid) : 0;
  if (a.new_refs != a.refs)
    for (int i = tid; i < nb; i += kPlanThreads) a.new_refs[i] = __ldcg(a.refs + i);   // (a fork ahead may have written them)
  const ForkRow x = fork_row_of(a, len, cap);
  int last = -1;   // the page that the row's tokens fill in part
  if (is_row && x.part > 0) {
    last = __ldg(a.tables + static_cast<int64_t>(tid) * a.max_blocks + x.full);
    if (last >= nb) last = -1;
  }
  if (is_row && x.bad) atomicOr(a.pool.err, PKV_DEVERR_POSITION);
  if (parent < -1 || parent >= a.num_rows) {
    atomicOr(a.pool.err, PKV_DEVERR_POSITION);
    parent = -1;
  }
  s_pages[tid] = is_row ? x.pages : 0;
  s_full[tid] = x.full;
  s_part[tid] = x.part;
  s_len[tid] = x.len;
  __syncthreads();
  if (parent >= 0) {
    atomicAdd(&s_kids[parent], 1);
    atomicMin(&s_first[parent], tid);
  }
  __syncthreads();
  s_from[tid] = s_kids[tid] == 1 ? x.full : 0;   // one child: the full pages' counts stay
  s_last[tid] = last;
  __syncthreads();
  for (int r0 = (tid >> 5) * kRowBatch; r0 < a.num_rows; r0 += kPlanThreads / 32 * kRowBatch) {
    int most = 0;
#pragma unroll
    for (int u = 0; u < kRowBatch; ++u) most = max(most, s_pages[r0 + u] - s_from[r0 + u]);   // (rows past the end have none)
    for (int j0 = lane; j0 < most; j0 += 32) {
      int pb[kRowBatch];
#pragma unroll
      for (int u = 0; u < kRowBatch; ++u) {
        const int j = s_from[r0 + u] + j0;
        pb[u] = j < s_pages[r0 + u] ? __ldg(a.tables + static_cast<int64_t>(r0 + u) * a.max_blocks + j) : 0;
      }
#pragma unroll
      for (int u = 0; u < kRowBatch; ++u) {
        const int j = s_from[r0 + u] + j0;
        if (j >= s_pages[r0 + u]) continue;
        const int k = s_kids[r0 + u], full = s_full[r0 + u];
        const int delta = j < full ? k - 1 : j == full && s_part[r0 + u] > 0 && k > 0 ? 0 : -1;
        if (pb[u] < 0 || pb[u] >= nb) atomicOr(a.pool.err, PKV_DEVERR_BLOCK_ID);
        else if (delta != 0) atomicAdd(a.new_refs + pb[u], delta);
      }
    }
  }
  __syncthreads();
  // Counts are final but for the partly filled pages; the first of them for the allocation are read with those pages'.
  int is_free[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) is_free[u] = 4 * tid + u < nb && refs[4 * tid + u] == 0;
  const bool settle = is_row && s_kids[tid] > 0 && x.part > 0;
  s_keeper[tid] = settle && last >= 0 && refs[last] == 1 ? s_first[tid] : -1;
  __syncthreads();
  int shared = 0, pages = 0;
  bool copies = false;
  if (is_child) {
    int held = 0;
    if (parent >= 0) {
      held = s_len[parent];
      const bool part = s_part[parent] > 0, keeps = part && s_keeper[parent] == tid;
      shared = s_full[parent] + (keeps ? 1 : 0);
      copies = part && !keeps;
    }
    pages = (min(max(new_cap, held), a.max_blocks * kBlockSize) + kBlockSize - 1) / kBlockSize;
  }
  const int need = max(0, pages - shared);
  int total;
  const int start = block_scan(need, s_warp, &total) - need;
  int found = 0;
  for (int base = 0; base < nb && found < total; base += 4 * kPlanThreads) {
    const int i = base + 4 * tid;
    int mine = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (base > 0) is_free[u] = i + u < nb && refs[i + u] == 0;
      mine += is_free[u];
    }
    int tot;
    int k = found + block_scan(mine, s_warp, &tot) - mine;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (is_free[u]) {
        if (k < total) {
          w.fresh[k] = i + u;
          a.new_refs[i + u] = 1;
        }
        ++k;
      }
    found += tot;
  }
  if (found < total && tid == 0) atomicOr(a.pool.err, PKV_DEVERR_NO_PAGES);
  // Partly filled pages whose children all copied them lose the row's ownership.
  if (settle && s_keeper[tid] < 0 && last >= 0) atomicAdd(a.new_refs + last, -1);
  if (is_child) {
    w.child[2 * tid] = make_int4(parent, shared, pages, start);
    w.child[2 * tid + 1] = make_int4(copies ? s_last[parent] : -1, copies ? s_part[parent] : 0,
                                     copies ? s_full[parent] : 0, min(found, total));
  }
}

// One CTA per child: its table row, and the copy of its parent's partly filled
// page, kCopyBatch chunks a thread at a time.  Bound by latency: its record, the
// fresh page's id, the page (4 children 4.2 us by itself, 240 children 5.6).
constexpr int kCopyBatch = 4;
__global__ void __launch_bounds__(256) fork_fill_kernel(const ForkArgs a) {
  const int i = blockIdx.x, tid = threadIdx.x;
  const int nb = a.pool.num_blocks;
  const ForkWs w = fork_ws(a.ws, a.num_rows, a.num_children, nb);
  griddep_wait();
  const int4 c0 = __ldcg(w.child + 2 * i), c1 = __ldcg(w.child + 2 * i + 1);
  const ForkFill c{c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
  const int32_t* old = a.tables + static_cast<int64_t>(max(c.parent, 0)) * a.max_blocks;
  int32_t* row = a.new_tables + static_cast<int64_t>(i) * a.max_blocks;
  auto fresh = [&](int j) {
    const int k = c.start + j - c.shared;
    return k < c.total ? __ldcg(w.fresh + k) : -1;
  };
  const int src = c.src, dst = c.src >= 0 && c.full < c.pages ? fresh(c.full) : -1;
  for (int j = tid; j < a.max_blocks; j += 256)
    row[j] = j < c.shared ? __ldg(old + j) : j < c.pages ? fresh(j) : -1;
  if (src < 0 || dst < 0) return;
  // Rows [0, part) of every KV head, K and V.
  const int row_chunks = a.pool.head_dim * a.pool.elem_bytes / 16;
  const int head = kBlockSize * row_chunks, live = c.part * row_chunks;
  const int64_t page = static_cast<int64_t>(a.pool.num_kv_heads) * head;
  const int chunks = 2 * a.pool.num_kv_heads * live;
  for (int e0 = tid; e0 < chunks; e0 += 256 * kCopyBatch) {
    uint4 v[kCopyBatch];
    uint4* pool[kCopyBatch];
    int64_t at[kCopyBatch];
#pragma unroll
    for (int k = 0; k < kCopyBatch; ++k) {
      const int e = e0 + 256 * k;
      const int u = e / live, ch = e - u * live;
      pool[k] = static_cast<uint4*>((u & 1) ? a.vp : a.kp);
      at[k] = static_cast<int64_t>(u >> 1) * head + ch;
      if (e < chunks) v[k] = pool[k][src * page + at[k]];
    }
#pragma unroll
    for (int k = 0; k < kCopyBatch; ++k)
      if (e0 + 256 * k < chunks) pool[k][dst * page + at[k]] = v[k];
  }
  if (a.pool.k_exps) {   // int8: the copied codes' exponents
    const int hkv = a.pool.num_kv_heads;
    for (int e = tid; e < 2 * hkv; e += 256) {
      int8_t* x = e < hkv ? a.pool.k_exps : a.pool.v_exps;
      const int g = e < hkv ? e : e - hkv;
      x[static_cast<int64_t>(dst) * hkv + g] = x[static_cast<int64_t>(src) * hkv + g];
    }
  }
  if (a.codes) {
    const int n = a.pool.num_kv_heads * 2 * a.pool.head_dim / 16;
    uint4* codes = reinterpret_cast<uint4*>(a.codes);
    for (int e = tid; e < n; e += 256) codes[static_cast<int64_t>(dst) * n + e] = codes[static_cast<int64_t>(src) * n + e];
    for (int e = tid; e < a.pool.num_kv_heads; e += 256)
      a.exps[static_cast<int64_t>(dst) * a.pool.num_kv_heads + e] = a.exps[static_cast<int64_t>(src) * a.pool.num_kv_heads + e];
  }
}

// A CTA copies kCopyBatch chunks a thread of a pair's page (K, then V), all loads
// before the stores.  Bound by HBM: 1024 pages of 64 KB in 23 us, 5.9 TB/s (a CTA a
// page with one load under way a thread: 31 us), 8192 in 166, 6.5 TB/s; 64 pages 4.3 us.
__global__ void __launch_bounds__(256) copy_blocks_kernel(const PoolView pool, uint4* kp, uint4* vp,
                                                          const int32_t* __restrict__ src,
                                                          const int32_t* __restrict__ dst, int8_t* codes,
                                                          int8_t* exps) {
  const int tid = threadIdx.x;
  griddep_wait();
  griddep_launch();
  const int s = __ldg(src + blockIdx.x), d = __ldg(dst + blockIdx.x);
  if (s < 0 || s >= pool.num_blocks || d < 0 || d >= pool.num_blocks) {
    if (tid == 0) atomicOr(pool.err, PKV_DEVERR_BLOCK_ID);
    return;
  }
  if (s == d) return;
  const int64_t page = static_cast<int64_t>(pool.num_kv_heads) * kBlockSize * pool.head_dim * pool.elem_bytes / 16;
  uint4 v[kCopyBatch];
#pragma unroll
  for (int k = 0; k < kCopyBatch; ++k) {
    const int64_t e = (static_cast<int64_t>(blockIdx.y) * kCopyBatch + k) * 256 + tid;
    if (e < 2 * page) v[k] = e < page ? kp[s * page + e] : vp[s * page + e - page];
  }
#pragma unroll
  for (int k = 0; k < kCopyBatch; ++k) {
    const int64_t e = (static_cast<int64_t>(blockIdx.y) * kCopyBatch + k) * 256 + tid;
    if (e < 2 * page) (e < page ? kp[d * page + e] : vp[d * page + e - page]) = v[k];
  }
  if (pool.k_exps && blockIdx.y == 0) {   // int8: the copied codes' exponents
    const int hkv = pool.num_kv_heads;
    for (int e = tid; e < 2 * hkv; e += 256) {
      int8_t* x = e < hkv ? pool.k_exps : pool.v_exps;
      const int g = e < hkv ? e : e - hkv;
      x[static_cast<int64_t>(d) * hkv + g] = x[static_cast<int64_t>(s) * hkv + g];
    }
  }
  if (codes && blockIdx.y == 0) {
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
// Bound by latency: positions, table, rows, a batch after another (one request,
// 6 kept tokens: 6.2 us; 128 requests of up to 14, 8 heads: 8.3).
constexpr int kMoveBatch = 8;
__global__ void __launch_bounds__(256) compact_kernel(const PoolView pool, uint4* kp, uint4* vp,
                                                      const int32_t* __restrict__ bt, int max_blocks, int num_reqs,
                                                      const int32_t* __restrict__ cu, const int32_t* __restrict__ src,
                                                      const int32_t* __restrict__ dst, int num_kept) {
  const int cpr = pool.head_dim * pool.elem_bytes / 16;   // 16-byte chunks of one head's row
  const int cols = 2 * pool.num_kv_heads * cpr;
  const int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int r = static_cast<int>(e / cols);
  griddep_wait();
  griddep_launch();
  if (e == 0) check_cu(cu, num_reqs, num_kept, pool.err);
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
  return (static_cast<size_t>(3) * num_rows + 3) / 4 * 4 + static_cast<size_t>(8) * num_children + num_blocks;
}

int launch_fork(const ForkArgs& a, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool small = a.num_rows <= kPlanThreads && a.num_children <= kPlanThreads;
  const cudaError_t e = small ? launch_dependent(fork_plan_small_kernel, dim3(1), kPlanThreads, 0, s, a)
                              : launch_dependent(fork_plan_kernel, dim3(1), kPlanThreads, 0, s, a);
  if (e != cudaSuccess || a.num_children == 0) return e;
  return launch_dependent(fork_fill_kernel, dim3(a.num_children), 256, 0, s, a);
}

int launch_copy_blocks(const PoolView& pool, void* kp, void* vp, const int32_t* src, const int32_t* dst, int n,
                       int8_t* codes, int8_t* exps, void* stream) {
  const int64_t chunks = static_cast<int64_t>(2) * pool.num_kv_heads * kBlockSize * pool.head_dim * pool.elem_bytes / 16;
  const dim3 grid(n, static_cast<unsigned>((chunks + 256 * kCopyBatch - 1) / (256 * kCopyBatch)));
  return launch_dependent(copy_blocks_kernel, grid, 256, 0, static_cast<cudaStream_t>(stream), pool,
                          static_cast<uint4*>(kp), static_cast<uint4*>(vp), src, dst, codes, exps);
}

int launch_compact(const PoolView& pool, void* kp, void* vp, const int32_t* block_tables, int max_blocks, int num_reqs,
                   const int32_t* cu_keep, const int32_t* src, const int32_t* dst, int num_kept, void* stream) {
  const int64_t cols = static_cast<int64_t>(2) * pool.num_kv_heads * (pool.head_dim * pool.elem_bytes / 16);
  const int64_t grid = (cols * num_reqs + 255) / 256;
  return launch_dependent(compact_kernel, dim3(static_cast<unsigned>(grid)), 256, 0, static_cast<cudaStream_t>(stream), pool,
                          static_cast<uint4*>(kp), static_cast<uint4*>(vp), block_tables, max_blocks, num_reqs, cu_keep,
                          src, dst, num_kept);
}

}  // namespace pkv
