// C entry points of the operators beside the causal paged attention: tree
// attention, block-selected attention, pages.  Their lengths, tables and masks
// are read on the device alone, so that the calls can be captured in a graph;
// they keep nothing from one call for the next and run on the caller's stream.
// A call of several kernels holds the pool's lock while it launches them, so that
// calls from two threads on one stream, which may share a workspace, follow one
// another.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "internal.h"
#include "ops.h"
#include "pool.h"
#include "sched.cuh"

using namespace pkv;

namespace {

// Makes the pool's device current for a call's launches.
class DeviceGuard {
 public:
  explicit DeviceGuard(int device) {
    if (cudaGetDevice(&prev_) != cudaSuccess) prev_ = device;
    if (prev_ != device) cudaSetDevice(device);
    device_ = device;
  }
  ~DeviceGuard() {
    if (prev_ != device_) cudaSetDevice(prev_);
  }
  DeviceGuard(const DeviceGuard&) = delete;
  DeviceGuard& operator=(const DeviceGuard&) = delete;

 private:
  int prev_ = 0, device_ = 0;
};

int check_tables(int max_blocks, int num_reqs, int num_tokens) {
  if (num_tokens < 0 || num_reqs < 0) return fail(PKV_EINVAL, "negative size");
  if (num_tokens == 0) return PKV_OK;
  if (num_reqs < 1 || max_blocks < 1) return fail(PKV_EINVAL, "num_reqs and max_blocks must be >= 1");
  // (Key positions, rounded up to a tile, stay below 2^31.)
  if (static_cast<int64_t>(max_blocks) * kBlockSize > (1ll << 31) - 1 - kTcKeys) return fail(PKV_EINVAL, "max_blocks too large");
  return PKV_OK;
}

int check_heads(const pkv_pool* pool, int num_q_heads) {
  if (num_q_heads < 1 || num_q_heads % pool->num_kv_heads)
    return fail(PKV_EINVAL, "num_q_heads must be a multiple of num_kv_heads");
  if (num_q_heads / pool->num_kv_heads > kTcRows) return fail(PKV_EUNSUPPORTED, "group size above 128");
  return PKV_OK;
}

int check_scale(float scale) {
  return scale > 0.f && scale <= 3.4e38f ? PKV_OK : fail(PKV_EINVAL, "scale must be positive and finite");
}

int check_top_k(int top_k) {
  return top_k >= 1 && top_k <= (1 << 27) ? PKV_OK : fail(PKV_EINVAL, "top_k must be in 1 .. 2^27");
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct TreeWs {
  size_t cuts, part_o, part_lse, total;
};
TreeWs tree_ws(const pkv_pool* pool, const TreeForm& f) {
  const size_t rows = static_cast<size_t>(f.slots) * f.slot_rows;
  TreeWs w;
  w.cuts = 0;
  w.part_o = align256(f.cuts * sizeof(TreeCut));
  w.part_lse = w.part_o + align256(rows * pool->head_dim * sizeof(float));
  w.total = w.part_lse + align256(rows * sizeof(float));
  return w;
}

TreeArgs tree_args(const pkv_pool* pool, const TreeForm& f, const TreeWs& w, void* workspace) {
  TreeArgs a{};
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.pool = pool->view();
  a.cuts = reinterpret_cast<TreeCut*>(ws + w.cuts);
  a.part_o = reinterpret_cast<float*>(ws + w.part_o);
  a.part_lse = reinterpret_cast<float*>(ws + w.part_lse);
  a.form = f;
  a.ctas = f.ctas;
  a.wait_ns = pool->wait_ns;
  a.withhold = pool->withhold;
  return a;
}

// Launches as many CTAs as `groups` groups of `blocks` blocks (key tiles) can
// occupy, both upper bounds: 16 blocks a CTA of the rows form, a tile a CTA of the
// tiles form (an even number: quads go to pairs of CTAs).  Whole groups, a CTA
// each, need no merge.  They are taken
//   - where groups are short (kWholeBlocks);
//   - where a CTA of twelve warps on every SM is no more than six blocks a warp
//     behind equal shares, if all groups are equally long (lists, one request; D =
//     128, us, shares / whole: 8 groups of 38 blocks 18.5 / 14.4, of 250 20.6 /
//     30.8; 32 lists of 64 24.7 / 22.7, of 128 26.7 / 28.7, of 256 28.9 / 37.9; 120
//     lists of 128 45.7 / 41.4);
//   - up to kNearBlocks blocks and a CTA an SM, if requests may differ: a longer
//     table may be that of one request of many, whose groups are then waited for (12
//     requests of 97 to 1236 blocks, 422 on average, 8 KV heads, a row tile each: bf16
//     64.6 / 103.5, FP8 48.0 / 94.6; 6 of 23 to 147: 24.8 / 22.8, 28.3 / 24.6; equally
//     long ones: 16 groups of 128 20.3 / 20.7, of 192 22.7 / 26.0; 64 of 96 24.7 /
//     18.6, of 128 25.1 / 22.6, of 256 41.8 / 36.9; 144 of 256 64.8 / 57.5);
//   - for lists, which are all equally long, where there are enough of them to keep
//     the memory busy (256 of 128 blocks: 91 us for selection and attention with
//     shares, 85 with whole groups).
// An SM holds twelve warps of this kernel: as one CTA, two or three, so that all
// groups are under way (selection and attention, us, three CTAs / two; 256 lists of
// 16 41.4 / 41.1, of 64 60.0 / 59.3, of 128 80.8 / 79.9, of 512 194 / 193, of 1024
// 328 / 324; 160 of 128 63.0 / 59.9, of 1024 257 / 229; 304 of 128 90.2 / 89.3, of 1024
// 378 / 379; FP8: 280 of 64 53.5 / 50.8, of 128 65.8 / 63.5, of 1024 242 / 198).
constexpr int kNearBlocks = 160;
void fit_ctas(TreeArgs& a, int64_t groups, int blocks, int num_sms) {
  const bool equal = a.sel || a.num_reqs == 1;
  const int64_t units = groups * (static_cast<int64_t>(blocks) + 2);
  const bool near = groups <= num_sms && blocks <= (equal ? 74 + std::max<int64_t>(48, groups * blocks / num_sms) : kNearBlocks);
  a.form.whole = !a.form.tensor && groups <= a.form.ctas && (blocks <= kWholeBlocks || near || (a.sel && groups >= num_sms));
  const int64_t want = a.form.whole ? groups : a.form.tensor ? (units + 1) / 2 * 2 : (units + 15) / 16;
  a.form.shrink(static_cast<int>(std::min<int64_t>(want < 2 ? 2 : want, a.form.ctas)));
  a.ctas = a.form.ctas;
  if (a.form.whole) a.form.warps = groups <= num_sms ? 12 : groups <= 2 * num_sms ? 6 : 4;
}

int check_workspace(const void* workspace, size_t have, size_t need, const char* size_fn) {
  if (!workspace || have < need) return fail(PKV_EINVAL, std::string("workspace missing or smaller than ") + size_fn);
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return fail(PKV_EINVAL, "workspace must be 256-byte aligned");
  return PKV_OK;
}

// Which form a batch takes, by its mean number of query rows a (request, KV
// head).  The rows form reads K and V once for every 16 rows, the tiles form once
// for 128 (or 256), but has more to start and, for FP8 pools, to widen.  Measured
// (rows / tiles, us): bf16, D = 128, 12 requests of 1.5 to 20 thousand tokens, 8
// KV heads: 16 rows 67 / 68, 24 rows 90 / 68, 64 rows 118 / 70; D = 64, 32 requests
// of 1 to 3 thousand, 8 KV heads: 32 rows 39 / 45, 48 rows 49 / 45; FP8, D = 128, the
// same 12 requests: 32 rows 66 / 85, 48 rows 80 / 86, 64 rows 96 / 87; 24 requests of
// 300 to 4000 tokens, 40 KV heads: 32 rows 136 / 216, 64 rows 256 / 235.
// A batch that gives every CTA of the rows form 16 blocks at most stays there
// (one request of 240 tokens, 2 KV heads, D = 64, 128 rows: 8.9 / 13.8).  The table's
// width stands for the contexts' lengths, which only the device knows.
bool tree_tensor(const pkv_pool* pool, int num_q_heads, int num_reqs, int num_tokens, int max_blocks) {
  if (pool->tree_form != 0) return pool->tree_form == 2;
  if (num_reqs < 1) return false;
  const int64_t rows = static_cast<int64_t>(num_tokens) * (num_q_heads / pool->num_kv_heads);
  const int64_t most = pool->elem_bytes == 1 ? 44 : pool->head_dim == 64 ? 40 : 20;
  const int64_t work = (rows / 16 + num_reqs) * pool->num_kv_heads * max_blocks;   // at most
  return rows > most * num_reqs && work > 16ll * 3 * pool->num_sms;
}

size_t select_ws(const pkv_pool* pool, int max_blocks, int num_tokens) {
  return align256(static_cast<size_t>(select_part(num_tokens, max_blocks, pool->num_kv_heads)) * max_blocks *
                  pool->num_kv_heads * sizeof(uint32_t));
}

int check_summary(const void* codes, const void* exps) {
  if (!codes || !exps) return fail(PKV_EINVAL, "NULL summary arrays");
  if (!aligned16(codes)) return fail(PKV_EINVAL, "summary codes must be 16-byte aligned");
  return PKV_OK;
}

}  // namespace

extern "C" {

int pkv_tree_mask(pkv_pool* pool, const int32_t* parents, const int32_t* cu_q_lens, int num_reqs, int num_tokens,
                  uint32_t* tree_mask, int mask_words, void* stream) {
  if (!pool) return fail(PKV_EINVAL, "pool is NULL");
  if (num_tokens < 0 || num_reqs < 0) return fail(PKV_EINVAL, "negative size");
  if (num_tokens == 0) return PKV_OK;
  if (num_reqs < 1) return fail(PKV_EINVAL, "num_reqs must be >= 1");
  if (mask_words < 1) return fail(PKV_EINVAL, "mask_words must be >= 1");
  if (!parents || !cu_q_lens || !tree_mask) return fail(PKV_EINVAL, "NULL device pointer");
  DeviceGuard guard(pool->device);
  const int rc = launch_tree_mask(parents, cu_q_lens, num_reqs, num_tokens, tree_mask, mask_words, pool->d_err, stream);
  if (rc != cudaSuccess) return cuda_fail(static_cast<cudaError_t>(rc), "tree mask launch");
  return PKV_OK;
}

int pkv_tree_attn_workspace_size(pkv_pool* pool, int num_q_heads, int max_blocks, int num_reqs, int num_tokens,
                                 size_t* bytes) {
  if (!pool || !bytes) return fail(PKV_EINVAL, "pool/bytes is NULL");
  const int rc = check_heads(pool, num_q_heads);
  if (rc) return rc;
  if (num_reqs < 0 || num_tokens < 0 || max_blocks < 0) return fail(PKV_EINVAL, "negative size");
  *bytes = tree_ws(pool, tree_form(tree_tensor(pool, num_q_heads, num_reqs, num_tokens, max_blocks), pool->num_sms)).total;
  return PKV_OK;
}

int pkv_tree_attn(pkv_pool* pool, const void* q, int num_q_heads, const int32_t* block_tables, int max_blocks,
                  const int32_t* ctx_lens, const int32_t* prefix_lens, const int32_t* cu_q_lens, int num_reqs,
                  int num_tokens, const uint32_t* tree_mask, int mask_words, float scale, void* o, float* lse,
                  void* workspace, size_t workspace_bytes, void* stream) {
  if (!pool) return fail(PKV_EINVAL, "pool is NULL");
  int rc = check_tables(max_blocks, num_reqs, num_tokens);
  if (rc || num_tokens == 0) return rc;
  if ((rc = check_heads(pool, num_q_heads)) || (rc = check_scale(scale))) return rc;
  if (!q || !block_tables || !ctx_lens || !prefix_lens || !cu_q_lens || !tree_mask || !o)
    return fail(PKV_EINVAL, "NULL device pointer");
  if (mask_words < 1) return fail(PKV_EINVAL, "mask_words must be >= 1");
  if (!aligned16(q) || !aligned16(o)) return fail(PKV_EINVAL, "q and o must be 16-byte aligned");
  if (static_cast<int64_t>(num_tokens) * num_q_heads >= (1ll << 31)) return fail(PKV_EUNSUPPORTED, "too many query rows");
  const TreeForm form = tree_form(tree_tensor(pool, num_q_heads, num_reqs, num_tokens, max_blocks), pool->num_sms);
  const TreeWs w = tree_ws(pool, form);
  if ((rc = check_workspace(workspace, workspace_bytes, w.total, "pkv_tree_attn_workspace_size()"))) return rc;
  DeviceGuard guard(pool->device);
  if ((rc = finish_swap_in(pool, stream))) return rc;
  std::lock_guard<std::mutex> lk(pool->mu);
  TreeArgs a = tree_args(pool, form, w, workspace);
  a.q = q;
  a.num_q_heads = num_q_heads;
  a.group = num_q_heads / pool->num_kv_heads;
  a.block_tables = block_tables;
  a.max_blocks = max_blocks;
  a.ctx_lens = ctx_lens;
  a.prefix_lens = prefix_lens;
  a.cu_q_lens = cu_q_lens;
  a.num_reqs = num_reqs;
  a.num_tokens = num_tokens;
  a.mask = tree_mask;
  a.mask_words = mask_words;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.o = o;
  a.lse = lse;
  a.tile_tokens = kTcRows / a.group;
  // No more CTAs than the largest batch of these sizes can use.
  const int64_t groups = (static_cast<int64_t>(num_tokens) * a.group / (form.tensor ? kTcRows : 16) + num_reqs) *
                         pool->num_kv_heads;
  fit_ctas(a, groups, form.tensor ? max_blocks / 8 + 1 : max_blocks, pool->num_sms);
  a.o_align32 = (reinterpret_cast<uintptr_t>(o) & 31u) == 0;
  if (form.tensor) {
    CUtensorMap tmap_q;
    if ((rc = make_q_tmap(&tmap_q, q, num_tokens, num_q_heads, pool->head_dim, a.group, &a.q_box_tokens))) return rc;
    rc = timed_launch(pool, 2, stream, [&] { return launch_tree_tc(a, &pool->tmap_k, &pool->tmap_v, &tmap_q, stream); });
  } else {
    rc = timed_launch(pool, 1, stream,
                      [&] { return launch_tree_rows(a, stream); });
  }
  if (rc != cudaSuccess) return cuda_fail(static_cast<cudaError_t>(rc), "tree attention launch");
  if (a.form.whole) return PKV_OK;
  rc = timed_launch(pool, 3, stream, [&] { return launch_tree_merge(a, stream); });
  if (rc != cudaSuccess) return cuda_fail(static_cast<cudaError_t>(rc), "tree merge launch");
  return PKV_OK;
}

int pkv_summarize(pkv_pool* pool, const int32_t* block_tables, int max_blocks, int num_reqs, const int32_t* cu_q_lens,
                  const int32_t* positions, const int32_t* ctx_lens, int num_tokens, int8_t* codes, int8_t* exps,
                  void* stream) {
  if (!pool) return fail(PKV_EINVAL, "pool is NULL");
  int rc = check_tables(max_blocks, num_reqs, num_tokens);
  if (rc || num_tokens == 0) return rc;
  if (!block_tables || !cu_q_lens || !positions || !ctx_lens) return fail(PKV_EINVAL, "NULL device pointer");
  if ((rc = check_summary(codes, exps))) return rc;
  if (static_cast<int64_t>(num_tokens) * pool->num_kv_heads >= (1ll << 31)) return fail(PKV_EUNSUPPORTED, "too many rows");
  DeviceGuard guard(pool->device);
  if ((rc = finish_swap_in(pool, stream))) return rc;
  SparseArgs a{};
  a.pool = pool->view();
  a.positions = positions;
  a.block_tables = block_tables;
  a.max_blocks = max_blocks;
  a.cu_q_lens = cu_q_lens;
  a.ctx_lens = ctx_lens;
  a.num_reqs = num_reqs;
  a.num_tokens = num_tokens;
  a.codes = codes;
  a.exps = exps;
  a.num_sms = pool->num_sms;
  rc = timed_launch(pool, 0, stream, [&] { return launch_summarize(a, stream); });
  if (rc != cudaSuccess) return cuda_fail(static_cast<cudaError_t>(rc), "summarize launch");
  return PKV_OK;
}

int pkv_select_blocks_workspace_size(pkv_pool* pool, int max_blocks, int num_tokens, size_t* bytes) {
  if (!pool || !bytes) return fail(PKV_EINVAL, "pool/bytes is NULL");
  const int rc = check_tables(max_blocks, 1, num_tokens);
  if (rc) return rc;
  *bytes = num_tokens == 0 ? 256 : select_ws(pool, max_blocks, num_tokens);
  return PKV_OK;
}

int pkv_select_blocks(pkv_pool* pool, const void* q, int num_q_heads, const int32_t* q_positions,
                      const int32_t* block_tables, int max_blocks, const int32_t* cu_q_lens, int num_reqs,
                      int num_tokens, const int8_t* codes, const int8_t* exps, int top_k, int sinks, int recent,
                      int32_t* selected, void* workspace, size_t workspace_bytes, void* stream) {
  if (!pool) return fail(PKV_EINVAL, "pool is NULL");
  int rc = check_tables(max_blocks, num_reqs, num_tokens);
  if (rc) return rc;
  if ((rc = check_top_k(top_k))) return rc;
  if (sinks < 0 || recent < 0) return fail(PKV_EINVAL, "need sinks >= 0, recent >= 0");
  if (num_tokens == 0) return PKV_OK;
  if ((rc = check_heads(pool, num_q_heads))) return rc;
  if (!q || !q_positions || !block_tables || !cu_q_lens || !selected) return fail(PKV_EINVAL, "NULL device pointer");
  if (!aligned16(q)) return fail(PKV_EINVAL, "q must be 16-byte aligned");
  if ((rc = check_summary(codes, exps))) return rc;
  if ((rc = check_workspace(workspace, workspace_bytes, select_ws(pool, max_blocks, num_tokens),
                            "pkv_select_blocks_workspace_size()")))
    return rc;
  DeviceGuard guard(pool->device);
  SparseArgs a{};
  a.pool = pool->view();
  a.q = q;
  a.num_q_heads = num_q_heads;
  a.group = num_q_heads / pool->num_kv_heads;
  a.positions = q_positions;
  a.block_tables = block_tables;
  a.max_blocks = max_blocks;
  a.cu_q_lens = cu_q_lens;
  a.num_reqs = num_reqs;
  a.num_tokens = num_tokens;
  a.codes = const_cast<int8_t*>(codes);
  a.exps = const_cast<int8_t*>(exps);
  a.sel = selected;
  a.top_k = top_k;
  a.sinks = std::min(sinks, max_blocks);
  a.recent = std::min(recent, max_blocks);
  a.num_sms = pool->num_sms;
  std::lock_guard<std::mutex> lk(pool->mu);
  a.keys = static_cast<uint32_t*>(workspace);
  a.tok_most = select_part(num_tokens, max_blocks, pool->num_kv_heads);
  rc = timed_launch(pool, 0, stream, [&] { return launch_select(a, stream); });
  if (rc != cudaSuccess) return cuda_fail(static_cast<cudaError_t>(rc), "block selection launch");
  return PKV_OK;
}

int pkv_sparse_attn_workspace_size(pkv_pool* pool, size_t* bytes) {
  if (!pool || !bytes) return fail(PKV_EINVAL, "pool/bytes is NULL");
  *bytes = tree_ws(pool, tree_form(false, pool->num_sms)).total;
  return PKV_OK;
}

int pkv_sparse_attn(pkv_pool* pool, const void* q, int num_q_heads, const int32_t* q_positions,
                    const int32_t* block_tables, int max_blocks, const int32_t* cu_q_lens, int num_reqs, int num_tokens,
                    const int32_t* selected, int top_k, float scale, void* o, float* lse, void* workspace,
                    size_t workspace_bytes, void* stream) {
  if (!pool) return fail(PKV_EINVAL, "pool is NULL");
  int rc = check_tables(max_blocks, num_reqs, num_tokens);
  if (rc) return rc;
  if ((rc = check_top_k(top_k))) return rc;
  if (num_tokens == 0) return PKV_OK;
  if ((rc = check_heads(pool, num_q_heads)) || (rc = check_scale(scale))) return rc;
  if (!q || !q_positions || !block_tables || !cu_q_lens || !selected || !o) return fail(PKV_EINVAL, "NULL device pointer");
  if (!aligned16(q) || !aligned16(o)) return fail(PKV_EINVAL, "q and o must be 16-byte aligned");
  const TreeForm form = tree_form(false, pool->num_sms);
  const TreeWs w = tree_ws(pool, form);
  if ((rc = check_workspace(workspace, workspace_bytes, w.total, "pkv_sparse_attn_workspace_size()"))) return rc;
  DeviceGuard guard(pool->device);
  if ((rc = finish_swap_in(pool, stream))) return rc;
  std::lock_guard<std::mutex> lk(pool->mu);
  TreeArgs a = tree_args(pool, form, w, workspace);
  a.q = q;
  a.num_q_heads = num_q_heads;
  a.group = num_q_heads / pool->num_kv_heads;
  a.positions = q_positions;
  a.block_tables = block_tables;
  a.max_blocks = max_blocks;
  a.cu_q_lens = cu_q_lens;
  a.num_reqs = num_reqs;
  a.num_tokens = num_tokens;
  a.sel = selected;
  a.top_k = top_k;
  fit_ctas(a, static_cast<int64_t>(num_tokens) * pool->num_kv_heads * ((a.group + 15) / 16), top_k, pool->num_sms);
  a.scale_log2 = scale * 1.4426950408889634f;
  a.o = o;
  a.lse = lse;
  rc = timed_launch(pool, 1, stream,
                    [&] { return launch_tree_rows(a, stream); });
  if (rc != cudaSuccess) return cuda_fail(static_cast<cudaError_t>(rc), "block-selected attention launch");
  if (a.form.whole) return PKV_OK;
  rc = timed_launch(pool, 3, stream, [&] { return launch_tree_merge(a, stream); });
  if (rc != cudaSuccess) return cuda_fail(static_cast<cudaError_t>(rc), "block-selected merge launch");
  return PKV_OK;
}

int pkv_fork_workspace_size(pkv_pool* pool, int num_rows, int num_children, size_t* bytes) {
  if (!pool || !bytes) return fail(PKV_EINVAL, "pool/bytes is NULL");
  if (num_rows < 0 || num_children < 0) return fail(PKV_EINVAL, "negative size");
  *bytes = align256(fork_ws_ints(pool->num_blocks, num_rows, num_children) * sizeof(int32_t));
  return PKV_OK;
}

int pkv_fork(pkv_pool* pool, const int32_t* tables, int num_rows, int max_blocks, const int32_t* lens,
             const int32_t* caps, const int32_t* parents, const int32_t* new_caps, int num_children,
             int32_t* new_tables, const int32_t* refs, int32_t* new_refs, int8_t* codes, int8_t* exps, void* workspace,
             size_t workspace_bytes, void* stream) {
  if (!pool) return fail(PKV_EINVAL, "pool is NULL");
  if (num_rows < 0 || num_children < 0) return fail(PKV_EINVAL, "negative size");
  if (max_blocks < 1 || static_cast<int64_t>(max_blocks) * kBlockSize > (1ll << 31) - 1 - kTcKeys)
    return fail(PKV_EINVAL, "max_blocks must be >= 1 and leave positions below 2^31");
  if ((num_rows > 0 && (!tables || !lens || !caps)) || (num_children > 0 && (!parents || !new_caps || !new_tables)) ||
      !refs || !new_refs)
    return fail(PKV_EINVAL, "NULL device pointer");
  if (num_rows > 0 && num_children > 0) {
    // A child's row is written while other children still read their parent's.
    const uintptr_t t0 = reinterpret_cast<uintptr_t>(tables), n0 = reinterpret_cast<uintptr_t>(new_tables);
    const uintptr_t tb = static_cast<uintptr_t>(num_rows) * max_blocks * 4, nb = static_cast<uintptr_t>(num_children) * max_blocks * 4;
    if (t0 < n0 + nb && n0 < t0 + tb) return fail(PKV_EINVAL, "new_tables must not overlap tables");
  }
  if ((codes == nullptr) != (exps == nullptr)) return fail(PKV_EINVAL, "give both summary arrays or neither");
  if (codes && !aligned16(codes)) return fail(PKV_EINVAL, "summary codes must be 16-byte aligned");
  const size_t need = fork_ws_ints(pool->num_blocks, num_rows, num_children) * sizeof(int32_t);
  if (!workspace || workspace_bytes < need)
    return fail(PKV_EINVAL, "workspace missing or smaller than pkv_fork_workspace_size()");
  if (reinterpret_cast<uintptr_t>(workspace) & 15u) return fail(PKV_EINVAL, "workspace must be 16-byte aligned");
  DeviceGuard guard(pool->device);
  int rc = finish_swap_in(pool, stream);
  if (rc) return rc;
  std::lock_guard<std::mutex> lk(pool->mu);
  ForkArgs a{pool->view(), pool->k, pool->v, tables, num_rows, max_blocks, lens, caps, parents, new_caps, num_children,
             new_tables, refs, new_refs, codes, exps, static_cast<int32_t*>(workspace)};
  rc = timed_launch(pool, 0, stream, [&] { return launch_fork(a, stream); });
  if (rc != cudaSuccess) return cuda_fail(static_cast<cudaError_t>(rc), "fork launch");
  return PKV_OK;
}

int pkv_copy_blocks(pkv_pool* pool, const int32_t* src, const int32_t* dst, int n, int8_t* codes, int8_t* exps,
                    void* stream) {
  if (!pool) return fail(PKV_EINVAL, "pool is NULL");
  if (n < 0) return fail(PKV_EINVAL, "negative count");
  if (n == 0) return PKV_OK;
  if (!src || !dst) return fail(PKV_EINVAL, "NULL device pointer");
  if ((codes == nullptr) != (exps == nullptr)) return fail(PKV_EINVAL, "give both summary arrays or neither");
  if (codes && !aligned16(codes)) return fail(PKV_EINVAL, "summary codes must be 16-byte aligned");
  DeviceGuard guard(pool->device);
  int rc = finish_swap_in(pool, stream);
  if (rc) return rc;
  rc = timed_launch(pool, 0, stream, [&] {
    return launch_copy_blocks(pool->view(), pool->k, pool->v, src, dst, n, codes, exps, stream);
  });
  if (rc != cudaSuccess) return cuda_fail(static_cast<cudaError_t>(rc), "block copy launch");
  return PKV_OK;
}

int pkv_compact(pkv_pool* pool, const int32_t* block_tables, int max_blocks, int num_reqs, const int32_t* cu_keep,
                const int32_t* src_positions, const int32_t* dst_starts, int num_kept, void* stream) {
  if (!pool) return fail(PKV_EINVAL, "pool is NULL");
  int rc = check_tables(max_blocks, num_reqs, num_kept);
  if (rc || num_kept == 0) return rc;
  if (!block_tables || !cu_keep || !src_positions || !dst_starts) return fail(PKV_EINVAL, "NULL device pointer");
  if (static_cast<int64_t>(num_reqs) * pool->num_kv_heads * pool->head_dim >= (1ll << 31))
    return fail(PKV_EUNSUPPORTED, "too many rows");
  DeviceGuard guard(pool->device);
  if ((rc = finish_swap_in(pool, stream))) return rc;
  rc = timed_launch(pool, 0, stream, [&] {
    return launch_compact(pool->view(), pool->k, pool->v, block_tables, max_blocks, num_reqs, cu_keep, src_positions,
                          dst_starts, num_kept, stream);
  });
  if (rc != cudaSuccess) return cuda_fail(static_cast<cudaError_t>(rc), "compact launch");
  return PKV_OK;
}

}  // extern "C"
