// Launchers of the operators beside the causal paged attention (tree
// attention, block-selected attention, pages); they return cudaError_t as int.
#pragma once
#include "internal.h"

namespace pkv {

struct TreeArgs;

// Launches a kernel that may be scheduled before the one ahead of it in the
// stream ends: it begins with griddep_wait().  What a kernel that releases its
// dependents early (griddep_launch) writes must not be read through the
// non-coherent path (__ldg) by the next: queries (they may be an output), mask
// words, lists, bounds, owners' counts and pool values are read with plain loads,
// __ldcg, cp.async or TMA, which see the writes behind griddep_wait().  Tables,
// lengths, positions and ids may be read with __ldg: of these calls only the
// fork's fill writes any (tables), and it lets nothing start before it ends.
// (summarize_kernel, which reads keys with __ldg, is launched without this.)
#ifdef __CUDACC__
template <class... Params, class... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, int threads, int smem, cudaStream_t s,
                             const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
#endif

// The two forms of the tree attention: warp-level MMA on 16 query rows, or
// tcgen05 on tiles of 128.
struct TreeForm {
  bool tensor;
  int ctas, cuts, slots, slot_rows;
  int many_groups;   // rows form: from so many groups on, a share a warp
  int whole;         // rows form: CTAs take whole groups, nothing is merged
  int warps;         // rows form: warps of a CTA (4; whole groups 4, 6 or 12)
  void shrink(int n) {
    cuts = cuts / ctas * n;
    ctas = n;
  }
};
TreeForm tree_form(bool tensor, int num_sms);
constexpr int kWholeBlocks = 32;   // blocks of a group up to which it stays whole
// Rows form: the record of a group that CTA `block` of W warps (`solo`: its warp
// `warp` by itself) begins and others go on with.  It is one of the CTA's own W
// records, which the CTA clears when it starts: no other CTA writes them.
#ifdef __CUDACC__
__host__ __device__
#endif
inline int cut_record(int block, int W, bool solo, int warp) { return block * W + (solo ? warp : 0); }
// tmk / tmv: the pool's block maps; tmq: q viewed as [T][Hq][D] in boxes of one tile.
// (launch_tree_rows also runs the attention over selected blocks.)
int launch_tree_rows(const TreeArgs& a, void* stream);
int launch_tree_tc(const TreeArgs& a, const void* tmk, const void* tmv, const void* tmq, void* stream);
int launch_tree_merge(const TreeArgs& a, void* stream);
int launch_score_merge(const TreeArgs& a, int row_tile, int64_t groups, void* stream);   // groups: at most, of the call
int launch_tree_mask(const int32_t* parents, const int32_t* cu, int num_reqs, int num_tokens, uint32_t* mask, int words,
                     unsigned* err, void* stream);

// One call of pkv_summarize or pkv_select_blocks.
struct SparseArgs {
  PoolView pool;
  const void* q;
  int num_q_heads, group;
  const int32_t* positions;
  const int32_t* block_tables;
  int max_blocks;
  const int32_t* cu_q_lens;
  const int32_t* ctx_lens;
  int num_reqs, num_tokens;
  int8_t* codes;     // [blocks][kv heads][2][D]: upper, lower
  int8_t* exps;      // [blocks][kv heads]
  int32_t* sel;      // [tokens][kv heads][top_k]
  int top_k, sinks, recent;
  int num_sms;
  // Selection: the keys [tokens of a part][kv heads][max_blocks] (workspace) of
  // tokens [tok_first, tok_first + tok_count), tok_most tokens a part.
  uint32_t* keys;
  int tok_first, tok_count, tok_most;
};
int launch_summarize(const SparseArgs& a, void* stream);
// The tokens of a part.
int select_part(int num_tokens, int max_blocks, int num_kv_heads);
int launch_select(const SparseArgs& a, void* stream);

// pkv_fork.
struct ForkArgs {
  PoolView pool;
  void* kp;
  void* vp;
  const int32_t* tables;
  int num_rows, max_blocks;
  const int32_t* lens;
  const int32_t* caps;
  const int32_t* parents;
  const int32_t* new_caps;
  int num_children;
  int32_t* new_tables;
  const int32_t* refs;
  int32_t* new_refs;
  int8_t* codes;      // summaries to copy along, or nullptr
  int8_t* exps;
  int32_t* ws;        // fork_ws_ints() ints
};
size_t fork_ws_ints(int num_blocks, int num_rows, int num_children);
int launch_fork(const ForkArgs& a, void* stream);
int launch_copy_blocks(const PoolView& pool, void* kp, void* vp, const int32_t* src, const int32_t* dst, int n,
                       int8_t* codes, int8_t* exps, void* stream);
int launch_compact(const PoolView& pool, void* kp, void* vp, const int32_t* block_tables, int max_blocks, int num_reqs,
                   const int32_t* cu_keep, const int32_t* src, const int32_t* dst, int num_kept, void* stream);
// pkv_score_attn: the form for few query rows, the form on tiles of 128.
struct ScoreArgs;
int launch_score_rows(const ScoreArgs& a, void* stream);
template <int D>
int launch_score_tc(const ScoreArgs& a, const void* tmk, const void* tmv, const void* tmq, void* stream);

// pkv_append_int8 (int8 pools), pkv_read_rows (any).
int launch_append_int8(const PoolView& pool, void* kp, void* vp, const int32_t* bt, int max_blocks, int num_reqs,
                       const int32_t* cu, const int32_t* pos, const int32_t* held, const void* k_new, const void* v_new,
                       int num_tokens, int num_sms, void* stream);
int launch_read_rows(const PoolView& pool, const int32_t* bt, int max_blocks, int num_reqs, const int32_t* cu,
                     const int32_t* pos, int num_tokens, void* k_out, void* v_out, int num_sms, void* stream);

}  // namespace pkv
