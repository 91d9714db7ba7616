// The pool object and the helpers that the C entry points share.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <mutex>
#include <string>
#include <vector>

#include "internal.h"

namespace pkv {

inline int fail(int code, const std::string& msg) { return set_last_error(code, msg); }
inline int cuda_fail(cudaError_t e, const char* what) {
  return set_last_error(PKV_ECUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

#define PKV_CUDA(call, what)                 \
  do {                                       \
    cudaError_t e_ = (call);                 \
    if (e_ != cudaSuccess) return pkv::cuda_fail(e_, what); \
  } while (0)

struct ProfRec {
  int kernel;
  cudaEvent_t a, b;
};

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace pkv

struct pkv_pool {
  int num_blocks = 0, block_size = 0, num_kv_heads = 0, head_dim = 0;
  int elem_bytes = 2;                 // 2: bf16; 1: fp8 e4m3 or int8 codes
  float k_scale = 1.f, v_scale = 1.f;
  int8_t* k_exps = nullptr;           // int8 pools (elem_bytes 1): exponents [num_blocks][num_kv_heads]
  int8_t* v_exps = nullptr;
  void* k = nullptr;
  void* v = nullptr;
  bool owns = false;
  unsigned* d_err = nullptr;
  int device = 0, num_sms = 0;
  CUtensorMap tmap_k;  // 64-byte aligned by its type
  CUtensorMap tmap_v;
  CUtensorMap dmap_k;  // split-KV kernel's maps (FP8, D = 128); copies of tmap_* otherwise
  CUtensorMap dmap_v;
  std::mutex mu;
  pkv::Plan plan;
  // Pinned, double-buffered staging for work-list uploads (allocated at
  // creation; a work list larger than one slot goes through pageable memory).
  static constexpr size_t kStagingBytes = size_t(4) << 20;
  uint8_t* pinned[2] = {nullptr, nullptr};
  cudaEvent_t pinned_done[2] = {nullptr, nullptr};
  int pinned_slot = 0;
  std::vector<uint8_t> staging;
  // The tensor-core kernel runs on `side`, concurrently with the split-KV
  // kernel on the caller's stream (fork / join through the two events).
  cudaStream_t side = nullptr;
  cudaEvent_t fork = nullptr, join = nullptr;
  // Recorded after each attention call's kernels: the next call's work-list
  // upload waits for it before rewriting the work lists.
  cudaEvent_t ws_free = nullptr;
  // Device copy of the work lists, owned by the pool (kStagingBytes): the
  // upload into it runs on the pool's copy stream, ordered after the previous
  // call's kernels only, so it overlaps the caller's earlier work (the
  // append, the next step's input copies) and never queues behind it.  The
  // caller's workspace, whose memory may still be in use by work queued on
  // the caller's stream, is written only by kernels on that stream.
  // Two buffers, used by alternate calls (with the pinned staging slots): an
  // upload then waits only for the call before the previous one, long done,
  // so it is ready to run when it is submitted and does not queue on the
  // copy engine behind transfers submitted after it (a serving loop's next
  // inputs).
  uint8_t* d_wl[2] = {nullptr, nullptr};
  cudaEvent_t wl_free[2] = {nullptr, nullptr};
  cudaStream_t copy = nullptr;
  cudaEvent_t up_done = nullptr;
  // Ahead-of-time swap-in: the copy engines bring the blocks into a device
  // staging buffer on the caller's copy stream (swap_ready), and the pool's
  // next call scatters them into place on its own stream (staged_free).
  std::mutex swap_mu;
  void* swap_staging = nullptr;
  size_t swap_staging_bytes = 0;
  cudaEvent_t swap_ready = nullptr, swap_staged_free = nullptr, swap_after = nullptr;
  bool swap_pending = false;
  unsigned long long swap_capture = 0;   // the capture that the pending transfer is part of (0: none)
  std::vector<int32_t> swap_ids;

  // Test and diagnostic settings (pkv_debug_set).
  uint64_t wait_ns = 1000000000ull;   // limit of every bounded wait in the kernels
  int withhold = 0;                   // see AttnArgs::withhold
  int fused_form = 0;                 // PKV_DEBUG_FUSED_FORM
  int tree_form = 0;                  // PKV_DEBUG_TREE_FORM

  // profiling (prof_mode 2: the two attention kernels run one after the other).
  // Not every call that launches holds `mu`: the lists have a lock of their own.
  std::atomic<bool> prof_on{false};
  std::atomic<int> prof_mode{0};
  std::mutex prof_mu;
  std::vector<cudaEvent_t> ev_free;
  std::vector<pkv::ProfRec> pending;
  pkv_profile totals{};

  pkv::PoolView view() const {
    return pkv::PoolView{k, v, num_blocks, num_kv_heads, head_dim, d_err, elem_bytes, k_scale, v_scale, k_exps, v_exps};
  }
  // Bytes of one physical block of K (or V): all KV heads.
  size_t block_bytes() const { return static_cast<size_t>(num_kv_heads) * pkv::kBlockSize * head_dim * elem_bytes; }

  cudaEvent_t take_event() {   // prof_mu held
    if (ev_free.empty()) {
      cudaEvent_t e;
      if (cudaEventCreate(&e) != cudaSuccess) return nullptr;
      return e;
    }
    cudaEvent_t e = ev_free.back();
    ev_free.pop_back();
    return e;
  }
};

namespace pkv {

// For calls that have no form for int8 pools.
inline int refuse_int8(const pkv_pool* pool, const char* call) {
  if (!pool->k_exps) return PKV_OK;
  return fail(PKV_EUNSUPPORTED, std::string(call) + " does not support int8 pools");
}

// Launch `fn` on `stream`, bracketed by profiling events when profiling is on (not in a capture: its events have no
// times, and would be in the way of those that do).
template <class F>
int timed_launch(pkv_pool* pool, int kernel, void* stream, F&& fn) {
  cudaEvent_t a = nullptr, b = nullptr;
  cudaStreamCaptureStatus capturing = cudaStreamCaptureStatusNone;
  if (pool->prof_on && cudaStreamIsCapturing(static_cast<cudaStream_t>(stream), &capturing) == cudaSuccess &&
      capturing == cudaStreamCaptureStatusNone) {
    {
      std::lock_guard<std::mutex> lk(pool->prof_mu);
      a = pool->take_event();
      b = pool->take_event();
    }
    if (a && b) cudaEventRecord(a, static_cast<cudaStream_t>(stream));
  }
  const int rc = fn();
  if (a && b) {
    cudaEventRecord(b, static_cast<cudaStream_t>(stream));
    std::lock_guard<std::mutex> lk(pool->prof_mu);
    pool->pending.push_back({kernel, a, b});
  }
  return rc;
}

// Lands a pending ahead-of-time swap-in on `stream`: waits for its transfer,
// then scatters the staged blocks into the pool.  Every call that reads or
// writes the pool starts with this.
int finish_swap_in(pkv_pool* pool, void* stream);

// Q viewed as [T][Hq][D] in boxes of one tile of kTcRows / group tokens (at most num_tokens: *box_tokens).
int make_q_tmap(CUtensorMap* map, const void* q, int num_tokens, int num_q_heads, int head_dim, int group,
                int* box_tokens);

}  // namespace pkv
