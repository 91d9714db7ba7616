// Host-only check of the profiling lists (compiled by tests/test_profile_lists_cpu.py
// against the library's own header, with stand-ins for the CUDA events): calls
// of one pool from several threads each leave their record, and no event is
// handed to two of them.
#include <cstdio>
#include <set>
#include <thread>
#include <vector>

#include "pool.h"

static std::atomic<uintptr_t> made{0};
extern "C" {
cudaError_t cudaEventCreate(cudaEvent_t* e) {
  *e = reinterpret_cast<cudaEvent_t>(16 * (1 + made.fetch_add(1)));
  return cudaSuccess;
}
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus* s) {
  *s = cudaStreamCaptureStatusNone;
  return cudaSuccess;
}
const char* cudaGetErrorString(cudaError_t) { return ""; }
}
int pkv::set_last_error(int code, const std::string&) { return code; }

int main() {
  constexpr int kThreads = 8, kCalls = 20000, kHad = 1000;
  pkv_pool pool;
  pool.prof_on = true;
  for (int i = 0; i < kHad; ++i) {
    cudaEvent_t e;
    cudaEventCreate(&e);
    pool.ev_free.push_back(e);
  }
  std::vector<std::thread> threads;
  for (int t = 0; t < kThreads; ++t)
    threads.emplace_back([&] {
      for (int i = 0; i < kCalls; ++i) pkv::timed_launch(&pool, 0, nullptr, [] { return 0; });
    });
  for (auto& t : threads) t.join();
  std::set<cudaEvent_t> events;
  for (const auto& r : pool.pending) {
    events.insert(r.a);
    events.insert(r.b);
  }
  const size_t n = size_t(kThreads) * kCalls;
  const bool ok = pool.pending.size() == n && events.size() == 2 * n && pool.ev_free.empty();
  std::printf("%s %zu records, %zu events\n", ok ? "ok" : "FAIL", pool.pending.size(), events.size());
  return ok ? 0 : 1;
}
