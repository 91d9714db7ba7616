// Attention over blocks that a cheap score selects for each query token.
//
// Bounds (pkv_summarize).  For each (block, KV head), over the block's written
// keys: the largest and the smallest value of every channel, rounded outwards
// to 8-bit codes of one power-of-two unit,
//   up_d = ceil(max_j K_j[d] / 2^e),  lo_d = floor(min_j K_j[d] / 2^e),
// e the smallest exponent >= -126 with max|K| <= 127 2^e.
//
// Score (pkv_select_blocks).  q_g . K_j <= sum_d max(q_d, 0) up_d + min(q_d, 0) lo_d
// (times 2^e) for every key j of the block.  Summed over the G heads of a
// group this needs the sums P_d = sum_g max(q_gd, 0) and N_d = sum_g min(q_gd, 0)
// alone: one product of length 2 D per block whatever the group.  q is taken as
// whole numbers of a power-of-two unit with G |q| < 2^15, so that the score is
// an exact 32-bit integer (P - N <= 32767 in
// each of at most 128 channels, codes of at most 127: below 2^30), rounded to fp32 once and scaled by
// 2^e exactly: the order of the blocks, ties included, does not depend on the
// order of any sum.
#include <cooperative_groups.h>
#include <cuda.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "internal.h"
#include "ops.h"
#include "ptx.cuh"
#include "sched.cuh"

namespace cg = cooperative_groups;

namespace pkv {
namespace {

// The request of token t (the last with cu <= t), or -1 for a token that belongs to none.
__device__ __forceinline__ int req_of(const int32_t* cu, int num_reqs, int t) {
  int lo = 0, hi = num_reqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(cu + mid) <= t) lo = mid; else hi = mid - 1;
  }
  return __ldg(cu + lo) <= t && t < __ldg(cu + lo + 1) ? lo : -1;
}

__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }   // -126 <= e <= 127

// x = m 2^e with m in [0.5, 1), for a normal x > 0.
__device__ __forceinline__ int exp_of(float x) { return static_cast<int>(__float_as_uint(x) >> 23) - 126; }
__device__ __forceinline__ float mant_of(float x) {
  return __uint_as_float((__float_as_uint(x) & 0x7fffffu) | 0x3f000000u);
}

// ---------------------------------------------------------------- bounds
// One warp per TOK consecutive tokens and KV head: it handles the blocks that
// these tokens open (the first of the request's consecutive tokens in a
// block).  Lane l holds channels [l D/32, (l + 1) D/32).
template <int D, bool F8, int TOK>
__global__ void __launch_bounds__(256) summarize_kernel(const SparseArgs a) {
  constexpr int kDPL = D / 32;
  const int lane = threadIdx.x & 31;
  const int Hkv = a.pool.num_kv_heads;
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int groups = (a.num_tokens + TOK - 1) / TOK;
  if (w >= static_cast<int64_t>(groups) * Hkv) return;
  const int g = static_cast<int>(w % Hkv), t0 = static_cast<int>(w / Hkv) * TOK;
  // Lane i: token t0 + i's request, and whether it opens a block.
  const int mine = t0 + lane;
  int my_req = -1;
  bool opens = false;
  if (lane < TOK && mine < a.num_tokens) {
    my_req = req_of(a.cu_q_lens, a.num_reqs, mine);
    opens = my_req >= 0 && (mine == __ldg(a.cu_q_lens + my_req) ||
                            (__ldg(a.positions + mine) >> 4) != (__ldg(a.positions + mine - 1) >> 4));
  }
  uint32_t todo = __ballot_sync(0xffffffffu, opens);
  while (todo) {
    const int i = __ffs(todo) - 1;
    todo &= todo - 1;
    const int t = t0 + i;
    const int r = __shfl_sync(0xffffffffu, my_req, i);
    const int p = __ldg(a.positions + t);
    const int ctx = min(__ldg(a.ctx_lens + r), a.max_blocks * kBlockSize);
    if (p < 0 || p >= ctx) {
      if (lane == 0) atomicOr(a.pool.err, PKV_DEVERR_POSITION);
      continue;
    }
    const int b = p >> 4;
    const int pb = __ldg(a.block_tables + static_cast<int64_t>(r) * a.max_blocks + b);
    if (pb < 0 || pb >= a.pool.num_blocks) {
      if (lane == 0) atomicOr(a.pool.err, PKV_DEVERR_BLOCK_ID);
      continue;
    }
    const int n = min(kBlockSize, ctx - b * kBlockSize);
    const int64_t chunk = static_cast<int64_t>(pb) * Hkv + g;
    const uint8_t* src = static_cast<const uint8_t*>(a.pool.k) + chunk * kBlockSize * D * (F8 ? 1 : 2) +
                         lane * kDPL * (F8 ? 1 : 2);
    float hi[kDPL], lo[kDPL];
#pragma unroll
    for (int d = 0; d < kDPL; ++d) { hi[d] = -CUDART_INF_F; lo[d] = CUDART_INF_F; }
#pragma unroll
    for (int j = 0; j < kBlockSize; ++j) {   // past the written keys: the last one again
      float x[kDPL];
      const uint8_t* row = src + min(j, n - 1) * D * (F8 ? 1 : 2);
      if constexpr (F8) {
        uint32_t h[2];
        if constexpr (kDPL == 4) e4m3x4_to_f16x4(__ldg(reinterpret_cast<const uint32_t*>(row)), h[0], h[1]);
        else h[0] = e4m3x2_lo_to_f16x2(__ldg(reinterpret_cast<const uint16_t*>(row)));
#pragma unroll
        for (int d = 0; d < kDPL; d += 2)
          asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.f32.f16 %0, x;\n\tcvt.f32.f16 %1, y;\n\t}"
              : "=f"(x[d]), "=f"(x[d + 1]) : "r"(h[d / 2]));
      } else {
        uint32_t v[2];
        if constexpr (kDPL == 4) {
          const uint2 y = __ldg(reinterpret_cast<const uint2*>(row));
          v[0] = y.x; v[1] = y.y;
        } else {
          v[0] = __ldg(reinterpret_cast<const uint32_t*>(row));
        }
#pragma unroll
        for (int d = 0; d < kDPL; d += 2) { x[d] = bf16lo_to_f32(v[d / 2]); x[d + 1] = bf16hi_to_f32(v[d / 2]); }
      }
#pragma unroll
      for (int d = 0; d < kDPL; ++d) {   // NaN: no change (fmaxf and fminf return the other operand)
        hi[d] = fmaxf(hi[d], x[d]);
        lo[d] = fminf(lo[d], x[d]);
      }
    }
    constexpr float kMost = 3.38953138925e38f;   // the largest finite bf16; infinities count as it
    float amax = 0.f;
#pragma unroll
    for (int d = 0; d < kDPL; ++d) {
      if (hi[d] < lo[d]) hi[d] = lo[d] = 0.f;   // NaN in every key
      hi[d] = fminf(fmaxf(hi[d], -kMost), kMost);
      lo[d] = fminf(fmaxf(lo[d], -kMost), kMost);
      amax = fmaxf(amax, fmaxf(fabsf(hi[d]), fabsf(lo[d])));
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, x));
    int e = -126;
    if (amax >= 1.17549435e-38f) e = max(e, exp_of(amax) - (mant_of(amax) <= 0.9921875f ? 7 : 6));
    const float inv = pow2f(-e);
    uint32_t up = 0, dn = 0;
#pragma unroll
    for (int d = 0; d < kDPL; ++d) {
      // Products below fp32's range round to 0, but outwards they are one unit.
      const int u = hi[d] > 0.f ? max(1, static_cast<int>(ceilf(hi[d] * inv))) : static_cast<int>(ceilf(hi[d] * inv));
      const int v = lo[d] < 0.f ? min(-1, static_cast<int>(floorf(lo[d] * inv))) : static_cast<int>(floorf(lo[d] * inv));
      up |= static_cast<uint32_t>(u & 0xff) << (8 * d);
      dn |= static_cast<uint32_t>(v & 0xff) << (8 * d);
    }
    int8_t* dst = a.codes + chunk * 2 * D + lane * kDPL;
    if constexpr (kDPL == 4) {
      *reinterpret_cast<uint32_t*>(dst) = up;
      *reinterpret_cast<uint32_t*>(dst + D) = dn;
    } else {
      *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(up);
      *reinterpret_cast<uint16_t*>(dst + D) = static_cast<uint16_t>(dn);
    }
    if (lane == 0) a.exps[chunk] = static_cast<int8_t>(e);
  }
}

// ---------------------------------------------------------------- selection
constexpr int kSelThreads = 256;
constexpr int kSelMost = 49152;   // scores a CTA keeps (192 KB)

// Order-preserving key of a score: larger score, larger key.  0 is below every score.
__device__ __forceinline__ uint32_t key_of(float f) {
  f += 0.f;   // -0 counts as 0
  const uint32_t u = __float_as_uint(f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// One cluster of CS CTAs per (token, KV head); CTA i scores the i-th part of
// the token's blocks into shared memory, then the cluster finds the top_k-th
// key with four 8-bit radix passes and writes the chosen blocks in order.
template <int D, int CS>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SparseArgs a) {
  extern __shared__ uint32_t keys[];
  __shared__ __align__(16) int16_t s_q[2 * D];   // P, then N
  __shared__ uint32_t s_hist[4][256];  // one histogram a pass
  __shared__ float s_red[8];
  __shared__ int s_cnt[2];             // keys above the threshold, equal to it
  __shared__ int s_scan[2][8];
  __shared__ int s_pick[2];            // radix pass: bin, keys above it
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int Hkv = a.pool.num_kv_heads, G = a.group;
  const int rank = CS > 1 ? static_cast<int>(blockIdx.x % CS) : 0;
  const int64_t th = blockIdx.x / CS;
  const int g = static_cast<int>(th % Hkv), t = static_cast<int>(th / Hkv);
  const int r = req_of_warp(a.cu_q_lens, a.num_reqs, t, lane);
  if (r < 0) return;   // cluster-uniform
  const int p = __ldg(a.positions + t);
  int32_t* out = a.sel + th * a.top_k;
  if (p < 0 || p >= a.max_blocks * kBlockSize) {
    if (rank == 0) {
      if (tid == 0) atomicOr(a.pool.err, PKV_DEVERR_POSITION);
      for (int i = tid; i < a.top_k; i += kSelThreads) out[i] = -1;
    }
    return;
  }
  const int n = (p >> 4) + 1;
  const int per = (n + CS - 1) / CS;
  const int b0 = min(n, rank * per), b1 = min(n, b0 + per);

  // Whole-number queries: unit 2^f, the smallest with |q| <= most 2^f, most = floor(32767 / G).
  const uint16_t* q = static_cast<const uint16_t*>(a.q) + (static_cast<int64_t>(t) * a.num_q_heads + g * G) * D;
  float amax = 0.f;
  for (int i = tid; i < G * D; i += kSelThreads) {
    const float x = fabsf(bf16lo_to_f32(__ldg(q + i)));
    if (x < CUDART_INF_F) amax = fmaxf(amax, x);   // values that are not finite count as 0
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, x));
  if (lane == 0) s_red[warp] = amax;
  for (int i = tid; i < 4 * 256; i += kSelThreads) (&s_hist[0][0])[i] = 0;
  if (tid < 2) s_cnt[tid] = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) amax = fmaxf(amax, s_red[w]);
  const float most = static_cast<float>(32767 / G);
  // Tiny queries (below 2^-100) count as 0: the unit stays a normal number.
  const bool none = !(amax >= 7.8886e-31f);
  const int f = none ? 0 : exp_of(amax) - exp_of(most) + (mant_of(amax) <= mant_of(most) ? 0 : 1);
  for (int d = tid; d < D; d += kSelThreads) {
    int P = 0, N = 0;
    for (int h = 0; h < G && !none; ++h) {
      const float x = bf16lo_to_f32(__ldg(q + h * D + d));
      // x 2^-f in two exact steps (2^-f alone may exceed the normal range)
      const int i = fabsf(x) < CUDART_INF_F ? static_cast<int>(rintf(x * pow2f(-f / 2) * pow2f(-(f - f / 2)))) : 0;
      if (i > 0) P += i; else N += i;
    }
    s_q[d] = static_cast<int16_t>(P);
    s_q[D + d] = static_cast<int16_t>(N);
  }
  __syncthreads();
  // Scores: four lanes a block, lane s of them the 16-byte pieces s, s + 4, ... of the 2 D codes.
  constexpr int kPieces = 2 * D / 64;
  const int sub = lane & 3;
  int qq[kPieces][8];
#pragma unroll
  for (int i = 0; i < kPieces; ++i)
#pragma unroll
    for (int w = 0; w < 8; ++w) qq[i][w] = reinterpret_cast<const int*>(s_q)[(i * 4 + sub) * 8 + w];
  const int32_t* bt_row = a.block_tables + static_cast<int64_t>(r) * a.max_blocks;
  // Two iterations' codes in flight, their block ids one more ahead.
  constexpr int kStep = kSelThreads / 4;
  const int first = b0 + warp * 8 + (lane >> 2);
  auto load_id = [&](int b) -> int { return b < b1 ? __ldg(bt_row + b) : -1; };
  struct Codes { uint4 c[kPieces]; int e; };
  auto load_codes = [&](int pb, Codes& k) {
    k.e = 0;
    if (pb >= 0 && pb < a.pool.num_blocks) {
      const int64_t chunk = static_cast<int64_t>(pb) * Hkv + g;
      const uint4* src = reinterpret_cast<const uint4*>(a.codes + chunk * 2 * D) + sub;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) k.c[i] = __ldg(src + i * 4);
      k.e = __ldg(a.exps + chunk);
    } else {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) k.c[i] = make_uint4(0, 0, 0, 0);
    }
  };
  auto score = [&](int b, int pb, const Codes& k) {
    int s = 0;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int w[4] = {static_cast<int>(k.c[i].x), static_cast<int>(k.c[i].y), static_cast<int>(k.c[i].z),
                        static_cast<int>(k.c[i].w)};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        s = __dp2a_lo(qq[i][2 * x], w[x], s);
        s = __dp2a_hi(qq[i][2 * x + 1], w[x], s);
      }
    }
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    if (sub == 0 && b < b1) {
      const bool there = pb >= 0 && pb < a.pool.num_blocks;
      if (!there) atomicOr(a.pool.err, PKV_DEVERR_BLOCK_ID);
      const bool forced = b < a.sinks || b >= n - a.recent;
      keys[b - b0] = !there ? 0u : forced ? 0xffffffffu : key_of(__int2float_rn(s) * pow2f(max(-126, k.e)));
    }
  };
  {
    const int iters = b1 > b0 + warp * 8 ? (b1 - b0 - warp * 8 + kStep - 1) / kStep : 0;   // warp-uniform
    int id0 = load_id(first), id1 = load_id(first + kStep), id2 = load_id(first + 2 * kStep);
    Codes k0, k1;
    load_codes(id0, k0);
    for (int i = 0; i < iters; i += 2) {
      load_codes(id1, k1);
      const int id3 = load_id(first + (i + 3) * kStep);
      score(first + i * kStep, id0, k0);
      id0 = id2;
      load_codes(id0, k0);
      id2 = load_id(first + (i + 4) * kStep);
      if (i + 1 < iters) score(first + (i + 1) * kStep, id1, k1);
      id1 = id3;
    }
  }
  __syncthreads();
  // The top_k-th largest key, 8 bits at a time.
  const int cnt = b1 - b0;
  uint32_t thr = 0;
  int need = min(a.top_k, n);       // keys still to be found at or below the current prefix
  if (n > a.top_k) {
    for (int pass = 0; pass < 4; ++pass) {
      const int shift = 24 - 8 * pass;
      for (int i = tid; i < cnt; i += kSelThreads) {
        const uint32_t k = keys[i];
        if (pass == 0 || (k >> (shift + 8)) == (thr >> (shift + 8))) atomicAdd(&s_hist[pass][(k >> shift) & 255u], 1u);
      }
      if constexpr (CS > 1) cg::this_cluster().sync(); else __syncthreads();
      // Thread i: bin 255 - i over the whole cluster, then an inclusive scan from the top bin.
      int c = 0;
#pragma unroll
      for (int x = 0; x < CS; ++x) {
        const uint32_t* h = &s_hist[pass][255 - tid];
        if constexpr (CS > 1) h = cg::this_cluster().map_shared_rank(h, x);
        c += static_cast<int>(*h);
      }
      int inc = c;
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, x);
        if (lane >= x) inc += y;
      }
      if (lane == 31) s_scan[0][warp] = inc;
      __syncthreads();
      for (int w = 0; w < warp; ++w) inc += s_scan[0][w];
      if (inc >= need && inc - c < need) {
        s_pick[0] = 255 - tid;
        s_pick[1] = inc - c;
      }
      __syncthreads();
      thr |= static_cast<uint32_t>(s_pick[0]) << shift;
      need -= s_pick[1];
      __syncthreads();
    }
  }
  if (thr == 0u) need = 0;   // all are taken but the entries without a block (key 0)
  // Count, then write in order: keys above thr, and the first `need` equal to it.
  int gt = 0, eq = 0;
  for (int i = tid; i < cnt; i += kSelThreads) {
    gt += keys[i] > thr;
    eq += keys[i] == thr;
  }
  if (gt) atomicAdd(&s_cnt[0], gt);
  if (eq) atomicAdd(&s_cnt[1], eq);
  if constexpr (CS > 1) cg::this_cluster().sync(); else __syncthreads();
  int eq_before = 0, at = 0, total = 0, eq_left = 0;
#pragma unroll
  for (int x = 0; x < CS; ++x) {
    const int* c = s_cnt;
    if constexpr (CS > 1) c = cg::this_cluster().map_shared_rank(c, x);
    const int cgt = c[0], ceq = c[1];
    const int take = min(max(need - eq_before, 0), ceq);
    if (x < rank) at += cgt + take;
    if (x == rank) eq_left = max(need - eq_before, 0);   // equal keys that this CTA may take
    total += cgt + take;
    eq_before += ceq;
  }
  for (int base = 0; base < cnt; base += kSelThreads) {
    const int i = base + tid;
    const uint32_t k = i < cnt ? keys[i] : 0u;
    const bool is_eq = i < cnt && k == thr, is_gt = i < cnt && k > thr;
    const uint32_t beq = __ballot_sync(0xffffffffu, is_eq), bgt = __ballot_sync(0xffffffffu, is_gt);
    if (lane == 0) { s_scan[0][warp] = __popc(beq); s_scan[1][warp] = __popc(bgt); }
    __syncthreads();
    int weq = 0, wgt = 0, teq = 0, tgt = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      if (w < warp) { weq += s_scan[0][w]; wgt += s_scan[1][w]; }
      teq += s_scan[0][w];
      tgt += s_scan[1][w];
    }
    const uint32_t below = (1u << lane) - 1u;
    const int peq = weq + __popc(beq & below), pgt = wgt + __popc(bgt & below);
    const bool take = is_gt || (is_eq && peq < eq_left);
    if (take) out[at + pgt + min(peq, eq_left)] = b0 + i;
    at += tgt + min(eq_left, teq);
    eq_left -= min(eq_left, teq);
    __syncthreads();
  }
  if (rank == 0)
    for (int i = total + tid; i < a.top_k; i += kSelThreads) out[i] = -1;
  if constexpr (CS > 1) cg::this_cluster().sync();   // no CTA leaves while another reads its shared memory
}

// Launches a kernel with clusters of CS CTAs.
template <class K, class... Args>
cudaError_t launch_cluster(K kernel, int cs, int64_t grid, int threads, int smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cs;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D, int CS>
int launch_select_t(const SparseArgs& a, cudaStream_t s) {
  cudaError_t e = smem_attr_once<select_kernel<D, CS>>(kSelMost * 4);
  if (e != cudaSuccess) return e;
  const int smem = (a.max_blocks + CS - 1) / CS * 4;
  return launch_cluster(select_kernel<D, CS>, CS, static_cast<int64_t>(a.num_tokens) * a.pool.num_kv_heads * CS,
                        kSelThreads, smem, s, a);
}

template <int D>
int launch_select_d(const SparseArgs& a, cudaStream_t s) {
  // The larger the cluster, the more of the machine a small batch uses; a
  // part has 256 blocks at least, and a CTA's scores have to fit.
  const int64_t th = static_cast<int64_t>(a.num_tokens) * a.pool.num_kv_heads;
  int cs = 1;
  while (cs < 8 && ((th * cs < 2 * a.num_sms && a.max_blocks / (2 * cs) >= 256) ||
                    (a.max_blocks + cs - 1) / cs > kSelMost))
    cs *= 2;
  switch (cs) {
    case 1: return launch_select_t<D, 1>(a, s);
    case 2: return launch_select_t<D, 2>(a, s);
    case 4: return launch_select_t<D, 4>(a, s);
    default: return launch_select_t<D, 8>(a, s);
  }
}

template <int D, bool F8>
int launch_summarize_d(const SparseArgs& a, cudaStream_t s) {
  // A warp of 16 tokens finds about one new block in a prompt; a batch of
  // single tokens opens one block a token and takes a warp for each.
  const int64_t one = static_cast<int64_t>(a.num_tokens) * a.pool.num_kv_heads;
  if (one <= 64ll * a.num_sms) {
    summarize_kernel<D, F8, 1><<<static_cast<unsigned>((one + 7) / 8), 256, 0, s>>>(a);
  } else {
    const int64_t w = static_cast<int64_t>((a.num_tokens + 15) / 16) * a.pool.num_kv_heads;
    summarize_kernel<D, F8, 16><<<static_cast<unsigned>((w + 7) / 8), 256, 0, s>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace

int launch_summarize(const SparseArgs& a, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool f8 = a.pool.elem_bytes == 1;
  if (a.pool.head_dim == 128) return f8 ? launch_summarize_d<128, true>(a, s) : launch_summarize_d<128, false>(a, s);
  return f8 ? launch_summarize_d<64, true>(a, s) : launch_summarize_d<64, false>(a, s);
}

int select_max_blocks() { return 8 * kSelMost; }

int launch_select(const SparseArgs& a, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return a.pool.head_dim == 128 ? launch_select_d<128>(a, s) : launch_select_d<64>(a, s);
}

}  // namespace pkv
