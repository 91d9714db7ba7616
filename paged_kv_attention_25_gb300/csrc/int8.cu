// The 8-bit cache with a power of two for each (block, KV head): the quantising
// write, and the reading back of rows (of pools of any type).
//
//   e  = max(e_old if the block keeps tokens, the smallest e' >= -126 with max |x| <= 127 2^e')
//   c  = rne(x / 2^e) for new rows x,   rne(c 2^(e_old - e)) for held codes
//
// A power of two instead of max|x| / 127: codes use six to seven bits, but x / 2^e
// is exact, so that a code does not hang on the rounding of a division; the value
// c 2^e is a bf16 value, so that reading back is exact; and a block that grows by
// a token at a time re-rounds its held codes only when the power changes (a scale
// of max|x| / 127 changes with every new maximum, about log 16 = 3 times a block).
#include <cuda_runtime.h>

#include "append.cuh"
#include "int8.cuh"
#include "internal.h"
#include "ops.h"
#include "ptx.cuh"
#include "sched.cuh"

namespace pkv {
namespace {

constexpr int kTokens = 16;    // tokens of a CTA
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr uint32_t kTop = 0x7f7eu;   // bf16 bits of 127 * 2^121

// The new tokens of one block: those that follow one another in the batch.
struct Run {
  int pb, held;         // block; the slots that held tokens before the call and keep them, as bits
  int tok[kBlockSize];  // the new row of each slot (the last of several), -1: none
};

// x of a bf16 pair (either half) times 2^-e, rounded to a whole number (ties to
// even) in the low byte: the product is exact and the sum has a step of one.
__device__ __forceinline__ uint32_t code_bits(float x, float inv) { return __float_as_uint(fmaf(x, inv, 12582912.f)); }
__device__ __forceinline__ uint32_t quant_int8x4(uint32_t w0, uint32_t w1, float inv) {
  const uint32_t a = __byte_perm(code_bits(bf16lo_to_f32(w0), inv), code_bits(bf16hi_to_f32(w0), inv), 0x0040);
  const uint32_t b = __byte_perm(code_bits(bf16lo_to_f32(w1), inv), code_bits(bf16hi_to_f32(w1), inv), 0x0040);
  return __byte_perm(a, b, 0x5410);
}
// The larger magnitude in each half (bf16 magnitudes order as their bits do).
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7fff7fffu); }
// Magnitudes above 127 * 2^121, infinities among them, become that; NaN becomes 0.
__device__ __forceinline__ uint32_t tame_half(uint32_t h) {
  const uint32_t mag = h & 0x7fffu;
  return mag > 0x7f80u ? 0u : mag > kTop ? ((h & 0x8000u) | kTop) : h;
}
__device__ __forceinline__ uint32_t tame(uint32_t w) { return tame_half(w & 0xffffu) | (tame_half(w >> 16) << 16); }
__device__ __forceinline__ uint32_t rescale_int8x4(uint32_t c, float f) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int v = static_cast<int8_t>((c >> (8 * i)) & 0xffu);
    r |= (code_bits(static_cast<float>(v), f) & 0xffu) << (8 * i);
  }
  return r;
}

// A CTA looks at 16 tokens and takes the blocks whose first new token (in the
// order of the batch) is among them; a warp takes the rows of one of these blocks,
// one KV head, K or V: up to 16 x D values in registers, their maximum, the codes.
// The y grid shares out (head, K or V).  Bound by HBM for prompts, by the chain of
// dependent loads (request, table, exponent) for a decode step.  28,870 tokens of 8
// heads, D = 128: 31.7 us in a row of such launches (5.6 TB/s); by itself, L2 flushed, from
// event to event, 40; four CTAs an SM spill a few registers, but two took 47 so, and
// reading the rows twice (the second time out of L1) with six 43.
template <int D>
__global__ void __launch_bounds__(kThreads, 4) append_int8_kernel(
    const PoolView pool, uint8_t* kp, uint8_t* vp, const int32_t* __restrict__ bt, int max_blocks, int num_reqs,
    const int32_t* __restrict__ cu, const int32_t* __restrict__ pos, const int32_t* __restrict__ held_lens,
    const uint8_t* k_new, const uint8_t* v_new, int num_tokens) {
  __shared__ Run s_run[kTokens];
  __shared__ int s_count;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int Hkv = pool.num_kv_heads;
  if (tid == 0) s_count = 0;
  griddep_wait();
  griddep_launch();
  if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) check_cu(cu, num_reqs, num_tokens, pool.err);
  __syncthreads();
  for (int i = warp; i < kTokens; i += kWarps) {
    const int64_t tl = static_cast<int64_t>(blockIdx.x) * kTokens + i;
    if (tl >= num_tokens) break;
    const int t = static_cast<int>(tl);
    // Positions of the tokens t .. t + 31 and of the one before.
    int p = lane < num_tokens - t ? __ldg(pos + t + lane) : -1;
    const int before = t > 0 ? __ldg(pos + t - 1) : -1;
    const int r = req_of_warp(cu, num_reqs, t, lane);
    if (r < 0) continue;
    const int p0 = __shfl_sync(0xffffffffu, p, 0);
    if (p0 < 0 || p0 >= max_blocks * kBlockSize) {
      if (lane == 0 && blockIdx.y == 0) atomicOr(pool.err, PKV_DEVERR_POSITION);
      continue;
    }
    if (t > max(__ldg(cu + r), 0) && (before >> 4) == (p0 >> 4)) continue;   // not the first of its block
    const int end = min(__ldg(cu + r + 1), num_tokens);
    const int pb = __ldg(bt + static_cast<int64_t>(r) * max_blocks + (p0 >> 4));
    if (pb < 0 || pb >= pool.num_blocks) {
      if (lane == 0 && blockIdx.y == 0) atomicOr(pool.err, PKV_DEVERR_BLOCK_ID);
      continue;
    }
    const int held = __ldg(held_lens + r) - (p0 & ~15);
    int at = 0;
    if (lane == 0) at = atomicAdd(&s_count, 1);
    at = __shfl_sync(0xffffffffu, at, 0);
    Run& run = s_run[at];
    if (lane < kBlockSize) run.tok[lane] = -1;
    __syncwarp();
    uint32_t written = 0;
    for (int base = t;;) {
      const uint32_t out = __ballot_sync(0xffffffffu, base + lane >= end || (p >> 4) != (p0 >> 4));
      const int n = out ? __ffs(out) - 1 : 32;
      if (lane < n) atomicMax(&run.tok[p & 15], base + lane);
      written |= __reduce_or_sync(0xffffffffu, lane < n ? 1u << (p & 15) : 0u);
      if (n < 32) break;
      base += 32;
      p = lane < num_tokens - base ? __ldg(pos + base + lane) : -1;
    }
    if (lane == 0) {
      run.pb = pb;
      run.held = static_cast<int>(low_bits(min(held, kBlockSize)) & ~written);
    }
  }
  __syncthreads();
  constexpr int kPer = D / 16;             // lanes of a row, 16 values each
  constexpr int kSlots = 32 / kPer;        // slots a step
  constexpr int kSteps = kBlockSize / kSlots;
  const int sub = lane / kPer, piece = lane % kPer;
  const int mine = (2 * Hkv - static_cast<int>(blockIdx.y) + static_cast<int>(gridDim.y) - 1) / static_cast<int>(gridDim.y);
  const int tasks = s_count * mine;
  for (int task = warp; task < tasks; task += kWarps) {
    const Run& run = s_run[task / mine];
    const int u = static_cast<int>(blockIdx.y) + task % mine * static_cast<int>(gridDim.y);
    const int g = u >> 1;
    const uint8_t* src = (u & 1) ? v_new : k_new;
    const int64_t chunk = static_cast<int64_t>(run.pb) * Hkv + g;
    uint8_t* codes = ((u & 1) ? vp : kp) + chunk * (kBlockSize * D) + piece * 16;
    int8_t* exps = ((u & 1) ? pool.v_exps : pool.k_exps) + chunk;
    const int e_old = run.held ? safe_exp(*exps) : kMinExp;
    uint4 x[kSteps][2];
    uint32_t m2 = 0;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int tok = run.tok[s * kSlots + sub];
      x[s][0] = x[s][1] = make_uint4(0, 0, 0, 0);
      if (tok >= 0) {
        const uint4* row = reinterpret_cast<const uint4*>(src + (static_cast<int64_t>(tok) * Hkv + g) * (2 * D)) + piece * 2;
        x[s][0] = row[0];
        x[s][1] = row[1];
      }
    }
    auto top = [&] {
      m2 = 0;
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          m2 = max_abs2(max_abs2(max_abs2(max_abs2(m2, x[s][h].x), x[s][h].y), x[s][h].z), x[s][h].w);
      return __reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16));
    };
    uint32_t m = top();
    if (m > kTop) {
      if (m >= 0x7f80u && lane == 0) atomicOr(pool.err, PKV_DEVERR_VALUE);
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          x[s][h] = make_uint4(tame(x[s][h].x), tame(x[s][h].y), tame(x[s][h].z), tame(x[s][h].w));
      m = top();
    }
    // max = (128 + f) 2^(E - 134) (a subnormal's is below 127 * 2^-126).
    const int E = static_cast<int>(m >> 7), f = static_cast<int>(m & 127u);
    const int e = max(e_old, E - 133 + (f == 127));
    const uint32_t held = run.held;
    if (held && e > e_old) {
      const float down = exp_f32(max(e_old - e, kMinExp));
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int slot = s * kSlots + sub;
        if ((held >> slot) & 1u) {
          uint4* c = reinterpret_cast<uint4*>(codes + slot * D);
          const uint4 v = *c;
          *c = make_uint4(rescale_int8x4(v.x, down), rescale_int8x4(v.y, down), rescale_int8x4(v.z, down),
                          rescale_int8x4(v.w, down));
        }
      }
    }
    const float inv = exp_f32(-e);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int slot = s * kSlots + sub;
      if (run.tok[slot] >= 0)
        *reinterpret_cast<uint4*>(codes + slot * D) =
            make_uint4(quant_int8x4(x[s][0].x, x[s][0].y, inv), quant_int8x4(x[s][0].z, x[s][0].w, inv),
                       quant_int8x4(x[s][1].x, x[s][1].y, inv), quant_int8x4(x[s][1].z, x[s][1].w, inv));
    }
    __syncwarp();   // every lane has read the old exponent
    if (lane == 0) *exps = static_cast<int8_t>(e);
  }
}

// Rows of a cache as bf16: a thread takes 16 values of a token's K or V row at a
// time, kBatch loads under way.  Bound by HBM (a row's codes are a whole line): 52
// thousand int8 tokens of 8 heads, D = 128, 54 us in a row of such launches (6.0 TB/s); by
// itself, L2 flushed, from event to event, 58 to 60.  Small CTAs and few loads a
// thread, so that an SM has 16 CTAs at different stages: with 256 threads, 16 tokens
// and 4 loads it was 68 us so.  A row's 32 bytes go out as one store: as two, 74 us.
constexpr int kBatch = 2, kReadTokens = 8, kReadThreads = 128;
template <int KIND>   // 0: bf16, 1: e4m3, 2: int8
__global__ void __launch_bounds__(kReadThreads, 2048 / kReadThreads) read_rows_kernel(const PoolView pool, const int32_t* __restrict__ bt,
                                                             int max_blocks, int num_reqs,
                                                             const int32_t* __restrict__ cu,
                                                             const int32_t* __restrict__ pos, int num_tokens,
                                                             uint8_t* k_out, uint8_t* v_out, bool align32) {
  __shared__ int s_pb[kReadTokens], s_slot[kReadTokens];   // block (-1: a slot that is not there, -2: no request)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int Hkv = pool.num_kv_heads, D = pool.head_dim;
  griddep_wait();
  griddep_launch();
  if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) check_cu(cu, num_reqs, num_tokens, pool.err);
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kReadTokens;
  const int here = static_cast<int>(min(static_cast<int64_t>(kReadTokens), num_tokens - t0));
  for (int i = warp; i < here; i += (kReadThreads / 32)) {
    const int t = static_cast<int>(t0) + i;
    const int p = __ldg(pos + t);
    const int r = req_of_warp(cu, num_reqs, t, lane);
    int pb = -2;
    if (r >= 0) {
      pb = -1;
      if (p < 0 || p >= max_blocks * kBlockSize) {
        if (lane == 0 && blockIdx.y == 0) atomicOr(pool.err, PKV_DEVERR_POSITION);
      } else {
        pb = __ldg(bt + static_cast<int64_t>(r) * max_blocks + (p >> 4));
        if (pb < 0 || pb >= pool.num_blocks) {
          pb = -1;
          if (lane == 0 && blockIdx.y == 0) atomicOr(pool.err, PKV_DEVERR_BLOCK_ID);
        }
      }
    }
    if (lane == 0) {
      s_pb[i] = pb;
      s_slot[i] = p & 15;
    }
  }
  __syncthreads();
  const int lg = D == 128 ? 3 : 2, per = 1 << lg;   // pieces of a head's row
  const int row = Hkv << lg;                        // ... of a token's K (or V)
  const int step = kReadThreads * static_cast<int>(gridDim.y);
  // Line i of 2 * here (K's tokens, then V's), piece x of its row; a step on without a division.
  const int first = static_cast<int>(blockIdx.y) * kReadThreads + tid, di = step / row, dx = step - di * row;
  int i = first / row, x = first - i * row;
  auto on = [&](int& i, int& x) {
    i += di;
    x += dx;
    if (x >= row) {
      x -= row;
      ++i;
    }
  };
  while (i < 2 * here) {
    uint4 c[kBatch], c2[kBatch];
    int ex[kBatch];
    int li = i, lx = x;
#pragma unroll
    for (int b = 0; b < kBatch; ++b, on(li, lx)) {
      c[b] = c2[b] = make_uint4(0, 0, 0, 0);
      ex[b] = 0;
      const bool is_v = li >= here;
      const int tok = is_v ? li - here : li;
      if (li >= 2 * here || s_pb[tok] < 0) continue;
      const int64_t chunk = static_cast<int64_t>(s_pb[tok]) * Hkv + (lx >> lg);
      const int64_t at = (((chunk << 4) + s_slot[tok]) << lg) + (lx & (per - 1));   // in pieces of 16 values
      const uint4* src = static_cast<const uint4*>(is_v ? pool.v : pool.k);
      if constexpr (KIND == 0) {
        c[b] = __ldcg(src + 2 * at);
        c2[b] = __ldcg(src + 2 * at + 1);
      } else {
        c[b] = __ldcg(src + at);
        if constexpr (KIND == 2) ex[b] = safe_exp((is_v ? pool.v_exps : pool.k_exps)[chunk]);
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b, on(i, x)) {
      const bool is_v = i >= here;
      const int tok = is_v ? i - here : i;
      if (i >= 2 * here || s_pb[tok] == -2) continue;
      uint4 lo = c[b], hi = c2[b];
      if constexpr (KIND != 0) {
        const uint32_t w[4] = {c[b].x, c[b].y, c[b].z, c[b].w};
        uint32_t o[8];
        if constexpr (KIND == 2) {
          const uint32_t f = exp_bf16x2(ex[b] + kWidenShift);   // (codes of a slot that is not there are zero)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            int8x4_to_bf16x4(w[k], o[2 * k], o[2 * k + 1]);
            o[2 * k] = mul_bf16x2(o[2 * k], f);
            o[2 * k + 1] = mul_bf16x2(o[2 * k + 1], f);
          }
        } else {
          const float f = is_v ? pool.v_scale : pool.k_scale;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t h[2];
            e4m3x4_to_f16x4(w[k], h[0], h[1]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float a, b2;
              asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.f32.f16 %0, x;\n\tcvt.f32.f16 %1, y;\n\t}"
                  : "=f"(a), "=f"(b2) : "r"(h[j]));
              o[2 * k + j] = pack_bf16x2(a * f, b2 * f);
            }
          }
        }
        lo = make_uint4(o[0], o[1], o[2], o[3]);
        hi = make_uint4(o[4], o[5], o[6], o[7]);
      }
      uint4* dst = reinterpret_cast<uint4*>(is_v ? v_out : k_out) + 2 * ((t0 + tok) * row + x);
      if (align32) {
        st_global_v8(dst, lo, hi);
      } else {
        dst[0] = lo;
        dst[1] = hi;
      }
    }
  }
}

// CTAs along y so that a small batch occupies the machine: at most `most`.
int spread(int64_t ctas, int most, int num_sms) {
  const int64_t want = (4ll * num_sms + ctas - 1) / ctas;
  return static_cast<int>(want < 1 ? 1 : want > most ? most : want);
}

}  // namespace

int launch_append_int8(const PoolView& pool, void* kp, void* vp, const int32_t* bt, int max_blocks, int num_reqs,
                       const int32_t* cu, const int32_t* pos, const int32_t* held, const void* k_new, const void* v_new,
                       int num_tokens, int num_sms, void* stream) {
  const int ctas = (num_tokens + kTokens - 1) / kTokens;
  const dim3 grid(ctas, spread(ctas, 2 * pool.num_kv_heads, num_sms));
  auto go = [&](auto kernel) {
    return launch_dependent(kernel, grid, kThreads, 0, static_cast<cudaStream_t>(stream), pool, static_cast<uint8_t*>(kp),
                            static_cast<uint8_t*>(vp), bt, max_blocks, num_reqs, cu, pos, held,
                            static_cast<const uint8_t*>(k_new), static_cast<const uint8_t*>(v_new), num_tokens);
  };
  return pool.head_dim == 128 ? go(append_int8_kernel<128>) : go(append_int8_kernel<64>);
}

int launch_read_rows(const PoolView& pool, const int32_t* bt, int max_blocks, int num_reqs, const int32_t* cu,
                     const int32_t* pos, int num_tokens, void* k_out, void* v_out, int num_sms, void* stream) {
  const int ctas = (num_tokens + kReadTokens - 1) / kReadTokens;
  const int64_t pieces = 2ll * kReadTokens * pool.num_kv_heads * (pool.head_dim / 16);
  const bool align32 = ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 31u) == 0;
  const dim3 grid(ctas, spread(ctas, static_cast<int>((pieces + kReadThreads - 1) / kReadThreads), num_sms));
  auto go = [&](auto kernel) {
    return launch_dependent(kernel, grid, kReadThreads, 0, static_cast<cudaStream_t>(stream), pool, bt, max_blocks, num_reqs,
                            cu, pos, num_tokens, static_cast<uint8_t*>(k_out), static_cast<uint8_t*>(v_out), align32);
  };
  return pool.k_exps ? go(read_rows_kernel<2>) : pool.elem_bytes == 1 ? go(read_rows_kernel<1>) : go(read_rows_kernel<0>);
}

}  // namespace pkv
