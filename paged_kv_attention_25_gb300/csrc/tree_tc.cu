// Tree attention on the tcgen05 tensor cores, for batches whose trees bring
// many query rows (drafted tokens x grouped heads) per KV head.
//
// One CTA per SM with the warp roles of the prefill kernel (K and V producers
// that gather blocks by TMA, one MMA issuer, two softmax warpgroups A and B,
// scores, P and O in TMEM), but no work list: lengths are read on the device,
// and a twelfth warp walks the CTA's share of the work and hands segments to
// the others through a ring in shared memory, ahead of their use (each role
// walking by itself cost 3 to 6 us a segment, most of it instruction misses).
//
// A request's query rows form tiles of 128 (whole tokens).  Two warpgroups keep
// the tensor pipe busy when there is something for both, so a step takes
//   quad    four tiles on two neighbouring CTAs, two tiles each (A and B share
//           every K/V tile): both CTAs read the same keys at about the same
//           time, the second one from L2;
//   pair    two tiles on one CTA;
//   single  one tile: A takes the even key tiles, B the odd ones, and A joins
//           B's state (read from its TMEM columns) at the end.
// Quads form one line of work, shared out over pairs of CTAs; pairs and singles
// form a second one over CTAs.  A key tile of a quad or a pair costs a CTA two S
// and two PV products (three units), one of a single half of that but the same
// copies (two units); every group costs kGroupUnits besides, for its start and
// its epilogue.
//
// Bound by the steps' order, not by one unit: a key tile of a pair takes 1.4 us, of
// which the MMAs are 1.23 at the clock under load (scores, exponentials and P of one
// group run while the other's products do).  12 requests of 1.5 to 40 thousand
// tokens, 40 to 64 nodes, 64 query and 8 KV heads, D = 128: 228 us, 1.18 PFLOP/s, and
// 16 for the merge.  Of these the shares' key tiles (391 units a CTA, a third of a
// pair's 1.4 us each) are 182; tiles filled in part are in them (1.16 times the rows).
//
// Masks: key tiles that end at or before the prefix are seen whole.  In the others
// each row's thread forms its 128 visibility bits from its mask words.  The V
// producer reads those tiles once in shared memory and clears elements that
// are not finite (a masked key must not reach a row as 0 * inf) and the rows
// past the context; rows that do see such an element get it added after their
// result is stored.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "internal.h"
#include "ops.h"
#include "ptx.cuh"
#include "rows.cuh"
#include "sched.cuh"
#include "tc.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 384;
constexpr int kBlkPerTile = kNK / kBlockSize;   // 8
constexpr int kSegSlots = 4;                    // segments handed out ahead
constexpr int kSegRing = 8;                     // V producer's reports (it is at most kSegSlots + 1 ahead)
constexpr int kSegReaders = 11;                 // warps that read a segment
constexpr int kPairUnits = 3, kSingleUnits = 2, kGroupUnits = 6;
using TcShare = Share<kPairUnits + kGroupUnits>;

template <int KS, int VS>
struct TreeBars {
  static constexpr int kKFull = 0, kKEmpty = KS, kKLanded = 2 * KS;
  static constexpr int kVFull = 3 * KS, kVEmpty = 3 * KS + VS, kVLanded = 3 * KS + 2 * VS;
  static constexpr int kT = 3 * KS + 3 * VS;
  static constexpr int kS = kT;             // + group: S of its next key tile in TMEM
  static constexpr int kP = kT + 2;         // + group: P written, O rescaled (128 arrivals)
  static constexpr int kPv = kT + 4;        // + group: its last PV of the segment done
  static constexpr int kQFull = kT + 6;     // + tile
  static constexpr int kQEmpty = kT + 8;    // + tile
  static constexpr int kQc = kT + 10;       // + tile: FP8: Q rows converted to f16 (128 arrivals)
  static constexpr int kMl = kT + 12;       // single: B's state is final (128 arrivals)
  static constexpr int kJoined = kT + 13;   // single: A has read it (128 arrivals)
  static constexpr int kDrain = kT + 14;
  static constexpr int kVDone = kT + 15;    // + segment % kSegRing: its V tiles are all handed over
  static constexpr int kSegFull = kT + 15 + kSegRing;               // + segment % kSegSlots: published
  static constexpr int kSegEmpty = kSegFull + kSegSlots;            // + segment % kSegSlots: read by every role
  static constexpr int kCount = kSegEmpty + kSegSlots;
};

// What one CTA does with one group: key tiles [kt0, kt1) of a request.
struct alignas(16) Seg {
  int req, g, prefix, ctx;
  int tok0, tok1, rows0, rows1;   // query tiles (rows1 = 0: single)
  int kt0, kt1, slot, flags;
};
static_assert(sizeof(Seg) == 48, "Seg layout: three 16-byte loads");
constexpr int kSegSingle = 1, kSegWhole = 2, kSegMissing = 4, kSegEnd = 8;

template <int D>
struct TreeSmem {
  using S = TcSmem<D>;
  using B = TreeBars<S::kKSt, S::kVSt>;
  static constexpr int kOffBar = S::kOffBar;
  static constexpr int kOffMl = kOffBar + ((B::kCount * 8 + 15) / 16) * 16;   // float2 [128]: B's m, l
  static constexpr int kOffSeg = kOffMl + kTcRows * 8;
  static constexpr int kOffMisc = kOffSeg + kSegSlots * static_cast<int>(sizeof(Seg));
  static constexpr int kTotal = kOffMisc + 64;
};
static_assert(TreeSmem<128>::kTotal <= 232448, "shared memory of the D = 128 kernel");

__device__ __forceinline__ int key_tiles(const TreeReq& q) { return max(1, (q.ctx + kNK - 1) / kNK); }
__device__ __forceinline__ int query_tiles(const TreeReq& q, int tile_tokens) {
  return (q.n + tile_tokens - 1) / tile_tokens;
}
__device__ __forceinline__ int64_t quad_units(const TreeReq& q, int tile_tokens, int hkv) {
  return static_cast<int64_t>(query_tiles(q, tile_tokens) / 4) * hkv * (kPairUnits * key_tiles(q) + kGroupUnits);
}
__device__ __forceinline__ int64_t rest_units(const TreeReq& q, int tile_tokens, int hkv) {
  const int rem = query_tiles(q, tile_tokens) % 4, kt = key_tiles(q);
  return static_cast<int64_t>(hkv) * ((rem >> 1) * (kPairUnits * kt + kGroupUnits) +
                                      (rem & 1) * (kSingleUnits * kt + kGroupUnits));
}

// Walks a CTA's two shares: the quads, then the rest.  Key tile k of a group
// that begins at unit 0 belongs to the worker that holds unit k * cost; the
// group's fixed units follow its last tile.
struct Walk {
  TreeShare sh[2];
  TreeReq rq;
  int line, req;
  bool fresh;   // rq is not the current request's yet

  // The next segment with key tiles.  cut: the record of a group that this CTA begins and others go on with.
  __device__ __forceinline__ bool next(const TreeArgs& a, Seg& s, TreeCut& cut) {
    const int hkv = a.pool.num_kv_heads, tt = a.tile_tokens;
    for (;;) {
      if (line == 0 && sh[0].u >= sh[0].end) {
        line = 1;
        fresh = true;
      }
      TreeShare h = line == 0 ? sh[0] : sh[1];
      if (h.u >= h.end) return false;
      if (fresh) {
        req = h.req;
        rq = tree_req(a, req);
        fresh = false;
      }
      for (;;) {
        const int64_t n = line == 0 ? quad_units(rq, tt, hkv) : rest_units(rq, tt, hkv);
        if (h.off < n) break;
        h.off -= n;
        if (++req >= a.num_reqs) return false;
        rq = tree_req(a, req);
      }
      const int kt = key_tiles(rq), nt = query_tiles(rq, tt), quads = nt / 4;
      const int pair_len = kPairUnits * kt + kGroupUnits;
      int x, tile, cost = kPairUnits, glen = pair_len;   // x: unit within the group
      bool single = false;
      if (line == 0) {
        const int64_t grp = h.off / pair_len;
        x = static_cast<int>(h.off - grp * pair_len);
        s.g = static_cast<int>(grp) / quads;
        tile = (static_cast<int>(grp) % quads) * 4 + 2 * (blockIdx.x & 1);
      } else {
        const int rem = nt % 4, pairs = rem >> 1;
        const int single_len = kSingleUnits * kt + kGroupUnits;
        const int w = pairs * pair_len + (rem & 1) * single_len;
        s.g = static_cast<int>(h.off / w);
        x = static_cast<int>(h.off - static_cast<int64_t>(s.g) * w);
        tile = quads * 4;
        if (x >= pairs * pair_len) {
          x -= pairs * pair_len;
          tile += rem & 2;
          cost = kSingleUnits;
          glen = single_len;
          single = true;
        }
      }
      const int len = static_cast<int>(min(static_cast<int64_t>(glen - x), h.end - h.u));
      const int kt0 = min(kt, (x + cost - 1) / cost), kt1 = min(kt, (x + len + cost - 1) / cost);
      const int64_t gbegin = h.u - x;
      h.u += len;
      h.off += len;
      if (line == 0) sh[0] = h; else sh[1] = h;
      if (kt0 >= kt1) continue;   // the group's fixed units only
      s.req = req;
      s.prefix = rq.prefix;
      s.ctx = rq.ctx;
      s.tok0 = rq.t0 + tile * tt;
      s.rows0 = min(tt, rq.n - tile * tt) * a.group;
      s.tok1 = s.tok0 + tt;
      s.rows1 = single ? 0 : min(tt, rq.n - (tile + 1) * tt) * a.group;
      s.kt0 = kt0;
      s.kt1 = kt1;
      s.slot = (static_cast<int>(blockIdx.x) * 2 + line) * 2 + (kt0 == 0 ? 1 : 0);
      s.flags = (single ? kSegSingle : 0) | (kt0 == 0 && kt1 == kt ? kSegWhole : 0);
      cut.count = 0;
      if (kt0 == 0 && kt1 < kt) {
        // The last tile's first unit names the last worker; the workers between each have a tile (a share is
        // longer than a tile).
        const int per = line ? 1 : 2;   // CTAs a worker
        const int wk = static_cast<int>(blockIdx.x) / per;
        cut.count = TcShare::owner(h.U, h.workers, gbegin + static_cast<int64_t>(kt - 1) * cost) - wk + 1;
        cut.first = s.slot;
        cut.next = ((static_cast<int>(blockIdx.x) + per) * 2 + line) * 2;
        cut.stride = per * 4;
        cut.tok_a = s.tok0;
        cut.rows_a = s.rows0;
        cut.tok_b = s.tok1;
        cut.rows_b = s.rows1;
        cut.f0 = 0;
        cut.g = s.g;
      }
      return true;
    }
  }
};

// V elements that are not finite, added to the stored result of a row that
// sees them (they were left out of the products).
template <int D, bool F8>
__device__ __noinline__ void add_odd(const TreeArgs& a, const Seg& s, const uint32_t* mrow, uint16_t* o, float* part) {
  const int64_t Hkv = a.pool.num_kv_heads;
  const int32_t* bt = a.block_tables + static_cast<int64_t>(s.req) * a.max_blocks;
  const int b0 = max(s.kt0 * kBlkPerTile, s.prefix / kBlockSize);
  const int b1 = min(s.kt1 * kBlkPerTile, (s.ctx + kBlockSize - 1) / kBlockSize);
  for (int b = b0; b < b1; ++b) {
    const int pb = __ldg(bt + b);
    if (pb < 0 || pb >= a.pool.num_blocks) continue;
    const uint32_t vis = tree_sees(s.prefix, s.ctx, mrow, a.mask_words, b * kBlockSize) & ~low_bits(s.prefix - b * kBlockSize);
    for (int k = 0; k < kBlockSize; ++k) {
      if (!((vis >> k) & 1u)) continue;
      for (int d = 0; d < D; ++d) {
        const float v = pool_v<D, F8>(a.pool, pb * Hkv + s.g, k, d);
        if (fabsf(v) < CUDART_INF_F) continue;
        if (part) part[d] += v;
        else o[d] = static_cast<uint16_t>(pack_bf16x2(bf16lo_to_f32(o[d]) + v, 0.f) & 0xffffu);
      }
    }
  }
}

template <int D, bool F8>
__global__ void __launch_bounds__(kThreads, 1)
tree_tc_kernel(const TreeArgs a, const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
               const __grid_constant__ CUtensorMap tmap_q) {
  using S = TcSmem<D>;
  using M = TreeSmem<D>;
  using B = typename M::B;
  constexpr int kKSt = S::kKSt, kVSt = S::kVSt;
  extern __shared__ __align__(1024) uint8_t smem[];
  griddep_wait();
  griddep_launch();   // the merge may take its place and wait
  if (threadIdx.x < 2) a.cuts[2 * blockIdx.x + threadIdx.x].count = 0;
  if ((smem_u32(smem) & 1023u) != 0) {   // swizzle atoms need 1024-byte alignment
    if (threadIdx.x == 0) atomicOr(a.pool.err, PKV_DEVERR_INTERNAL);
    return;
  }
  const unsigned err0 = *reinterpret_cast<volatile unsigned*>(a.pool.err);
  if (__syncthreads_or((err0 & PKV_DEVERR_TIMEOUT) != 0)) return;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + M::kOffBar);
  float2* s_ml = reinterpret_cast<float2*>(smem + M::kOffMl);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + M::kOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + M::kOffMisc + 8);
  volatile int* s_odd = reinterpret_cast<volatile int*>(smem + M::kOffMisc + 16);   // [kSegRing]
  Seg* s_seg = reinterpret_cast<Seg*>(smem + M::kOffSeg);   // [kSegSlots]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.group, Hkv = a.pool.num_kv_heads;
  Walk walk;
  {
    // The CTA's shares (scratch in the query buffer, before its first copy).
    TreeShare (&sh)[2] = walk.sh;
    int64_t U[2], off[2];
    int reqs[2];
    auto share = [&](const int64_t (&len)[2], int line) {   // line 0: of this CTA's pair, line 1: of the CTA
      TreeShare& t = sh[line];
      t.U = len[line];
      t.workers = TcShare::workers(t.U, line ? a.ctas : a.ctas / 2);
      const int w = line ? static_cast<int>(blockIdx.x) : static_cast<int>(blockIdx.x >> 1);
      t.u = t.end = 0;
      if (t.U > 0 && w < t.workers) {
        t.u = TcShare::begin(t.U, t.workers, w);
        t.end = TcShare::begin(t.U, t.workers, w + 1);
      }
    };
    tree_scan<kThreads, 2, 2>(
        a, reinterpret_cast<int64_t*>(smem), U, reqs, off,
        [&](const TreeReq& q, int line) {
          return line == 0 ? quad_units(q, a.tile_tokens, Hkv) : rest_units(q, a.tile_tokens, Hkv);
        },
        [&](const int64_t (&len)[2], int p, int& line, int64_t& unit) {
          share(len, p);
          line = p;
          unit = sh[p].u < sh[p].end ? sh[p].u : -1;
        });
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      sh[i].req = reqs[i];
      sh[i].off = off[i];
    }
    if (sh[0].u >= sh[0].end && sh[1].u >= sh[1].end) return;   // block-uniform
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kKSt; ++i) {
      mbar_init(&bars[B::kKFull + i], 1);
      mbar_init(&bars[B::kKEmpty + i], 1);
      mbar_init(&bars[B::kKLanded + i], 1);
    }
    for (int i = 0; i < kVSt; ++i) {
      mbar_init(&bars[B::kVFull + i], 1);
      mbar_init(&bars[B::kVEmpty + i], 1);
      mbar_init(&bars[B::kVLanded + i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars[B::kS + t], 1);
      mbar_init(&bars[B::kP + t], 128);
      mbar_init(&bars[B::kPv + t], 1);
      mbar_init(&bars[B::kQFull + t], 1);
      mbar_init(&bars[B::kQEmpty + t], 1);
      mbar_init(&bars[B::kQc + t], 128);
    }
    mbar_init(&bars[B::kMl], 128);
    mbar_init(&bars[B::kJoined], 128);
    mbar_init(&bars[B::kDrain], 1);
    for (int i = 0; i < kSegRing; ++i) mbar_init(&bars[B::kVDone + i], 1);
    for (int i = 0; i < kSegSlots; ++i) {
      mbar_init(&bars[B::kSegFull + i], 1);
      mbar_init(&bars[B::kSegEmpty + i], kSegReaders);
    }
    *s_abort = 0;
    fence_mbar_init();
  }
  if (warp == 8 && lane == 0) {
    prefetch_tmap(&tmap_q);
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
  }
  if (warp == 9) {
    tmem_alloc(s_tmem, kTmemCols);
    tmem_relinquish();
  }
  // The scratch words above are generic writes to the query buffer, which TMA fills next.
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const uint32_t sQ = smem_u32(smem + S::kOffQ);
  const uint32_t sK = smem_u32(smem + S::kOffK);
  const uint32_t sV = smem_u32(smem + S::kOffV);
  // The CTA's r-th segment: waits until it is published, reads it and frees its slot.  false: gave up, or no more (`ok`
  // tells which).
  Seg sg;
  bool ok = true;
  auto take = [&](int r) -> bool {
    const int slot = r % kSegSlots;
    if (!(ok = mbar_wait_warp(&bars[B::kSegFull + slot], (r / kSegSlots) & 1, s_abort, a.wait_ns))) return false;
    sg = s_seg[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[B::kSegEmpty + slot]);
    return (sg.flags & kSegEnd) == 0;
  };

  if (warp == 8 || warp == 10) {
    // ------------------------------------------------------------ producers: warp 8 K (and Q), warp 10 V
    const bool is_k = warp == 8;
    const int nst = is_k ? kKSt : kVSt;
    uint8_t* const stages = smem + (is_k ? S::kOffK : S::kOffV);
    const int bar_full = is_k ? B::kKFull : B::kVFull, bar_empty = is_k ? B::kKEmpty : B::kVEmpty;
    const int bar_landed = is_k ? B::kKLanded : B::kVLanded;
    const CUtensorMap* const tm = is_k ? &tmap_k : &tmap_v;
    int cnt = 0;      // tiles issued in the launch
    int fin = 0;      // FP8: tiles widened and handed over
    int nq = 0;       // segments whose query tiles have been issued
    uint32_t landed_par = 0;
    for (int r = 0; ok && take(r); ++r) {
      if (is_k) {
        for (int t = 0; t < 2 && ok; ++t) {
          if (!(ok = mbar_wait_warp(&bars[B::kQEmpty + t], (r & 1) ^ 1, s_abort, a.wait_ns))) break;
          if (lane == 0) {
            if ((t ? sg.rows1 : sg.rows0) > 0) {
              mbar_arrive_expect_tx(&bars[B::kQFull + t], static_cast<uint32_t>(D * 2 * G * a.q_box_tokens));
              uint8_t* qt = smem + S::kOffQ + t * S::kQ;
#pragma unroll
              for (int hf = 0; hf < S::kHalves; ++hf)
                tma_load_3d(qt + hf * (kTcRows * 128), &tmap_q, hf * 64, sg.g * G, t ? sg.tok1 : sg.tok0,
                            &bars[B::kQFull + t]);
            } else {
              mbar_arrive(&bars[B::kQFull + t]);
            }
          }
          __syncwarp();
        }
        if (!ok) break;
        nq = r + 1;
      }
      const int32_t* bt_row = a.block_tables + static_cast<int64_t>(sg.req) * a.max_blocks;
      const int nblk = (sg.ctx + kBlockSize - 1) / kBlockSize;
      // Lane l holds block 32 w + l of the segment (window w: four key tiles), the next window in flight.
      auto load_window = [&](int w) -> int {
        const int b = sg.kt0 * kBlkPerTile + w * 32 + lane;
        return b < nblk && b < sg.kt1 * kBlkPerTile ? __ldg(bt_row + b) : -1;
      };
      auto check_window = [&](int pb) -> int { return pb >= 0 && pb < a.pool.num_blocks ? pb : -1; };
      int win = 0;
      int ids_cur = check_window(load_window(0)), ids_next = load_window(1);
      // Lane l < 8: chunk index of key tile j's block l, or -1.
      auto block_chunk = [&](int j) -> int {
        const int rel = j - sg.kt0;
        if ((rel >> 2) != win) {
          win = rel >> 2;
          ids_cur = check_window(ids_next);
          ids_next = load_window(win + 1);
        }
        const int pb = __shfl_sync(0xffffffffu, ids_cur, (rel & 3) * kBlkPerTile + (lane & 7));
        return lane < kBlkPerTile && pb >= 0 ? pb * Hkv + sg.g : -1;
      };
      int seg_odd = 0;
      // V tiles that some row does not see whole: clear the rows without a key
      // (past the context, or of a block that is not there) and, behind the
      // prefix, elements that are not finite.  have: blocks that were copied.
      auto clean_v = [&](uint8_t* stage, int j, uint32_t have) {
        constexpr int kCh = S::kHalves * 8;   // 16-byte chunks of a key's row
        const int ch = lane % kCh;
        uint8_t* col = stage + (ch / 8) * S::kHS;
        const int live = sg.ctx - j * kNK;
        const int first = have == 0xffu ? max(0, sg.prefix - j * kNK) & ~(32 / kCh - 1) : 0;
        const int pre = sg.prefix - j * kNK;
        bool odd = false;
#pragma unroll 4
        for (int key = first + lane / kCh; key < kNK; key += 32 / kCh) {
          uint4* p = reinterpret_cast<uint4*>(col + (key / 8) * S::kGS + (key % 8) * 128 + (((ch % 8) ^ (key % 8)) * 16));
          if (key >= live || !((have >> (key / kBlockSize)) & 1u)) {
            *p = make_uint4(0, 0, 0, 0);
            continue;
          }
          if (key < pre) continue;
          uint4 v = *p;
          bool any = false;
          v.x = finite_pair<F8>(v.x, any);
          v.y = finite_pair<F8>(v.y, any);
          v.z = finite_pair<F8>(v.z, any);
          v.w = finite_pair<F8>(v.w, any);
          if (any) {
            *p = v;
            odd = true;
          }
        }
        if (__any_sync(0xffffffffu, odd)) seg_odd = 1;
      };
      // Which tiles need it: a tile that ends behind the prefix, or lacks a block.
      auto needs_clean = [&](int j, uint32_t have) { return (j + 1) * kNK > sg.prefix || have != 0xffu; };
      if constexpr (!F8) {
        for (int j = sg.kt0; j < sg.kt1; ++j, ++cnt) {
          const int y = block_chunk(j);
          const int st = cnt % nst;
          const uint32_t have = __ballot_sync(0xffffffffu, y >= 0);
          if (!(ok = mbar_wait_warp(&bars[bar_empty + st], ((cnt / nst) & 1) ^ 1, s_abort, a.wait_ns))) break;
          // Test hook: CTA 0 never issues its first K tile, so that the issuer's bounded wait for it runs out.
          if (a.withhold == 2 && is_k && cnt == 0 && blockIdx.x == 0) continue;
          const bool clean = !is_k && needs_clean(j, have);
          uint64_t* bar = &bars[(clean ? bar_landed : bar_full) + st];
          if (lane == 0)
            mbar_arrive_expect_tx(bar, static_cast<uint32_t>(__popc(have)) * (S::kHalves * kBlockSize * 128));
          __syncwarp();
          uint8_t* stage = stages + st * S::kKV;
          if (y >= 0) {
            if constexpr (D == 128) tma_load_4d(stage + lane * S::kBlkBytes, tm, 0, 0, 0, 2 * y, bar);
            else tma_load_2d(stage + lane * S::kBlkBytes, tm, 0, y * kBlockSize, bar);
          }
          if (clean) {
            const uint32_t par = (landed_par >> st) & 1u;
            landed_par ^= 1u << st;
            if (!mbar_wait_warp(bar, par, s_abort, a.wait_ns)) {
              (void)mbar_wait(bar, par, nullptr, a.wait_ns);   // let this tile's copies land
              ok = false;
              break;
            }
            clean_v(stage, j, have);
            fence_proxy_async_smem();   // read by the tensor cores
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[bar_full + st]);
          }
        }
        if (!ok) break;
      } else {
        // Codes land in the upper half of a stage and are widened in place; a
        // copy is issued as soon as a stage is free and widened as soon as it
        // has landed, whichever is ready.
        int jl = sg.kt0, jw = sg.kt0;
        uint32_t have_ring = 0;   // blocks copied, 8 bits per stage (at most four stages)
        uint64_t idle0 = 0;
        while (jw < sg.kt1) {
          bool moved = false;
          if (jl < sg.kt1 && cnt - fin < nst && mbar_test_warp(&bars[bar_empty + cnt % nst], ((cnt / nst) & 1) ^ 1)) {
            const int y = block_chunk(jl), st = cnt % nst;
            const uint32_t have = __ballot_sync(0xffffffffu, y >= 0);
            have_ring = (have_ring & ~(0xffu << (8 * st))) | (have << (8 * st));
            uint64_t* bar = &bars[bar_landed + st];
            const bool withheld = a.withhold == 2 && is_k && cnt == 0 && blockIdx.x == 0;   // test hook (above)
            if (lane == 0 && !withheld) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(__popc(have)) * (kBlockSize * D));
            __syncwarp();
            if (y >= 0 && !withheld)
              tma_load_2d(stages + st * S::kKV + S::kKV / 2 + lane * (kBlockSize * D), tm, 0, y * kBlockSize, bar);
            ++cnt;
            ++jl;
            moved = true;
          }
          if (fin < cnt && mbar_test_warp(&bars[bar_landed + fin % nst], (fin / nst) & 1)) {
            const int st = fin % nst;
            uint8_t* stage = stages + st * S::kKV;
            widen_stage<D>(stage, lane);
            const uint32_t have = (have_ring >> (8 * st)) & 0xffu;
            if (!is_k && needs_clean(jw, have)) {
              __syncwarp();
              clean_v(stage, jw, have);
            }
            fence_proxy_async_smem();   // read by the tensor cores
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[bar_full + st]);
            ++fin;
            ++jw;
            moved = true;
          }
          if (moved) {
            idle0 = 0;
          } else {
            const uint64_t now = globaltimer_ns();
            if (idle0 == 0) idle0 = now;
            if (__any_sync(0xffffffffu, *s_abort != 0 || now - idle0 > a.wait_ns)) {
              ok = false;
              break;
            }
          }
        }
      }
      if (ok && !is_k && lane == 0) {
        s_odd[r % kSegRing] = seg_odd;
        mbar_arrive(&bars[B::kVDone + r % kSegRing]);
      }
      __syncwarp();
    }
    if (!ok) {   // gave up: flag it and let copies already issued land
      if (lane == 0) atomicOr(a.pool.err, PKV_DEVERR_TIMEOUT);
      *s_abort = 1;
      if constexpr (F8) {
        for (int i = fin; i < cnt; ++i) (void)mbar_wait(&bars[bar_landed + i % nst], (i / nst) & 1, nullptr, a.wait_ns);
      } else {
        for (int i = max(0, cnt - nst); i < cnt; ++i)
          (void)mbar_wait(&bars[bar_full + i % nst], (i / nst) & 1, nullptr, a.wait_ns);
      }
      if (is_k && nq > 0) {
        for (int t = 0; t < 2; ++t) (void)mbar_wait(&bars[B::kQFull + t], (nq - 1) & 1, nullptr, a.wait_ns);
      }
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t idesc_s = F8 ? make_idesc_f16(128, kNK, false) : make_idesc_bf16(128, kNK, false);
    constexpr uint32_t idesc_o = F8 ? make_idesc_f16(128, D, true) : make_idesc_bf16(128, D, true);
    const uint64_t dk = make_sdesc_sw128(sK, 16, S::kGS);
    const uint64_t dv = make_sdesc_sw128(sV, S::kHS, S::kGS);
    const uint64_t dqA = make_sdesc_sw128(sQ, 16, 1024), dqB = make_sdesc_sw128(sQ + S::kQ, 16, 1024);
    auto k_desc = [&](int gk) { return dk + static_cast<uint64_t>(((gk % kKSt) * S::kKV) >> 4); };
    auto v_desc = [&](int gv) { return dv + static_cast<uint64_t>(((gv % kVSt) * S::kKV) >> 4); };
    const uint32_t lead = elect_one();   // every lane runs the issue code, the elected one issues
    auto release = [&](int bar) { tc_commit_lead(lead, &bars[bar]); };
    // S of group t = (query tile) K^T
    auto issue_s = [&](int t, uint64_t dq, uint64_t kd) {
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const int hf = ks / 4, kk = ks % 4;
        tc_mma_lead(lead, tmem + t * kNK, dq + static_cast<uint64_t>((hf * (kTcRows * 128) + kk * 32) >> 4),
                    kd + static_cast<uint64_t>((hf * S::kHS + kk * 32) >> 4), idesc_s, ks > 0 ? 1u : 0u);
      }
      release(B::kS + t);
    };
    // O of group t (+)= P V
    auto issue_pv = [&](int t, bool acc, uint64_t vd) {
#pragma unroll
      for (int ks = 0; ks < kNK / 16; ++ks)
        tc_mma_ts_lead(lead, tmem + kColO + t * 128, tmem + t * kNK + ks * 8,
                       vd + static_cast<uint64_t>((ks * 2 * S::kGS) >> 4), idesc_o, (acc || ks > 0) ? 1u : 0u);
    };
    constexpr int kQReady = F8 ? B::kQc : B::kQFull;
    int kc = 0, vc = 0;          // K / V tiles consumed
    uint32_t pc0 = 0, pc1 = 0;   // P phases of group A / B waited so far
    auto wait_k = [&] { return mbar_wait_warp(&bars[B::kKFull + kc % kKSt], (kc / kKSt) & 1, s_abort, a.wait_ns); };
    auto wait_v = [&] { return mbar_wait_warp(&bars[B::kVFull + vc % kVSt], (vc / kVSt) & 1, s_abort, a.wait_ns); };
    auto wait_p = [&](int t) {
      const bool o = mbar_wait_warp(&bars[B::kP + t], (t ? pc1 : pc0) & 1, s_abort, a.wait_ns);
      if (t) ++pc1; else ++pc0;
      return o;
    };
    for (int r = 0; ok && take(r); ++r) {
      const int n = sg.kt1 - sg.kt0;   // >= 1
      if (!(ok = mbar_wait_warp(&bars[kQReady], r & 1, s_abort, a.wait_ns) &&
                 mbar_wait_warp(&bars[kQReady + 1], r & 1, s_abort, a.wait_ns)))
        break;
      if (!(sg.flags & kSegSingle)) {
        // Both groups use every key tile: PV_A(j) S_A(j+1) PV_B(j) S_B(j+1).
        if (!(ok = wait_k())) break;
        tc_fence_after();
        issue_s(0, dqA, k_desc(kc));
        issue_s(1, dqB, k_desc(kc));
        if (n == 1) {
          release(B::kQEmpty);
          release(B::kQEmpty + 1);
        }
        release(B::kKEmpty + kc % kKSt);
        ++kc;
        for (int j = 0; ok && j < n; ++j) {
          if (!(ok = wait_v())) break;
          const uint64_t vd = v_desc(vc), kd = k_desc(kc);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!(ok = wait_p(t))) break;
            tc_fence_after();
            issue_pv(t, j > 0, vd);
            if (j == n - 1) release(B::kPv + t);
            if (j + 1 < n) {
              if (t == 0 && !(ok = wait_k())) break;
              issue_s(t, t ? dqB : dqA, kd);
              if (j + 1 == n - 1) release(B::kQEmpty + t);
            }
          }
          if (!ok) break;
          if (j + 1 < n) {
            release(B::kKEmpty + kc % kKSt);
            ++kc;
          }
          release(B::kVEmpty + vc % kVSt);
          ++vc;
        }
      } else {
        // Group j % 2 uses key tile j: S_A(0) S_B(1), then PV(j) S(j+2).
        release(B::kQEmpty + 1);   // no second query tile
        for (int j = 0; ok && j < 2 && j < n; ++j) {
          if (!(ok = wait_k())) break;
          tc_fence_after();
          issue_s(j, dqA, k_desc(kc));
          if (j == n - 1) release(B::kQEmpty);
          release(B::kKEmpty + kc % kKSt);
          ++kc;
        }
        for (int j = 0; ok && j < n; ++j) {
          const int t = j & 1;
          if (!(ok = wait_v() && wait_p(t))) break;
          tc_fence_after();
          if (t) issue_pv(1, j > 1, v_desc(vc)); else issue_pv(0, j > 1, v_desc(vc));
          if (j + 2 >= n) release(B::kPv + t);
          release(B::kVEmpty + vc % kVSt);
          ++vc;
          if (j + 2 < n) {
            if (!(ok = wait_k())) break;
            if (t) issue_s(1, dqA, k_desc(kc)); else issue_s(0, dqA, k_desc(kc));
            if (j + 2 == n - 1) release(B::kQEmpty);
            release(B::kKEmpty + kc % kKSt);
            ++kc;
          }
        }
      }
    }
    if (!ok) {
      if (lane == 0) atomicOr(a.pool.err, PKV_DEVERR_TIMEOUT);
      *s_abort = 1;
    }
    // Drain: every MMA issued has completed before TMEM is released.
    release(B::kDrain);
    (void)mbar_wait_warp(&bars[B::kDrain], 0, nullptr, a.wait_ns);
  } else if (warp == 11) {
    // ------------------------------------------------------------ scheduler
    walk.line = 0;
    walk.fresh = true;
    for (int r = 0;; ++r) {
      Seg s;
      TreeCut cut;
      const bool more = walk.next(a, s, cut);
      if (more) {
        if (cut.count > 0 && lane == 0) a.cuts[2 * blockIdx.x + walk.line] = cut;
        // Blocks that are not there: flagged here, and only then looked for by the softmax warps.
        const int32_t* bt_row = a.block_tables + static_cast<int64_t>(s.req) * a.max_blocks;
        const int end = min(s.kt1 * kBlkPerTile, (s.ctx + kBlockSize - 1) / kBlockSize);
        bool gone = false;
        for (int b = s.kt0 * kBlkPerTile + lane; b < end; b += 32) {
          const int pb = __ldg(bt_row + b);
          gone |= pb < 0 || pb >= a.pool.num_blocks;
        }
        if (__any_sync(0xffffffffu, gone)) {
          s.flags |= kSegMissing;
          if (lane == 0) atomicOr(a.pool.err, PKV_DEVERR_BLOCK_ID);
        }
      } else {
        s.flags = kSegEnd;
      }
      const int slot = r % kSegSlots;
      if (!(ok = mbar_wait_warp(&bars[B::kSegEmpty + slot], ((r / kSegSlots) & 1) ^ 1, s_abort, a.wait_ns))) break;
      if (lane == 0) {
        s_seg[slot] = s;
        mbar_arrive(&bars[B::kSegFull + slot]);
      }
      __syncwarp();
      if (!more) break;
    }
    if (!ok) {
      if (lane == 0) atomicOr(a.pool.err, PKV_DEVERR_TIMEOUT);
      *s_abort = 1;
    }
  } else {
    // ------------------------------------------------------------ softmax / epilogue of group X
    const int X = (warp >> 2) & 1;
    const int row = threadIdx.x & 127;        // row within the tile (TMEM lane)
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t colS = X * kNK, colO = kColO + X * 128;
    const float sl2 = F8 ? a.scale_log2 * a.pool.k_scale : a.scale_log2;
    uint32_t sc = 0, pvc = 0, joins = 0;      // phases waited so far
    for (int r = 0; ok && take(r); ++r) {
      const int g = sg.g;
      const bool single = (sg.flags & kSegSingle) != 0, whole = (sg.flags & kSegWhole) != 0;
      const bool mine = X == 0 || !single;               // stores its rows
      const int nrows = X && !single ? sg.rows1 : sg.rows0;
      const int tok = X && !single ? sg.tok1 : sg.tok0;
      const bool valid = row < nrows;
      const int t_row = tok + (valid ? row / G : 0);
      const uint32_t* mrow = a.mask + static_cast<int64_t>(t_row) * a.mask_words;
      const int step = single ? 2 : 1;
      const int n = sg.kt1 - sg.kt0;
      const int nt = single ? (n + 1 - X) / 2 : n;    // key tiles of this group
      if constexpr (F8) {
        // Operands of one MMA share a type: this thread's Q row to f16, in place (exact within f16's range).
        ok = mbar_wait_warp(&bars[B::kQFull + X], r & 1, s_abort, a.wait_ns);
        if (ok && mine) {
          uint8_t* qrow = smem + S::kOffQ + X * S::kQ + row * 128;
#pragma unroll
          for (int hf = 0; hf < S::kHalves; ++hf) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              uint4* q16 = reinterpret_cast<uint4*>(qrow + hf * (kTcRows * 128) + c * 16);
              uint4 v = *q16;
              v.x = pack_f16x2(bf16lo_to_f32(v.x), bf16hi_to_f32(v.x));
              v.y = pack_f16x2(bf16lo_to_f32(v.y), bf16hi_to_f32(v.y));
              v.z = pack_f16x2(bf16lo_to_f32(v.z), bf16hi_to_f32(v.z));
              v.w = pack_f16x2(bf16lo_to_f32(v.w), bf16hi_to_f32(v.w));
              *q16 = v;
            }
          }
          fence_proxy_async_smem();   // read by the tensor cores
        }
        mbar_arrive(&bars[B::kQc + X]);
      }
      // Blocks that are not there, as bits: window of 32 blocks (four key tiles) at a time.
      const int32_t* bt_row = a.block_tables + static_cast<int64_t>(sg.req) * a.max_blocks;
      const int nblk = (sg.ctx + kBlockSize - 1) / kBlockSize;
      auto missing_of = [&](int w) -> uint32_t {
        const int b = sg.kt0 * kBlkPerTile + w * 32 + lane;
        bool gone = false;
        if (b < nblk && b < sg.kt1 * kBlkPerTile) {
          const int pb = __ldg(bt_row + b);
          gone = pb < 0 || pb >= a.pool.num_blocks;
        }
        return __ballot_sync(0xffffffffu, gone);
      };
      const bool any_missing = (sg.flags & kSegMissing) != 0;
      uint32_t missing = any_missing ? missing_of(0) : 0u;
      float m = -CUDART_INF_F, l = 0.f;
      for (int i = 0; ok && i < nt; ++i) {
        const int rel = single ? 2 * i + X : i;
        const int key0 = (sg.kt0 + rel) * kNK;
        if (any_missing && rel > 0 && (rel & 3) < step) missing = missing_of(rel >> 2);
        const uint32_t gone = (missing >> ((rel & 3) * kBlkPerTile)) & 0xffu;
        const bool masked = key0 + kNK > sg.prefix || gone != 0;
        uint32_t vis[4];
        if (masked) {   // the mask words are on their way while the scores are computed
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            vis[w] = tree_sees(sg.prefix, sg.ctx, mrow, a.mask_words, key0 + 32 * w);
            if ((gone >> (2 * w)) & 1u) vis[w] &= 0xffff0000u;
            if ((gone >> (2 * w)) & 2u) vis[w] &= 0x0000ffffu;
          }
        }
        if (!(ok = mbar_wait_warp(&bars[B::kS + X], sc & 1, s_abort, a.wait_ns))) break;
        ++sc;
        tc_fence_after();
        float s[kNK];
#pragma unroll
        for (int c = 0; c < kNK; c += 16) tmem_ld16(tmem + lane_base + colS + c, s + c);
        tmem_wait_ld();
        if (masked) {
#pragma unroll
          for (int w = 0; w < 4; ++w)
#pragma unroll
            for (int c = 0; c < 32; ++c) s[32 * w + c] = (vis[w] >> c) & 1u ? s[32 * w + c] : -CUDART_INF_F;
        }
        float mx8[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) mx8[k] = fmaxf(s[2 * k], s[2 * k + 1]);
#pragma unroll
        for (int c = 16; c < kNK; c += 2) mx8[(c >> 1) & 7] = max3f(mx8[(c >> 1) & 7], s[c], s[c + 1]);
        const float mx = max3f(max3f(mx8[0], mx8[1], mx8[2]), max3f(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7]));
        // Lazy rescaling: a row keeps its reference while the tile's maximum
        // stays within 2^kRescaleLog2 of it.  (Rows of the tile that are not the
        // segment's, other requests' or whatever the buffer held, have no say:
        // they would move the warp's references, and with them roundings.)
        const float m_tile = valid ? mx * sl2 : -CUDART_INF_F;
        const bool grow = __any_sync(0xffffffffu, m_tile > m + kRescaleLog2);
        const float m_new = grow ? fmaxf(m, m_tile) : m;
        const float neg_m = m_new == -CUDART_INF_F ? 0.f : -m_new;
        float rs0[4] = {0.f, 0.f, 0.f, 0.f}, rs1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int cc = 0; cc < kNK; cc += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int c = cc; c < cc + 32; c += 2) {
            float x0 = s[c], x1 = s[c + 1];
            fma2(x0, x1, sl2, neg_m);
            const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
            add2(rs0[(c >> 1) & 3], rs1[(c >> 1) & 3], p0, p1);
            pk[(c - cc) / 2] = F8 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
          }
          tmem_st16(tmem + lane_base + colS + cc / 2, reinterpret_cast<const float*>(pk));
        }
        const float rsum = ((rs0[0] + rs1[0]) + (rs0[1] + rs1[1])) + ((rs0[2] + rs1[2]) + (rs0[3] + rs1[3]));
        const float alpha = grow && m != -CUDART_INF_F ? fast_exp2(m + neg_m) : 1.f;
        if (grow && i > 0) {   // O is complete: S was issued after the group's previous PV
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            float o[32];
            tmem_ld16(tmem + lane_base + colO + c, o);
            tmem_ld16(tmem + lane_base + colO + c + 16, o + 16);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= alpha;
            tmem_st16(tmem + lane_base + colO + c, o);
            tmem_st16(tmem + lane_base + colO + c + 16, o + 16);
          }
        }
        l = l * alpha + rsum;
        m = m_new;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bars[B::kP + X]);
      }
      if (!ok) break;
      if (nt > 0) {
        if (!(ok = mbar_wait_warp(&bars[B::kPv + X], pvc & 1, s_abort, a.wait_ns))) break;
        ++pvc;
        tc_fence_after();
      }
      float wa = 1.f, wb = 0.f;   // weights of A's and B's accumulators
      bool join = false;
      if (single) {
        if (X == 1) {
          s_ml[row] = make_float2(m, l);
          tc_fence_before();
          mbar_arrive(&bars[B::kMl]);
          ok = mbar_wait_warp(&bars[B::kJoined], joins & 1, s_abort, a.wait_ns);
          ++joins;
          tc_fence_after();
          // Its rows are A's to store; the segment's flag is still to be passed.
          if (ok) ok = mbar_wait_warp(&bars[B::kVDone + r % kSegRing], (r / kSegRing) & 1, s_abort, a.wait_ns);
          continue;
        }
        if (!(ok = mbar_wait_warp(&bars[B::kMl], joins & 1, s_abort, a.wait_ns))) break;
        ++joins;
        tc_fence_after();
        join = n > 1;
        const float2 b = s_ml[row];
        if (join && b.y != 0.f) {   // l = 0: B saw no key of this row
          if (l == 0.f) {
            wa = 0.f;
            wb = 1.f;
            m = b.x;
            l = b.y;
          } else {
            const float mm = fmaxf(m, b.x);
            wa = fast_exp2(m - mm);
            wb = fast_exp2(b.x - mm);
            l = l * wa + b.y * wb;
            m = mm;
          }
        }
      }
      const float inv = l == 0.f ? 0.f : (F8 ? a.pool.v_scale : 1.f) / l;
      const float lse2 = l == 0.f ? -CUDART_INF_F : m + fast_log2(l);
      const int h = g * G + row % G;
      const int64_t prow = static_cast<int64_t>(sg.slot) * 256 + X * 128 + row;
      const int64_t orow = static_cast<int64_t>(t_row) * a.num_q_heads + h;
      uint4* dst_o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + orow * D);
      float4* dst_p = reinterpret_cast<float4*>(a.part_o + prow * D);
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += 32) {
        float ob[32];
        tmem_ld16(tmem + lane_base + colO + c0, ob);
        tmem_ld16(tmem + lane_base + colO + c0 + 16, ob + 16);
        if (join) {   // warp-uniform
          float oc[32];
          tmem_ld16(tmem + lane_base + kColO + 128 + c0, oc);
          tmem_ld16(tmem + lane_base + kColO + 128 + c0 + 16, oc + 16);
          tmem_wait_ld();
          // (a weight of 0 stands for a state without keys: its columns may hold anything)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            ob[e] = (wa == 0.f ? 0.f : ob[e] * wa) + (wb == 0.f ? 0.f : oc[e] * wb);
        } else {
          tmem_wait_ld();
        }
        if (valid && l != 0.f) {
#pragma unroll
          for (int e = 0; e < 32; ++e) ob[e] *= inv;
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) ob[e] = 0.f;
        }
        if (valid) {
          if (whole) {
#pragma unroll
            for (int e = 0; e < 32; e += 16) {
              uint4 w0, w1;
              w0.x = pack_bf16x2(ob[e], ob[e + 1]);       w0.y = pack_bf16x2(ob[e + 2], ob[e + 3]);
              w0.z = pack_bf16x2(ob[e + 4], ob[e + 5]);   w0.w = pack_bf16x2(ob[e + 6], ob[e + 7]);
              w1.x = pack_bf16x2(ob[e + 8], ob[e + 9]);   w1.y = pack_bf16x2(ob[e + 10], ob[e + 11]);
              w1.z = pack_bf16x2(ob[e + 12], ob[e + 13]); w1.w = pack_bf16x2(ob[e + 14], ob[e + 15]);
              // A thread writes its own row: 32 bytes a store, a whole sector, where o allows it.
              if (a.o_align32) {
                st_global_v8(dst_o + (c0 + e) / 8, w0, w1);
              } else {
                dst_o[(c0 + e) / 8] = w0;
                dst_o[(c0 + e) / 8 + 1] = w1;
              }
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              const uint32_t* w = reinterpret_cast<const uint32_t*>(ob + e);
              st_global_v8(dst_p + (c0 + e) / 4, make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7]));
            }
          }
        }
      }
      if (single) {
        tc_fence_before();
        mbar_arrive(&bars[B::kJoined]);   // B's columns have been read
      }
      if (valid) {
        if (whole) {
          if (a.lse) a.lse[orow] = lse2 * 0.69314718055994530942f;
        } else {
          a.part_lse[prow] = lse2;
        }
      }
      if (!(ok = mbar_wait_warp(&bars[B::kVDone + r % kSegRing], (r / kSegRing) & 1, s_abort, a.wait_ns))) break;
      if (s_odd[r % kSegRing] && valid)
        add_odd<D, F8>(a, sg, mrow, static_cast<uint16_t*>(a.o) + orow * D, whole ? nullptr : a.part_o + prow * D);
    }
    if (!ok) {
      if (lane == 0) atomicOr(a.pool.err, PKV_DEVERR_TIMEOUT);
      *s_abort = 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, bool F8>
int launch_t(const TreeArgs& a, const CUtensorMap* tk, const CUtensorMap* tv, const CUtensorMap* tq, cudaStream_t s) {
  const int smem = TreeSmem<D>::kTotal;
  cudaError_t e = smem_attr_once<tree_tc_kernel<D, F8>>(smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(tree_tc_kernel<D, F8>, dim3(a.ctas), kThreads, smem, s, a, *tk, *tv, *tq);
}

}  // namespace

int launch_tree_tc(const TreeArgs& a, const void* tmk, const void* tmv, const void* tmq, void* stream) {
  const CUtensorMap* k = static_cast<const CUtensorMap*>(tmk);
  const CUtensorMap* v = static_cast<const CUtensorMap*>(tmv);
  const CUtensorMap* q = static_cast<const CUtensorMap*>(tmq);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool f8 = a.pool.elem_bytes == 1;
  if (a.pool.head_dim == 128) return f8 ? launch_t<128, true>(a, k, v, q, s) : launch_t<128, false>(a, k, v, q, s);
  return f8 ? launch_t<64, true>(a, k, v, q, s) : launch_t<64, false>(a, k, v, q, s);
}

}  // namespace pkv
