// Attention of a chunk of new tokens over a paged key/value cache.
//
// For query row (token i, head h) of sequence s with n keys, q_len of them new:
//   o = softmax(scale * q K^T) V over keys j < n, and j <= n - q_len + i if causal,
// one pass over the keys with a running maximum and sum, as in fa_fwd.cu, whose
// building blocks these are: TMA into 128-byte-swizzled shared tiles, S = Q K^T and
// O += P V as tcgen05 MMAs into tensor memory, P over S as bf16, lazy rescaling.
//
// Bounds: a long chunk is bound by the tensor cores (4 d FLOP a query row and key),
// a single token by the read of K and V (4 d G FLOP for 4 d bytes a key).  Both
// are served by putting the G query heads that share a key head into the rows of
// one tile: row r of a tile is token r / G, head r mod G, so K and V are read once
// for all of them.
//
// Work: a unit is one key head's block of one or two 128-row query tiles and all
// key tiles (128 keys) it sees.  The key tiles of all units, one unit after the
// other, are cut into equal runs, one per CTA, whatever mix of lengths a step
// brings; lengths are read on the device, so the host knows none of them and one
// captured graph serves every step.  A cut that falls near a unit's border moves
// there.  A unit that is cut leaves unnormalised partial outputs (fp32) with
// their maxima and sums in the workspace, at most two a CTA, and a second kernel
// (a programmatic dependent) merges them in a fixed order: no atomics on results.
//
// Two forms of a unit share the code:
//   two tiles  256 rows against each key tile: warpgroup t owns query tile t
//   one tile   128 rows or fewer: warpgroup t takes every other key tile of the
//              same rows, with S and O of its own, merged at the unit's end.
//              A single token's softmax is one warp's work of about 2000 cycles a
//              key tile, latency that two key tiles in flight hide behind the
//              ~2800 cycles in which the SM's share of HBM brings 64 KiB.
// The kernel for short chunks (WIDE = false) has one query buffer's worth of
// tile and a deeper K / V ring; the other takes both forms.
//
// Roles (12 warps): 0-3 and 4-7 softmax warpgroups, 8 producer, 9 MMA issuer,
// 10 clears the rows of V behind a sequence's end (what lies there in a page is
// not the sequence's, and 0 * NaN is NaN; K needs none of it, its scores are
// masked), 11 idle.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/fa.h"
#include "fa_common.cuh"
#include "fa_paged.cuh"
#include "fa_paged_plan.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

using namespace paged;

template <int D, bool WIDE>
struct PagedCfg {
  static constexpr int kTileBytes = kTileRows * D * 2;
  static constexpr int kBlocks = D / 64;
  static constexpr int kQTiles = WIDE ? 2 : 1;
  static constexpr int kStages = D == 128 ? (WIDE ? 2 : 3) : (WIDE ? 5 : 6);
  static constexpr int kThreads = 384;
  // Register split of the forward kernel: 2 x 128 x 200 + 128 x 104 = 384 x 168.
  static constexpr int kLaunchRegs = 168;
  static constexpr int kAuxRegs = 104;
  static constexpr int kSoftmaxRegs = 200;
  static_assert(2 * 128 * kSoftmaxRegs + 128 * kAuxRegs <= kThreads * kLaunchRegs, "register split");
  static constexpr int kTmemCols = 512;
  static constexpr int kColS = 0;    // + 128 t, P over it
  static constexpr int kColO = 256;  // + 128 t
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + kQTiles * kTileBytes;
  static constexpr int kOffV = kOffK + kStages * kTileBytes;
  static constexpr int kOffMl = kOffV + kStages * kTileBytes;  // [2][128] (m, l) of the two halves of a one-tile unit
  static constexpr int kOffPlan = kOffMl + 2 * 128 * 8;
  static constexpr int kPlanBytes = 192;
  static constexpr int kOffBar = kOffPlan + kPlanBytes;
  static constexpr int kNumBars = 4 + 5 * kStages + 6 + 3;
  static constexpr int kOffTmemSlot = kOffBar + 8 * kNumBars;
  static constexpr int kOffAbort = kOffTmemSlot + 4;
  static constexpr int kSmemBytes = kOffAbort + 4;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

// ------------------------------------------------------------------- the plan --
// The kernel's arguments as a walk (fa_paged_plan.cuh) sees them.
struct Work {
  const int* cu;
  const int* lens;
  int S, Hk, T, cap, causal;
  __device__ __forceinline__ explicit Work(const PagedParams& p)
      : cu(p.cu_seqlens), lens(p.kv_lens), S(p.S), Hk(p.Hk), T(p.T), cap(p.max_pages << p.page_log2),
        causal(p.causal) {}
  __device__ __forceinline__ Seq seq(int s, bool& bad) const {
    return make_seq(__ldg(cu + s), __ldg(cu + s + 1), __ldg(lens + s), T, cap, bad);
  }
  __device__ __forceinline__ Seq seq(int s) const {
    bool bad = false;
    return seq(s, bad);
  }
};

// The CTA's run in shared memory.
struct Plan {
  long long x[2];   // its borders in the row of all key tiles
  int s, hk, b, j;  // where the first one lies
  int status;
  int pad;
  long long scan[16];
};
static_assert(sizeof(Plan) <= 192, "plan size");

// Sum over the block of one value a thread: the exclusive prefix, and the total.
template <int THREADS>
__device__ long long block_scan(long long v, long long* warps, long long* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x / 32;
  long long inc = v;
#pragma unroll
  for (int off = 1; off < 32; off *= 2) {
    const long long u = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += u;
  }
  __syncthreads();  // the previous use of `warps` has been read
  if (lane == 31) warps[w] = inc;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) {
    const long long x = warps[i];
    before += i < w ? x : 0;
    all += x;
  }
  *total = all;
  return before + inc - v;
}

// Every thread of the CTA.  Fills *plan: the run of this CTA.  The borders are
// computed alike by the CTAs on both sides of them.
template <int THREADS>
__device__ void make_plan(const PagedParams& p, int ut, Plan* plan) {
  const Work work(p);
  const int tid = threadIdx.x;
  bool bad = false;
  Seq q = {0, 0, 0};
  long long per_head = 0, before = 0, total = 0;
  const int chunks = (p.S + THREADS - 1) / THREADS;
  for (int c = 0; c < chunks; ++c) {
    const int s = c * THREADS + tid;
    per_head = 0;
    if (s < p.S) {
      q = work.seq(s, bad);
      per_head = seq_tiles(q, ut, p.causal);
    }
    long long part;
    before = total + block_scan<THREADS>(per_head * p.Hk, plan->scan, &part);
    total += part;
  }
  if (bad) atomicExch(p.status, FA_ERR_DEVICE_INDEX);
  const int ctas = (int)(total < gridDim.x ? total : gridDim.x);  // at least one tile a CTA
  const long long tol = snap_tolerance(total, ctas);
  if (tid == 0) {
    plan->x[0] = plan->x[1] = total;
    plan->s = p.S;
    plan->hk = plan->b = plan->j = 0;
  }
  __syncthreads();
  long long run = 0;
  for (int c = 0; c < chunks; ++c) {
    if (chunks > 1) {  // (with one chunk the values of the first pass are still here)
      const int s = c * THREADS + tid;
      per_head = 0;
      if (s < p.S) {
        q = work.seq(s);
        per_head = seq_tiles(q, ut, p.causal);
      }
      long long part;
      before = run + block_scan<THREADS>(per_head * p.Hk, plan->scan, &part);
      run += part;
    }
#pragma unroll 1
    for (int e = 0; e < 2; ++e) {
      if ((int)blockIdx.x + e > ctas) continue;
      const long long x = border(total, blockIdx.x + e, ctas);
      // the sequence it lies in (none for x == total: as set above)
      if (x < before || x >= before + per_head * p.Hk) continue;
      int hk, b, j;
      plan->x[e] = x + place(q, x - before, per_head, ut, p.causal, tol, hk, b, j);
      if (e == 0) {
        plan->s = c * THREADS + tid;
        plan->hk = hk;
        plan->b = b;
        plan->j = j;
      }
    }
  }
  __syncthreads();
}

struct PagedBars {
  uint64_t* q_full;    // [2] per query tile (two buffers of the one-tile kernel)
  uint64_t* q_empty;   // [2]
  uint64_t* k_full;    // [stages]
  uint64_t* v_full;
  uint64_t* k_empty;
  uint64_t* v_empty;
  uint64_t* s_full;    // [2]
  uint64_t* p_full;    // [2]
  uint64_t* o_full;    // [2]
  uint64_t* v_clear;   // [stages] the rows behind the sequence's end are zero (one phase a tile that has such rows)
  uint64_t* ml_full;   // one-tile units: both halves' (m, l) are in shared memory
  uint64_t* ml_empty;  // ... and both halves' outputs have been read
  uint64_t* mma_done;
};

template <int D, bool WIDE>
__global__ void __launch_bounds__(384, 1)
    paged_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedParams p) {
  using C = PagedCfg<D, WIDE>;
  // A negative scale: S is computed negated and the softmax uses |c2|.
  const uint32_t s_negate = p.c2 < 0.f ? kIdescNegateA : 0u;
  const float c2 = fabsf(p.c2);
  int* status = p.status;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (!smem_base_ok(smem_raw, status)) return;
  uint8_t* sm = smem_raw;

  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::kOffBar);
  PagedBars B;
  B.q_full = bars;
  B.q_empty = B.q_full + 2;
  B.k_full = B.q_empty + 2;
  B.v_full = B.k_full + C::kStages;
  B.k_empty = B.v_full + C::kStages;
  B.v_empty = B.k_empty + C::kStages;
  B.s_full = B.v_empty + C::kStages;
  B.p_full = B.s_full + 2;
  B.o_full = B.p_full + 2;
  B.v_clear = B.o_full + 2;
  B.ml_full = B.v_clear + C::kStages;
  B.ml_empty = B.ml_full + 1;
  B.mma_done = B.ml_empty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::kOffTmemSlot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + C::kOffAbort);
  Plan* plan = reinterpret_cast<Plan*>(sm + C::kOffPlan);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int tt = p.tile_tokens;
  const int ut = C::kQTiles * tt;  // tokens a unit

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B.q_full[i], 1);
      mbar_init(&B.q_empty[i], 1);
      mbar_init(&B.s_full[i], 1);
      mbar_init(&B.p_full[i], 128);
      mbar_init(&B.o_full[i], 1);
    }
    for (int st = 0; st < C::kStages; ++st) {
      mbar_init(&B.k_full[st], 1);
      mbar_init(&B.v_full[st], 1);
      mbar_init(&B.k_empty[st], 1);
      mbar_init(&B.v_empty[st], 2);  // the MMA issuer and warp 10
      mbar_init(&B.v_clear[st], 1);
    }
    mbar_init(B.ml_full, 256);
    mbar_init(B.ml_empty, 256);
    mbar_init(B.mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_map(&tm_q);
    tma_prefetch_map(&tm_k);
    tma_prefetch_map(&tm_v);
  }
  make_plan<C::kThreads>(p, ut, plan);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  const Work work(p);
  // Whether the segment's unit has one query tile: both warpgroups share its rows.
  auto one_tile = [&](const Segment& g) { return !WIDE || g.ntok <= tt; };

  if (warp >= 8) {
    regs_dec<C::kAuxRegs>();
    // Query buffers: [tile] in the two-tile kernel, a ring of q_bufs in the other.
    const int q_blk = (!WIDE && p.q_bufs == 2) ? kSwzBlockBytes / 2 : kSwzBlockBytes;
    const int q_bytes = q_blk * C::kBlocks;
    const int q_bufs = WIDE ? 1 : p.q_bufs;
    if (warp == 8) {
      // ------------------------------------------------------------ producer --
      Walk w = walk_start(work, plan->x[1] - plan->x[0], plan->s, plan->hk, plan->b, plan->j, ut);
      Segment g;
      const int box_rows = min(1 << p.page_log2, kTileRows);
      const int per_tile = kTileRows / box_rows;   // pages of a key tile (1 if pages are longer)
      const uint32_t box_bytes = box_rows * 128;
      const uint32_t q_box = tt * p.G * 128;
      uint32_t qcnt[2] = {0, 0}, kv_it = 0;
      bool ok = true, lost = false;
      while (ok && walk_get(work, w, ut, g)) {
        const bool one = one_tile(g);
        const int* table = p.page_table + (size_t)w.s * p.max_pages;
        // this lane's page of key tile j: outside the pool, the copy reads past the
        // map's last page and fills with zeros
        auto page_of = [&](int j) {
          int id = p.num_pages;
          if (lane < per_tile) {
            const int first = j * kTileRows + lane * box_rows;
            if (first < w.q.kv) {
              id = __ldg(table + (first >> p.page_log2));
              if (id < 0 || id >= p.num_pages) {
                id = p.num_pages;
                lost = true;
              }
            }
          }
          return id;
        };
        int page = page_of(g.j0);
#pragma unroll
        for (int t = 0; t < C::kQTiles; ++t) {
          if (!ok || (t == 1 && one)) continue;
          if (WIDE && !one && t == 0 && tile0_count(w.q, g, tt, p.causal) == 0) continue;
          const int bi = WIDE ? t : qcnt[0] % q_bufs;
          const uint32_t use = WIDE ? qcnt[t] : qcnt[0] / q_bufs;
          if (!(ok = mbar_wait_warp(&B.q_empty[bi], (use & 1) ^ 1, status))) break;
          if (lane == 0) {
            uint8_t* dst = sm + C::kOffQ + bi * q_bytes;
            mbar_expect_tx(&B.q_full[bi], q_box * C::kBlocks);
            for (int kb = 0; kb < C::kBlocks; ++kb)
              tma_load_4d(dst + kb * q_blk, &tm_q, &B.q_full[bi], 64 * kb, 0, w.hk, w.q.q0 + g.tok0 + t * tt);
          }
          __syncwarp();
          ++qcnt[WIDE ? t : 0];
        }
        for (int j = g.j0; j < g.j1 && ok; ++j, ++kv_it) {
          const int st = kv_it % C::kStages;
          const uint32_t ph = (kv_it / C::kStages) & 1;
          const int left = w.q.kv - j * kTileRows;  // keys from this tile on
          const int boxes = left <= 0 ? 0 : min(per_tile, (left + box_rows - 1) / box_rows);
          const int row = per_tile == 1 ? (j * kTileRows) & ((1 << p.page_log2) - 1) : 0;
          const int cur = page;
          if (j + 1 < g.j1) page = page_of(j + 1);
          if (!(ok = mbar_wait_warp(&B.k_empty[st], ph ^ 1, status))) break;
          if (lane == 0) mbar_expect_tx(&B.k_full[st], boxes * box_bytes * C::kBlocks);
          __syncwarp();
          if (lane < boxes) {
            uint8_t* dst = sm + C::kOffK + st * C::kTileBytes + lane * box_bytes;
            for (int kb = 0; kb < C::kBlocks; ++kb)
              tma_load_4d(dst + kb * kSwzBlockBytes, &tm_k, &B.k_full[st], 64 * kb, row, w.hk, cur);
          }
          __syncwarp();
          if (!(ok = mbar_wait_warp(&B.v_empty[st], ph ^ 1, status))) {
            // the K copy of this tile is in flight: it lands before the block ends
            mbar_wait_warp(&B.k_full[st], ph, status);
            break;
          }
          if (lane == 0) mbar_expect_tx(&B.v_full[st], boxes * box_bytes * C::kBlocks);
          __syncwarp();
          if (lane < boxes) {
            uint8_t* dst = sm + C::kOffV + st * C::kTileBytes + lane * box_bytes;
            for (int kb = 0; kb < C::kBlocks; ++kb)
              tma_load_4d(dst + kb * kSwzBlockBytes, &tm_v, &B.v_full[st], 64 * kb, row, w.hk, cur);
          }
          __syncwarp();
        }
        if (__any_sync(0xffffffffu, aborted(abort_flag))) ok = false;
        if (ok) walk_next(work, w, ut, g);
      }
      if (!ok) *abort_flag = 1;
      if (lost) atomicExch(status, FA_ERR_DEVICE_INDEX);
      // Drain: every copy this warp started lands before the block ends.
#pragma unroll
      for (int t = 0; t < (WIDE ? 2 : 1); ++t) {
        const uint32_t bufs = q_bufs;
        for (uint32_t x = qcnt[t] > bufs ? qcnt[t] - bufs : 0; x < qcnt[t]; ++x)
          mbar_wait_warp(&B.q_full[WIDE ? t : x % bufs], (x / bufs) & 1, status);
      }
      for (uint32_t i = kv_it > (uint32_t)C::kStages ? kv_it - C::kStages : 0; i < kv_it; ++i) {
        mbar_wait_warp(&B.k_full[i % C::kStages], (i / C::kStages) & 1, status);
        mbar_wait_warp(&B.v_full[i % C::kStages], (i / C::kStages) & 1, status);
      }
    } else if (warp == 9) {
      // ---------------------------------------------------------- MMA issuer --
      Walk w = walk_start(work, plan->x[1] - plan->x[0], plan->s, plan->hk, plan->b, plan->j, ut);
      Segment g;
      const uint32_t idS = idesc_bf16(128, 128, 0, 0) | s_negate;  // S = (+/-) Q K^T, both K-major
      constexpr uint32_t kIdO = idesc_bf16(128, D, 0, 1);            // O += P V, V is MN-major
      const uint32_t q_s = smem_addr(sm + C::kOffQ);
      const uint32_t k_s = smem_addr(sm + C::kOffK);
      const uint32_t v_s = smem_addr(sm + C::kOffV);
      uint32_t qcnt[2] = {0, 0}, pcnt[2] = {0, 0}, kv_it = 0, clears = 0;  // clears: bit st = parity of v_clear[st]
      bool ok = true;
      auto issue_s = [&](int t, uint32_t qa, uint32_t it) {
        const uint32_t ka = k_s + (it % C::kStages) * C::kTileBytes;
#pragma unroll
        for (int kb = 0; kb < C::kBlocks; ++kb)
          mma_ss_run_w<4, 2, 2>(tbase + C::kColS + 128 * t, sdesc(qa + kb * q_blk, 16, 1024),
                                sdesc(ka + kb * kSwzBlockBytes, 16, 1024), idS, kb > 0);
        mma_commit_w(&B.s_full[t]);
      };
      auto wait_k = [&](uint32_t it) {
        if (!mbar_wait_warp(&B.k_full[it % C::kStages], (it / C::kStages) & 1, status)) return false;
        tc_fence_after();
        return true;
      };
      auto issue_pv = [&](int t, uint32_t it, bool accumulate) {
        mma_ts_run_w<8, 8, 128>(tbase + C::kColO + 128 * t, tbase + C::kColS + 128 * t,
                                sdesc(v_s + (it % C::kStages) * C::kTileBytes, kSwzBlockBytes, 1024), kIdO,
                                accumulate);
      };
      while (ok && walk_get(work, w, ut, g)) {
        const bool one = one_tile(g);
        const int nt = g.j1 - g.j0;
        const int tail = w.q.kv - (last_tile(w.q.kv) << 7) < kTileRows ? last_tile(w.q.kv) : -1;
        // V of key tile j: cleared behind the end where the sequence ends in it
        auto wait_v = [&](int i) {
          const uint32_t it = kv_it + i;
          const int st = it % C::kStages;
          if (g.j0 + i == tail) {
            const uint32_t parity = (clears >> st) & 1;
            clears ^= 1u << st;
            return mbar_wait_warp(&B.v_clear[st], parity, status);
          }
          return mbar_wait_warp(&B.v_full[st], (it / C::kStages) & 1, status);
        };
        if (one) {
          const int bi = WIDE ? 0 : qcnt[0] % q_bufs;
          const uint32_t qa = q_s + bi * q_bytes;
          ok = mbar_wait_warp(&B.q_full[bi], (qcnt[0] / q_bufs) & 1, status);
          ++qcnt[0];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (!ok || i >= nt || !(ok = wait_k(kv_it + i))) continue;
            issue_s(i, qa, kv_it + i);
            mma_commit_w(&B.k_empty[(kv_it + i) % C::kStages]);
            if (i + 1 == nt) mma_commit_w(&B.q_empty[bi]);  // the last S of the segment
          }
          for (int i = 0; i < nt && ok; ++i) {
            const int t = i & 1;
            ok = mbar_wait_warp(&B.p_full[t], (t ? pcnt[1] : pcnt[0]) & 1, status);
            if (t)
              ++pcnt[1];
            else
              ++pcnt[0];
            if (!ok || !(ok = wait_v(i))) break;
            tc_fence_after();
            issue_pv(t, kv_it + i, i >= 2);
            mma_commit_w(&B.v_empty[(kv_it + i) % C::kStages]);
            if (i + 2 < nt) {
              if (!(ok = wait_k(kv_it + i + 2))) break;
              issue_s(t, qa, kv_it + i + 2);
              mma_commit_w(&B.k_empty[(kv_it + i + 2) % C::kStages]);
              if (i + 3 == nt) mma_commit_w(&B.q_empty[bi]);
            } else {
              mma_commit_w(&B.o_full[t]);
            }
          }
        } else if constexpr (WIDE) {
          const int cnt[2] = {tile0_count(w.q, g, tt, p.causal), nt};
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!ok || cnt[t] == 0) continue;
            ok = mbar_wait_warp(&B.q_full[t], qcnt[t] & 1, status);
            ++qcnt[t];
          }
          if (ok) ok = wait_k(kv_it);
          if (ok) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (cnt[t] == 0) continue;
              issue_s(t, q_s + t * q_bytes, kv_it);
              if (cnt[t] == 1) mma_commit_w(&B.q_empty[t]);
            }
            mma_commit_w(&B.k_empty[kv_it % C::kStages]);
          }
          for (int i = 0; i < nt && ok; ++i) {
            bool v_ready = false, k_ready = false;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (!ok || i >= cnt[t]) continue;
              ok = mbar_wait_warp(&B.p_full[t], pcnt[t] & 1, status);
              ++pcnt[t];
              if (ok && !v_ready) {
                ok = wait_v(i);
                v_ready = true;
              }
              if (!ok) break;
              tc_fence_after();
              issue_pv(t, kv_it + i, i > 0);
              if (i + 1 < cnt[t]) {
                if (!k_ready && !(ok = wait_k(kv_it + i + 1))) break;
                k_ready = true;
                issue_s(t, q_s + t * q_bytes, kv_it + i + 1);
                if (i + 2 == cnt[t]) mma_commit_w(&B.q_empty[t]);  // the last S of this tile
              } else {
                mma_commit_w(&B.o_full[t]);
              }
            }
            if (ok) {
              mma_commit_w(&B.v_empty[(kv_it + i) % C::kStages]);
              if (i + 1 < nt) mma_commit_w(&B.k_empty[(kv_it + i + 1) % C::kStages]);
            }
          }
        }
        kv_it += nt;
        if (__any_sync(0xffffffffu, aborted(abort_flag))) ok = false;
        if (ok) walk_next(work, w, ut, g);
      }
      if (!ok) *abort_flag = 1;
      mma_commit_w(B.mma_done);
      mbar_wait_warp(B.mma_done, 0, status);
    } else if (warp == 10) {
      // ------------------------------------------- rows behind a sequence's end --
      // Follows every V tile (a parity wait must not run ahead of the ring, nor
      // the ring ahead of it: a slot is released by this warp as well).
      Walk w = walk_start(work, plan->x[1] - plan->x[0], plan->s, plan->hk, plan->b, plan->j, ut);
      Segment g;
      uint32_t kv_it = 0;
      bool ok = true;
      while (ok && walk_get(work, w, ut, g)) {
        const int last = last_tile(w.q.kv), used = w.q.kv - (last << 7);
        for (int j = g.j0; j < g.j1; ++j, ++kv_it) {
          const int st = kv_it % C::kStages;
          if (!(ok = mbar_wait_warp(&B.v_full[st], (kv_it / C::kStages) & 1, status))) break;
          if (j == last && used < kTileRows) {
            for (int kb = 0; kb < C::kBlocks; ++kb) {
              uint4* rows = reinterpret_cast<uint4*>(sm + C::kOffV + st * C::kTileBytes + kb * kSwzBlockBytes);
              for (int i = used * 8 + lane; i < kTileRows * 8; i += 32) rows[i] = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.v_clear[st]);
          }
          if (lane == 0) mbar_arrive(&B.v_empty[st]);
          __syncwarp();
        }
        if (__any_sync(0xffffffffu, aborted(abort_flag))) ok = false;
        if (ok) walk_next(work, w, ut, g);
      }
      if (!ok) *abort_flag = 1;
    }
  } else {
    regs_inc<C::kSoftmaxRegs>();
    // -------------------------------------------------------------- softmax --
    const int t = warp / 4, quarter = warp % 4;
    const int r = quarter * 32 + lane;  // row of the tile
    const int rtok = r / p.G;           // its token in the tile
    const int rhead = r - rtok * p.G;
    const uint32_t t_s = tmem_lane_col(tbase, quarter * 32, C::kColS + 128 * t);
    const uint32_t t_o = tmem_lane_col(tbase, quarter * 32, C::kColO + 128 * t);
    float2* ml = reinterpret_cast<float2*>(sm + C::kOffMl);
    uint32_t scnt = 0, ocnt = 0, merges = 0;
    bool ok = true;
    int tail_row0 = 0, tail_tok = 0, tail_hk = 0, has_tail = 0, has_head = 0;  // for the header
    Walk w = walk_start(work, plan->x[1] - plan->x[0], plan->s, plan->hk, plan->b, plan->j, ut);
    Segment g;
    while (ok && walk_get(work, w, ut, g)) {
      const bool one = one_tile(g);
      const int nt = g.j1 - g.j0;
      const int tok = g.tok0 + (one ? 0 : t * tt) + rtok;         // in the sequence
      const int tile_rows = min(tt, g.ntok - (one ? 0 : t * tt)) * p.G;
      const bool valid = r < tile_rows;
      const bool busy = quarter * 32 < tile_rows;                 // any row of this warp
      const int cnt = one ? (nt + 1 - t) / 2 : t ? nt : tile0_count(w.q, g, tt, p.causal);
      const int jfirst = g.j0 + (one ? t : 0), jstep = one ? 2 : 1;
      const int past = w.q.kv - w.q.qn;
      const int lim = !valid ? -1 : p.causal ? min(past + tok, w.q.kv - 1) : w.q.kv - 1;  // last key it sees
      // the first row's: up to it no tile needs a mask
      const int lim0 = p.causal ? min(past + tok - rtok, w.q.kv - 1) : w.q.kv - 1;
      float m_run = -INFINITY, l_run = 0.f;  // log2 units
      for (int i = 0; i < cnt; ++i) {
        if (!(ok = mbar_wait_warp(&B.s_full[t], scnt & 1, status))) break;
        ++scnt;
        if (busy) {
          tc_fence_after();
          uint32_t sv[128];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(t_s + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&sv[32 * c]));
          tmem_wait_ld();
          float* s = reinterpret_cast<float*>(sv);
          const int kbase = (jfirst + i * jstep) * kTileRows;
          if (kbase + kTileRows - 1 > lim0) {
            const int cut = lim - kbase;  // key kbase + c is seen iff c <= cut
#pragma unroll
            for (int c = 0; c < 128; ++c) s[c] = (c > cut) ? -INFINITY : s[c];
          }
          float pm[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) pm[e] = max3f(s[2 * e], s[2 * e + 1], -INFINITY);
#pragma unroll
          for (int c = 16; c < 128; c += 2) pm[(c / 2) & 7] = max3f(pm[(c / 2) & 7], s[c], s[c + 1]);
          const float mx2 =
              max3f(max3f(pm[0], pm[1], pm[2]), max3f(pm[3], pm[4], pm[5]), fmaxf(pm[6], pm[7])) * c2;
          if (i == 0) {
            m_run = mx2;
          } else {
            const bool need = mx2 > m_run + kRescaleThreshold;
            if (__any_sync(0xffffffffu, need)) {
              // O_t is quiescent: S_t(i) was committed after P V of this half's last tile
              const float m_new = fmaxf(m_run, mx2);
              const float alpha = (m_run == -INFINITY) ? 0.f : ex2(m_run - m_new);
              l_run *= alpha;
              m_run = m_new;
              const uint64_t a2 = f2_pack(alpha, alpha);
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                uint32_t v[16];
                tmem_ld16(t_o + 16 * c, v);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  float lo, hi;
                  f2_unpack(f2_mul(f2_pack(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), a2), lo, hi);
                  v[2 * k] = __float_as_uint(lo);
                  v[2 * k + 1] = __float_as_uint(hi);
                }
                tmem_st16(t_o + 16 * c, v);
              }
            }
          }
          // P = 2^(s c2 - m) (0 where masked: a row that has seen no key has m = -inf and
          // every score -inf), summed in fp32 before its rounding to bf16 for P V
          const float mref = (m_run == -INFINITY) ? 0.f : m_run;
          const uint64_t c2x2 = f2_pack(c2, c2), negm = f2_pack(-mref, -mref);
          uint64_t ls[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const int c = 32 * h + 2 * k;
              float x0, x1;
              f2_unpack(f2_fma(f2_pack(s[c], s[c + 1]), c2x2, negm), x0, x1);
              const uint64_t e2 = f2_pack(ex2(x0), ex2(x1));
              ls[k & 3] = f2_add(ls[k & 3], e2);
              float p0, p1;
              f2_unpack(e2, p0, p1);
              pk[k] = pack_bf16x2(p0, p1);
            }
            tmem_st16(t_s + 16 * h, pk);
          }
          float a0, a1;
          f2_unpack(f2_add(f2_add(ls[0], ls[1]), f2_add(ls[2], ls[3])), a0, a1);
          l_run += a0 + a1;
          tmem_wait_st();
          tc_fence_before();
        }
        if (i == 0 && merges > 0) {
          // both halves must have read the last merged unit's O before P V overwrites it
          if (!(ok = mbar_wait_warp(B.ml_empty, (merges - 1) & 1, status))) break;
        }
        mbar_arrive(&B.p_full[t]);
      }
      if (ok && cnt > 0) {
        ok = mbar_wait_warp(&B.o_full[t], ocnt & 1, status);
        ++ocnt;
      }
      if (!ok) break;
      tc_fence_after();
      // One-tile unit of two or more tiles: both halves' (m, l), then each half
      // writes one half of the columns from both outputs.
      const bool merge = one && nt > 1;
      float w0 = 1.f, w1 = 0.f, m_out = m_run, l_out = l_run;  // weights of this half's and the other's output
      if (merge) {
        ml[t * 128 + r] = make_float2(m_run, l_run);
        mbar_arrive(B.ml_full);
        if (!(ok = mbar_wait_warp(B.ml_full, merges & 1, status))) break;
        ++merges;
        const float2 other = ml[(1 - t) * 128 + r];
        m_out = fmaxf(m_run, other.x);
        w0 = (m_run == -INFINITY) ? 0.f : ex2(m_run - m_out);
        w1 = (other.x == -INFINITY) ? 0.f : ex2(other.x - m_out);
        l_out = l_run * w0 + other.y * w1;
      }
      const bool whole = g.j0 == 0 && g.j1 == g.n;
      const bool writes = one && !merge ? t == 0 : true;  // (a single key tile: half 0 alone)
      if (writes && busy) {
        const bool empty = l_out == 0.f;  // saw no key: zero, whatever O holds
        const float scale_o = whole ? (empty ? 0.f : 1.f / l_out) : 1.f;
        w0 *= scale_o;
        w1 *= scale_o;
        const size_t row = (size_t)(w.q.q0 + tok) * (p.Hk * p.G) + w.hk * p.G + rhead;
        const int slot = g.j0 > 0 ? 0 : 1;
        const int prow = (one ? 0 : t * 128) + r;
        const size_t part = ((size_t)blockIdx.x * 2 + slot) * kPagedRows + prow;
        const int c_lo = merge ? t * (D / 2) : 0, c_hi = merge ? c_lo + D / 2 : D;
        const uint32_t t_o1 = tmem_lane_col(tbase, quarter * 32, C::kColO + 128 * (1 - t));
        const bool has_o = cnt > 0;
#pragma unroll 1
        for (int c = c_lo; c < c_hi; c += 16) {
          uint32_t v[16];
          float x[16];
          if (has_o) {
            tmem_ld16(t_o + c, v);
            if (merge) {
              uint32_t u[16];
              tmem_ld16(t_o1 + c, u);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                // a half that saw no key has weight 0 and an O of zeros times V
                const float a = w0 == 0.f ? 0.f : w0 * __uint_as_float(v[k]);
                x[k] = w1 == 0.f ? a : fmaf(w1, __uint_as_float(u[k]), a);
              }
            } else {
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) x[k] = empty ? 0.f : w0 * __uint_as_float(v[k]);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) x[k] = 0.f;
          }
          if (!valid) continue;
          if (whole) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + row * D + c);
#pragma unroll
            for (int k = 0; k < 2; ++k)
              dst[k] = make_uint4(pack_bf16x2(x[8 * k], x[8 * k + 1]), pack_bf16x2(x[8 * k + 2], x[8 * k + 3]),
                                  pack_bf16x2(x[8 * k + 4], x[8 * k + 5]), pack_bf16x2(x[8 * k + 6], x[8 * k + 7]));
          } else {
            float4* dst = reinterpret_cast<float4*>(p.part_o + part * D + c);
#pragma unroll
            for (int k = 0; k < 4; ++k) dst[k] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
          }
        }
        if (valid && (!merge || t == 0)) {
          if (!whole)
            reinterpret_cast<float2*>(p.part_ml)[part] = make_float2(m_out, l_out);
          else if (p.lse)
            p.lse[row] = empty ? -INFINITY : (m_out + __log2f(l_out)) * kLn2;
        }
      }
      if (merge) {
        tc_fence_before();
        mbar_arrive(B.ml_empty);
      }
      if (g.j0 > 0) {
        has_head = g.j1 == g.n ? 2 : 1;
      } else if (g.j1 < g.n) {
        has_tail = 1;
        tail_row0 = w.q.q0 + g.tok0;
        tail_tok = g.ntok;
        tail_hk = w.hk;
      }
      tc_fence_before();
      if (aborted(abort_flag)) ok = false;
      if (ok) walk_next(work, w, ut, g);
    }
    if (!ok) *abort_flag = 1;
    if (threadIdx.x == 0) {
      int4* hdr = reinterpret_cast<int4*>(p.hdr + (size_t)blockIdx.x * kPagedHdr);
      hdr[0] = make_int4(has_tail, tail_row0, tail_tok, tail_hk);
      hdr[1] = make_int4(has_head, 0, 0, 0);
    }
  }

  // The merge kernel (a programmatic dependent) may start launching; it waits
  // for this grid's results before it reads them.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tbase, C::kTmemCols);
  }
}

// Merges the units that were cut: block (c, y) takes rows of the unit that CTA
// c began and did not end.  Its parts are CTA c's second slot and the first
// slots of the CTAs behind it up to the one that ended it.  A warp a row.
template <int D>
__global__ void __launch_bounds__(256) paged_merge_kernel(const PagedParams p, int ctas) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x;
  const int lane = threadIdx.x & 31;
  const int4 h = *reinterpret_cast<const int4*>(p.hdr + (size_t)c * kPagedHdr);
  if (!h.x) return;
  // the first CTA behind c whose first slot ends its unit
  int last = ctas - 1;
  for (int at = c + 1; at < ctas; at += 32) {
    const bool ends = at + lane < ctas && p.hdr[(size_t)(at + lane) * kPagedHdr + 4] != 1;
    const unsigned found = __ballot_sync(0xffffffffu, ends);
    if (found) {
      last = at + __ffs(found) - 1;
      break;
    }
  }
  const int parts = last - c + 1;
  auto slot = [&](int i) { return ((size_t)(c + i) * 2 + (i == 0 ? 1 : 0)) * kPagedRows; };
  const int tt = p.tile_tokens, tile = tt * p.G;
  const int rows = h.z * p.G;  // valid rows, densely numbered
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
  constexpr int kPer = D / 32;
  for (int n = blockIdx.y * 8 + threadIdx.x / 32; n < rows; n += gridDim.y * 8) {
    const int prow = n < tile ? n : 128 + n - tile;
    float m = -INFINITY;
    for (int i = lane; i < parts; i += 32) m = fmaxf(m, ml[slot(i) + prow].x);
#pragma unroll
    for (int off = 16; off > 0; off /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    float l = 0.f, acc[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
      const float2 x = ml[slot(i) + prow];
      const float w = x.x == -INFINITY ? 0.f : ex2(x.x - m);
      l = fmaf(w, x.y, l);
      const float* src = p.part_o + (slot(i) + prow) * D + kPer * lane;
      if constexpr (kPer == 4) {
        const float4 v = *reinterpret_cast<const float4*>(src);
        acc[0] = fmaf(w, v.x, acc[0]);
        acc[1] = fmaf(w, v.y, acc[1]);
        acc[2] = fmaf(w, v.z, acc[2]);
        acc[3] = fmaf(w, v.w, acc[3]);
      } else {
        const float2 v = *reinterpret_cast<const float2*>(src);
        acc[0] = fmaf(w, v.x, acc[0]);
        acc[1] = fmaf(w, v.y, acc[1]);
      }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const int tok = n / p.G;
    const size_t row = (size_t)(h.y + tok) * (p.Hk * p.G) + h.w * p.G + (n - tok * p.G);
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) + row * D) + (kPer / 2) * lane;
#pragma unroll
    for (int e = 0; e < kPer / 2; ++e) dst[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    if (lane == 0 && p.lse) p.lse[row] = l > 0.f ? (m + __log2f(l)) * kLn2 : -INFINITY;
  }
}

template <int D, bool WIDE>
cudaError_t launch_paged_t(const PagedLaunch& a, cudaStream_t stream) {
  using C = PagedCfg<D, WIDE>;
  auto kern = paged_kernel<D, WIDE>;
  // The register split inside the kernel assumes it was built with exactly
  // kLaunchRegs registers a thread: refuse to launch any other build.
  static const bool regs_ok = [&] {
    cudaFuncAttributes attr;
    return cudaFuncGetAttributes(&attr, kern) == cudaSuccess && attr.numRegs == C::kLaunchRegs;
  }();
  if (!regs_ok) return cudaErrorInvalidKernelImage;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  kern<<<a.grid, C::kThreads, C::kSmemBytes, stream>>>(a.tm_q, a.tm_k, a.tm_v, a.p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.grid, WIDE ? 8 : 4);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_merge_kernel<D>, a.p, a.grid);
}

}  // namespace

cudaError_t launch_paged(const PagedLaunch& a, cudaStream_t stream) {
  if (a.d == 64) return a.wide ? launch_paged_t<64, true>(a, stream) : launch_paged_t<64, false>(a, stream);
  return a.wide ? launch_paged_t<128, true>(a, stream) : launch_paged_t<128, false>(a, stream);
}

}  // namespace fa
