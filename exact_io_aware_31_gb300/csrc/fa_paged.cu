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
// key tiles (128 keys) it sees.  The units, one after the other, are cut into
// runs of equal cost, one per CTA, whatever mix of lengths a step brings; lengths
// are read on the device, so the host knows none of them and one captured graph
// serves every step.  A cut that falls near a unit's border moves there.  A unit
// that is cut leaves unnormalised partial outputs (fp32) with their maxima and
// sums in the workspace, at most two a CTA, and a second kernel (a programmatic
// dependent) merges them in a fixed order: no atomics on results.
//
// Three forms of a unit, by its query rows; warpgroups t = 0, 1:
//   two tiles   up to 256 rows against each key tile: warpgroup t owns tile t
//   one tile    33 to 128 rows: warpgroup t takes every other key tile of the
//               same rows, with S and O of its own, merged at the unit's end
//   four copies up to 32 rows (single tokens): as one tile, and the rows are
//               copied into each quarter of the tile, whose warp takes a quarter
//               of the columns (its P is zero in the others).  A warp that had
//               32 rows to itself spent about 2000 cycles a key tile on one
//               lane's 128 exponentials while three warps idled: 64 sequences
//               of 256 to 1024 keys, 8 tokens each, 16 heads, d = 64 ran in 68 us
//               (41 now).  The eight partial rows are merged through the unit's
//               own query buffer, which is dead by then.
// SHORT kernels hold only the last form: the host takes them where it was told
// that chunks are short; a longer chunk is then a row of small units.
//
// Rounding: scores, maxima, sums and O are fp32.  P is rounded to bf16 once, as the
// MMA takes it (its sum takes the fp32 values), for single tokens, too, which run the
// same MMAs: outputs are 2.0e-3 to 2.3e-3 off (norm of the error by the norm) where
// the rounding of the output alone makes 1.65e-3.  MMAs that take more of P (tf32)
// want V in 32 bits as well: twice its shared memory at half the rate.
//
// Measured (GB300, d = 128, 32 query and 8 key heads): 2 x 2048 tokens against 16384
// and 8789 keys 458 to 471 us, 1.66 PFLOP/s (86% of the dense rate; the softmax between
// the MMAs), and 508 in a loop of seconds, when the power limit holds the clock near
// 1.8 of 2.07 GHz (89% of the rate then); 64 single tokens against up to 8192 keys
// 219 us, 6.1 TB/s (91% of the copy rate); one token, 16 heads, 16384 keys 32 us (7 us
// until the first tile, 4 us of merge).  Small units are bound by the chain from one
// unit's last tile to the next one's first scores (2 us) and by instruction fetch.
//
// Roles (12 warps): 0-3 and 4-7 softmax warpgroups, 8 producer, 9 MMA issuer,
// 10 clears the rows of V behind a sequence's end (what lies there in a page is
// not the sequence's, and 0 * NaN is NaN; K needs none of it, its scores are
// masked), 11 (short chunks) walks the run for the others.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "fa_common.cuh"
#include "fa_paged.cuh"
#include "fa_paged_plan.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

using namespace paged;

#ifdef FA_TEST_HOOKS
// Test builds only (-DFA_TEST_HOOKS, never the default library).  1: softmax
// warpgroup 0 withholds its first "P ready" arrival of every unit, so that the
// waits behind it run out.  2: every CTA takes its shared memory for misaligned.
static __device__ int g_fa_test_paged;
#endif

template <int D>
struct PagedCfg {
  static constexpr int kTileBytes = kTileRows * D * 2;
  static constexpr int kBlocks = D / 64;
  // Slots of the K and V rings; the rest is two query buffers.  A K slot is
  // free once S is done, long before its V slot; the next K is what the MMA
  // issuer waits for first.
  static constexpr int kKSlots = D == 128 ? 3 : 6;
  static constexpr int kVSlots = D == 128 ? 2 : 5;
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
  static constexpr int kOffK = kOffQ + 2 * kTileBytes;
  static constexpr int kOffV = kOffK + kKSlots * kTileBytes;
  static constexpr int kOffMl = kOffV + kVSlots * kTileBytes;  // [2 buffers][8 warps][8 rows] (m, l)
  static constexpr int kOffPlan = kOffMl + 2 * 64 * 8;
  static constexpr int kPlanBytes = 192;
  static constexpr int kOffSegs = kOffPlan + kPlanBytes;  // (short chunks) [kSegs] segments
  static constexpr int kSegs = 4;
  static constexpr int kOffBar = kOffSegs + kSegs * 48;
  static constexpr int kNumBars = 4 + 4 + 2 * kKSlots + 3 * kVSlots + 8 + 1 + 2 * kSegs;
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
  int S, Hk, T, cap;
  __device__ __forceinline__ explicit Work(const PagedParams& p)
      : cu(p.cu_seqlens), lens(p.kv_lens), S(p.S), Hk(p.Hk), T(p.T), cap(p.max_pages << p.page_log2) {}
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
  Spot at[2];      // its borders
  Seq q[2];        // the sequences they lie in
  long long y[2];  // while it is made: places in the cost of their key heads
  long long scan[12];
};
static_assert(sizeof(Plan) <= 192, "plan size");

// Token of a row: row / G for rows up to 256 and G up to 128.  With m = 65536 / G + 1
// the product is row / G + row * e / (65536 G) for an e of 1 .. G: too little to
// reach the next integer while row * e < 65536.
__device__ __forceinline__ int token_of(const PagedParams& p, int row) { return (row * p.g_inverse) >> 16; }

// n / d for positive n: 32 bits where they do (a 64-bit division is a long
// stretch of code in front of a CTA's first copy).
__device__ __forceinline__ long long div_long(long long n, long long d) {
  if (((n | d) >> 32) == 0) return (unsigned)n / (unsigned)d;
  return n / d;
}

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
template <int D, int THREADS>
__device__ void make_plan(const PagedParams& p, const Shape& sh, Plan* plan) {
  const Work work(p);
  const int tid = threadIdx.x;
  bool bad = false;
  Seq q = {0, 0, 0};
  long long per_head = 0, before = 0, total = 0;
  const int chunks = (p.S + THREADS - 1) / THREADS;
  if (tid < 2) plan->at[tid] = {p.S, 0, 0, 0};  // a border at the end
  for (int c = 0; c < chunks; ++c) {
    const int s = c * THREADS + tid;
    per_head = 0;
    if (s < p.S) {
      q = work.seq(s, bad);
      per_head = cost_of_seq<D>(q, sh);
    }
    long long part;
    before = total + block_scan<THREADS>(per_head * p.Hk, plan->scan, &part);
    total += part;
  }
  if (bad) record_index(p.status);
  // The sequences that the borders lie in.
  const int ctas = ctas_for<D>(total, gridDim.x);
  const long long share = ctas > 0 ? div_long(total, ctas) : 0;
  long long run = 0;
  for (int c = 0; c < chunks; ++c) {
    if (chunks > 1) {  // (with one chunk the values of the first pass are still here)
      const int s = c * THREADS + tid;
      per_head = 0;
      if (s < p.S) {
        q = work.seq(s);
        per_head = cost_of_seq<D>(q, sh);
      }
      long long part;
      before = run + block_scan<THREADS>(per_head * p.Hk, plan->scan, &part);
      run += part;
    }
#pragma unroll 1
    for (int e = 0; e < 2; ++e) {
      const long long x = border(total, share, blockIdx.x + e, ctas);
      if ((int)blockIdx.x + e > ctas || x < before || x >= before + per_head * p.Hk) continue;
      const int hk = (int)div_long(x - before, per_head);
      plan->at[e] = {c * THREADS + tid, hk, 0, 0};
      plan->y[e] = x - before - hk * per_head;
      plan->q[e] = q;
    }
  }
  __syncthreads();
  // Their blocks: every thread tries some.
#pragma unroll 1
  for (int e = 0; e < 2; ++e) {
    if (plan->at[e].s >= p.S) continue;
    const Seq sq = plan->q[e];
    for (int b = tid; b * sh.ut < sq.qn; b += THREADS) {
      int j;
      if (place<D>(sq, plan->y[e], b, sh, j)) {
        plan->at[e].b = b;
        plan->at[e].j = j;
      }
    }
  }
  __syncthreads();
}

struct PagedBars {
  uint64_t* q_full;   // [2] per query buffer
  uint64_t* q_empty;  // [2] a two-tile unit's last S has read it
  uint64_t* x_done;   // [2] a one-tile unit's partial rows are merged: its query buffer is free
  uint64_t* x_full;   // both warpgroups' partial rows are in shared memory
  uint64_t* x_next;   // ... and have been read: the unit's next eight rows may follow
  uint64_t* k_full;   // [K slots]
  uint64_t* k_empty;
  uint64_t* v_full;   // [V slots]
  uint64_t* v_empty;
  uint64_t* v_clear;  // the rows behind the sequence's end are zero (one phase a tile that has such rows)
  uint64_t* s_full;   // [2]
  uint64_t* p_full;   // [2]
  uint64_t* p_half;   // [2] (not with four copies) P of the first 64 keys is there
  uint64_t* o_full;   // [2]
  uint64_t* mma_done;
  uint64_t* seg_full;   // [segments] (short chunks) warp 11 has written it
  uint64_t* seg_empty;  // every warp that walks has read it
};

// 32 bytes of a row, 32-byte aligned: rows of the workspace (an output of the caller's
// is only 16-byte aligned).
__device__ __forceinline__ void store32(void* dst, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// A warp's bounded wait.  SMALL: mbar_wait_warp in fewer instructions.  Small units
// pass through all code of their roles and wait for instructions a good part of
// their time, so what is shorter is faster: 64 sequences of 8 tokens, d = 64, took
// 43.5 us and 42.7 with it; 2 chunks of 509 tokens among 14 single ones 60.3 and
// 57.8, with d = 64 49.4 and 42.8.  The softmax of long chunks comes out slower with
// it (2 x 2048 tokens: 468 -> 480 us) and has the other one.
template <bool SMALL>
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, int* status) {
  if constexpr (!SMALL) return mbar_wait_warp(bar, parity, status);
  const uint32_t a = smem_addr(bar);
  uint32_t t0 = 0;
#pragma unroll 1
  for (uint32_t n = 0;; ++n) {
    if (__all_sync(0xffffffffu, mbar_test(a, parity))) return true;
    if (n & 31) continue;
    const uint32_t now = (uint32_t)(global_ns() >> 10);  // (about a microsecond)
    if (n == 0) t0 = now;
    if (__any_sync(0xffffffffu, now - t0 > (uint32_t)(kWaitLimitNs >> 10))) {
      atomicExch(status, kDevTimeout);
      return false;
    }
  }
}

template <int D, bool SHORT>
__global__ void __launch_bounds__(384, 1)
    paged_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_q4,
                 const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                 const __grid_constant__ PagedParams p) {
  using C = PagedCfg<D>;
  // A negative scale: S is computed negated and the softmax uses |c2|.
  const uint32_t s_negate = p.c2 < 0.f ? kIdescNegateA : 0u;
  const float c2 = fabsf(p.c2);
  int* status = p.status;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  bool start_ok = smem_base_ok(smem_raw, status);
#ifdef FA_TEST_HOOKS
  if (*reinterpret_cast<volatile int*>(&g_fa_test_paged) == 2) {
    if (threadIdx.x == 0) atomicExch(status, kDevInternal);
    start_ok = false;
  }
#endif
  if (!start_ok) {  // nothing for the merge kernel, whatever the workspace holds
    if (threadIdx.x < kPagedHdr) p.hdr[(size_t)blockIdx.x * kPagedHdr + threadIdx.x] = 0;
    return;
  }
  uint8_t* sm = smem_raw;
  // The merge kernel (a programmatic dependent) may start launching: its blocks
  // take the room of CTAs that are done, and wait for this grid's results.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::kOffBar);
  PagedBars B;
  B.q_full = bars;
  B.q_empty = B.q_full + 2;
  B.x_done = B.q_empty + 2;
  B.x_full = B.x_done + 2;
  B.x_next = B.x_full + 1;
  B.k_full = B.x_next + 1;
  B.k_empty = B.k_full + C::kKSlots;
  B.v_full = B.k_empty + C::kKSlots;
  B.v_empty = B.v_full + C::kVSlots;
  B.v_clear = B.v_empty + C::kVSlots;
  B.s_full = B.v_clear + C::kVSlots;
  B.p_full = B.s_full + 2;
  B.p_half = B.p_full + 2;
  B.o_full = B.p_half + 2;
  B.mma_done = B.o_full + 2;
  B.seg_full = B.mma_done + 1;
  B.seg_empty = B.seg_full + C::kSegs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::kOffTmemSlot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + C::kOffAbort);
  Plan* plan = reinterpret_cast<Plan*>(sm + C::kOffPlan);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int tt = p.tile_tokens, t4 = p.copy_tokens;
  const Shape sh = {SHORT ? t4 : 2 * tt, tt, t4, p.causal};

  if (warp == 0) {
    for (int i = lane; i < C::kNumBars; i += 32) {
      uint64_t* bar = bars + i;
      const bool merge = bar == B.x_full || bar == B.x_next || bar == B.x_done || bar == B.x_done + 1;
      const bool p_full = bar >= B.p_full && bar < B.p_full + 4;  // p_half too
      const bool v_empty = bar >= B.v_empty && bar < B.v_empty + C::kVSlots;  // the MMA issuer and warp 10
      mbar_init(bar, merge ? 256 : p_full ? 128 : bar >= B.seg_empty ? 11 : v_empty ? 2 : 1);
    }
    if (lane == 0) *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_map(&tm_q);
    tma_prefetch_map(&tm_q4);
    tma_prefetch_map(&tm_k);
    tma_prefetch_map(&tm_v);
  }
  // Short chunks: the plan behind the barrier (64 sequences of 8 tokens against up to
  // 1024 keys, d = 64: 47.3 -> 45.4 us).  The other way round with the other forms,
  // whose softmax loops come out slower so (2 x 2048 tokens: 458 -> 463 us).
  if constexpr (!SHORT) make_plan<D, C::kThreads>(p, sh, plan);
  tc_fence_before();
  __syncthreads();
  if constexpr (SHORT) make_plan<D, C::kThreads>(p, sh, plan);
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  const Work work(p);
  auto form_of = [&](const Segment& g) { return SHORT ? kFourCopies : sh.form(g.ntok); };
  // The roles' walk through the run: `step` goes to the next segment, the first one
  // included.  With short chunks warp 11 walks for all and the others read what it
  // wrote: one copy of that code instead of five, and out of the chain between one
  // unit's outputs and the next one's scores.
  struct Place {
    Walk w;
    Segment g;
    uint32_t count;
  };
  auto start = [&] {
    Place a;
    a.count = 0;
    if constexpr (!SHORT) a.w = walk_start(work, plan->at[0], plan->at[1], plan->q[0], sh);
    return a;
  };
  auto step = [&](Place& a, bool& ok) {
    if (!ok) return false;
    if constexpr (SHORT) {
      const int slot = a.count % C::kSegs;
      ok = wait_warp<SHORT>(&B.seg_full[slot], (a.count / C::kSegs) & 1, status);
      if (!ok) return false;
      ++a.count;
      const int4* e = reinterpret_cast<const int4*>(sm + C::kOffSegs) + 3 * slot;
      const int4 x = e[0], y = e[1], z = e[2];
      __syncwarp();
      if (lane == 0) mbar_arrive(&B.seg_empty[slot]);
      a.w = {{x.x, x.y, 0, 0}, {x.z, x.w, y.x}};
      a.g = {y.y, y.z, y.w, z.x, z.y};
      return z.z != 0;
    } else {
      if (a.count++ > 0) walk_next(work, a.w, plan->at[1], sh, a.g);
      return walk_get(work, a.w, plan->at[1], sh, a.g);
    }
  };

  if (warp >= 8) {
    regs_dec<C::kAuxRegs>();
    if (warp == 8) {
      // ------------------------------------------------------------ producer --
      Place place = start();
      const Walk& w = place.w;
      const Segment& g = place.g;
      const int box_rows = min(1 << p.page_log2, kTileRows);
      const int per_tile = kTileRows / box_rows;  // pages of a key tile (1 if pages are longer)
      const uint32_t box_bytes = box_rows * 128;
      // Query buffers: two-tile units take both (buffer t for tile t), the
      // others one in turn.  What frees a buffer depends on its last user.
      uint32_t q_uses[2] = {0, 0};            // copies into each buffer
      uint32_t by_mma[2] = {0, 0}, by_merge[2] = {0, 0};
      bool merged[2] = {false, false};
      uint32_t turn = 0, kv_it = 0;
      bool ok = true, lost = false;
      auto wait_q = [&](int b) {
        if (merged[b]) return wait_warp<true>(&B.x_done[b], (by_merge[b] - 1) & 1, status);
        return by_mma[b] == 0 || wait_warp<true>(&B.q_empty[b], (by_mma[b] - 1) & 1, status);
      };
      while (step(place, ok)) {
        const Form form = form_of(g);
        const int* table = p.page_table + (size_t)w.at.s * p.max_pages;
        const int pages = (w.q.kv + (1 << p.page_log2) - 1) >> p.page_log2;
        // this lane's page of key tile j, asked for a tile ahead
        auto page_at = [&](int j) {
          const int at = (j * kTileRows + lane * box_rows) >> p.page_log2;
          return lane < per_tile && at < pages ? __ldg(table + at) : 0;
        };
        int next = page_at(g.j0);
        const int q_row = w.q.q0 + g.tok0;
        auto load_q = [&](int b, const CUtensorMap* map, int copies, uint32_t box, int row) {
          if (lane == 0) {
            uint8_t* dst = sm + C::kOffQ + b * C::kTileBytes;
            mbar_expect_tx(&B.q_full[b], copies * box * C::kBlocks);
#pragma unroll 1
            for (int kb = 0; kb < C::kBlocks; ++kb)
#pragma unroll 1
              for (int c = 0; c < copies; ++c)
                tma_load_4d(dst + kb * kSwzBlockBytes + c * (kSwzBlockBytes / 4), map, &B.q_full[b], 64 * kb, 0, w.at.hk,
                            row);
          }
          __syncwarp();
        };
        if (form == kTwoTiles) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!ok || (t == 0 && tile0_count(w.q, g, sh) == 0)) continue;
            if (!(ok = wait_q(t))) break;
            load_q(t, &tm_q, 1, tt * p.G * 128, q_row + t * tt);
            ++q_uses[t];
            ++by_mma[t];
            merged[t] = false;
          }
        } else {
          const int b = turn & 1;
          ++turn;
          ok = b ? wait_q(1) : wait_q(0);
          if (!ok) break;
          if (form == kFourCopies)
            load_q(b, &tm_q4, 4, t4 * p.G * 128, q_row);
          else
            load_q(b, &tm_q, 1, tt * p.G * 128, q_row);
          if (b) {
            ++q_uses[1], ++by_merge[1], merged[1] = true;
          } else {
            ++q_uses[0], ++by_merge[0], merged[0] = true;
          }
        }
        for (int j = g.j0; j < g.j1 && ok; ++j, ++kv_it) {
          const int left = w.q.kv - j * kTileRows;  // keys from this tile on
          const int boxes = left <= 0 ? 0 : min(per_tile, (left + box_rows - 1) / box_rows);
          const int row = per_tile == 1 ? (j * kTileRows) & ((1 << p.page_log2) - 1) : 0;
          int page = next;
          if (j + 1 < g.j1) next = page_at(j + 1);
          if (page < 0 || page >= p.num_pages) {
            // outside the pool: the copy reads past the map's last page and fills with zeros
            page = p.num_pages;
            lost = lost || lane < boxes;
          }
          const int ks = kv_it % C::kKSlots, vs = kv_it % C::kVSlots;
          const uint32_t kph = (kv_it / C::kKSlots) & 1, vph = (kv_it / C::kVSlots) & 1;
          if (!(ok = wait_warp<true>(&B.k_empty[ks], kph ^ 1, status))) break;
          if (lane == 0) mbar_expect_tx(&B.k_full[ks], boxes * box_bytes * C::kBlocks);
          __syncwarp();
          if (lane < boxes) {
            uint8_t* dst = sm + C::kOffK + ks * C::kTileBytes + lane * box_bytes;
            for (int kb = 0; kb < C::kBlocks; ++kb)
              tma_load_4d(dst + kb * kSwzBlockBytes, &tm_k, &B.k_full[ks], 64 * kb, row, w.at.hk, page);
          }
          __syncwarp();
          if (!(ok = wait_warp<true>(&B.v_empty[vs], vph ^ 1, status))) {
            // the K copy of this tile is in flight: it lands before the block ends
            wait_warp<true>(&B.k_full[ks], kph, status);
            break;
          }
          if (lane == 0) mbar_expect_tx(&B.v_full[vs], boxes * box_bytes * C::kBlocks);
          __syncwarp();
          if (lane < boxes) {
            uint8_t* dst = sm + C::kOffV + vs * C::kTileBytes + lane * box_bytes;
            for (int kb = 0; kb < C::kBlocks; ++kb)
              tma_load_4d(dst + kb * kSwzBlockBytes, &tm_v, &B.v_full[vs], 64 * kb, row, w.at.hk, page);
          }
          __syncwarp();
        }
        if (__any_sync(0xffffffffu, aborted(abort_flag))) ok = false;
      }
      if (!ok) *abort_flag = 1;
      if (lost) record_index(status);
      // Drain: every copy this warp started lands before the block ends.
#pragma unroll
      for (int b = 0; b < 2; ++b)
        if (q_uses[b] > 0) wait_warp<true>(&B.q_full[b], (q_uses[b] - 1) & 1, status);
      for (uint32_t i = kv_it > (uint32_t)C::kKSlots ? kv_it - C::kKSlots : 0; i < kv_it; ++i)
        wait_warp<true>(&B.k_full[i % C::kKSlots], (i / C::kKSlots) & 1, status);
      for (uint32_t i = kv_it > (uint32_t)C::kVSlots ? kv_it - C::kVSlots : 0; i < kv_it; ++i)
        wait_warp<true>(&B.v_full[i % C::kVSlots], (i / C::kVSlots) & 1, status);
    } else if (warp == 9) {
      // ---------------------------------------------------------- MMA issuer --
      Place place = start();
      const Walk& w = place.w;
      const Segment& g = place.g;
      const uint32_t idS = idesc_bf16(128, 128, 0, 0) | s_negate;  // S = (+/-) Q K^T, both K-major
      constexpr uint32_t kIdO = idesc_bf16(128, D, 0, 1);            // O += P V, V is MN-major
      const uint32_t q_s = smem_addr(sm + C::kOffQ);
      const uint32_t k_s = smem_addr(sm + C::kOffK);
      const uint32_t v_s = smem_addr(sm + C::kOffV);
      uint32_t q_uses[2] = {0, 0}, pcnt[2] = {0, 0}, hcnt[2] = {0, 0}, turn = 0, kv_it = 0;
      uint32_t clears = 0;  // bit st: parity of v_clear[st]
      bool ok = true;
      auto issue_s = [&](int t, uint32_t qa, uint32_t it) {
        const uint32_t ka = k_s + (it % C::kKSlots) * C::kTileBytes;
#pragma unroll(SHORT ? 1 : C::kBlocks)
        for (int kb = 0; kb < C::kBlocks; ++kb)
          mma_ss_run_w<4, 2, 2>(tbase + C::kColS + 128 * t, sdesc(qa + kb * kSwzBlockBytes, 16, 1024),
                                sdesc(ka + kb * kSwzBlockBytes, 16, 1024), idS, kb > 0);
        mma_commit_w(&B.s_full[t]);
      };
      auto wait_k = [&](uint32_t it) {
        if (!wait_warp<true>(&B.k_full[it % C::kKSlots], (it / C::kKSlots) & 1, status)) return false;
        tc_fence_after();
        return true;
      };
      // O_t (+)= P_t V: the first or second 64 keys (4 steps of 16), or all
      auto issue_pv_half = [&](int t, uint32_t it, int h, bool accumulate) {
        mma_ts_run_w<4, 8, 128>(tbase + C::kColO + 128 * t, tbase + C::kColS + 128 * t + 32 * h,
                                sdesc(v_s + (it % C::kVSlots) * C::kTileBytes + h * (kSwzBlockBytes / 2),
                                      kSwzBlockBytes, 1024),
                                kIdO, accumulate);
      };
      auto issue_pv = [&](int t, uint32_t it, bool accumulate) {
        mma_ts_run_w<8, 8, 128>(tbase + C::kColO + 128 * t, tbase + C::kColS + 128 * t,
                                sdesc(v_s + (it % C::kVSlots) * C::kTileBytes, kSwzBlockBytes, 1024), kIdO,
                                accumulate);
      };
      while (step(place, ok)) {
        const Form form = form_of(g);
        const int nt = g.j1 - g.j0;
        const int last = last_tile(w.q.kv);
        const int tail = w.q.kv - (last << 7) < kTileRows ? last - g.j0 : -1;
        // V of the segment's key tile i: cleared behind the end where the sequence ends in it
        auto wait_v = [&](int i) {
          const uint32_t it = kv_it + i;
          const int st = it % C::kVSlots;
          if (i == tail) {
            const uint32_t parity = (clears >> st) & 1;
            clears ^= 1u << st;
            return wait_warp<true>(&B.v_clear[st], parity, status);
          }
          return wait_warp<true>(&B.v_full[st], (it / C::kVSlots) & 1, status);
        };
        if (form != kTwoTiles) {
          const int b = turn & 1;
          ++turn;
          const uint32_t qa = q_s + b * C::kTileBytes;
          ok = wait_warp<true>(&B.q_full[b], (b ? q_uses[1] : q_uses[0]) & 1, status);
          if (b)
            ++q_uses[1];
          else
            ++q_uses[0];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (!ok || i >= nt || !(ok = wait_k(kv_it + i))) continue;
            issue_s(i, qa, kv_it + i);
            mma_commit_w(&B.k_empty[(kv_it + i) % C::kKSlots]);
          }
          for (int i = 0; i < nt && ok; ++i) {
            const int t = i & 1;
            const bool halves = !SHORT && form == kOneTile;
            if (halves) {
              ok = wait_warp<true>(&B.p_half[t], (t ? hcnt[1] : hcnt[0]) & 1, status);
              if (t)
                ++hcnt[1];
              else
                ++hcnt[0];
              if (!ok || !(ok = wait_v(i))) break;
              tc_fence_after();
              issue_pv_half(t, kv_it + i, 0, i >= 2);
            }
            ok = wait_warp<true>(&B.p_full[t], (t ? pcnt[1] : pcnt[0]) & 1, status);
            if (t)
              ++pcnt[1];
            else
              ++pcnt[0];
            if (!ok || (!halves && !(ok = wait_v(i)))) break;
            tc_fence_after();
            if (halves)
              issue_pv_half(t, kv_it + i, 1, true);
            else
              issue_pv(t, kv_it + i, i >= 2);
            mma_commit_w(&B.v_empty[(kv_it + i) % C::kVSlots]);
            if (i + 2 < nt) {
              if (!(ok = wait_k(kv_it + i + 2))) break;
              issue_s(t, qa, kv_it + i + 2);
              mma_commit_w(&B.k_empty[(kv_it + i + 2) % C::kKSlots]);
            } else {
              mma_commit_w(&B.o_full[t]);  // covers the segment's last S too: issued before
            }
          }
        } else if constexpr (!SHORT) {
          const int cnt[2] = {tile0_count(w.q, g, sh), nt};
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!ok || cnt[t] == 0) continue;
            ok = wait_warp<true>(&B.q_full[t], q_uses[t] & 1, status);
            ++q_uses[t];
          }
          if (ok) ok = wait_k(kv_it);
          if (ok) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (cnt[t] == 0) continue;
              issue_s(t, q_s + t * C::kTileBytes, kv_it);
              if (cnt[t] == 1) mma_commit_w(&B.q_empty[t]);
            }
            mma_commit_w(&B.k_empty[kv_it % C::kKSlots]);
          }
          for (int i = 0; i < nt && ok; ++i) {
            bool v_ready = false, k_ready = false;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (!ok || i >= cnt[t]) continue;
              ok = wait_warp<true>(&B.p_half[t], hcnt[t] & 1, status);
              ++hcnt[t];
              if (ok && !v_ready) {
                ok = wait_v(i);
                v_ready = true;
              }
              if (!ok) break;
              tc_fence_after();
              issue_pv_half(t, kv_it + i, 0, i > 0);
              ok = wait_warp<true>(&B.p_full[t], pcnt[t] & 1, status);
              ++pcnt[t];
              if (!ok) break;
              tc_fence_after();
              issue_pv_half(t, kv_it + i, 1, true);
              if (i + 1 < cnt[t]) {
                if (!k_ready && !(ok = wait_k(kv_it + i + 1))) break;
                k_ready = true;
                issue_s(t, q_s + t * C::kTileBytes, kv_it + i + 1);
                if (i + 2 == cnt[t]) mma_commit_w(&B.q_empty[t]);  // the last S of this tile
              } else {
                mma_commit_w(&B.o_full[t]);
              }
            }
            if (ok) {
              mma_commit_w(&B.v_empty[(kv_it + i) % C::kVSlots]);
              if (i + 1 < nt) mma_commit_w(&B.k_empty[(kv_it + i + 1) % C::kKSlots]);
            }
          }
        }
        kv_it += nt;
        if (__any_sync(0xffffffffu, aborted(abort_flag))) ok = false;
      }
      if (!ok) *abort_flag = 1;
      mma_commit_w(B.mma_done);
      wait_warp<true>(B.mma_done, 0, status);
    } else if (warp == 10) {
      // ------------------------------------------- rows behind a sequence's end --
      // Follows every V tile (a parity wait must not run ahead of the ring, nor
      // the ring ahead of it: a slot is released by this warp as well).
      Place place = start();
      const Walk& w = place.w;
      const Segment& g = place.g;
      uint32_t kv_it = 0;
      bool ok = true;
      while (step(place, ok)) {
        const int last = last_tile(w.q.kv), used = w.q.kv - (last << 7);
        for (int j = g.j0; j < g.j1; ++j, ++kv_it) {
          const int st = kv_it % C::kVSlots;
          if (!(ok = wait_warp<true>(&B.v_full[st], (kv_it / C::kVSlots) & 1, status))) break;
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
      }
      if (!ok) *abort_flag = 1;
    } else if constexpr (SHORT) {
      // ------------------------------------------------------------ the walk --
      Walk w = walk_start(work, plan->at[0], plan->at[1], plan->q[0], sh);
      Segment g = {};
      for (uint32_t i = 0;; ++i) {
        const bool more = !__any_sync(0xffffffffu, aborted(abort_flag)) && walk_get(work, w, plan->at[1], sh, g);
        const int slot = i % C::kSegs;
        if (!wait_warp<true>(&B.seg_empty[slot], ((i / C::kSegs) & 1) ^ 1, status)) break;
        if (lane == 0) {
          int4* e = reinterpret_cast<int4*>(sm + C::kOffSegs) + 3 * slot;
          e[0] = make_int4(w.at.s, w.at.hk, w.q.q0, w.q.qn);
          e[1] = make_int4(w.q.kv, g.tok0, g.ntok, g.n);
          e[2] = make_int4(g.j0, g.j1, more, 0);
          mbar_arrive(&B.seg_full[slot]);
        }
        __syncwarp();
        if (!more) break;
        walk_next(work, w, plan->at[1], sh, g);
      }
    }
  } else {
    regs_inc<C::kSoftmaxRegs>();
    // -------------------------------------------------------------- softmax --
    const int t = warp / 4, quarter = warp % 4;
    const int r = quarter * 32 + lane;  // row of the tile
    const uint32_t t_s = tmem_lane_col(tbase, quarter * 32, C::kColS + 128 * t);
    const uint32_t t_o = tmem_lane_col(tbase, quarter * 32, C::kColO + 128 * t);
    uint32_t scnt = 0, ocnt = 0, turn = 0;
    uint32_t x_uses[2] = {0, 0};  // one-tile units that took each query buffer
    uint32_t fills = 0, nexts = 0;
    bool guard = false;  // the other half may still read this half's O of the last (one-tile) unit
    bool ok = true;
    int tail_row0 = 0, tail_tok = 0, tail_hk = 0, has_tail = 0, has_head = 0;  // for the header
    float m_run = -INFINITY, l_run = 0.f;  // running maximum (log2 units) and sum of this row, in this warp's columns
    // Of rescaling (log2 units).  Infinite for a row that is no token's: what such rows
    // hold (neighbours' queries, leftovers where G does not divide 32) must not decide
    // when the warp rescales, as that is seen in the last bits of the others.
    float threshold = kRescaleThreshold;
    // One key tile: NC columns from c0 on; MASK: column c is seen iff c <= cut.
    auto tile = [&](auto nc, auto masked, int c0, bool first, int cut) {
      constexpr int NC = decltype(nc)::value;
      tc_fence_after();
      uint32_t sv[NC];
#pragma unroll
      for (int c = 0; c < NC / 32; ++c) tmem_ld32(t_s + c0 + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&sv[32 * c]));
      tmem_wait_ld();
      float* s = reinterpret_cast<float*>(sv);
      if constexpr (decltype(masked)::value) {
#pragma unroll
        for (int c = 0; c < NC; ++c) s[c] = (c > cut) ? -INFINITY : s[c];
      }
      float pm[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) pm[e] = max3f(s[2 * e], s[2 * e + 1], -INFINITY);
#pragma unroll
      for (int c = 16; c < NC; c += 2) pm[(c / 2) & 7] = max3f(pm[(c / 2) & 7], s[c], s[c + 1]);
      const float mx2 = max3f(max3f(pm[0], pm[1], pm[2]), max3f(pm[3], pm[4], pm[5]), fmaxf(pm[6], pm[7])) * c2;
      if (first) {
        m_run = mx2;
      } else {
        const bool need = mx2 > m_run + threshold;
        if (__any_sync(0xffffffffu, need)) {
          // O_t is quiescent: this S was committed after P V of this half's last tile
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
      for (int h = 0; h < NC / 32; ++h) {
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
        tmem_st16(t_s + c0 / 2 + 16 * h, pk);
        if (NC == 128 && h == 1) {  // P V of the first 64 keys may start
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&B.p_half[t]);
        }
      }
      if constexpr (NC == 32) {  // this copy of the rows takes no other columns
        const uint32_t zero[16] = {};
#pragma unroll
        for (int h = 1; h < 4; ++h) tmem_st16(t_s + ((c0 / 2 + 16 * h) & 63), zero);
      }
      float a0, a1;
      f2_unpack(f2_add(f2_add(ls[0], ls[1]), f2_add(ls[2], ls[3])), a0, a1);
      l_run += a0 + a1;
      tmem_wait_st();
      tc_fence_before();
    };
    Place place = start();
    const Walk& w = place.w;
    const Segment& g = place.g;
    while (step(place, ok)) {
      const Form form = form_of(g);
      const bool two = form == kTwoTiles, four = form == kFourCopies;
      const int nt = g.j1 - g.j0;
      const int row = four ? lane : r;              // among the query tile's rows
      const int rtok = token_of(p, row), rhead = row - rtok * p.G;
      const int tile0 = two ? t * tt : 0;           // the query tile's first token in the unit
      const int tok = g.tok0 + tile0 + rtok;        // in the sequence
      const int tile_rows = min(tt, g.ntok - tile0) * p.G;
      const bool valid = row < tile_rows;
      const bool busy = four || quarter * 32 < tile_rows;  // any row of this warp
      const int cnt = two ? (t ? nt : tile0_count(w.q, g, sh)) : (nt + 1 - t) / 2;
      const int jfirst = g.j0 + (two ? 0 : t), jshift = two ? 0 : 1;  // every second key tile
      const int past = w.q.kv - w.q.qn;
      const int lim = !valid ? -1 : p.causal ? min(past + tok, w.q.kv - 1) : w.q.kv - 1;  // last key it sees
      // the tile's first row's: up to it no key tile needs a mask
      const int lim0 = p.causal ? min(past + g.tok0 + tile0, w.q.kv - 1) : w.q.kv - 1;
      threshold = valid ? kRescaleThreshold : INFINITY;
      m_run = -INFINITY;
      l_run = 0.f;
      if (!SHORT && cnt > 0 && guard) {
        // both halves must have read that O before P V overwrites it
        const int b = ~turn & 1;  // that unit's buffer: the one in front of the next
        if (!(ok = wait_warp<SHORT>(&B.x_done[b], ((b ? x_uses[1] : x_uses[0]) - 1) & 1, status))) break;
        guard = false;
      }
      // Key tiles [0, free) need no mask, the others come behind them: two loops, so
      // that the first has no masking in it (4% of a long chunk's time).
      const int free = min(cnt, max(0, ((lim0 + 1) >> 7) - jfirst + jshift) >> jshift);
      auto tiles = [&](auto nc, auto masked, int c0, int from, int to) {
        for (int i = from; i < to && ok; ++i) {
          if (!(ok = wait_warp<SHORT>(&B.s_full[t], scnt & 1, status))) break;
          ++scnt;
          tile(nc, masked, c0, i == 0, lim - (jfirst + (i << jshift)) * kTileRows - c0);
#ifdef FA_TEST_HOOKS
          if (t == 0 && i == 0 && *reinterpret_cast<volatile int*>(&g_fa_test_paged) == 1) continue;
#endif
          mbar_arrive(&B.p_full[t]);
        }
      };
      constexpr std::false_type kFree{};
      constexpr std::true_type kMasked{};
      if (four) {
        constexpr std::integral_constant<int, 32> kQuarter{};
        tiles(kQuarter, kMasked, 32 * quarter, 0, cnt);  // (one loop: less code, see wait_warp)
      } else if constexpr (!SHORT) {
        constexpr std::integral_constant<int, 128> kAll{};
        if (busy) {
          tiles(kAll, kFree, 0, 0, free);
          tiles(kAll, kMasked, 0, free, cnt);
        } else {
          for (int i = 0; i < cnt && ok; ++i) {
            if (!(ok = wait_warp<SHORT>(&B.s_full[t], scnt & 1, status))) break;
            ++scnt;
            mbar_arrive(&B.p_half[t]);
            mbar_arrive(&B.p_full[t]);
          }
        }
      }
      if (ok && cnt > 0) {
        ok = wait_warp<SHORT>(&B.o_full[t], ocnt & 1, status);
        ++ocnt;
      }
      if (!ok) break;
      tc_fence_after();
      const bool whole = g.j0 == 0 && g.j1 == g.n;
      const size_t out_row = (size_t)(w.q.q0 + tok) * (p.Hk * p.G) + w.at.hk * p.G + rhead;
      const size_t slot = ((size_t)blockIdx.x * 2 + (g.j0 > 0 ? 0 : 1)) * kPagedRows;
      if (four) {
        // Up to eight partial rows (four if there was one key tile) for each query row: eight
        // query rows at a time, every warp writes its unnormalised outputs to the dead query
        // buffer (16-byte chunk c of row rr at c ^ rr) with their (m, l); a thread adds up one
        // chunk of one row.
        const int b = turn & 1;
        ++turn;
        float4* xs = reinterpret_cast<float4*>(sm + C::kOffQ + b * C::kTileBytes);
        float2* ml = reinterpret_cast<float2*>(sm + C::kOffMl) + 64 * b;
        const int parts = nt > 1 ? 8 : 4;
        constexpr int kChunks = D / 4;
        for (int r0 = 0; r0 < tile_rows; r0 += 8) {
          if (cnt > 0) {
            const bool mine = lane >= r0 && lane < r0 + 8 && valid;
            const int rr = lane & 7;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t v[32];
              tmem_ld32(t_o + 32 * c, v);
              tmem_wait_ld();
              if (mine) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  xs[(warp * 8 + rr) * kChunks + ((8 * c + k) ^ rr)] =
                      make_float4(__uint_as_float(v[4 * k]), __uint_as_float(v[4 * k + 1]),
                                  __uint_as_float(v[4 * k + 2]), __uint_as_float(v[4 * k + 3]));
              }
            }
            if (mine) ml[warp * 8 + rr] = make_float2(m_run, l_run);
          }
          mbar_arrive(B.x_full);
          if (!(ok = wait_warp<SHORT>(B.x_full, fills & 1, status))) break;
          ++fills;
          guard = false;  // everyone is past the last unit
          const int rr = threadIdx.x / kChunks, c = threadIdx.x % kChunks, q_row = r0 + rr;
          if (rr < 8 && q_row < tile_rows) {
            float m = -INFINITY;
            float2 part[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              part[i] = i < parts ? ml[i * 8 + rr] : make_float2(-INFINITY, 0.f);
              m = fmaxf(m, part[i].x);
            }
            float l = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if (part[i].y == 0.f) continue;  // saw no key (a row of NaN has a maximum of -inf, too)
              const float wt = ex2(part[i].x - m);
              const float4 x = xs[(i * 8 + rr) * kChunks + (c ^ rr)];
              l = fmaf(wt, part[i].y, l);
              o.x = fmaf(wt, x.x, o.x), o.y = fmaf(wt, x.y, o.y), o.z = fmaf(wt, x.z, o.z), o.w = fmaf(wt, x.w, o.w);
            }
            if (whole) {
              const int qt = token_of(p, q_row);
              const size_t at = (size_t)(w.q.q0 + g.tok0 + qt) * (p.Hk * p.G) + w.at.hk * p.G + (q_row - qt * p.G);
              const float inv = l == 0.f ? 0.f : 1.f / l;
              reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + at * D)[c] =
                  make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
              if (c == 0 && p.lse) p.lse[at] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
            } else {
              reinterpret_cast<float4*>(p.part_o + (slot + q_row) * D)[c] = o;
              if (c == 0) reinterpret_cast<float2*>(p.part_ml)[slot + q_row] = make_float2(m, l);
            }
          }
          if (r0 + 8 < tile_rows) {
            mbar_arrive(B.x_next);
            if (!(ok = wait_warp<SHORT>(B.x_next, nexts & 1, status))) break;
            ++nexts;
          }
        }
        if (!ok) break;
        fence_proxy_async_smem();  // the next copy into the buffer comes behind these accesses
        mbar_arrive(&B.x_done[b]);
        if (b)
          ++x_uses[1];
        else
          ++x_uses[0];
      } else if constexpr (!SHORT) {
        // One-tile unit of two or more key tiles: both halves' (m, l) through the dead query
        // buffer, then each half writes half of the columns from both outputs.  With one
        // key tile half 1 has nothing to add, but waits as well: it must not run ahead, and
        // arrive on x_done for the unit after the next in half 0's place.
        const bool merge = !two && nt > 1;
        float w0 = 1.f, w1 = 0.f, m_out = m_run, l_out = l_run;  // weights of this half's and the other's output
        const int b = turn & 1;
        if (!two) {
          float2* ml = reinterpret_cast<float2*>(sm + C::kOffQ + b * C::kTileBytes);
          if (merge) ml[t * 128 + r] = make_float2(m_run, l_run);
          mbar_arrive(B.x_full);
          if (!(ok = wait_warp<SHORT>(B.x_full, fills & 1, status))) break;
          ++fills;
          if (merge) {
            const float2 other = ml[(1 - t) * 128 + r];
            m_out = fmaxf(m_run, other.x);
            w0 = l_run == 0.f ? 0.f : ex2(m_run - m_out);
            w1 = other.y == 0.f ? 0.f : ex2(other.x - m_out);
            l_out = l_run * w0 + other.y * w1;
          }
        }
        if (busy && (two || merge || t == 0)) {  // (a single key tile: half 0 alone)
          const bool empty = l_out == 0.f;       // saw no key: zero, whatever O holds
          const float scale_o = whole ? (empty ? 0.f : 1.f / l_out) : 1.f;
          w0 *= scale_o;
          w1 *= scale_o;
          const size_t part = slot + (two ? t * 128 : 0) + r;
          const int c_lo = merge ? t * (D / 2) : 0, c_hi = merge ? c_lo + D / 2 : D;
          const uint32_t t_o1 = tmem_lane_col(tbase, quarter * 32, C::kColO + 128 * (1 - t));
#pragma unroll 1
          for (int c = c_lo; c < c_hi; c += 32) {
            uint32_t v[32];
            if (cnt > 0) {
              tmem_ld32(t_o + c, v);
              if (merge) {
                uint32_t u[32];
                tmem_ld32(t_o1 + c, u);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                  // a half that saw no key has weight 0 and an O of zeros times V
                  const float x = w0 == 0.f ? 0.f : w0 * __uint_as_float(v[k]);
                  v[k] = __float_as_uint(w1 == 0.f ? x : fmaf(w1, __uint_as_float(u[k]), x));
                }
              } else {
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 32; ++k) v[k] = empty ? 0u : __float_as_uint(w0 * __uint_as_float(v[k]));
              }
            } else {
#pragma unroll
              for (int k = 0; k < 32; ++k) v[k] = 0u;
            }
            if (!valid) continue;
            if (whole) {
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                uint32_t y[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  y[k] = pack_bf16x2(__uint_as_float(v[8 * h + 2 * k]), __uint_as_float(v[8 * h + 2 * k + 1]));
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + out_row * D + c + 8 * h) =
                    make_uint4(y[0], y[1], y[2], y[3]);
              }
            } else {
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                uint32_t y[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) y[k] = v[8 * h + k];
                store32(p.part_o + part * D + c + 8 * h, y);
              }
            }
          }
          if (valid && (!merge || t == 0)) {
            if (!whole)
              reinterpret_cast<float2*>(p.part_ml)[part] = make_float2(m_out, l_out);
            else if (p.lse)
              p.lse[out_row] = empty ? -INFINITY : (m_out + __log2f(l_out)) * kLn2;
          }
        }
        if (!two) {
          ++turn;
          tc_fence_before();
          fence_proxy_async_smem();
          mbar_arrive(&B.x_done[b]);
          if (b)
            ++x_uses[1];
          else
            ++x_uses[0];
          guard = true;
        }
      }
      if (g.j0 > 0) {
        has_head = g.j1 == g.n ? 2 : 1;
      } else if (g.j1 < g.n) {
        has_tail = 1;
        tail_row0 = w.q.q0 + g.tok0;
        tail_tok = g.ntok;
        tail_hk = w.at.hk;
      }
      tc_fence_before();
      if (__any_sync(0xffffffffu, aborted(abort_flag))) ok = false;
    }
    if (!ok) *abort_flag = 1;
    if (threadIdx.x == 0) {
      int4* hdr = reinterpret_cast<int4*>(p.hdr + (size_t)blockIdx.x * kPagedHdr);
      hdr[0] = make_int4(has_tail, tail_row0, tail_tok, tail_hk);
      hdr[1] = make_int4(has_head, 0, 0, 0);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tbase, C::kTmemCols);
  }
}

// Merges the units that were cut: blocks (c, y) take rows of the unit that CTA c
// began and did not end.  Its parts are CTA c's second slot and the first slots
// of the CTAs behind it up to the one that ended it, added in a fixed order.
// D / 8 lanes a row.  Of few parts a warp adds up all, AHEAD of them asked for at
// once: two where the rows are many (40 MB in all where every CTA cut a unit of 256
// rows), eight for the few rows of short chunks.  More parts (a long cache and few
// heads) are shared by a block's warps, eight parts at a time, and the rows by the
// blocks of all CTAs that worked on the unit: one warp after 46 parts of a unit
// (267 tokens, one head, 5885 keys, d = 64) took most of that call's 39 us.
template <int D, int AHEAD>
__global__ void __launch_bounds__(256, AHEAD == 2 ? 4 : 2) paged_merge_kernel(const PagedParams p, int ctas) {
  constexpr int kLanes = D / 8, kRowsAWarp = 32 / kLanes, kRowsABlock = 8 * kRowsAWarp;
  const int lane = threadIdx.x & 31, l8 = lane % kLanes;
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
  int c = blockIdx.x;  // the CTA that began the unit
  auto slot = [&](int i) { return ((size_t)(c + i) * 2 + (i == 0 ? 1 : 0)) * kPagedRows; };
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int4 h = *reinterpret_cast<const int4*>(p.hdr + (size_t)c * kPagedHdr);
  const int inside = p.hdr[(size_t)c * kPagedHdr + 4];
  int ends = c + 1 + lane < ctas ? p.hdr[(size_t)(c + 1 + lane) * kPagedHdr + 4] : 2;
  if (!h.x) {
    if (inside != 1) return;
    // this CTA's run lies within a unit: the nearest one in front that began one
    for (int at = c - 1;; at -= 32) {
      const unsigned found = __ballot_sync(0xffffffffu, at >= lane && p.hdr[(size_t)(at - lane) * kPagedHdr] != 0);
      if (found) {
        c = at - (__ffs(found) - 1);
        break;
      }
      if (at < 32) return;
    }
    h = *reinterpret_cast<const int4*>(p.hdr + (size_t)c * kPagedHdr);
    ends = c + 1 + lane < ctas ? p.hdr[(size_t)(c + 1 + lane) * kPagedHdr + 4] : 2;
  }
  // the first CTA behind c whose first slot ends its unit
  int last = ctas - 1;
  for (int at = c + 1;; at += 32) {
    const unsigned found = __ballot_sync(0xffffffffu, ends != 1);
    if (found) {
      last = min(last, at + __ffs(found) - 1);
      break;
    }
    ends = at + 32 + lane < ctas ? p.hdr[(size_t)(at + 32 + lane) * kPagedHdr + 4] : 2;
  }
  const int parts = last - c + 1;
  const int tile = p.tile_tokens * p.G;
  const int rows = h.z * p.G;  // valid rows, densely numbered
  auto put = [&](int n, float m, float l, const float (&acc)[8]) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int tok = token_of(p, n);
    const size_t row = (size_t)(h.y + tok) * (p.Hk * p.G) + h.w * p.G + (n - tok * p.G);
    reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + row * D)[l8] =
        make_uint4(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv),
                   pack_bf16x2(acc[4] * inv, acc[5] * inv), pack_bf16x2(acc[6] * inv, acc[7] * inv));
    if (l8 == 0 && p.lse) p.lse[row] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
  };
  auto add = [](float (&acc)[8], float w, const float4& a, const float4& b) {
    acc[0] = fmaf(w, a.x, acc[0]), acc[1] = fmaf(w, a.y, acc[1]), acc[2] = fmaf(w, a.z, acc[2]);
    acc[3] = fmaf(w, a.w, acc[3]), acc[4] = fmaf(w, b.x, acc[4]), acc[5] = fmaf(w, b.y, acc[5]);
    acc[6] = fmaf(w, b.z, acc[6]), acc[7] = fmaf(w, b.w, acc[7]);
  };
  if (parts > (AHEAD == 2 ? 4 : 8)) {
    __shared__ float4 sum[8][32][2];
    __shared__ float2 stat[8][32];
    const int wp = threadIdx.x / 32, blocks = (last - c) * gridDim.y;
    for (int q = (blockIdx.x - c) * gridDim.y + blockIdx.y; q * kRowsAWarp < rows; q += blocks) {
      const int n = min(q * kRowsAWarp + lane / kLanes, rows - 1);  // (rows past the end repeat the last one)
      const int prow = n < tile ? n : 128 + n - tile;
      float m = -INFINITY, l = 0.f, acc[8] = {};
      float4 v0 = {}, v1 = {};
      float2 x = {-INFINITY, 0.f};
      auto load = [&](int i) {
        const float4* src = reinterpret_cast<const float4*>(p.part_o + (slot(i) + prow) * D) + 2 * l8;
        v0 = src[0], v1 = src[1], x = ml[slot(i) + prow];
      };
      if (wp < parts) load(wp);
      for (int i = wp; i < parts; i += 8) {
        const float4 u0 = v0, u1 = v1;
        const float2 y = x;
        if (i + 8 < parts) load(i + 8);
        if (y.y == 0.f) continue;  // saw no key
        const float m_new = fmaxf(m, y.x);
        const float old = m == -INFINITY ? 0.f : ex2(m - m_new), w = ex2(y.x - m_new);
        l = fmaf(w, y.y, l * old);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] *= old;
        add(acc, w, u0, u1);
        m = m_new;
      }
      sum[wp][lane][0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      sum[wp][lane][1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
      stat[wp][lane] = make_float2(m, l);
      __syncthreads();
      if (wp == 0) {
        for (int k = 1; k < 8; ++k) m = fmaxf(m, stat[k][lane].x);
        l = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
        for (int k = 0; k < 8; ++k) {
          const float2 y = stat[k][lane];
          if (y.y == 0.f) continue;
          const float w = ex2(y.x - m);
          l = fmaf(w, y.y, l);
          add(acc, w, sum[k][lane][0], sum[k][lane][1]);
        }
        if (q * kRowsAWarp + lane / kLanes < rows) put(n, m, l, acc);
      }
      __syncthreads();
    }
    return;
  }
  if (c != (int)blockIdx.x) return;
  for (int n0 = blockIdx.y * kRowsABlock + threadIdx.x / 32 * kRowsAWarp; n0 < rows; n0 += gridDim.y * kRowsABlock) {
    const int n = min(n0 + lane / kLanes, rows - 1);  // (rows past the end repeat the last one)
    const int prow = n < tile ? n : 128 + n - tile;
    float4 v[AHEAD][2];
    float2 x[AHEAD];
    auto load = [&](int i, int k) {
      const float4* src = reinterpret_cast<const float4*>(p.part_o + (slot(i) + prow) * D) + 2 * l8;
      v[k][0] = src[0];
      v[k][1] = src[1];
      x[k] = ml[slot(i) + prow];
    };
    float m = -INFINITY;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (k < 2 || k < parts) load(k, k);  // a cut unit has two parts at least
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (k < 2 || k < parts) m = fmaxf(m, x[k].x);
    if (AHEAD < 4 && parts > AHEAD) {
      for (int i = AHEAD + l8; i < parts; i += kLanes) m = fmaxf(m, ml[slot(i) + prow].x);
#pragma unroll
      for (int off = kLanes / 2; off > 0; off /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    }
    float l = 0.f, acc[8] = {};
    for (int i = 0; i < parts; i += AHEAD) {
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        if (i + k >= parts) continue;
        const float w = x[k].y == 0.f ? 0.f : ex2(x[k].x - m);
        l = fmaf(w, x[k].y, l);
        add(acc, w, v[k][0], v[k][1]);
        if (i + k + AHEAD < parts) load(i + k + AHEAD, k);
      }
    }
    if (n0 + lane / kLanes < rows) put(n, m, l, acc);
  }
}

template <int D, bool SHORT>
cudaError_t launch_paged_t(const PagedLaunch& a, cudaStream_t stream) {
  using C = PagedCfg<D>;
  auto kern = paged_kernel<D, SHORT>;
  // The register split inside the kernel assumes it was built with exactly
  // kLaunchRegs registers a thread: refuse to launch any other build.
  static const bool regs_ok = [&] {
    cudaFuncAttributes attr;
    return cudaFuncGetAttributes(&attr, kern) == cudaSuccess && attr.numRegs == C::kLaunchRegs;
  }();
  if (!regs_ok) return cudaErrorInvalidKernelImage;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  kern<<<a.grid, C::kThreads, C::kSmemBytes, stream>>>(a.tm_q, a.tm_q4, a.tm_k, a.tm_v, a.p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  // Units of up to three key tiles are never cut (fa_paged_plan.cuh, place()).
  if (((long long)a.p.max_pages << a.p.page_log2) <= kNeverCut * kTileRows) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.grid, SHORT ? 2 : 4);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_merge_kernel<D, SHORT ? 8 : 2>, a.p, a.grid);
}

}  // namespace

cudaError_t launch_paged(const PagedLaunch& a, cudaStream_t stream) {
  if (a.d == 64) return a.is_short ? launch_paged_t<64, true>(a, stream) : launch_paged_t<64, false>(a, stream);
  return a.is_short ? launch_paged_t<128, true>(a, stream) : launch_paged_t<128, false>(a, stream);
}

}  // namespace fa

#ifdef FA_TEST_HOOKS
// Test builds only: sets what g_fa_test_paged says (0: nothing).
extern "C" int fa_test_paged(int mode) {
  return cudaMemcpyToSymbol(fa::g_fa_test_paged, &mode, sizeof(int)) == cudaSuccess ? 0 : 4;
}
#endif
