// Attention of a few rows over a paged cache: the entries of a batch whose sequences
// share keys (fa_paged_shared.cu) that have at most 16 (or 32) query rows a key head:
// single tokens, mostly, behind their group's shared keys.
//
// Bound: the read of K and V (4 d bytes a key for 4 d G FLOP; 64 single tokens of 8192 keys,
// 32 + 8 heads, d = 128, pages of 128: 320 us for 2.15 GB, 6.7 TB/s, the rate of a copy;
// pages of 16: 330).  The units are short, a few hundred keys, so what matters is that loads
// never wait for the end of one.  The
// 128-row tiles of paged_kernel take 2 us from a unit's last key tile to the next one's
// first scores (tensor memory, barriers between the roles, eight partial rows merged by
// the whole CTA); here a unit's end costs the loads nothing:
//
//   a producer warp goes from unit to unit on its own, up to eight ahead of the others; ten
//     stages of 16 KB (32 keys of d = 128, 64 of d = 64) an SM, in two CTAs
//   five warps take the stages in turn, each alone: S = Q K^T by 16 x 8 x 16 MMAs whose
//     results stay in registers (mma.sync: 16 rows are an eighth of tcgen05's smallest
//     tile, and the way through tensor memory and back is most of a short unit's time;
//     the MMAs here are busy a fifth of the time that the loads take), a running maximum
//     and sum of its own, P from the registers of S, O += P V.  More rows than a tile or two
//     are paged_kernel's: 64 would keep these MMAs busy three quarters of the time
//   where a unit has up to 32 rows a second team of five warps takes the other 16: it reads
//     the same stages, a warp of each team a stage (one warp for both tiles took 1.9 us a
//     stage, and five warps 1.9 us to join a unit: 51 sequences of 5 tokens, 20 + 4 heads,
//     in 4 groups 46.5 us, 40.6 with two teams)
//   the stages of the next unit go on where those of the last one ended, so that units of
//     a stage or two run side by side; the warp that is the last to put its partial rows
//     into shared memory joins them, while the others are at the next unit
//
// Units are (piece, key head) pairs in the order of a list; CTAs take them from a
// counter, as paged_kernel's CTAs leave their SMs to this kernel one after the other.  Which
// CTA computes a unit has no part in its result: its stages go to the
// warps in the order of the unit, and are joined in that order, too.
//
// Rounding as in paged_kernel: scores, maxima, sums and O in fp32, P to bf16 once for the
// second product.
//
// Registers: 168, what the room for two CTAs (or one of eleven warps) leaves a thread; of it
// d = 128 with two row tiles spills 20 bytes, with one 4, d = 64 with one 8.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_common.cuh"
#include "fa_context.h"
#include "fa_paged.cuh"
#include "fa_paged_plan.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

using namespace paged;

#ifdef FA_TEST_HOOKS
// Test builds only (-DFA_TEST_HOOKS, never the default library).  1: warp 0 withholds its
// arrival where the partial rows are joined, so that the waits there run out.  2: every CTA
// takes its shared memory for misaligned.
static __device__ int g_fa_test_rows;
#endif

template <int D, int MT>
struct RowsCfg {
  static constexpr int kRows = kFewRows * MT;
  static constexpr int kKeys = rows_keys(D);
  static constexpr int kBlocks = D / 64;
  static constexpr int kKvBytes = kKeys * D * 2;      // K or V of a stage
  static constexpr int kStageBytes = 2 * kKvBytes;
  static constexpr int kStages = MT == 1 ? 5 : 10;
  static constexpr int kCtas = rows_ctas(kRows);      // an SM
  // Warps that compute.  The stages are a multiple of a team's, so that a stage's buffer has
  // one reader in each: a warp that came for a buffer's next contents while another one still
  // waited for these would take the one's for the other's (a wait knows odd from even).  Two
  // that both read all of its contents cannot come apart so far.
  static constexpr int kWarps = 5;                    // of a team, which has 16 rows
  static constexpr int kAll = MT * kWarps;
  static_assert(kStages % kWarps == 0, "one reader a buffer and team");
  static constexpr int kThreads = 32 * (kAll + 1);
  static constexpr int kJoinFloats = 512;             // room of a warp for partial rows
  static constexpr int kItems = 8;                    // units that the producer may be ahead
  static constexpr int kOffJoin = kStages * kStageBytes;                  // [2][warps][kJoinFloats]
  static constexpr int kOffMl = kOffJoin + 2 * kWarps * kJoinFloats * 4;  // [2][warps][rows] (m, l)
  static constexpr int kOffItem = kOffMl + 2 * kWarps * kRows * 8;        // [kItems] 64 bytes
  static constexpr int kOffBar = kOffItem + kItems * 64;
  static constexpr int kNumBars = 2 * kStages + 2 * kItems + 2 * 2 + kWarps;
  static constexpr int kOffArrived = kOffBar + 8 * kNumBars;  // [2] warps whose rows are in the room
  static constexpr int kOffAbort = kOffArrived + 8;
  static constexpr int kSmemBytes = kOffAbort + 8;
  static_assert(kStageBytes == 16384 && (kSmemBytes + 1024) * kCtas <= 233472, "shared memory of an SM");
};

// A tiled load of five dimensions global -> shared, completion counted in bytes on `bar`.
__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2,
                                            int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_rows(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A warp's bounded wait.  The time is looked at every 64 tests only (in front of the second
// test it took 38.1 us instead of 37.9: 64 single tokens of 330 keys, 32 + 8 heads, d = 128).
__device__ __forceinline__ bool wait_short(uint64_t* bar, uint32_t parity, int* status) {
  const uint32_t a = smem_addr(bar);
  uint32_t t0 = 0;
#pragma unroll 1
  for (uint32_t n = 1;; ++n) {
    if (__all_sync(0xffffffffu, mbar_test(a, parity))) return true;
    if (n & 63) continue;
    const uint32_t now = (uint32_t)(global_ns() >> 10);  // (about a microsecond)
    if (n == 64) t0 = now;
    if (__any_sync(0xffffffffu, now - t0 > (uint32_t)(kWaitLimitNs >> 10))) {
      atomicExch(status, kDevTimeout);
      return false;
    }
  }
}

// What the producer tells the others of a unit.
struct Item {
  int q0, qn, kv, kind;
  int k0, stages, hk, slot;  // slot: place of its partial rows, -1: not split
  int parts, which, base, end;  // base: stages of this CTA before; end: there is no unit
};

template <int D, int MT>
__global__ void __launch_bounds__(RowsCfg<D, MT>::kThreads, RowsCfg<D, MT>::kCtas)
    rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                const __nv_bfloat16* __restrict__ queries, const long long q_stride_t, const long long q_stride_h,
                const __grid_constant__ PagedParams p) {
  using C = RowsCfg<D, MT>;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw;
  int* status = p.status;
  bool start_ok = smem_base_ok(smem_raw, status);
#ifdef FA_TEST_HOOKS
  if (*reinterpret_cast<volatile int*>(&g_fa_test_rows) == 2) {
    if (threadIdx.x == 0) atomicExch(status, kDevInternal);
    start_ok = false;
  }
#endif
  if (!start_ok) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (threadIdx.x == 0) p.plan->failed = 1;
    return;
  }
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::kOffBar);  // [stages] K and V are there
  uint64_t* empty = full + C::kStages;                            // the warps that took it are done
  uint64_t* item_full = empty + C::kStages;                       // [items]
  uint64_t* item_empty = item_full + C::kItems;
  uint64_t* room_free = item_empty + C::kItems;                   // [2] its rows have been joined
  uint64_t* room_full = room_free + 2;                            // [2] (many rows) every warp's part is there
  uint64_t* last_read = room_full + 2;                            // [warps] (many rows) all teams' are done with their last stage
  int* arrived = reinterpret_cast<int*>(sm + C::kOffArrived);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + C::kOffAbort);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (warp == 0) {
    for (int i = lane; i < C::kNumBars; i += 32) {
      uint64_t* bar = full + i;
      mbar_init(bar, bar >= last_read                      ? MT
                     : bar >= room_full                    ? 32 * C::kAll
                     : bar >= item_empty                   ? C::kAll
                     : bar >= empty && bar < item_full     ? MT
                                                           : 1);
    }
    if (lane == 0) *abort_flag = 0, arrived[0] = arrived[1] = 0;
    fence_mbar_init();
  }
  if (warp == C::kAll && lane == 0) {
    tma_prefetch_map(&tm_k);
    tma_prefetch_map(&tm_v);
  }
  __syncthreads();
  // The lists are there: the launch in front waited for them before it let this one begin, or,
  // where there is none between, is the one that makes them.
  if (p.T * (long long)p.G <= p.few_rows) asm volatile("griddepcontrol.wait;" ::: "memory");

  if (warp == C::kAll) {
    // ---------------------------------------------------------------- producer --
    const SharedPiece* list = reinterpret_cast<const SharedPiece*>(reinterpret_cast<const uint8_t*>(p.plan) +
                                                                   shared_lists(p.S, p.num_groups, p.sms).pieces);
    const unsigned Hk = p.Hk, total = (unsigned)__ldcg(&p.plan->pieces) * Hk;
    const int box_rows = imin(1 << p.page_log2, C::kKeys), boxes = C::kKeys / box_rows;
    const uint32_t box_bytes = box_rows * 128 * C::kBlocks;
    // This lane's copy of a stage: K or V, a box of rows.  (A warp issues its lanes' copies one
    // after the other, so there are as few as can be.)
    const int copies = 2 * boxes, my_box = lane & (boxes - 1), my_v = lane >= boxes;
    const uint32_t my_offset = my_v * C::kKvBytes + my_box * box_bytes;
    uint32_t it = 0, count = 0;  // stages and units of this CTA
    bool ok = true, lost = false;
    // A unit's number is asked for two units ahead, its piece one, its first pages while the
    // stages of the one in front are copied.  (No further: what a CTA has taken no other one
    // does.)
    auto split = [&](unsigned i, int& hk) {  // i = piece * Hk + hk
      unsigned x = __umulhi(i, p.hk_inverse), rest = i - x * Hk;
      while (rest >= Hk) rest -= Hk, ++x;  // (once or twice at most: the inverse is rounded down)
      hk = (int)rest;
      return x;
    };
    auto fetch = [&](unsigned i, int& hk) {
      SharedPiece e = {};
      if (i < total) {
        const SharedPiece* from = list + split(i, hk);
        e.seq = __ldcg(&from->seq), e.part = __ldcg(&from->part);
      }
      return e;
    };
    auto page_at = [&](const SharedPiece& e, int i) {  // this lane's of stage i
      const int key = e.part.x + i * C::kKeys + my_box * box_rows;
      return lane < copies && key < e.part.y
                 ? __ldg(p.page_table + (size_t)e.seq.z * p.max_pages + e.seq.w + (key >> p.page_log2))
                 : 0;
    };
    // (All from the counter: CTAs that wait for paged_kernel's SMs find nothing left.)
    auto take = [&] { return lane == 0 ? atomicAdd(&p.plan->next, 1u) : 0u; };
    unsigned at = __shfl_sync(0xffffffffu, take(), 0), after = take();
    int hk = 0, hk1 = 0;
    SharedPiece e = fetch(at, hk);
    int page = page_at(e, 0), page1 = 0;
    unsigned next = __shfl_sync(0xffffffffu, after, 0);
    for (;; ++count) {
      const int slot = count % C::kItems;
      const bool end = at >= total;
      if (!(ok = wait_short(&item_empty[slot], ((count / C::kItems) & 1) ^ 1, status))) break;
      const int k0 = e.part.x, k1 = e.part.y;
      const int stages = end ? 0 : (k1 - k0 + C::kKeys - 1) / C::kKeys;
      if (lane == 0) {
        int4* to = reinterpret_cast<int4*>(sm + C::kOffItem + slot * 64);
        const unsigned said = e.part.w;
        to[0] = make_int4((int)((unsigned)e.seq.x >> 2), (int)(said & 31) + 1, e.seq.y, e.seq.x & 3);
        to[1] = make_int4(k0, stages, hk, e.part.z);
        to[2] = make_int4((int)(said >> 18), (int)(said >> 5 & 8191), (int)it, end);
        mbar_arrive(&item_full[slot]);
      }
      __syncwarp();
      if (end) break;
      after = take();
      const SharedPiece e1 = fetch(next, hk1);
      for (int i = 0; i < stages; ++i, ++it) {
        const int key = k0 + i * C::kKeys, st = it % C::kStages;
        const int live = imin(boxes, (k1 - key + box_rows - 1) / box_rows);  // boxes with keys
        const bool mine = lane < copies && my_box < live;
        int from = page;
        if (from < 0 || from >= p.num_pages) {
          // outside the pool: the copy reads past the map's last page and fills with zeros
          from = p.num_pages;
          lost = lost || mine;
        }
        if (i + 1 < stages) page = page_at(e, i + 1);
        if (i == 2) page1 = page_at(e1, 0);
        if (!(ok = wait_short(&empty[st], ((it / C::kStages) & 1) ^ 1, status))) break;
        if (lane == 0) mbar_expect_tx(&full[st], live * box_bytes * 2);
        __syncwarp();
        if (mine)
          tma_load_5d(sm + st * C::kStageBytes + my_offset, my_v ? &tm_v : &tm_k, &full[st], 0,
                      (key + my_box * box_rows) & ((1 << p.page_log2) - 1), 0, hk, from);
        __syncwarp();
      }
      if (!ok || __any_sync(0xffffffffu, aborted(abort_flag))) {
        ok = false;
        break;
      }
      at = next;
      next = __shfl_sync(0xffffffffu, after, 0);
      e = e1, hk = hk1;
      page = stages > 2 ? page1 : page_at(e, 0);
    }
    if (!ok) *abort_flag = 1;
    if (lost) record_index(status);
    // Drain: every copy this warp started lands before the block ends.
    for (uint32_t i = it > (uint32_t)C::kStages ? it - C::kStages : 0; i < it; ++i)
      wait_short(&full[i % C::kStages], (i / C::kStages) & 1, status);
  } else {
    // ----------------------------------------------------------------- the others --
    const float c2 = p.c2;
    const uint32_t stage0 = smem_addr(sm);
    // A box holds its rows' first 64 columns, then the others: bytes between 64 columns, and
    // between 16 keys (of d = 128; of d = 64 a stage's rows lie one after the other).
    const uint32_t half = imin(1 << p.page_log2, C::kKeys) * 128;
    const uint32_t keys16 = D == 64 ? 2048 : half == 2048 ? 4096 : 2048;
    const int g = lane / 4, c = lane % 4;  // rows g and g + 8, columns 2 c and 2 c + 1 of a result's tile
    const int team = MT > 1 ? warp / C::kWarps : 0, mine = warp - team * C::kWarps, row0 = kFewRows * team;
    uint32_t rooms = 0, fulls = 0, reads = 0;  // uses of the rooms, of last_read; bit r: parity of room_full[r]
    bool ok = true;
    const size_t all = (size_t)p.T * p.Hk * p.G;
    const size_t rows0 = (size_t)p.sms * (2 * kPagedRows);
    for (uint32_t count = 0; ok; ++count) {
      const int slot = count % C::kItems;
      if (!(ok = wait_short(&item_full[slot], (count / C::kItems) & 1, status))) break;
      const int4* e = reinterpret_cast<const int4*>(sm + C::kOffItem + slot * 64);
      const int4 e0 = e[0], e1 = e[1], e2 = e[2];
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_empty[slot]);
      const Item u = {e0.x, e0.y, e0.z, e0.w, e1.x, e1.y, e1.z, e1.w, e2.x, e2.y, e2.z, e2.w};
      if (u.end) break;
      const int valid = u.qn * p.G;  // rows
      // This warp's stages: place, place + kWarps, .. of the unit; `takers` warps have some.
      const int place = (mine + C::kWarps - u.base % C::kWarps) % C::kWarps;
      const int takers = imax(1, imin(u.stages, C::kWarps));
      // Rows that fit into a room are joined by the last warp to bring its part; more of them by
      // all, out of the buffers of their last stages, which the producer gets back then.
      const bool fits = valid * D <= C::kJoinFloats, hold = !fits && takers > 1;
      if (place >= takers && (fits || takers == 1)) {  // nothing to do but to keep count
        if (takers > 1) {
          const uint32_t use = rooms++;
          if (!(ok = wait_short(&room_free[use & 1], ((use >> 1) & 1) ^ 1, status))) break;
          if (lane == 0) mbar_arrive(&room_free[use & 1]);
        }
        continue;
      }
      const bool causal = p.causal && u.kind != kPrefix;
      const int past = u.kv - u.qn;
      const int lim0 = causal ? imin(past, u.kv - 1) : u.kv - 1;  // last key that all rows see
      const bool idle = row0 >= valid;  // this team has no rows: it keeps count
      int lim[2];
      float m[2], l[2], o[D / 8][4];
      // The queries, in the layout of an MMA's first operand; rows that are no token's are zero.
      uint32_t qa[D / 16][4];
      const __nv_bfloat16* q_head = queries + (size_t)u.hk * p.G * q_stride_h;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = row0 + g + 8 * i, tok = (row * p.g_inverse) >> 16;
        const uint32_t* src = reinterpret_cast<const uint32_t*>(q_head + (size_t)(u.q0 + tok) * q_stride_t +
                                                                (size_t)(row - tok * p.G) * q_stride_h) + c;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const bool there = row < valid && place < takers;
          qa[k][i] = there ? __ldg(src + 8 * k) : 0u;
          qa[k][2 + i] = there ? __ldg(src + 8 * k + 4) : 0u;
        }
        lim[i] = causal ? imin(past + tok, u.kv - 1) : u.kv - 1;
        m[i] = -INFINITY;
        l[i] = 0.f;
      }
#pragma unroll
      for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
      for (int i = place; i < u.stages; i += C::kWarps) {
        const uint32_t it = (uint32_t)u.base + i;
        const int st = it % C::kStages;
        if (!(ok = wait_short(&full[st], (it / C::kStages) & 1, status))) break;
        if (MT > 1 && idle) {
          __syncwarp();
          if (lane == 0 && !(hold && i + C::kWarps >= u.stages)) mbar_arrive(&empty[st]);
          continue;
        }
        const uint32_t k_s = stage0 + st * C::kStageBytes, v_s = k_s + C::kKvBytes;
        const int key0 = u.k0 + i * C::kKeys, used = u.kv - key0;  // keys of the stage that the entry has
        if (used < C::kKeys) {
          // what lies behind the end in a page is not the entry's, and 0 * NaN is NaN
          for (int x = used * 8 + lane; x < C::kKeys * 8; x += 32)
#pragma unroll
            for (int kb = 0; kb < C::kBlocks; ++kb)
              *reinterpret_cast<uint4*>(sm + st * C::kStageBytes + C::kKvBytes + kb * half + (x / 128) * keys16 +
                                        x % 128 * 16) = make_uint4(0, 0, 0, 0);
          __syncwarp();
        }
        // S = Q K^T: 8 keys a tile
        float s[C::kKeys / 8][4];
#pragma unroll
        for (int n = 0; n < C::kKeys / 8; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
        for (int k2 = 0; k2 < D / 32; ++k2)  // 32 columns
#pragma unroll
          for (int n = 0; n < C::kKeys / 8; ++n) {
            uint32_t kf[4];
            const int row = lane & 7, chunk = 4 * (k2 & 1) + (lane >> 3);
            ldsm4(k_s + (k2 >> 1) * half + (n >> 1) * keys16 + ((n & 1) * 8 + row) * 128 + ((chunk ^ row) << 4), kf);
            mma_rows(s[n], qa[2 * k2], kf[0], kf[1]);
            mma_rows(s[n], qa[2 * k2 + 1], kf[2], kf[3]);
          }
        // in log2 units; -inf where masked
        float mx[2];
        bool need = false;
        const bool masked = key0 + C::kKeys - 1 > lim0;
#pragma unroll
        for (int i2 = 0; i2 < 2; ++i2) {
          float t = -INFINITY;
          const int last = lim[i2] - key0 - 2 * c;
#pragma unroll
          for (int n = 0; n < C::kKeys / 8; ++n) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float& y = s[n][2 * i2 + x];
              y *= c2;
              if (masked) y = 8 * n + x > last ? -INFINITY : y;
              t = fmaxf(t, y);
            }
          }
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
          mx[i2] = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
          need = need || mx[i2] > m[i2] + kRescaleThreshold;
        }
        // A row's maximum moves by what the row itself holds, whatever makes the warp come here.
        if (__any_sync(0xffffffffu, need)) {
#pragma unroll
          for (int i2 = 0; i2 < 2; ++i2) {
            const bool moves = mx[i2] > m[i2] + kRescaleThreshold;
            const float alpha = !moves ? 1.f : m[i2] == -INFINITY ? 0.f : ex2(m[i2] - mx[i2]);
            m[i2] = moves ? mx[i2] : m[i2];
            l[i2] *= alpha;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) o[n][2 * i2] *= alpha, o[n][2 * i2 + 1] *= alpha;
          }
        }
        // P = 2^(s - m) (0 where masked), summed before its rounding; O += P V: 16 keys at a time
        uint32_t pa[C::kKeys / 16][4];
#pragma unroll
        for (int i2 = 0; i2 < 2; ++i2) {
          const float ref = m[i2] == -INFINITY ? 0.f : m[i2];
          float sum = 0.f;
#pragma unroll
          for (int n = 0; n < C::kKeys / 8; ++n) {
            const float p0 = ex2(s[n][2 * i2] - ref), p1 = ex2(s[n][2 * i2 + 1] - ref);
            sum += p0 + p1;
            pa[n / 2][2 * (n & 1) + i2] = pack_bf16x2(p0, p1);
          }
          l[i2] += sum;
        }
#pragma unroll
        for (int k = 0; k < C::kKeys / 16; ++k)
#pragma unroll
          for (int n2 = 0; n2 < D / 16; ++n2) {
            uint32_t vf[4];
            const int row = lane & 15, chunk = 2 * (n2 & 3) + (lane >> 4);
            ldsm4t(v_s + (n2 >> 2) * half + k * keys16 + row * 128 + ((chunk ^ (row & 7)) << 4), vf);
            mma_rows(o[2 * n2], pa[k], vf[0], vf[1]);
            mma_rows(o[2 * n2 + 1], pa[k], vf[2], vf[3]);
          }
        if (used < C::kKeys) fence_proxy_async_smem();  // the next copy comes behind the zeros
        __syncwarp();
        if (lane == 0 && !(hold && i + C::kWarps >= u.stages)) mbar_arrive(&empty[st]);
      }
      if (!ok) break;
#pragma unroll
      for (int i2 = 0; i2 < 2; ++i2) {
        l[i2] += __shfl_xor_sync(0xffffffffu, l[i2], 1);
        l[i2] += __shfl_xor_sync(0xffffffffu, l[i2], 2);
      }
      // Where a row of the unit goes: the output if it has no other parts, else the workspace.
      float2* out_ml = reinterpret_cast<float2*>(p.part_ml);
      const bool direct = u.slot < 0 && u.kind == kAlone;
      auto out_row = [&](int row) {
        const int tok = (row * p.g_inverse) >> 16;
        return (size_t)(u.q0 + tok) * (p.Hk * p.G) + u.hk * p.G + (row - tok * p.G);
      };
      auto part_row = [&](int row, size_t at) {
        return u.slot < 0 ? rows0 + (u.kind == kPrefix ? 0 : all) + at
                          : rows0 + 2 * all + (size_t)(u.slot + u.hk) * p.few_rows + row;
      };
      auto put_ml = [&](int row, size_t at, float top, float sum) {
        const size_t apart = rows0 + (u.kind == kPrefix ? 0 : all) + at;
        if (direct) {
          if (p.lse) p.lse[at] = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * kLn2;
          out_ml[apart] = make_float2(0.f, kRowDone);
        } else {
          out_ml[part_row(row, at)] = make_float2(top, sum);
          if (u.slot >= 0 && u.which == 0)
            out_ml[apart] = make_float2(__int_as_float((((u.slot + u.hk) << 13 | u.parts) << 5) | row),
                                        u.kind == kRest ? kRowPartsOfRest : kRowParts);
        }
      };
      if (takers == 1) {  // nothing to join
#pragma unroll
        for (int i2 = 0; i2 < 2; ++i2) {
          const int row = row0 + g + 8 * i2;
          if (row >= valid) continue;
          const size_t at = out_row(row);
          if (c == 0) put_ml(row, at, m[i2], l[i2]);
          if (direct) {
            const float inv = l[i2] == 0.f ? 0.f : 1.f / l[i2];  // (saw no key: zero)
            uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) + at * D) + c;
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
              out[4 * n] = pack_bf16x2(o[n][2 * i2] * inv, o[n][2 * i2 + 1] * inv);
          } else {
            float2* out = reinterpret_cast<float2*>(p.part_o + part_row(row, at) * D) + c;
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
              out[4 * n] = make_float2(o[n][2 * i2], o[n][2 * i2 + 1]);
          }
        }
        __syncwarp();
        continue;
      }
      // The buffers of the last stages are written to next: all teams have read them.
      if (MT > 1 && hold && place < takers) {
        if (lane == 0) mbar_arrive(&last_read[mine]);
        if (!(ok = wait_short(&last_read[mine], reads++ & 1, status))) break;
      }
      // This warp's (m, l) and rows.  (Every warp takes part in every use of a room, if only by
      // its arrival, so that none is a use ahead or behind.)
      const uint32_t use = rooms++, r = use & 1;
      if (!(ok = wait_short(&room_free[r], ((use >> 1) & 1) ^ 1, status))) break;
      float2* ml = reinterpret_cast<float2*>(sm + C::kOffMl) + r * (C::kWarps * C::kRows);
      auto rows_of = [&](int w) {  // of the w-th taker
        return hold ? reinterpret_cast<float*>(
                          sm + ((u.base + w + (u.stages - 1 - w) / C::kWarps * C::kWarps) % C::kStages) * C::kStageBytes)
                    : reinterpret_cast<float*>(sm + C::kOffJoin) + (r * C::kWarps + w) * C::kJoinFloats;
      };
      if (place < takers) {
        float* to = rows_of(place);
#pragma unroll
        for (int i2 = 0; i2 < 2; ++i2) {
          const int row = row0 + g + 8 * i2;
          if (row >= valid) continue;
          if (c == 0) ml[place * C::kRows + row] = make_float2(m[i2], l[i2]);
#pragma unroll
          for (int n = 0; n < D / 8; ++n)
            *reinterpret_cast<float2*>(to + row * D + ((8 * n + 2 * c) ^ (8 * (row & 3)))) =
                make_float2(o[n][2 * i2], o[n][2 * i2 + 1]);
        }
      }
      // Four columns of a row, joined in the order of the unit's stages.
      auto join = [&](int x) {
        const int row = x / (D / 4), col = x % (D / 4) * 4;
        float2 part[C::kWarps];
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < C::kWarps; ++w) {
          part[w] = w < takers ? ml[w * C::kRows + row] : make_float2(-INFINITY, 0.f);
          top = fmaxf(top, part[w].x);
        }
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < C::kWarps; ++w) {
          if (part[w].y == 0.f) continue;  // saw no key (a row of NaN has a maximum of -inf, too)
          const float wt = ex2(part[w].x - top);
          const float4 v = *reinterpret_cast<const float4*>(rows_of(w) + row * D + (col ^ (8 * (row & 3))));
          sum = fmaf(wt, part[w].y, sum);
          y.x = fmaf(wt, v.x, y.x), y.y = fmaf(wt, v.y, y.y), y.z = fmaf(wt, v.z, y.z), y.w = fmaf(wt, v.w, y.w);
        }
        const size_t at = out_row(row);
        if (direct) {
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + at * D + col) =
              make_uint2(pack_bf16x2(y.x * inv, y.y * inv), pack_bf16x2(y.z * inv, y.w * inv));
        } else {
          *reinterpret_cast<float4*>(p.part_o + part_row(row, at) * D + col) = y;
        }
        if (col == 0) put_ml(row, at, top, sum);
      };
      // Counts the warps that came here in this use.
      auto came = [&] {
        __threadfence_block();
        __syncwarp();
        int before = lane == 0 ? atomicAdd(&arrived[r], 1) : 0;
        before = __shfl_sync(0xffffffffu, before, 0);
        __threadfence_block();
        return before + 1;
      };
#ifdef FA_TEST_HOOKS
      if (warp == 0 && *reinterpret_cast<volatile int*>(&g_fa_test_rows) == 1) continue;
#endif
      if (hold) {
        mbar_arrive(&room_full[r]);
        if (!(ok = wait_short(&room_full[r], fulls >> r & 1, status))) break;
        fulls ^= 1u << r;
        for (int x = threadIdx.x; x < valid * (D / 4); x += 32 * C::kAll) join(x);
        fence_proxy_async_smem();  // the next copies come behind these accesses
        if (came() == C::kAll) {
          if (lane < takers)
            for (int j = 0; j < MT; ++j)
              mbar_arrive(&empty[(u.base + lane + (u.stages - 1 - lane) / C::kWarps * C::kWarps) % C::kStages]);
          if (lane == 0) arrived[r] = 0;
        }
      } else if (!idle && came() == takers) {
        for (int x = lane; x < valid * (D / 4); x += 32) join(x);
        if (lane == 0) arrived[r] = 0;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&room_free[r]);
      if (__any_sync(0xffffffffu, aborted(abort_flag))) ok = false;
    }
    if (!ok) *abort_flag = 1;
  }
  __syncthreads();
  if (threadIdx.x == 0 && aborted(abort_flag)) p.plan->failed = 1;
  // The launch behind waits for this one alone: so this one is done after paged_kernel.
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int D, int MT>
cudaError_t launch_rows_t(const PagedLaunch& a, cudaStream_t stream) {
  using C = RowsCfg<D, MT>;
  auto kern = rows_kernel<D, MT>;
  static std::atomic<unsigned long long> allowed{0};
  const cudaError_t e = allow_shared(reinterpret_cast<const void*>(kern), C::kSmemBytes, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C::kCtas * a.grid);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a.tm_kr, a.tm_vr, static_cast<const __nv_bfloat16*>(a.q), a.q_stride_t,
                            a.q_stride_h, a.p);
}

}  // namespace

cudaError_t launch_shared_rows(const PagedLaunch& a, cudaStream_t stream) {
  const bool once = a.p.few_rows <= kFewRows;
  if (a.d == 64) return once ? launch_rows_t<64, 1>(a, stream) : launch_rows_t<64, 2>(a, stream);
  return once ? launch_rows_t<128, 1>(a, stream) : launch_rows_t<128, 2>(a, stream);
}

}  // namespace fa

#ifdef FA_TEST_HOOKS
// Test builds only: sets what g_fa_test_rows says (0: nothing).
extern "C" int fa_test_rows(int mode) {
  return cudaMemcpyToSymbol(fa::g_fa_test_rows, &mode, sizeof(int)) == cudaSuccess ? 0 : 4;
}
#endif
