// Attention of a few rows over a paged cache: the entries of a batch whose sequences
// share keys (fa_paged_shared.cu) that have at most 16 (or 32) query rows a key head:
// single tokens, mostly, behind their group's shared keys.
//
// Bound: the read of K and V (4 d bytes a key for 4 d G FLOP).  The units are short, a
// few hundred keys, so what matters is that loads never wait for the end of one.  The
// 128-row tiles of paged_kernel take 2 us from a unit's last key tile to the next one's
// first scores (tensor memory, barriers between the roles, eight partial rows merged by
// the whole CTA); here a unit's end costs the loads nothing:
//
//   a producer warp goes from unit to unit on its own, two units ahead of the loads;
//     ten stages of 16 KB (32 keys of d = 128, 64 of d = 64) an SM, in two CTAs
//   five warps take the stages in turn, each alone: S = Q K^T by 16 x 8 x 16 MMAs whose
//     results stay in registers (mma.sync: 16 rows are an eighth of tcgen05's smallest
//     tile, and the way through tensor memory and back is most of a short unit's time;
//     the MMAs here are busy a fifth of the time that the loads take), a running maximum
//     and sum of its own, P from the registers of S, O += P V
//   at the unit's end their partial rows are joined through shared memory, while the
//     next units' stages arrive
//
// Units are (piece, key head) pairs in the order of a list; CTAs take them from a
// counter.  Which CTA computes a unit has no part in its result: its stages go to the
// warps in the order of the unit, and are joined in that order, too.
//
// Rounding as in paged_kernel: scores, maxima, sums and O in fp32, P to bf16 once for the
// second product.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_common.cuh"
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
  static constexpr int kHalf = kKeys * 128;           // bytes of a block of 64 columns of K or V
  static constexpr int kBlocks = D / 64;
  static constexpr int kKvBytes = kBlocks * kHalf;    // K or V of a stage
  static constexpr int kStageBytes = 2 * kKvBytes;
  static constexpr int kStages = MT == 1 ? 5 : 10;
  static constexpr int kCtas = MT == 1 ? 2 : 1;       // an SM
  // Warps that compute.  The stages are a multiple of them, so that a stage's buffer has
  // one reader: a warp that came for a buffer's next contents while another one still waited
  // for these would take the one's for the other's (a wait knows odd from even).
  static constexpr int kWarps = 5;
  static_assert(kStages % kWarps == 0, "one reader a buffer");
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int kQHalf = kRows * 128;
  static constexpr int kQBytes = kBlocks * kQHalf;
  static constexpr int kJoinFloats = 512;             // of a warp's partial rows at a time
  static constexpr int kItems = 4;                    // units that the producer may be ahead
  static constexpr int kOffQ = kStages * kStageBytes;  // [2]
  static constexpr int kOffJoin = kOffQ + 2 * kQBytes; // [2][warps][kJoinFloats]
  static constexpr int kOffMl = kOffJoin + 2 * kWarps * kJoinFloats * 4;  // [2][warps][rows] (m, l)
  static constexpr int kOffItem = kOffMl + 2 * kWarps * kRows * 8;        // [kItems] 64 bytes
  static constexpr int kOffBar = kOffItem + kItems * 64;
  static constexpr int kNumBars = 2 * kStages + 2 * 2 + 2 * kItems + 2;
  static constexpr int kOffAbort = kOffBar + 8 * kNumBars;
  static constexpr int kSmemBytes = kOffAbort + 8;
  static_assert(kStageBytes == 16384 && (kSmemBytes + 1024) * kCtas <= 233472, "shared memory of an SM");
};

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

// A warp's bounded wait (paged_kernel's for small units).
__device__ __forceinline__ bool wait_short(uint64_t* bar, uint32_t parity, int* status) {
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

// What the producer tells the others of a unit.
struct Item {
  int q0, qn, kv, kind;
  int k0, stages, hk, slot;  // slot: place of its partial rows, -1: not split
  int parts, which, base, end;  // base: stages of this CTA before; end: there is no unit
};

template <int D, int MT>
__global__ void __launch_bounds__(RowsCfg<D, MT>::kThreads, RowsCfg<D, MT>::kCtas)
    rows_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedParams p) {
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
    if (threadIdx.x == 0) p.plan->failed = 1;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::kOffBar);  // [stages] K and V are there
  uint64_t* empty = full + C::kStages;                            // the warp that took it is done
  uint64_t* q_full = empty + C::kStages;                          // [2]
  uint64_t* q_empty = q_full + 2;                                 // every warp is done with it
  uint64_t* item_full = q_empty + 2;                              // [items]
  uint64_t* item_empty = item_full + C::kItems;
  uint64_t* joined = item_empty + C::kItems;                      // [2] every warp's partial rows are there
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + C::kOffAbort);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (warp == 0) {
    for (int i = lane; i < C::kNumBars; i += 32) {
      uint64_t* bar = full + i;
      const bool all = (bar >= q_empty && bar < q_empty + 2) || (bar >= item_empty && bar < item_empty + C::kItems);
      mbar_init(bar, bar >= joined ? 32 * C::kWarps : all ? C::kWarps : 1);
    }
    if (lane == 0) *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == C::kWarps && lane == 0) {
    tma_prefetch_map(&tm_q);
    tma_prefetch_map(&tm_k);
    tma_prefetch_map(&tm_v);
  }
  __syncthreads();
  const int few = p.few_rows / p.G;  // tokens of a unit at most

  if (warp == C::kWarps) {
    // ---------------------------------------------------------------- producer --
    const SharedPiece* list = reinterpret_cast<const SharedPiece*>(reinterpret_cast<const uint8_t*>(p.plan) +
                                                                   shared_lists(p.S, p.num_groups, p.sms).pieces);
    const unsigned Hk = p.Hk, total = (unsigned)__ldcg(&p.plan->pieces) * Hk;
    const int box_rows = imin(1 << p.page_log2, C::kKeys), boxes = C::kKeys / box_rows;
    const uint32_t box_bytes = box_rows * 128;
    // This lane's copy of a stage: K or V, a block of 64 columns, a box of rows.
    const int copies = 2 * C::kBlocks * boxes;
    const int my_box = lane % boxes, my_block = lane / boxes % C::kBlocks, my_v = lane / (boxes * C::kBlocks);
    uint32_t it = 0, count = 0;  // stages and units of this CTA
    bool ok = true, lost = false;
    // The unit, the next one's piece and the one behind's number are asked for ahead.
    unsigned at = blockIdx.x, next = at + gridDim.x;
    int4 s = {}, h = {}, t = {};
    auto fetch = [&](unsigned i) {
      if (i < total) {
        const SharedPiece* e = list + i / Hk;
        s = __ldcg(&e->seq), h = __ldcg(&e->how), t = __ldcg(&e->part);
      }
    };
    fetch(at);
    for (;; ++count) {
      const int slot = count % C::kItems, b = count & 1;
      const bool end = at >= total;
      if (!(ok = wait_short(&item_empty[slot], ((count / C::kItems) & 1) ^ 1, status))) break;
      const int hk = (int)(at % Hk), k0 = h.z, k1 = h.w, row = s.w, page0 = h.x, q0 = s.x;
      const int stages = end ? 0 : (k1 - k0 + C::kKeys - 1) / C::kKeys;
      if (lane == 0) {
        int4* e = reinterpret_cast<int4*>(sm + C::kOffItem + slot * 64);
        e[0] = make_int4(s.x, s.y, s.z, h.y);
        e[1] = make_int4(k0, stages, hk, t.x);
        e[2] = make_int4(t.y, t.z, (int)it, end);
        mbar_arrive(&item_full[slot]);
      }
      __syncwarp();
      if (end) break;
      unsigned after = 0;
      if (lane == 0) after = atomicAdd(&p.plan->next, 1u);
      fetch(next);
      if (!(ok = wait_short(&q_empty[b], ((count >> 1) & 1) ^ 1, status))) break;
      if (lane == 0) {
        mbar_expect_tx(&q_full[b], few * p.G * 128 * C::kBlocks);
        for (int kb = 0; kb < C::kBlocks; ++kb)
          tma_load_4d(sm + C::kOffQ + b * C::kQBytes + kb * C::kQHalf, &tm_q, &q_full[b], 64 * kb, 0, hk, q0);
      }
      __syncwarp();
      const int* table = p.page_table + (size_t)row * p.max_pages + page0;
      auto page_at = [&](int i) {
        const int key = k0 + i * C::kKeys + my_box * box_rows;
        return lane < copies && key < k1 ? __ldg(table + (key >> p.page_log2)) : 0;
      };
      int page = page_at(0);
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
        if (i + 1 < stages) page = page_at(i + 1);
        if (!(ok = wait_short(&empty[st], ((it / C::kStages) & 1) ^ 1, status))) break;
        if (lane == 0) mbar_expect_tx(&full[st], live * box_bytes * C::kBlocks * 2);
        __syncwarp();
        if (mine)
          tma_load_4d(sm + st * C::kStageBytes + my_v * C::kKvBytes + my_block * C::kHalf + my_box * box_bytes,
                      my_v ? &tm_v : &tm_k, &full[st], 64 * my_block, (key + my_box * box_rows) & ((1 << p.page_log2) - 1),
                      hk, from);
        __syncwarp();
      }
      if (!ok || __any_sync(0xffffffffu, aborted(abort_flag))) {
        ok = false;
        ++count;  // (its queries are on their way)
        break;
      }
      at = next;
      next = __shfl_sync(0xffffffffu, after, 0);
    }
    if (!ok) *abort_flag = 1;
    if (lost) record_index(status);
    // Drain: every copy this warp started lands before the block ends.
    for (uint32_t i = count > 2 ? count - 2 : 0; i < count; ++i) wait_short(&q_full[i & 1], (i >> 1) & 1, status);
    for (uint32_t i = it > (uint32_t)C::kStages ? it - C::kStages : 0; i < it; ++i)
      wait_short(&full[i % C::kStages], (i / C::kStages) & 1, status);
  } else {
    // ----------------------------------------------------------------- the others --
    const float c2 = p.c2;
    const uint32_t stage0 = smem_addr(sm);
    const int g = lane / 4, c = lane % 4;  // rows g and g + 8, columns 2 c and 2 c + 1 of a result's tile
    uint32_t joins = 0;
    bool ok = true;
    const size_t all = (size_t)p.T * p.Hk * p.G;
    const size_t rows0 = (size_t)p.sms * (2 * kPagedRows);
    for (uint32_t count = 0; ok; ++count) {
      const int slot = count % C::kItems, b = count & 1;
      if (!(ok = wait_short(&item_full[slot], (count / C::kItems) & 1, status))) break;
      const int4* e = reinterpret_cast<const int4*>(sm + C::kOffItem + slot * 64);
      const int4 e0 = e[0], e1 = e[1], e2 = e[2];
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_empty[slot]);
      const Item u = {e0.x, e0.y, e0.z, e0.w, e1.x, e1.y, e1.z, e1.w, e2.x, e2.y, e2.z, e2.w};
      if (u.end) break;
      const int valid = u.qn * p.G;  // rows
      const bool causal = p.causal && u.kind != kPrefix;
      const int past = u.kv - u.qn;
      const int lim0 = causal ? imin(past, u.kv - 1) : u.kv - 1;  // last key that all rows see
      int lim[2 * MT];
      float m[2 * MT], l[2 * MT], o[MT][D / 8][4];
#pragma unroll
      for (int i = 0; i < 2 * MT; ++i) {
        const int row = g + 8 * i, tok = (row * p.g_inverse) >> 16;
        lim[i] = row >= valid ? -1 : causal ? imin(past + tok, u.kv - 1) : u.kv - 1;
        m[i] = -INFINITY;
        l[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int n = 0; n < D / 8; ++n) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
      // This warp's stages: place, place + kWarps, .. of the unit.
      const int place = (warp + C::kWarps - u.base % C::kWarps) % C::kWarps;
      const uint32_t q_s = smem_addr(sm + C::kOffQ + b * C::kQBytes);
      auto q_frag = [&](int i, int k, uint32_t (&a)[4]) {  // rows 16 i .. + 15, columns 16 k .. + 15
        const int row = 16 * i + (lane & 15), chunk = 2 * (k & 3) + (lane >> 4);
        ldsm4(q_s + (k >> 2) * C::kQHalf + row * 128 + ((chunk ^ (row & 7)) << 4), a);
      };
      constexpr bool kKeepQ = MT == 1;
      uint32_t qa[kKeepQ ? D / 16 : 1][4];
      // (one waits in any case: were all free to go on, they could hand back the buffer
      // before the producer has taken it, and it would wait for the next time)
      if (place == 0 || place < u.stages) {
        if (!(ok = wait_short(&q_full[b], (count >> 1) & 1, status))) break;
        if constexpr (kKeepQ) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) q_frag(0, k, qa[k]);
        }
      }
      if constexpr (kKeepQ) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_empty[b]);
      }
      for (int i = place; i < u.stages; i += C::kWarps) {
        const uint32_t it = (uint32_t)u.base + i;
        const int st = it % C::kStages;
        if (!(ok = wait_short(&full[st], (it / C::kStages) & 1, status))) break;
        const uint32_t k_s = stage0 + st * C::kStageBytes, v_s = k_s + C::kKvBytes;
        const int key0 = u.k0 + i * C::kKeys, used = u.kv - key0;  // keys of the stage that the entry has
        if (used < C::kKeys) {
          // what lies behind the end in a page is not the entry's, and 0 * NaN is NaN
          for (int x = used * 8 + lane; x < C::kKeys * 8; x += 32)
#pragma unroll
            for (int kb = 0; kb < C::kBlocks; ++kb)
              reinterpret_cast<uint4*>(sm + st * C::kStageBytes + C::kKvBytes + kb * C::kHalf)[x] =
                  make_uint4(0, 0, 0, 0);
          __syncwarp();
        }
        // S = Q K^T: 8 keys a tile
        float s[MT][C::kKeys / 8][4];
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int n = 0; n < C::kKeys / 8; ++n) s[j][n][0] = s[j][n][1] = s[j][n][2] = s[j][n][3] = 0.f;
#pragma unroll
        for (int k2 = 0; k2 < D / 32; ++k2) {  // 32 columns
          uint32_t a0[MT][4], a1[MT][4];
#pragma unroll
          for (int j = 0; j < MT; ++j) {
            if constexpr (kKeepQ) {
#pragma unroll
              for (int x = 0; x < 4; ++x) a0[j][x] = qa[2 * k2][x], a1[j][x] = qa[2 * k2 + 1][x];
            } else {
              q_frag(j, 2 * k2, a0[j]);
              q_frag(j, 2 * k2 + 1, a1[j]);
            }
          }
#pragma unroll
          for (int n = 0; n < C::kKeys / 8; ++n) {
            uint32_t kf[4];
            const int row = 8 * n + (lane & 7), chunk = 4 * (k2 & 1) + (lane >> 3);
            ldsm4(k_s + (k2 >> 1) * C::kHalf + row * 128 + ((chunk ^ (row & 7)) << 4), kf);
#pragma unroll
            for (int j = 0; j < MT; ++j) {
              mma_rows(s[j][n], a0[j], kf[0], kf[1]);
              mma_rows(s[j][n], a1[j], kf[2], kf[3]);
            }
          }
        }
        // in log2 units; -inf where masked
        float mx[2 * MT];
        bool need = false;
        const bool masked = key0 + C::kKeys - 1 > lim0;
#pragma unroll
        for (int i2 = 0; i2 < 2 * MT; ++i2) {
          float t = -INFINITY;
          const int last = lim[i2] - key0 - 2 * c;
#pragma unroll
          for (int n = 0; n < C::kKeys / 8; ++n) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float& y = s[i2 / 2][n][2 * (i2 & 1) + x];
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
          for (int i2 = 0; i2 < 2 * MT; ++i2) {
            if (!(mx[i2] > m[i2] + kRescaleThreshold)) continue;
            const float alpha = m[i2] == -INFINITY ? 0.f : ex2(m[i2] - mx[i2]);
            m[i2] = mx[i2];
            l[i2] *= alpha;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) o[i2 / 2][n][2 * (i2 & 1)] *= alpha, o[i2 / 2][n][2 * (i2 & 1) + 1] *= alpha;
          }
        }
        // P = 2^(s - m) (0 where masked), summed before its rounding; O += P V: 16 keys at a time
        uint32_t pa[MT][C::kKeys / 16][4];
#pragma unroll
        for (int i2 = 0; i2 < 2 * MT; ++i2) {
          const float ref = m[i2] == -INFINITY ? 0.f : m[i2];
          float sum = 0.f;
#pragma unroll
          for (int n = 0; n < C::kKeys / 8; ++n) {
            const float p0 = ex2(s[i2 / 2][n][2 * (i2 & 1)] - ref), p1 = ex2(s[i2 / 2][n][2 * (i2 & 1) + 1] - ref);
            sum += p0 + p1;
            pa[i2 / 2][n / 2][2 * (n & 1) + (i2 & 1)] = pack_bf16x2(p0, p1);
          }
          l[i2] += sum;
        }
#pragma unroll
        for (int k = 0; k < C::kKeys / 16; ++k)
#pragma unroll
          for (int n2 = 0; n2 < D / 16; ++n2) {
            uint32_t vf[4];
            const int row = 16 * k + (lane & 15), chunk = 2 * (n2 & 3) + (lane >> 4);
            ldsm4t(v_s + (n2 >> 2) * C::kHalf + row * 128 + ((chunk ^ (row & 7)) << 4), vf);
#pragma unroll
            for (int j = 0; j < MT; ++j) {
              mma_rows(o[j][2 * n2], pa[j][k], vf[0], vf[1]);
              mma_rows(o[j][2 * n2 + 1], pa[j][k], vf[2], vf[3]);
            }
          }
        if (used < C::kKeys) fence_proxy_async_smem();  // the next copy comes behind the zeros
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
      }
      if (!ok) break;
      if constexpr (!kKeepQ) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_empty[b]);
      }
      // The warps' rows: (m, l), then as many columns of O at a time as there is room for.
      float2* ml = reinterpret_cast<float2*>(sm + C::kOffMl) + b * C::kWarps * C::kRows;
#pragma unroll
      for (int i2 = 0; i2 < 2 * MT; ++i2) {
        l[i2] += __shfl_xor_sync(0xffffffffu, l[i2], 1);
        l[i2] += __shfl_xor_sync(0xffffffffu, l[i2], 2);
        if (c == 0) ml[place * C::kRows + g + 8 * i2] = make_float2(m[i2], l[i2]);
      }
      const int rows_log2 = valid <= 4 ? 2 : valid <= 8 ? 3 : valid <= 16 ? 4 : 5;
      const int cols = imin(D, C::kJoinFloats >> rows_log2);
      const int mine_row = threadIdx.x / (cols / 4), mine_col = threadIdx.x % (cols / 4);  // 4 columns
      for (int c0 = 0; c0 < D; c0 += cols) {
        float* room = reinterpret_cast<float*>(sm + C::kOffJoin) + (joins & 1) * (C::kWarps * C::kJoinFloats);
        if (place < u.stages) {
#pragma unroll
          for (int i2 = 0; i2 < 2 * MT; ++i2) {
            const int row = g + 8 * i2;
            if (row >= valid) continue;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
              const int col = 8 * n + 2 * c - c0;
              if (col < 0 || col >= cols) continue;
              *reinterpret_cast<float2*>(room + place * C::kJoinFloats + row * cols + (col ^ (8 * (row & 1) & (cols - 1)))) =
                  make_float2(o[i2 / 2][n][2 * (i2 & 1)], o[i2 / 2][n][2 * (i2 & 1) + 1]);
            }
          }
        }
#ifdef FA_TEST_HOOKS
        if (warp != 0 || *reinterpret_cast<volatile int*>(&g_fa_test_rows) != 1)
#endif
          mbar_arrive(&joined[joins & 1]);
        if (!(ok = wait_short(&joined[joins & 1], (joins >> 1) & 1, status))) break;
        ++joins;
        if (mine_row >= valid) continue;
        float2 part[C::kWarps];
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < C::kWarps; ++w) {
          part[w] = ml[w * C::kRows + mine_row];
          top = fmaxf(top, part[w].x);
        }
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < C::kWarps; ++w) {
          if (part[w].y == 0.f) continue;  // saw no key (a row of NaN has a maximum of -inf, too)
          const float wt = ex2(part[w].x - top);
          const float4 x = *reinterpret_cast<const float4*>(room + w * C::kJoinFloats + mine_row * cols +
                                                            ((4 * mine_col) ^ (8 * (mine_row & 1) & (cols - 1))));
          sum = fmaf(wt, part[w].y, sum);
          y.x = fmaf(wt, x.x, y.x), y.y = fmaf(wt, x.y, y.y), y.z = fmaf(wt, x.z, y.z), y.w = fmaf(wt, x.w, y.w);
        }
        const int tok = (mine_row * p.g_inverse) >> 16, col = c0 + 4 * mine_col;
        const size_t at = (size_t)(u.q0 + tok) * (p.Hk * p.G) + u.hk * p.G + (mine_row - tok * p.G);
        float2* out_ml = reinterpret_cast<float2*>(p.part_ml);
        const size_t apart = rows0 + (u.kind == kPrefix ? 0 : all) + at;
        if (u.slot < 0 && u.kind == kAlone) {
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + at * D + col) =
              make_uint2(pack_bf16x2(y.x * inv, y.y * inv), pack_bf16x2(y.z * inv, y.w * inv));
          if (col == 0) {
            if (p.lse) p.lse[at] = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * kLn2;
            out_ml[apart] = make_float2(0.f, kRowDone);
          }
        } else {
          const size_t part_row = u.slot < 0 ? apart : rows0 + 2 * all + (size_t)(u.slot + u.hk) * kPartRows + mine_row;
          *reinterpret_cast<float4*>(p.part_o + part_row * D + col) = y;
          if (col == 0) {
            out_ml[part_row] = make_float2(top, sum);
            if (u.slot >= 0 && u.which == 0)
              out_ml[apart] = make_float2(__int_as_float((((u.slot + u.hk) << 13 | u.parts) << 5) | mine_row),
                                          u.kind == kRest ? kRowPartsOfRest : kRowParts);
          }
        }
      }
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
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(rows_ctas(a.p.few_rows, a.grid));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a.tm_qr, a.tm_kr, a.tm_vr, a.p);
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
