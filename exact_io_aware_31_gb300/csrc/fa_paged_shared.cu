// Attention of a batch whose sequences share their first keys: what the work is, and
// the merge of its parts.
//
// The sequences of a group have the same first e keys.  A softmax over [0, n) is put
// together from those over [0, e) and [e, n), each with its maximum m, sum l and
// unnormalised output o (m in log2 units):
//   m = max(m1, m2),  o = (o1 2^(m1 - m) + o2 2^(m2 - m)) / (l1 2^(m1 - m) + l2 2^(m2 - m))
// so the shared keys are an entry of the work of their own, with the tokens of all the
// group's sequences (they lie one after the other) as its rows: K and V are read once
// for up to 256 rows of them instead of once a sequence, and the MMAs' tiles are full
// where a single token fills G rows of 128.  All of those keys are visible to all of
// those tokens, as e is cut to what every sequence has in front of its new tokens.
//
// Four launches, each begun while the one in front runs:
//   shared_plan_kernel   one block: the entries, in two lists, and their costs
//   paged_kernel         (fa_paged.cu) entries of many rows, the shared keys among them,
//                        on as many CTAs as are their share of all work
//   rows_kernel          (fa_paged_rows.cu) entries of few rows, on the other SMs: single
//                        tokens behind their group's keys
//   shared_merge_kernel  the rows that have parts
//
// Measured (GB300; in brackets fa_fwd_paged on the same batch): 64 single tokens, 8192
// shared keys and up to 512 of their own, 32 + 8 heads, d = 128: 47 us (299); 256 behind
// 2 x 2048, up to 1024 of their own: 130 (281), 5.3 TB/s; 128 behind 1021, 16 heads, d = 64:
// 28 (90); 48 x 5 behind 4 prompts of up to 4093, 20 + 4 heads, d = 128: 41 (49); 4 behind
// 512: 13 (13.8); 8 x 509 tokens behind 16384: 703 (711), both at the tensor cores' rate.
// Small batches are a chain: plan 5 us (9 with more than 256 entries, 13 with 514, 18 with
// 1026), beginnings and ends of units 6 us each, merge 6 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_common.cuh"
#include "fa_paged.cuh"
#include "fa_paged_plan.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

using namespace paged;

constexpr size_t kGroupBytes = 8 + 7 * 4;  // of the plan's shared memory
constexpr int kMaxCtas = 178;  // (their parts' places are below 2^13, as a row's mark has room for)
static_assert(kMaxCtas * kMaxParts < 1 << 13, "a row's mark");
// What paged_kernel takes until its first tile and behind its last, what of it between two units,
// and what rows_kernel takes (a tenth of a microsecond, as all costs).
constexpr int kTileStart = 150, kTileEnds = 80, kRowsStart = 60;
// Cost of a unit of rows_kernel: its share of an SM's copies for 128 keys, and its beginning and
// end (more where all warps join its rows).  Like all that only decides how work is divided, in
// fp32: the block's time is that of its arithmetic, one step after the other.
template <int D>
__device__ __forceinline__ float rows_cost(int keys, int rows) {
  return (D == 128 ? 14.f : 7.f) * (keys + 32) + 128.f * (rows > kFewRows ? 40 : rows * D > 512 ? 12 : 6);
}

// ------------------------------------------------------------------ the lists --
// Sums of a thread's values over those in front of it; *total grows by all.
struct Sums {
  long long cost;  // of the entries with many rows
  float keys;      // of those with few
  float few;       // their cost
};
struct Counts {
  int entries, pieces, places, unused;
};
__device__ __forceinline__ Sums operator+(const Sums& x, const Sums& y) {
  return {x.cost + y.cost, x.keys + y.keys, x.few + y.few};
}
__device__ __forceinline__ Counts operator+(const Counts& x, const Counts& y) {
  return {x.entries + y.entries, x.pieces + y.pieces, x.places + y.places, 0};
}
__device__ __forceinline__ Sums shfl_up(const Sums& x, int off) {
  return {__shfl_up_sync(0xffffffffu, x.cost, off), __shfl_up_sync(0xffffffffu, x.keys, off),
          __shfl_up_sync(0xffffffffu, x.few, off)};
}
__device__ __forceinline__ Counts shfl_up(const Counts& x, int off) {
  return {__shfl_up_sync(0xffffffffu, x.entries, off), __shfl_up_sync(0xffffffffu, x.pieces, off),
          __shfl_up_sync(0xffffffffu, x.places, off), 0};
}

template <int THREADS, class T>
__device__ __forceinline__ T scan(const T& v, T* warps, T* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x / 32;
  T s = v;
#pragma unroll
  for (int off = 1; off < 32; off *= 2) {
    const T x = shfl_up(s, off);
    if (lane >= off) s = s + x;
  }
  T before = shfl_up(s, 1);
  if (lane == 0) before = T{};
  __syncthreads();  // the previous use of `warps` has been read
  if (lane == 31) warps[w] = s;
  __syncthreads();
  T front = *total;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) {
    const T x = warps[i];
    if (i == w) before = front + before;
    front = front + x;
  }
  *total = front;
  return before;
}

// A piece in 32 bytes: tokens lie below 2^30 and are at most 32, parts are fewer than 2^13.
__device__ __forceinline__ SharedPiece pack_piece(const SharedSeq& q, int k0, int k1, int slot, int parts, int which) {
  SharedPiece e;
  e.seq = make_int4((int)((unsigned)q.q0 << 2 | q.kind), q.kv, q.row, q.page0);
  e.part = make_int4(k0, k1, slot, parts << 18 | which << 5 | (q.qn - 1));
  return e;
}

// One block.  Cuts each group's shared keys to whole pages that all of its sequences with
// new tokens and keys have in front of those, and drops them where computing them once costs
// no less.  Thread by thread the entries are the groups' shared keys, then the sequences; with
// no more entries than threads each is looked at once.
template <int D, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) shared_plan_kernel(const PagedParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ unsigned long long plan_smem[];
  const int S = p.S, NG = p.num_groups, N = NG + S, tid = threadIdx.x, lane = tid & 31;
  unsigned long long* apart = plan_smem;            // [NG] cost of a key tile for each of its sequences by itself
  int* start = reinterpret_cast<int*>(apart + NG);  // [NG + 1]
  int* front = start + NG + 1;                      // [NG] keys in front of the new tokens, the fewest
  int* first = front + NG;                          // [NG] first sequence with new tokens and keys
  int* row = first + NG;                            // [NG] its first row
  int* row_end = row + NG;                          // [NG] behind the last one's rows
  int* members = row_end + NG;                      // [NG] how many there are
  int* keys = members + NG;                         // [NG] shared keys
  __shared__ Sums warps[THREADS / 32];
  __shared__ Counts warp_counts[THREADS / 32];
  __shared__ unsigned all_units;        // of a key head, with many rows
  __shared__ unsigned long long best;   // see below
  const Shape sh = {2 * p.tile_tokens, p.tile_tokens, p.copy_tokens, p.causal};
  const int cap = p.max_pages << p.page_log2, few = p.few_rows / p.G;
  const bool once = N <= THREADS;
  bool bad = false;
  auto sequence = [&](int s, bool& b) {
    return make_seq(__ldg(p.cu_seqlens + s), __ldg(p.cu_seqlens + s + 1), __ldg(p.kv_lens + s), p.T, cap, b);
  };
  // Everything that the first of each thread's entries needs is asked for at once.
  Seq mine = {0, 0, 0};
  if (tid >= NG && tid < N) mine = sequence(tid - NG, bad);
  const int row0 = imin(imax(__ldg(p.cu_seqlens), 0), p.T), row1 = imin(imax(__ldg(p.cu_seqlens + S), 0), p.T);
  const int want = tid < NG ? __ldg(p.prefix_lens + tid) : 0;
  for (int g = tid; g <= NG && NG > 0; g += THREADS) {
    const int at = __ldg(p.groups + g);
    start[g] = imin(imax(at, 0), S);
    bad = bad || start[g] != at || (g > 0 && at < __ldg(p.groups + g - 1));
    if (g < NG) front[g] = first[g] = row[g] = 0x7fffffff, row_end[g] = members[g] = 0, apart[g] = 0;
  }
  if (tid == 0) all_units = 0, best = ~0ull;
  __syncthreads();
  // A sequence's group: the last one that begins at it or in front (-1: none).
  auto group_of = [&](int s) {
    int lo = 0, hi = NG + 1;  // start[lo - 1] <= s < start[hi]
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (start[mid] <= s)
        lo = mid + 1;
      else
        hi = mid;
    }
    return lo - 1 < NG ? lo - 1 : -1;
  };
  // A sequence without keys (left out of the step, as its pages were not there) sees nothing, and
  // keeps the others from sharing nothing: its rows are its own entry's.
  auto in_group = [](const Seq& q) { return q.qn > 0 && q.kv > 0; };
  int my_group = -1;  // of the sequence that `mine` is
  if (NG > 0) {
    for (int i0 = 0; i0 < N; i0 += THREADS) {
      const int i = i0 + tid, s = i - NG;
      int g = -1, f = 0x7fffffff, q0 = 0, q1 = 0, cost = 0;
      if (i >= NG && i < N) {
        const Seq q = i0 == 0 ? mine : sequence(s, bad);
        if (in_group(q) && (g = group_of(s)) >= 0) {
          f = imax(0, p.causal ? q.kv - q.qn : q.kv);
          q0 = q.q0, q1 = q.q0 + q.qn;
          const int full = q.qn / sh.ut, rest = q.qn - full * sh.ut;
          cost = full * tile_cost<D>(sh.form(sh.ut)) + (rest > 0 ? tile_cost<D>(sh.form(rest)) : 0);
        }
      }
      if (i0 == 0) my_group = g;
      // most warps hold sequences of one group alone
      const unsigned in = __ballot_sync(0xffffffffu, g >= 0);
      if (in == 0) continue;
      const int g0 = __shfl_sync(0xffffffffu, g, __ffs(in) - 1);
      if (__all_sync(0xffffffffu, g < 0 || g == g0)) {
        const int least = __reduce_min_sync(0xffffffffu, f), end = __reduce_max_sync(0xffffffffu, q1);
        const int sum = __reduce_add_sync(0xffffffffu, cost);
        if (lane == __ffs(in) - 1) {
          atomicMin(&front[g0], least);
          atomicMin(&first[g0], s);
          atomicMin(&row[g0], q0);
          atomicMax(&row_end[g0], end);
          atomicAdd(&members[g0], __popc(in));
          atomicAdd(&apart[g0], (unsigned long long)sum);
        }
      } else if (g >= 0) {
        atomicMin(&front[g], f);
        atomicMin(&first[g], s);
        atomicMin(&row[g], q0);
        atomicMax(&row_end[g], q1);
        atomicAdd(&members[g], 1);
        atomicAdd(&apart[g], (unsigned long long)cost);
      }
    }
    __syncthreads();
  }
  // A group's entry: `n` keys of its first sequence, all rows from that one's to the last one's.
  auto prefix_of = [&](int g, int n) {
    SharedSeq q;
    q.q0 = row[g];
    q.qn = row_end[g] - row[g];
    q.kv = n;
    q.row = first[g];
    q.page0 = 0;
    q.kind = kPrefix;
    return q;
  };
  for (int g = tid; g < NG; g += THREADS) {
    const int x = g == tid ? want : __ldg(p.prefix_lens + g);
    bad = bad || x < 0 || x > cap;
    int n = imin(imax(x, 0), front[g]) >> p.page_log2 << p.page_log2;
    if (members[g] < 2) n = 0;
    if (n > 0) {
      const SharedSeq q = prefix_of(g, n);
      const float cost = q.qn <= few ? rows_cost<D>(n, q.qn * p.G) : (float)cost_of_seq<D>(q, sh);
      if (cost >= (float)apart[g] * n) n = 0;
    }
    keys[g] = n;
  }
  if (NG > 0) __syncthreads();
  auto entry = [&](int i) {
    SharedSeq q;
    q.q0 = q.qn = q.kv = q.row = q.page0 = q.kind = 0;
    if (i < NG) {
      if (keys[i] > 0) q = prefix_of(i, keys[i]);
    } else if (i < N) {
      static_cast<Seq&>(q) = i == tid ? mine : sequence(i - NG, bad);  // (without groups the first look at it)
      if (q.qn > 0) {
        const int g = i == tid ? my_group : NG > 0 && in_group(q) ? group_of(i - NG) : -1;
        const int n = g >= 0 ? keys[g] : 0;
        q.row = i - NG;
        q.page0 = n >> p.page_log2;
        q.kv -= n;
        q.kind = n > 0 ? kRest : kAlone;
      }
    }
    return q;
  };
  // Costs and keys in front of each entry.
  SharedSeq q;
  Sums front_of = {0, 0.f, 0.f}, sum = {0, 0.f, 0.f};
  auto values = [&] {
    const bool few_rows = q.qn > 0 && q.qn <= few;
    const Sums v = {q.qn > few ? cost_of_seq<D>(q, sh) : 0, few_rows ? (float)q.kv : 0.f,
                    few_rows ? rows_cost<D>(q.kv, q.qn * p.G) : 0.f};
    return v;
  };
  for (int i0 = 0; i0 < N; i0 += THREADS) {
    q = entry(i0 + tid);
    const unsigned units = __reduce_add_sync(0xffffffffu, q.qn > few ? (unsigned)blocks_of(q, sh.ut) : 0u);
    if (lane == 0 && units > 0) atomicAdd(&all_units, units);
    front_of = scan<THREADS>(values(), warps, &sum);
  }
  const float few_all = sum.few * p.Hk, all_keys = sum.keys * p.Hk;
  const long long many_all = sum.cost * p.Hk;
  // The CTAs that paged_kernel's entries are given to: all that they can be given to, or, with
  // others beside them, as many as let both kernels end at the same time.
  const int most = ctas_for<D>(many_all, p.sms);
  if (few_all > 0.f && tid > 0 && tid <= most && tid < p.sms) {
    // (rows_kernel is bound by device memory, of which an SM can use almost twice its share
    // where it has two CTAs; paged_kernel's tiles take longer beside it)
    const float tiles = 1.4f * many_all / tid + 128 * kTileStart;
    const float mine = few_all * (p.few_rows > kFewRows ? 1.f : 0.6f) / (p.sms - tid);
    const float rows = fmaxf(mine, few_all / p.sms) + 128 * kRowsStart;
    atomicMin(&best, (unsigned long long)__float_as_uint(fmaxf(tiles, rows)) << 8 | tid);  // (positive: in order as bits)
  }
  const SharedLists at = shared_lists(S, NG, p.sms);
  uint8_t* base = reinterpret_cast<uint8_t*>(p.plan);
  long long* costs = reinterpret_cast<long long*>(base + at.cost);
  SharedEntry* list = reinterpret_cast<SharedEntry*>(base + at.list);
  SharedPiece* pieces = reinterpret_cast<SharedPiece*>(base + at.pieces);
  Sums again = {0, 0.f, 0.f};
  Counts total = {0, 0, 0, 0};
  for (int i0 = 0; i0 < N; i0 += THREADS) {
    if (!once) {
      q = entry(i0 + tid);
      front_of = scan<THREADS>(values(), warps, &again);
    }
    const bool few_rows = q.qn > 0 && q.qn <= few, many_rows = q.qn > few;
    int part = 1, parts = 0;
    if (few_rows) {
      part = part_keys(front_of.keys * p.Hk, all_keys, p.few_rows / kFewRows, p.sms);
      parts = parts_of_keys(q.kv, part);
    }
    const Counts before = scan<THREADS>(Counts{many_rows, parts, parts > 1 ? parts : 0, 0}, warp_counts, &total);
    if (many_rows) {
      costs[before.entries] = front_of.cost * p.Hk;
      list[before.entries].seq = make_int4(q.q0, q.qn, q.kv, q.row);
      list[before.entries].how = make_int4(q.page0, q.kind, 0, 0);
    }
    for (int k = 0; k < parts; ++k)
      pieces[before.pieces + k] = pack_piece(q, k * part, k + 1 < parts ? (k + 1) * part : q.kv,
                                             parts > 1 ? (before.places + k) * p.Hk : -1, parts, k);
  }
  if (tid == 0) {
    costs[total.entries] = many_all;
    // (a multiple of the units where that costs less than it gives: units of one cost are then
    // cut into the same parts, and no CTA has the end of one and the beginning of the next,
    // which take it 6 us each.  13 sequences, 5 of them of 196 tokens, behind 20318 keys, 10
    // heads on 2, d = 64: 122 us on 80 CTAs, the only multiple of 80 units, 79 on 152)
    int ctas = few_all > 0.f && most > 0 ? (int)(best & 255) : most;
    const unsigned long long units = (unsigned long long)all_units * p.Hk;
    if (units > 0 && units < (unsigned long long)ctas) {
      const int fewer = ctas - ctas % (int)units;
      if (1.4f * many_all * (1.f / fewer - 1.f / ctas) <= 128 * kTileEnds) ctas = fewer;
    }
    int4* head = reinterpret_cast<int4*>(p.plan);
    head[0] = make_int4(total.entries, total.pieces, ctas, 0);
    head[1] = make_int4(row0, row1, 0, 0);
  }
  if (bad) record_index(p.status);
}

// ------------------------------------------------------------------ the merge --
// D / 8 lanes a row of the output (a token's query head).  Bound by latency: a row's mark,
// the end of a unit that was cut, its parts, one after the other; so every warp takes rows
// of its own, asks for eight parts at once, and all rows of a step are under way at the same
// time.  Where rows are many (MANY) most are done and the others have few parts: a warp looks at
// 32 marks at a time, and there are twice as many warps.  Where rows are so few that the warps outnumber them, the eight of a block share a
// row's parts (a group's keys, cut into a part a CTA).  Parts are added in a fixed order:
// those of the sequence's own keys, then those of the shared ones.
template <int D, int SPLIT, bool MANY>
__global__ void __launch_bounds__(256, MANY ? 4 : 2) shared_merge_kernel(const PagedParams p) {
  constexpr int kLanes = D / 8, kRowsAWarp = 32 / kLanes, kAtOnce = MANY ? 2 : 8;
  static_assert(SPLIT == 1 || !MANY, "no such form");
  __shared__ float4 sum[SPLIT > 1 ? 8 : 1][32][2];
  __shared__ float2 stat[SPLIT > 1 ? 8 : 1][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, l8 = lane % kLanes;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 head0 = __ldcg(reinterpret_cast<const int4*>(p.plan));
  const int4 head1 = __ldcg(reinterpret_cast<const int4*>(p.plan) + 1);
  const int Hq = p.Hk * p.G;
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
  const size_t slots = (size_t)p.sms * (2 * kPagedRows), all = (size_t)p.T * Hq;
  const int few_rows = imax(p.few_rows, kFewRows), places = shared_parts(p.sms) * kPartRows / few_rows;
  // Rows of a warp (or, split, of a block): the next `chunk`.
  constexpr int chunk = MANY ? 32 : kRowsAWarp;
  const size_t stride = (size_t)gridDim.x * (SPLIT > 1 ? 1 : 8) * chunk;
  size_t n0 = ((size_t)blockIdx.x * (SPLIT > 1 ? 1 : 8) + (SPLIT > 1 ? 0 : warp)) * chunk;
  unsigned todo = 0;
  bool fresh = true;
  for (;;) {
    if (fresh) {
      if (n0 >= all) break;
      todo = (1u << (chunk - 1) << 1) - 1;
      if (MANY)
        todo = __ballot_sync(0xffffffffu, n0 + lane < all && __ldcg(&ml[slots + all + n0 + lane].y) != kRowDone);
    }
    // the lane groups' rows: the first ones of those left (a group without one goes along)
    int at_row = -1;
#pragma unroll
    for (int k = 0; k < kRowsAWarp; ++k) {
      if (lane / kLanes == k) at_row = __ffs(todo) - 1;
      todo &= todo - 1;
    }
    const bool has = at_row >= 0 && n0 + at_row < all;
    const size_t row = n0 + (has ? at_row : 0);
    fresh = todo == 0;
    if (fresh) n0 += stride;
    const float2 own = __ldcg(ml + slots + all + row), shared = __ldcg(ml + slots + row);
    // (behind the loads: asked for at the same time as the first of them.  The last one: a CTA
    // gave up, and what the workspace says is not this call's)
    const int ctas = head0.z;
    if (head1.y <= head1.x || head1.z) return;
    const bool done = !has || row < (size_t)head1.x * Hq || row >= (size_t)head1.y * Hq || own.y == kRowDone;
    if (SPLIT > 1 ? __syncthreads_and(done) : __all_sync(0xffffffffu, done)) continue;
    // Where the parts are: `count` of a unit cut from CTA c on, of an entry's parts from place
    // c on, or one in the row's own place.  (What is said is cut to what there is room for.)
    enum { kHere, kCut, kPlaces };
    struct Parts {
      int how, c, at, count;
    };
    auto parts_of = [&](float2 x) {
      const int said = __float_as_int(x.x);
      Parts u = {kHere, 0, 0, 1};
      if (x.y == kRowCut || x.y == kRowCutOfRest) {
        u.how = kCut;
        u.c = imin(imax(said / kPagedRows, 0), p.sms - 1);
        u.at = said & (kPagedRows - 1);
      } else if (x.y == kRowParts || x.y == kRowPartsOfRest) {
        u.how = kPlaces;
        u.at = said & (few_rows - 1);
        u.count = said >> 5 & 8191;
        u.c = imax(said >> 18, 0);
      }
      return u;
    };
    Parts a = parts_of(own), b = {kHere, 0, 0, 0};
    if (done)
      a = {kHere, 0, 0, 0};
    else if (own.y != kRowCut && own.y != kRowParts)
      b = parts_of(shared);
    // A cut unit's parts: up to the first CTA behind c whose first slot ends its unit.
    bool open_a = a.how == kCut, open_b = b.how == kCut;
    for (int k = 1; __any_sync(0xffffffffu, open_a || open_b); k += kLanes) {
      const int ca = a.c + k + l8, cb = b.c + k + l8;
      const bool on_a = open_a && ca < ctas - 1 && __ldcg(p.hdr + (size_t)ca * kPagedHdr + 4) == 1;
      const bool on_b = open_b && cb < ctas - 1 && __ldcg(p.hdr + (size_t)cb * kPagedHdr + 4) == 1;
      auto end = [&](Parts& u, bool& open, bool on) {
        const unsigned ends = __ballot_sync(0xffffffffu, open && !on) >> (lane / kLanes * kLanes) & ((1u << (kLanes - 1) << 1) - 1);
        if (!open || !ends) return;
        u.count = imax(imin(u.c + k + __ffs(ends) - 1, imax(ctas, 1) - 1) - u.c + 1, 1);
        open = false;
      };
      end(a, open_a, on_a);
      end(b, open_b, on_b);
    }
    const int count = a.count + b.count;
    auto place = [&](int i) {
      const bool of_b = i >= a.count;
      const Parts& u = of_b ? b : a;
      const int k = of_b ? i - a.count : i;
      if (u.how == kHere) return slots + (of_b ? 0 : all) + row;
      if (u.how == kPlaces) return slots + 2 * all + (size_t)imin(u.c + k * p.Hk, places - 1) * few_rows + u.at;
      return ((size_t)imin(u.c + k, p.sms - 1) * 2 + (k == 0 ? 1 : 0)) * kPagedRows + u.at;
    };
    float m = -INFINITY, l = 0.f, acc[8] = {};
    auto add = [&](float w, const float4& u, const float4& v) {
      acc[0] = fmaf(w, u.x, acc[0]), acc[1] = fmaf(w, u.y, acc[1]), acc[2] = fmaf(w, u.z, acc[2]);
      acc[3] = fmaf(w, u.w, acc[3]), acc[4] = fmaf(w, v.x, acc[4]), acc[5] = fmaf(w, v.y, acc[5]);
      acc[6] = fmaf(w, v.z, acc[6]), acc[7] = fmaf(w, v.w, acc[7]);
    };
    for (int i0 = SPLIT > 1 ? warp : 0; i0 < count; i0 += kAtOnce * SPLIT) {
      float4 v[kAtOnce][2];
      float2 x[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        x[k] = make_float2(-INFINITY, 0.f);
        if (i0 + k * SPLIT >= count) continue;
        const size_t at = place(i0 + k * SPLIT);
        const float4* src = reinterpret_cast<const float4*>(p.part_o + at * D) + 2 * l8;
        v[k][0] = __ldcg(src), v[k][1] = __ldcg(src + 1), x[k] = __ldcg(ml + at);
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        if (x[k].y == 0.f) continue;  // saw no key
        const float m_new = fmaxf(m, x[k].x);
        const float old = m == -INFINITY ? 0.f : ex2(m - m_new), w = ex2(x[k].x - m_new);
        l = fmaf(w, x[k].y, l * old);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] *= old;
        add(w, v[k][0], v[k][1]);
        m = m_new;
      }
    }
    if constexpr (SPLIT > 1) {
      sum[warp][lane][0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      sum[warp][lane][1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
      stat[warp][lane] = make_float2(m, l);
      __syncthreads();
      if (warp == 0) {
        for (int k = 1; k < SPLIT; ++k) m = fmaxf(m, stat[k][lane].x);
        l = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
        for (int k = 0; k < SPLIT; ++k) {
          const float2 y = stat[k][lane];
          if (y.y == 0.f) continue;
          const float w = ex2(y.x - m);
          l = fmaf(w, y.y, l);
          add(w, sum[k][lane][0], sum[k][lane][1]);
        }
      }
    }
    if ((SPLIT == 1 || warp == 0) && !done) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + row * D)[l8] =
          make_uint4(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv),
                     pack_bf16x2(acc[4] * inv, acc[5] * inv), pack_bf16x2(acc[6] * inv, acc[7] * inv));
      if (l8 == 0 && p.lse) p.lse[row] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
    }
    if constexpr (SPLIT > 1) __syncthreads();
  }
}

template <int D>
cudaError_t launch_merge_t(const PagedLaunch& a, cudaStream_t stream) {
  if (a.grid > kMaxCtas) return cudaErrorInvalidConfiguration;
  const size_t rows = (size_t)a.p.T * a.p.Hk * a.p.G;
  constexpr int kRowsAWarp = 32 / (D / 8);
  const bool few = rows <= (size_t)a.grid * 2 * kRowsAWarp;        // (as many blocks as there is room for)
  const bool many = rows > (size_t)a.grid * 2 * 8 * kRowsAWarp * 4;  // (four times the rows that there is room for)
  const size_t a_block = few ? kRowsAWarp : many ? 32 * 8 : kRowsAWarp * 8;
  const size_t blocks = (rows + a_block - 1) / a_block, most = (size_t)a.grid * 32;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks < most ? blocks : most));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few    ? shared_merge_kernel<D, 8, false>
                                  : many ? shared_merge_kernel<D, 1, true>
                                         : shared_merge_kernel<D, 1, false>,
                            a.p);
}

template <int D, int THREADS>
cudaError_t launch_plan_t(const PagedLaunch& a, cudaStream_t stream) {
  const size_t bytes = (size_t)a.p.num_groups * kGroupBytes + sizeof(int);
  if (bytes > 32768) {  // (more than a kernel may have without asking, with what it has besides)
    const cudaError_t e = cudaFuncSetAttribute(shared_plan_kernel<D, THREADS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)(kMaxGroups * kGroupBytes + sizeof(int)));
    if (e != cudaSuccess) return e;
  }
  shared_plan_kernel<D, THREADS><<<1, THREADS, bytes, stream>>>(a.p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_shared_plan(const PagedLaunch& a, cudaStream_t stream) {
  // (its sums over the block take longer with more threads)
  if (a.p.S + a.p.num_groups <= 256) return a.d == 64 ? launch_plan_t<64, 256>(a, stream) : launch_plan_t<128, 256>(a, stream);
  return a.d == 64 ? launch_plan_t<64, 512>(a, stream) : launch_plan_t<128, 512>(a, stream);
}

cudaError_t launch_shared_merge(const PagedLaunch& a, cudaStream_t stream) {
  return a.d == 64 ? launch_merge_t<64>(a, stream) : launch_merge_t<128>(a, stream);
}

}  // namespace fa
