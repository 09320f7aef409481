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
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_common.cuh"
#include "fa_paged.cuh"
#include "fa_paged_plan.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

using namespace paged;

constexpr size_t kGroupBytes = 8 + 5 * 4;  // of the plan's shared memory
constexpr int kMaxCtas = 255;  // (what a row's mark has room for)
// Least cost of a CTA's share of paged_kernel where other CTAs have the rest (a tenth of a
// microsecond, as all costs): what a CTA takes until its first tile and behind its last.
constexpr int kLeastShare = 60;
// Fewest keys of a part of an entry with few rows.
constexpr int kLeastPart = 256;

// ------------------------------------------------------------------ the lists --
// Sums over the block of four values a thread: those in front of it; *total grows by all.
struct Sums {
  long long cost, keys;
  int entries, pieces;
};

template <int THREADS>
__device__ __forceinline__ Sums scan4(const Sums& v, Sums* warps, Sums* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x / 32;
  Sums s = v;
#pragma unroll
  for (int off = 1; off < 32; off *= 2) {
    const long long cost = __shfl_up_sync(0xffffffffu, s.cost, off), keys = __shfl_up_sync(0xffffffffu, s.keys, off);
    const int entries = __shfl_up_sync(0xffffffffu, s.entries, off);
    const int pieces = __shfl_up_sync(0xffffffffu, s.pieces, off);
    if (lane >= off) s.cost += cost, s.keys += keys, s.entries += entries, s.pieces += pieces;
  }
  __syncthreads();  // the previous use of `warps` has been read
  if (lane == 31) warps[w] = s;
  __syncthreads();
  s.cost += total->cost - v.cost;
  s.keys += total->keys - v.keys;
  s.entries += total->entries - v.entries;
  s.pieces += total->pieces - v.pieces;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) {
    const Sums x = warps[i];
    if (i < w) s.cost += x.cost, s.keys += x.keys, s.entries += x.entries, s.pieces += x.pieces;
    total->cost += x.cost, total->keys += x.keys, total->entries += x.entries, total->pieces += x.pieces;
  }
  return s;
}

// One block.  Cuts each group's shared keys to whole pages that all of its sequences with
// new tokens have in front of those, and drops them where computing them once costs no
// less.  Entries of few rows are split where there are too few of them for all CTAs.
template <int D, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) shared_plan_kernel(const PagedParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ unsigned long long plan_smem[];
  const int S = p.S, NG = p.num_groups, tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
  unsigned long long* apart = plan_smem;            // [NG] cost of a key tile for each of its sequences by itself
  int* start = reinterpret_cast<int*>(apart + NG);  // [NG + 1]
  int* front = start + NG + 1;                      // [NG] keys in front of the new tokens, the fewest
  int* first = front + NG;                          // [NG] first sequence with new tokens
  int* members = first + NG;                        // [NG] how many there are
  int* keys = members + NG;                         // [NG] shared keys
  __shared__ Sums warps[THREADS / 32];
  const Shape sh = {2 * p.tile_tokens, p.tile_tokens, p.copy_tokens, p.causal};
  const int cap = p.max_pages << p.page_log2, few = p.few_rows / p.G;
  bool bad = false;
  auto sequence = [&](int s, bool& b) {
    return make_seq(__ldg(p.cu_seqlens + s), __ldg(p.cu_seqlens + s + 1), __ldg(p.kv_lens + s), p.T, cap, b);
  };
  // The first of each thread's sequences and groups, asked for at once.
  Seq mine = {0, 0, 0};
  if (tid < S) mine = sequence(tid, bad);
  auto sequence_again = [&](int s) {
    bool unused = false;
    return s == tid ? mine : sequence(s, unused);
  };
  const int want0 = tid < NG ? __ldg(p.prefix_lens + tid) : 0;
  for (int g = tid; g <= NG && NG > 0; g += THREADS) {
    const int at = __ldg(p.groups + g);
    start[g] = imin(imax(at, 0), S);
    bad = bad || start[g] != at || (g > 0 && at < __ldg(p.groups + g - 1));
    if (g < NG) front[g] = first[g] = 0x7fffffff, members[g] = 0, apart[g] = 0;
  }
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
  if (NG > 0) {
    for (int s0 = 0; s0 < S; s0 += THREADS) {
      const int s = s0 + tid;
      int g = -1, f = 0x7fffffff, cost = 0;
      if (s < S) {
        const Seq q = sequence_again(s);
        if (s0 > 0) sequence(s, bad);
        if (q.qn > 0 && (g = group_of(s)) >= 0) {
          f = imax(0, p.causal ? q.kv - q.qn : q.kv);
          const int full = q.qn / sh.ut, rest = q.qn - full * sh.ut;
          cost = full * tile_cost<D>(sh.form(sh.ut)) + (rest > 0 ? tile_cost<D>(sh.form(rest)) : 0);
        }
      }
      // most warps hold sequences of one group alone
      const unsigned in = __ballot_sync(0xffffffffu, g >= 0);
      if (in == 0) continue;
      const int g0 = __shfl_sync(0xffffffffu, g, __ffs(in) - 1);
      if (__all_sync(0xffffffffu, g < 0 || g == g0)) {
        const int least = __reduce_min_sync(0xffffffffu, f);
        const int sum = __reduce_add_sync(0xffffffffu, cost);
        if (lane == 0) {
          atomicMin(&front[g0], least);
          atomicMin(&first[g0], s0 + warp * 32 + __ffs(in) - 1);
          atomicAdd(&members[g0], __popc(in));
          atomicAdd(&apart[g0], (unsigned long long)sum);
        }
      } else if (g >= 0) {
        atomicMin(&front[g], f);
        atomicMin(&first[g], s);
        atomicAdd(&members[g], 1);
        atomicAdd(&apart[g], (unsigned long long)cost);
      }
    }
    __syncthreads();
  }
  // The group's entry, `n` keys of its first sequence.
  auto prefix_of = [&](int g, int n) {
    SharedSeq q;
    const int end = imin(imax(__ldg(p.cu_seqlens + start[g + 1]), 0), p.T);
    q.q0 = imin(imax(__ldg(p.cu_seqlens + first[g]), 0), p.T);
    q.qn = imax(0, end - q.q0);
    q.kv = n;
    q.row = first[g];
    q.page0 = 0;
    q.kind = kPrefix;
    return q;
  };
  // Cost of a key head of an entry.
  auto cost_of_entry = [&](const SharedSeq& q) {
    return q.qn <= few ? cost_of<D>(1, q.kv, kShortCopies) : cost_of_seq<D>(q, sh);
  };
  for (int g = tid; g < NG; g += THREADS) {
    const int want = g == tid ? want0 : __ldg(p.prefix_lens + g);
    bad = bad || want < 0 || want > cap;
    int n = imin(imax(want, 0), front[g]) >> p.page_log2 << p.page_log2;
    if (members[g] < 2) n = 0;
    if (n > 0) {
      const SharedSeq q = prefix_of(g, n);
      if (q.qn == 0 || cost_of_entry(q) >= (long long)apart[g] * n) n = 0;
    }
    keys[g] = n;
  }
  __syncthreads();
  // Entry i: the groups' shared keys, then the sequences.
  auto entry = [&](int i) {
    SharedSeq q;
    q.q0 = q.qn = q.kv = q.row = q.page0 = q.kind = 0;
    if (i < NG) {
      if (keys[i] > 0) q = prefix_of(i, keys[i]);
    } else if (i < NG + S) {
      const int s = i - NG;
      static_cast<Seq&>(q) = sequence_again(s);
      if (q.qn > 0) {
        const int g = NG > 0 ? group_of(s) : -1;
        const int n = g >= 0 ? keys[g] : 0;
        q.row = s;
        q.page0 = n >> p.page_log2;
        q.kv -= n;
        q.kind = n > 0 ? kRest : kAlone;
      }
    }
    return q;
  };
  // Of the entries with few rows: all keys, and what a part of them is to hold.
  Sums total = {0, 0, 0, 0};
  long long rows_cost = 0;
  for (int i0 = 0; i0 < NG + S; i0 += THREADS) {
    const SharedSeq q = entry(i0 + tid);
    const bool few_rows = q.qn > 0 && q.qn <= few;
    const Sums v = {few_rows ? cost_of_entry(q) : 0, few_rows ? q.kv : 0, 0, 0};
    scan4<THREADS>(v, warps, &total);
  }
  rows_cost = total.cost * p.Hk;
  const long long share = total.keys * p.Hk / (kPartsASm * p.sms);
  const int part = imax(kLeastPart, (int)imin(0x3fffff00, (int)(share > 0x3fffff00 ? 0x3fffff00 : share) + 127) / 128 * 128);
  const SharedLists at = shared_lists(S, NG, p.sms);
  uint8_t* base = reinterpret_cast<uint8_t*>(p.plan);
  long long* costs = reinterpret_cast<long long*>(base + at.cost);
  SharedEntry* list = reinterpret_cast<SharedEntry*>(base + at.list);
  SharedPiece* pieces = reinterpret_cast<SharedPiece*>(base + at.pieces);
  // The lists.  `keys` of the sums counts the parts of split entries here.
  total = {0, 0, 0, 0};
  for (int i0 = 0; i0 < NG + S; i0 += THREADS) {
    const SharedSeq q = entry(i0 + tid);
    const bool few_rows = q.qn > 0 && q.qn <= few, many_rows = q.qn > few;
    const int parts = few_rows ? imax(1, (q.kv + part - 1) / part) : 0;
    const Sums v = {many_rows ? cost_of_entry(q) * p.Hk : 0, parts > 1 ? parts : 0, many_rows, parts};
    const Sums before = scan4<THREADS>(v, warps, &total);
    if (many_rows) {
      costs[before.entries] = before.cost;
      list[before.entries].seq = make_int4(q.q0, q.qn, q.kv, q.row);
      list[before.entries].how = make_int4(q.page0, q.kind, 0, 0);
    }
    for (int k = 0; k < parts; ++k) {
      SharedPiece& e = pieces[before.pieces + k];
      e.seq = make_int4(q.q0, q.qn, q.kv, q.row);
      e.how = make_int4(q.page0, q.kind, k * part, k + 1 < parts ? (k + 1) * part : q.kv);
      e.part = make_int4(parts > 1 ? ((int)before.keys + k) * p.Hk : -1, parts, k, 0);
    }
  }
  if (tid == 0) {
    costs[total.entries] = total.cost;
    int ctas = ctas_for<D>(total.cost, p.sms);
    if (rows_cost > 0 && ctas > 1) {
      const long long even = (total.cost + rows_cost) / p.sms, least = 128ll * kLeastShare;
      const long long each = even > least ? even : least;
      const long long most = (total.cost + each - 1) / each;
      ctas = most < ctas ? (int)most : ctas;
    }
    const int row0 = imin(imax(__ldg(p.cu_seqlens), 0), p.T);
    const int row1 = imin(imax(__ldg(p.cu_seqlens + S), 0), p.T);
    int4* head = reinterpret_cast<int4*>(p.plan);
    head[0] = make_int4(total.entries, total.pieces, ctas, 2 * rows_ctas(p.few_rows, p.sms));
    head[1] = make_int4(row0, row1, 0, 0);
  }
  if (bad) record_index(p.status);
}

// ------------------------------------------------------------------ the merge --
// D / 8 lanes a row of the output (a token's query head).  SPLIT warps share a row's
// parts: all eight of a block where rows are few and a group's keys may be cut into
// many parts, one where rows are many.  Parts are added in a fixed order: those of
// the sequence's own keys, then those of the shared ones.
template <int D, int SPLIT>
__global__ void __launch_bounds__(256) shared_merge_kernel(const PagedParams p) {
  constexpr int kLanes = D / 8, kRowsAWarp = 32 / kLanes, kRowsABlock = kRowsAWarp * 8 / SPLIT;
  __shared__ short ends[kMaxCtas + 1];  // the CTA that ends the unit that CTA c began
  __shared__ float4 sum[SPLIT > 1 ? 8 : 1][32][2];
  __shared__ float2 stat[SPLIT > 1 ? 8 : 1][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, l8 = lane % kLanes;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int ctas = __ldcg(&p.plan->ctas);
  const int4 plan = __ldcg(reinterpret_cast<const int4*>(p.plan) + 1);
  const int Hq = p.Hk * p.G;
  const size_t rows = (size_t)(plan.y - plan.x) * Hq, row0 = (size_t)plan.x * Hq;
  // (the last one: a CTA gave up, and what the workspace says is not this call's)
  if (plan.y <= plan.x || (size_t)blockIdx.x * kRowsABlock >= rows || plan.z) return;
  if ((int)threadIdx.x < ctas) ends[threadIdx.x] = (short)__ldcg(p.hdr + (size_t)threadIdx.x * kPagedHdr + 4);
  __syncthreads();
  {
    const int c = threadIdx.x;
    int last = c + 1;
    while (last < ctas - 1 && ends[last] == 1) ++last;
    __syncthreads();
    if (c < ctas) ends[c] = (short)imin(last, ctas - 1);
    __syncthreads();
  }
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
  const size_t slots = (size_t)p.sms * (2 * kPagedRows), all = (size_t)p.T * Hq;
  const int places = shared_parts(p.sms);
  for (size_t n0 = (size_t)blockIdx.x * kRowsABlock; n0 < rows; n0 += (size_t)gridDim.x * kRowsABlock) {
    const size_t n = n0 + (SPLIT > 1 ? 0 : warp * kRowsAWarp) + lane / kLanes;
    const size_t row = row0 + (n < rows ? n : rows - 1);
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
        u.c = imin(imax(said / kPagedRows, 0), imax(ctas, 1) - 1);
        u.at = said & (kPagedRows - 1);
        u.count = ctas > 0 ? imax(1, ends[u.c] - u.c + 1) : 1;
      } else if (x.y == kRowParts || x.y == kRowPartsOfRest) {
        u.how = kPlaces;
        u.at = said & (kPartRows - 1);
        u.count = said >> 5 & 8191;
        u.c = imax(said >> 18, 0);
      }
      return u;
    };
    const float2 own = __ldcg(ml + slots + all + row), head = __ldcg(ml + slots + row);
    const bool done = own.y == kRowDone;
    Parts a = parts_of(own), b = {kHere, 0, 0, 0};
    if (done)
      a.count = 0;
    else if (own.y != kRowCut && own.y != kRowParts)
      b = parts_of(head);
    const int count = a.count + b.count;
    auto place = [&](int i) {
      const bool of_b = i >= a.count;
      const Parts& u = of_b ? b : a;
      const int k = of_b ? i - a.count : i;
      if (u.how == kHere) return slots + (of_b ? 0 : all) + row;
      if (u.how == kPlaces) return slots + 2 * all + (size_t)imin(u.c + k * p.Hk, places - 1) * kPartRows + u.at;
      return ((size_t)imin(u.c + k, p.sms - 1) * 2 + (k == 0 ? 1 : 0)) * kPagedRows + u.at;
    };
    float m = -INFINITY, l = 0.f, acc[8] = {};
    float4 v0 = {}, v1 = {};
    float2 x = {-INFINITY, 0.f};
    auto load = [&](int i) {
      const size_t at = place(i);
      const float4* src = reinterpret_cast<const float4*>(p.part_o + at * D) + 2 * l8;
      v0 = __ldcg(src), v1 = __ldcg(src + 1), x = __ldcg(ml + at);
    };
    auto add = [&](float w, const float4& u, const float4& v) {
      acc[0] = fmaf(w, u.x, acc[0]), acc[1] = fmaf(w, u.y, acc[1]), acc[2] = fmaf(w, u.z, acc[2]);
      acc[3] = fmaf(w, u.w, acc[3]), acc[4] = fmaf(w, v.x, acc[4]), acc[5] = fmaf(w, v.y, acc[5]);
      acc[6] = fmaf(w, v.z, acc[6]), acc[7] = fmaf(w, v.w, acc[7]);
    };
    const int i0 = SPLIT > 1 ? warp : 0;
    if (i0 < count) load(i0);
    for (int i = i0; i < count; i += SPLIT) {
      const float4 u0 = v0, u1 = v1;
      const float2 y = x;
      if (i + SPLIT < count) load(i + SPLIT);
      if (y.y == 0.f) continue;  // saw no key
      const float m_new = fmaxf(m, y.x);
      const float old = m == -INFINITY ? 0.f : ex2(m - m_new), w = ex2(y.x - m_new);
      l = fmaf(w, y.y, l * old);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] *= old;
      add(w, u0, u1);
      m = m_new;
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
    if ((SPLIT == 1 || warp == 0) && n < rows && !done) {
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
  const bool few = rows <= 8192;
  const size_t a_block = few ? kRowsAWarp : kRowsAWarp * 8;
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
  return cudaLaunchKernelEx(&cfg, few ? shared_merge_kernel<D, 8> : shared_merge_kernel<D, 1>, a.p);
}

template <int D, int THREADS>
cudaError_t launch_plan_t(const PagedLaunch& a, cudaStream_t stream) {
  const size_t bytes = (size_t)a.p.num_groups * kGroupBytes + sizeof(int);
  const cudaError_t e = cudaFuncSetAttribute(shared_plan_kernel<D, THREADS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)(kMaxGroups * kGroupBytes + sizeof(int)));
  if (e != cudaSuccess) return e;
  shared_plan_kernel<D, THREADS><<<1, THREADS, bytes, stream>>>(a.p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_shared_plan(const PagedLaunch& a, cudaStream_t stream) {
  // (its sums over the block take longer with more threads)
  if (a.p.S + a.p.num_groups <= 256) return a.d == 64 ? launch_plan_t<64, 256>(a, stream) : launch_plan_t<128, 256>(a, stream);
  return a.d == 64 ? launch_plan_t<64, 1024>(a, stream) : launch_plan_t<128, 1024>(a, stream);
}

cudaError_t launch_shared_merge(const PagedLaunch& a, cudaStream_t stream) {
  return a.d == 64 ? launch_merge_t<64>(a, stream) : launch_merge_t<128>(a, stream);
}

}  // namespace fa
