// Attention of a batch whose sequences share their first keys: what the work is, and
// the merge of its parts.  The attention itself is paged_kernel (fa_paged.cu).
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
// Three launches, each begun while the one in front runs: the list of entries with
// their costs (one block), the attention over all entries cut into runs of equal cost
// (the shared keys of a group are cut as any other unit), and the merge.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_common.cuh"
#include "fa_paged.cuh"
#include "fa_paged_plan.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

using namespace paged;

constexpr int kPlanThreads = 1024;
constexpr size_t kGroupBytes = 8 + 5 * 4;  // of the plan's shared memory
constexpr int kMaxCtas = 1024;

__device__ __forceinline__ long long* plan_costs(SharedPlan* plan) { return reinterpret_cast<long long*>(plan + 1); }

// ------------------------------------------------------------------- the list --
// One block.  Cuts each group's shared keys to whole key tiles and pages that all of
// its sequences with new tokens have in front of those, and drops them where
// computing them once costs no less.
template <int D>
__global__ void __launch_bounds__(kPlanThreads, 1) shared_plan_kernel(const PagedParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ unsigned long long plan_smem[];
  const int S = p.S, NG = p.num_groups, tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
  unsigned long long* apart = plan_smem;          // [NG] cost of a key tile for each of its sequences by itself
  int* start = reinterpret_cast<int*>(apart + NG);  // [NG + 1]
  int* front = start + NG + 1;                      // [NG] keys in front of the new tokens, the fewest
  int* first = front + NG;                          // [NG] first sequence with new tokens
  int* members = first + NG;                        // [NG] how many there are
  int* keys = members + NG;                         // [NG] shared keys
  __shared__ long long warp_cost[kPlanThreads / 32];
  __shared__ int warp_count[kPlanThreads / 32];
  const Shape sh = {2 * p.tile_tokens, p.tile_tokens, p.copy_tokens, p.causal};
  const int cap = p.max_pages << p.page_log2;
  bool bad = false;
  auto sequence = [&](int s, bool& b) {
    return make_seq(__ldg(p.cu_seqlens + s), __ldg(p.cu_seqlens + s + 1), __ldg(p.kv_lens + s), p.T, cap, b);
  };
  for (int g = tid; g <= NG; g += kPlanThreads) {
    const int at = __ldg(p.groups + g);
    start[g] = imin(imax(at, 0), S);
    bad = bad || start[g] != at || (g > 0 && at < __ldg(p.groups + g - 1));
  }
  for (int g = tid; g < NG; g += kPlanThreads) front[g] = first[g] = 0x7fffffff, members[g] = 0, apart[g] = 0;
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
    for (int s0 = 0; s0 < S; s0 += kPlanThreads) {
      const int s = s0 + tid;
      int g = -1, f = 0x7fffffff, cost = 0;
      if (s < S) {
        bool unused = false;
        const Seq q = sequence(s, unused);
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
  const int step = imax(kTileRows, 1 << p.page_log2);
  // The group's entry, `keys` of its first sequence.
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
  for (int g = tid; g < NG; g += kPlanThreads) {
    const int want = __ldg(p.prefix_lens + g);
    bad = bad || want < 0 || want > cap;
    int n = imin(imax(want, 0), front[g]) / step * step;
    if (members[g] < 2) n = 0;
    if (n > 0) {
      const SharedSeq q = prefix_of(g, n);
      if (q.qn == 0 || cost_of_seq<D>(q, sh) >= (long long)apart[g] * n) n = 0;
    }
    keys[g] = n;
  }
  __syncthreads();
  // The entries that have tokens, groups in front, and the cost of those before each.
  long long* costs = plan_costs(p.plan);
  SharedEntry* list = reinterpret_cast<SharedEntry*>(costs + shared_plan_costs(S + NG));
  long long total = 0;
  int entries = 0;
  for (int i0 = 0; i0 < NG + S; i0 += kPlanThreads) {
    const int i = i0 + tid;
    SharedSeq q;
    long long cost = 0;
    q.qn = 0;
    if (i < NG) {
      if (keys[i] > 0) q = prefix_of(i, keys[i]);
    } else if (i < NG + S) {
      const int s = i - NG;
      static_cast<Seq&>(q) = sequence(s, bad);
      if (q.qn > 0) {
        const int g = NG > 0 ? group_of(s) : -1;
        const int n = g >= 0 ? keys[g] : 0;
        q.row = s;
        q.page0 = n >> p.page_log2;
        q.kv -= n;
        q.kind = n > 0 ? kRest : kAlone;
      }
    }
    const bool live = q.qn > 0;
    if (live) cost = cost_of_seq<D>(q, sh) * p.Hk;
    long long before = cost;
    const unsigned votes = __ballot_sync(0xffffffffu, live);
#pragma unroll
    for (int off = 1; off < 32; off *= 2) {
      const long long u = __shfl_up_sync(0xffffffffu, before, off);
      if (lane >= off) before += u;
    }
    if (lane == 31) warp_cost[warp] = before, warp_count[warp] = __popc(votes);
    __syncthreads();
    before += total - cost;
    int at = entries + __popc(votes & ((1u << lane) - 1));
    for (int k = 0; k < kPlanThreads / 32; ++k) {
      const long long c = warp_cost[k];
      const int n = warp_count[k];
      if (k < warp) before += c, at += n;
      total += c;
      entries += n;
    }
    if (live) {
      costs[at] = before;
      list[at].seq = make_int4(q.q0, q.qn, q.kv, q.row);
      list[at].how = make_int4(q.page0, q.kind, 0, 0);
    }
    __syncthreads();  // before the next sums
  }
  if (tid == 0) {
    costs[entries] = total;
    const int row0 = imin(imax(__ldg(p.cu_seqlens), 0), p.T);
    const int row1 = imin(imax(__ldg(p.cu_seqlens + S), 0), p.T);
    *reinterpret_cast<int4*>(p.plan) = make_int4(entries, row0, row1, 0);
  }
  if (bad) record_index(p.status);
}

// ------------------------------------------------------------------ the merge --
// D / 8 lanes a row of the output (a token's query head).  SPLIT warps share a row's
// parts: all eight of a block where rows are few and a group's keys may be cut into
// many parts, one where rows are many.  Parts are added in a fixed order: those of
// the sequence's own keys, then those of the shared ones.
template <int D, int SPLIT>
__global__ void __launch_bounds__(256) shared_merge_kernel(const PagedParams p, int ctas) {
  constexpr int kLanes = D / 8, kRowsAWarp = 32 / kLanes, kRowsABlock = kRowsAWarp * 8 / SPLIT;
  __shared__ short ends[kMaxCtas];  // the CTA that ends the unit that CTA c began
  __shared__ float4 sum[SPLIT > 1 ? 8 : 1][32][2];
  __shared__ float2 stat[SPLIT > 1 ? 8 : 1][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, l8 = lane % kLanes;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 plan = __ldcg(reinterpret_cast<const int4*>(p.plan));
  const int Hq = p.Hk * p.G;
  const size_t rows = (size_t)(plan.z - plan.y) * Hq, row0 = (size_t)plan.y * Hq;
  if (plan.z <= plan.y || (size_t)blockIdx.x * kRowsABlock >= rows) return;
  bool ended = true;
  for (int c = threadIdx.x; c < ctas; c += 256) {
    const int* hdr = p.hdr + (size_t)c * kPagedHdr;
    ends[c] = (short)__ldcg(hdr + 4);
    ended = ended && __ldcg(hdr + kPagedEnded) == 1;
  }
  if (!__syncthreads_and(ended)) return;  // a CTA gave up: what the workspace says is not this call's
  {
    int last[kMaxCtas / 256];
#pragma unroll
    for (int k = 0; k < kMaxCtas / 256; ++k) {
      const int c = threadIdx.x + 256 * k;
      last[k] = c + 1;
      while (last[k] < ctas - 1 && ends[last[k]] == 1) ++last[k];
      if (last[k] > ctas - 1) last[k] = ctas - 1;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kMaxCtas / 256; ++k)
      if (threadIdx.x + 256 * k < ctas) ends[threadIdx.x + 256 * k] = (short)last[k];
    __syncthreads();
  }
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
  const size_t slots = (size_t)ctas * (2 * kPagedRows), all = (size_t)p.T * Hq;
  for (size_t n0 = (size_t)blockIdx.x * kRowsABlock; n0 < rows; n0 += (size_t)gridDim.x * kRowsABlock) {
    const size_t n = n0 + (SPLIT > 1 ? 0 : warp * kRowsAWarp) + lane / kLanes;
    const size_t row = row0 + (n < rows ? n : rows - 1);
    // Where the parts are: `count` of a unit cut from CTA c on, or one in the row's own place.
    struct Parts {
      int c, at, count;
    };
    auto cut = [&](float m) {
      const int said = __float_as_int(m);
      Parts u;
      u.c = imin(imax(said / kPagedRows, 0), ctas - 1);
      u.at = said & (kPagedRows - 1);
      u.count = imax(1, ends[u.c] - u.c + 1);
      return u;
    };
    const float2 own = __ldcg(ml + slots + all + row), head = __ldcg(ml + slots + row);
    const bool done = own.y == kRowDone;
    const bool own_cut = own.y == kRowCut || own.y == kRowCutOfRest;
    Parts a = {-1, 0, done ? 0 : 1}, b = {-1, 0, 0};
    if (own_cut) a = cut(own.x);
    if (!done && own.y != kRowCut) {
      b.count = 1;
      if (head.y == kRowCut) b = cut(head.x);
    }
    const int count = a.count + b.count;
    auto place = [&](int i) {
      const bool of_b = i >= a.count;
      const int c = of_b ? b.c : a.c, k = of_b ? i - a.count : i, at = of_b ? b.at : a.at;
      if (c < 0) return slots + (of_b ? 0 : all) + row;
      return ((size_t)imin(c + k, ctas - 1) * 2 + (k == 0 ? 1 : 0)) * kPagedRows + at;
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
  return cudaLaunchKernelEx(&cfg, few ? shared_merge_kernel<D, 8> : shared_merge_kernel<D, 1>, a.p, a.grid);
}

template <int D>
cudaError_t launch_plan_t(const PagedLaunch& a, cudaStream_t stream) {
  const size_t bytes = (size_t)a.p.num_groups * kGroupBytes + sizeof(int);
  const cudaError_t e = cudaFuncSetAttribute(shared_plan_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)(kMaxGroups * kGroupBytes + sizeof(int)));
  if (e != cudaSuccess) return e;
  shared_plan_kernel<D><<<1, kPlanThreads, bytes, stream>>>(a.p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_shared_plan(const PagedLaunch& a, cudaStream_t stream) {
  return a.d == 64 ? launch_plan_t<64>(a, stream) : launch_plan_t<128>(a, stream);
}

cudaError_t launch_shared_merge(const PagedLaunch& a, cudaStream_t stream) {
  return a.d == 64 ? launch_merge_t<64>(a, stream) : launch_merge_t<128>(a, stream);
}

}  // namespace fa
