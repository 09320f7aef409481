// A paged cache's tables, kept on the device: pages for the tokens of a step, and back.
//
// extend: for sequence s of a step (request r = requests[s] of length L, n new tokens)
//   rows cu[s] .. cu[s] + n - 1 of the step, cu the running sum of n
//   pages ceil(L / P) .. ceil((L + n) / P) - 1 of r from the top of the pool's stack,
//     in the order of the batch: the running sum of their numbers says which
//   slot of its token at position x: page[x / P] * P + x mod P
// release: pages ceil(keep / P) .. ceil(L / P) - 1 of r onto the stack, so that they
//   would be taken again in the same order.
//
// Bounds: a few words a sequence and one a page in use; nothing but latency until the
// batch holds some 10^5 pages.  So one launch: every block adds up the lengths of all
// sequences itself (three running sums in shared memory), takes a share of the pages
// and tokens, found by bisection, and the last block to be done writes the requests'
// lengths and the pool's count, which the others have read by then.
//
// Measured (GB300; a step and its return, two launches): 1 request 8.0 us, 256 of up to
// 8192 keys in pages of 16 14.4 (what they move takes 0.1), 1024 of up to 32768 keys 24.2
// (1.6); 3 us of each launch are the kernel's own begin and end, the rest a chain of loads
// (lengths, sums, entries, pages).  1024 threads a block measured no faster.
#include <cuda_runtime.h>

#include "fa_paged_tables.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kPiece = 256;   // table entries that a warp takes at once
constexpr int kTokens = 128;  // tokens

struct Sums {
  long long a, b;
};

// Running sums over the block of two values a thread, without its own; `total` grows by all.
__device__ __forceinline__ Sums scan2(long long a, long long b, Sums* warps, Sums* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x / 32;
  Sums s = {a, b};
#pragma unroll
  for (int off = 1; off < 32; off *= 2) {
    const long long x = __shfl_up_sync(0xffffffffu, s.a, off), y = __shfl_up_sync(0xffffffffu, s.b, off);
    if (lane >= off) s.a += x, s.b += y;
  }
  __syncthreads();  // the previous use of `warps` has been read
  if (lane == 31) warps[w] = s;
  __syncthreads();
  s.a += total->a - a;
  s.b += total->b - b;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    const Sums x = warps[i];
    if (i < w) s.a += x.a, s.b += x.b;
    total->a += x.a;
    total->b += x.b;
  }
  return s;
}

// Last index i < n with sums[i] <= x; sums[0] <= x.
__device__ __forceinline__ int find(const int* sums, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (sums[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int clamp(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }

// The first sequence of each request, by request (others of the same request are refused).
__device__ __forceinline__ void find_owners(const TablesParams& p, int* owner) {
  for (int r = threadIdx.x; r < p.R; r += kThreads) owner[r] = 0x7fffffff;
  __syncthreads();
  for (int s = threadIdx.x; s < p.S; s += kThreads) {
    const int r = __ldg(p.requests + s);
    if (r >= 0 && r < p.R) atomicMin(&owner[r], s);
  }
  __syncthreads();
}

// Whether this block is the last one: what it writes then no other block will read.
__device__ __forceinline__ bool last_block(const TablesParams& p) {
  if (gridDim.x == 1) {
    __syncthreads();
    return true;
  }
  __threadfence();
  __syncthreads();
  int mine = 0;
  if (threadIdx.x == 0) mine = atomicInc(reinterpret_cast<unsigned*>(p.pool + 1), gridDim.x - 1) == gridDim.x - 1;
  mine = __syncthreads_or(mine);
  __threadfence();
  return mine;
}

// A sequence as the blocks keep it.
struct Rows {
  int* request;  // -1: none, or left out
  int* old;      // its length before
  int* cu;       // [S + 1] first row
  int* before;   // pages that those in front take, or give
  int* piece;    // [S + 1] pieces of table entries in front
  int* owner;    // [R]
  __device__ Rows(int* sm, int S) {
    request = sm;
    old = request + S;
    before = old + S;
    cu = before + S;
    piece = cu + S + 1;
    owner = piece + S + 1;
  }
};

__global__ void __launch_bounds__(kThreads, 1) extend_kernel(const TablesParams p) {
  extern __shared__ int tables_smem[];
  __shared__ Sums warps[kWarps];
  __shared__ int taken;
  const Rows seq(tables_smem, p.S);
  const int S = p.S, T = p.T, lg = p.page_log2, tid = threadIdx.x, lane = tid & 31;
  const long long cap = (long long)p.max_pages << lg;
  const int said = *reinterpret_cast<volatile int*>(p.pool), count = clamp(said, 0, p.num_pages);
  bool bad = said != count;
  if (tid == 0) taken = 0;
  find_owners(p, seq.owner);
  Sums rows = {0, 0}, pages = {0, 0};
  for (int s0 = 0; s0 < S; s0 += kThreads) {
    const int s = s0 + tid;
    int r = -1, n = 0, len = 0;
    if (s < S) {
      r = max(__ldg(p.requests + s), -1);
      const int want = __ldg(p.lens + s);
      n = r >= 0 && want > 0 ? want : 0;  // (negative: a place without a request)
      bad = bad || r >= p.R || (r >= 0 && want < 0);
      if (r >= p.R || (r >= 0 && seq.owner[r] != s)) r = -2;
      if (r >= 0) len = *reinterpret_cast<volatile int*>(p.request_lens + r);
    }
    const Sums at = scan2(n, 0, warps, &rows);
    if (s < S) seq.cu[s] = (int)(at.a < T ? at.a : T);
    bool in = r >= 0 && len >= 0 && len + (long long)n <= cap && (n == 0 || at.a + n <= T);
    const int page0 = in ? (int)((len + (1ll << lg) - 1) >> lg) : 0;
    const int page1 = in ? (int)((len + (long long)n + (1ll << lg) - 1) >> lg) : 0;
    const Sums got = scan2(page1 - page0, (page1 + kPiece - 1) / kPiece, warps, &pages);
    if (in && page1 > page0 && got.a + (page1 - page0) > count) in = false;  // not enough pages
    if (s < S) {
      bad = bad || (!in && r != -1);
      seq.request[s] = in ? r : -1;
      seq.old[s] = len;
      seq.before[s] = in ? (int)(got.a < count ? got.a : count) : 0;
      seq.piece[s] = (int)got.b;
    }
    // the pool's top goes down by what those that came in take
    const int top = in && page1 > page0 ? (int)(got.a + (page1 - page0)) : 0;
    const int most = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0 && most > 0) atomicMax(&taken, most);
  }
  if (tid == 0) {
    seq.cu[S] = (int)(rows.a < T ? rows.a : T);
    seq.piece[S] = (int)pages.b;
  }
  __syncthreads();
  const int* stack = p.pool + kPoolHead;
  const int pieces = seq.piece[S], end = seq.cu[S];
  // Page x of sequence s: its request's, or the next one of the stack.
  auto page_of = [&](int s, int r, int x) {
    const int held = (int)((seq.old[s] + (1ll << lg) - 1) >> lg);
    return x < held ? __ldg(p.request_table + (size_t)r * p.max_pages + x)
                    : __ldg(stack + clamp(count - 1 - (seq.before[s] + x - held), 0, p.num_pages - 1));
  };
  // What the caller's rows hold, and through release() the stack, may be no page: its tokens have
  // no slot (the caller writes to its own cache by them), and each entry in use is looked at below.
  auto is_page = [&](int x) { return (unsigned)x < (unsigned)p.num_pages; };
  bool lost = false;
  const long long items = (long long)pieces + (T + (long long)kTokens - 1) / kTokens;  // (T goes up to 2^31 - 1)
  for (long long i = (long long)blockIdx.x * kWarps + tid / 32; i < items; i += (long long)gridDim.x * kWarps) {
    if (i < pieces) {
      const int s = find(seq.piece, S, (int)i), r = seq.request[s];
      if (r < 0) continue;
      const int n = seq.cu[s + 1] - seq.cu[s], x0 = ((int)i - seq.piece[s]) * kPiece;
      const int held = (int)((seq.old[s] + (1ll << lg) - 1) >> lg);
      const int used = (int)((seq.old[s] + (long long)n + (1ll << lg) - 1) >> lg);
      int page[kPiece / 32];  // all asked for before the first is written
#pragma unroll
      for (int k = 0; k < kPiece / 32; ++k) {
        const int x = x0 + 32 * k + lane;
        page[k] = x < used ? page_of(s, r, x) : 0;
      }
#pragma unroll
      for (int k = 0; k < kPiece / 32; ++k) {
        const int x = x0 + 32 * k + lane;
        if (x >= used) continue;
        lost = lost || !is_page(page[k]);
        p.page_table[(size_t)s * p.max_pages + x] = page[k];
        if (x >= held) p.request_table[(size_t)r * p.max_pages + x] = page[k];
      }
    } else {
      int pos[kTokens / 32];
      long long slot[kTokens / 32];
#pragma unroll
      for (int k = 0; k < kTokens / 32; ++k) {
        const long long t = (i - pieces) * kTokens + 32 * k + lane;
        pos[k] = 0;
        slot[k] = -1;
        if (t < end) {
          const int s = find(seq.cu, S, (int)t), r = seq.request[s];
          pos[k] = -1;
          if (r >= 0) {
            pos[k] = seq.old[s] + ((int)t - seq.cu[s]);
            const int page = page_of(s, r, pos[k] >> lg);
            if (is_page(page)) slot[k] = ((long long)page << lg) + (pos[k] & ((1 << lg) - 1));
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kTokens / 32; ++k) {
        const long long t = (i - pieces) * kTokens + 32 * k + lane;
        if (t >= T) continue;
        if (p.positions) p.positions[t] = pos[k];
        if (p.slots) p.slots[t] = slot[k];
      }
    }
  }
  if (blockIdx.x == 0) {
    for (int s = tid; s <= S; s += kThreads) {
      p.cu_seqlens[s] = seq.cu[s];
      if (s < S) p.kv_lens[s] = seq.request[s] >= 0 ? seq.old[s] + seq.cu[s + 1] - seq.cu[s] : 0;
    }
    lost = lost || bad;
  }
  if (lost) record_index(p.status);
  if (!last_block(p)) return;
  for (int s = tid; s < S; s += kThreads)
    if (seq.request[s] >= 0) p.request_lens[seq.request[s]] = seq.old[s] + seq.cu[s + 1] - seq.cu[s];
  if (tid == 0) p.pool[0] = count - taken;
}

__global__ void __launch_bounds__(kThreads, 1) release_kernel(const TablesParams p) {
  extern __shared__ int tables_smem[];
  __shared__ Sums warps[kWarps];
  const Rows seq(tables_smem, p.S);
  const int S = p.S, lg = p.page_log2, tid = threadIdx.x, lane = tid & 31;
  const long long cap = (long long)p.max_pages << lg;
  const int said = *reinterpret_cast<volatile int*>(p.pool), count = clamp(said, 0, p.num_pages);
  bool bad = said != count;
  find_owners(p, seq.owner);
  Sums given = {0, 0};
  for (int s0 = 0; s0 < S; s0 += kThreads) {
    const int s = s0 + tid;
    int r = -1, keep = 0, first = 0, n = 0;
    if (s < S && (r = __ldg(p.requests + s)) >= 0) {
      const int want = p.lens ? __ldg(p.lens + s) : 0;
      const bool in = r < p.R && seq.owner[r] == s;
      const int len = in ? *reinterpret_cast<volatile int*>(p.request_lens + r) : 0;
      const int kept = in && p.kept_pages ? __ldg(p.kept_pages + r) : 0;
      if (in && len >= 0 && len <= cap && want >= 0 && want <= len && kept >= 0 && kept <= p.max_pages) {
        keep = want;
        first = max((int)((keep + (1ll << lg) - 1) >> lg), kept);
        n = (int)((len + (1ll << lg) - 1) >> lg) - first;
        if (n < 0) n = 0;
      } else {
        bad = true;
        r = -1;
      }
    }
    const Sums at = scan2(n, (n + kPiece - 1) / kPiece, warps, &given);
    if (s < S) {
      seq.request[s] = r < 0 ? -1 : r;
      seq.old[s] = keep;
      seq.cu[s] = first;
      seq.before[s] = (int)(at.a < (1 << 30) ? at.a : 1 << 30);
      seq.piece[s] = (int)at.b;
    }
  }
  // More pages than there is room for: some were given back before, or were never taken.
  const bool fits = given.a <= p.num_pages - count;
  bad = bad || !fits;
  if (tid == 0) seq.piece[S] = fits ? (int)given.b : 0;
  __syncthreads();
  const int total = fits ? (int)given.a : 0;
  int* stack = p.pool + kPoolHead;
  for (int i = blockIdx.x * kWarps + tid / 32; i < seq.piece[S]; i += gridDim.x * kWarps) {
    const int s = find(seq.piece, S, i), r = seq.request[s], x0 = (i - seq.piece[s]) * kPiece;
    const int n = (s + 1 < S ? seq.before[s + 1] : total) - seq.before[s];
    int page[kPiece / 32];  // all asked for before the first is written
#pragma unroll
    for (int k = 0; k < kPiece / 32; ++k) {
      const int x = x0 + 32 * k + lane;
      page[k] = x < n ? __ldg(p.request_table + (size_t)r * p.max_pages + seq.cu[s] + x) : 0;
    }
#pragma unroll
    for (int k = 0; k < kPiece / 32; ++k) {
      const int x = x0 + 32 * k + lane;
      if (x >= n) continue;
      bad = bad || page[k] < 0 || page[k] >= p.num_pages;
      stack[count + total - 1 - (seq.before[s] + x)] = page[k];
    }
  }
  if (bad) record_index(p.status);
  if (!last_block(p) || !fits) return;
  for (int s = tid; s < S; s += kThreads)
    if (seq.request[s] >= 0) p.request_lens[seq.request[s]] = seq.old[s];
  if (tid == 0) p.pool[0] = count + total;
}

template <class K>
cudaError_t launch(K kern, const TablesParams& p, int sms, long long items, cudaStream_t stream) {
  const size_t bytes = (5 * (size_t)p.S + 2 + p.R) * sizeof(int);
  constexpr size_t kMost = (5 * (size_t)kMaxSequences + 2 + kMaxRequests) * sizeof(int);
  if (bytes > 32768) {  // (more than a kernel may have without asking, with what it has besides)
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMost);
    if (e != cudaSuccess) return e;
  }
  const long long blocks = (items + kWarps - 1) / kWarps;
  kern<<<(unsigned)(blocks < 1 ? 1 : blocks < sms ? blocks : sms), kThreads, bytes, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

// A block a sixteen pieces or groups of tokens that there may be.
cudaError_t launch_paged_extend(const TablesParams& p, int sms, cudaStream_t stream) {
  const long long items =
      (long long)p.S * ((p.max_pages + kPiece - 1) / kPiece) + (p.T + (long long)kTokens - 1) / kTokens;
  return launch(extend_kernel, p, sms, items, stream);
}

cudaError_t launch_paged_release(const TablesParams& p, int sms, cudaStream_t stream) {
  return launch(release_kernel, p, sms, (long long)p.S * ((p.max_pages + kPiece - 1) / kPiece), stream);
}

}  // namespace fa
