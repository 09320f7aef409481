// Launch interface of the paged attention kernels (fa_paged.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>

namespace fa {

// The plan of a batch whose sequences share keys, in the workspace: what the work is, one
// entry after the other, with the cost of all entries in front of each.
struct SharedPlan {
  int entries;        // how many there are
  int row0, row1;     // tokens that belong to a sequence
  int pad;
  // long long cost[S + num_groups + 1], then SharedEntry[S + num_groups] (16-byte aligned)
};
struct SharedEntry {
  int4 seq;  // first token, tokens, keys, row of the page table
  int4 how;  // its first entry there, kind
};
static_assert(sizeof(SharedPlan) == 16 && sizeof(SharedEntry) == 32, "16-byte reads");

struct PagedParams {
  void* o;                // [T, Hq, d] bf16
  float* lse;             // [T, Hq] fp32 or null
  const int* page_table;  // [S, max_pages]
  const int* cu_seqlens;  // [S + 1]
  const int* kv_lens;     // [S]
  int T, S, Hk, G;        // G query heads a key head
  int num_pages, page_log2, max_pages;
  int g_inverse;          // 65536 / G + 1
  int causal;
  float c2;               // scale * log2(e)
  int tile_tokens;        // tokens of a 128-row query tile: G * tile_tokens <= 128
  int copy_tokens;        // tokens whose rows fit a quarter of it (0: none)
  int* hdr;               // [grid][kPagedHdr]
  float* part_ml;         // [grid][2][rows][2]: running maximum (log2 units), sum
  float* part_o;          // [grid][2][rows][d]: unnormalised output
  int* status;
  // Sequences that share keys (fa_paged_shared.cu); null and 0 otherwise
  const int* groups;       // [num_groups + 1] first sequence of each group, and its end
  const int* prefix_lens;  // [num_groups] keys that its sequences share
  int num_groups;
  SharedPlan* plan;
};

// ints of a CTA's header in the workspace
constexpr int kPagedHdr = 8;
constexpr int kPagedEnded = 5;  // (shared keys) which of them says that the CTA did its work
// query rows of a unit at most
constexpr int kPagedRows = 256;

struct PagedLaunch {
  CUtensorMap tm_q;   // [T, Hk, G, d]: boxes of 64 columns x G x 1 x tile_tokens
  CUtensorMap tm_q4;  // ... x copy_tokens
  CUtensorMap tm_k;  // [pages, Hk, page_size, d]: boxes of 64 columns x min(page_size, 128) rows
  CUtensorMap tm_v;
  PagedParams p;
  int d;
  int is_short;  // units of copy_tokens only
  int is_shared;
  int grid;
};

cudaError_t launch_paged(const PagedLaunch& a, cudaStream_t stream);

// Groups of a batch at most.
constexpr int kMaxGroups = 4096;

// Partial rows of a batch whose sequences share keys lie behind the CTAs' slots: first
// those of the shared keys, one a row of the output, then those of the rest.  Where a
// row's partial outputs are instead is said by a sum that no row can have:
constexpr float kRowCut = -1.f;         // in the slots: the maximum holds the CTA that began the unit and the row there
constexpr float kRowDone = -2.f;        // in the output already
constexpr float kRowCutOfRest = -3.f;   // as kRowCut, and there are shared keys, too

inline __host__ __device__ size_t shared_plan_costs(int entries) { return ((size_t)entries + 2) / 2 * 2; }

cudaError_t launch_shared_plan(const PagedLaunch& a, cudaStream_t stream);
cudaError_t launch_shared_merge(const PagedLaunch& a, cudaStream_t stream);

}  // namespace fa
