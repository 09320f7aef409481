// Launch interface of the paged attention kernels (fa_paged.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>

#include "fa_paged_plan.cuh"

namespace fa {

// The plan of a batch whose sequences share keys, in the workspace: what the work is, one
// entry after the other, with the cost of all entries in front of each.
struct SharedPlan {
  int entries;      // of paged_kernel's list
  int pieces;       // of rows_kernel's
  int ctas;         // that paged_kernel's work is given to
  unsigned next;    // rows_kernel: the next of its pieces' heads that no CTA has taken
  int row0, row1;   // tokens that belong to a sequence
  int failed;       // a CTA gave up: the workspace's rows are not this call's
  int pad;
};
struct SharedEntry {
  int4 seq;  // first token, tokens, keys, row of the page table
  int4 how;  // its first entry there, kind
};
// Of an entry with few rows, or a part of its keys.
struct SharedPiece {
  int4 seq;   // first token and kind, keys, row of the page table, first entry there
  int4 part;  // keys [x, y) of the entry, place of its partial rows (-1: not split), parts, which one, tokens
};
static_assert(sizeof(SharedPlan) == 32 && sizeof(SharedEntry) == 32 && sizeof(SharedPiece) == 32, "16-byte reads");

using paged::kMaxParts;
using paged::kPartRows;
using paged::shared_parts;

// Where the lists lie behind the head: costs in front of the entries, entries, pieces.
struct SharedLists {
  size_t cost, list, pieces, bytes;
};
inline __host__ __device__ SharedLists shared_lists(int S, int groups, int sms) {
  const size_t n = (size_t)S + groups;
  SharedLists w;
  w.cost = sizeof(SharedPlan);
  w.list = w.cost + (n + 2) / 2 * 2 * sizeof(long long);
  w.pieces = w.list + n * sizeof(SharedEntry);
  w.bytes = w.pieces + (n + shared_parts(sms)) * sizeof(SharedPiece);
  return w;
}

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
  int sms;
  unsigned hk_inverse;     // (2^32 - 1) / Hk
  int few_rows;            // entries of at most so many rows of a key head go to rows_kernel (0: none)
};

// ints of a CTA's header in the workspace
constexpr int kPagedHdr = 8;
// query rows of a unit at most
constexpr int kPagedRows = 256;

struct PagedLaunch {
  CUtensorMap tm_q;   // [T, Hk, G, d]: boxes of 64 columns x G x 1 x tile_tokens
  CUtensorMap tm_q4;  // ... x copy_tokens
  CUtensorMap tm_k;  // [pages, Hk, page_size, d]: boxes of 64 columns x min(page_size, 128) rows
  CUtensorMap tm_v;
  CUtensorMap tm_kr;  // shared keys: boxes of rows_kernel's rows
  CUtensorMap tm_vr;
  const void* q;
  long long q_stride_t, q_stride_h;
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
// those of the shared keys, one a row of the output, then those of the rest, then
// few_rows for each head of a part of rows_kernel.  Where a row's partial outputs are
// instead is said by a sum that no row can have:
constexpr float kRowDone = -1.f;         // in the output already
constexpr float kRowCut = -2.f;          // in the slots: the maximum holds the CTA that began the unit and the row there
constexpr float kRowCutOfRest = -3.f;    // as kRowCut, and there are shared keys, too
constexpr float kRowParts = -4.f;        // in parts: the maximum holds their first place, their number and the row there
constexpr float kRowPartsOfRest = -5.f;  // as kRowParts, and there are shared keys, too

// Rows of a 16-row matrix tile: what rows_kernel takes at a time, once or twice.
constexpr int kFewRows = 16;
// Its CTAs an SM.
inline __host__ __device__ constexpr int rows_ctas(int few_rows) { return few_rows <= kFewRows ? 2 : 1; }
// Keys of a stage: 16 KB of K and V.
inline __host__ __device__ constexpr int rows_keys(int d) { return d == 128 ? 32 : 64; }

cudaError_t launch_shared_plan(const PagedLaunch& a, cudaStream_t stream);
cudaError_t launch_shared_rows(const PagedLaunch& a, cudaStream_t stream);
cudaError_t launch_shared_merge(const PagedLaunch& a, cudaStream_t stream);

}  // namespace fa
