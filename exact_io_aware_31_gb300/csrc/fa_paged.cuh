// Launch interface of the paged attention kernels (fa_paged.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>

namespace fa {

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
  PagedParams p;
  int d;
  int is_short;  // units of copy_tokens only
  int grid;
};

cudaError_t launch_paged(const PagedLaunch& a, cudaStream_t stream);

}  // namespace fa
