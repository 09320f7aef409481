// Launch interface of the kernels that keep a paged cache's tables (fa_paged_tables.cu).
#pragma once

#include <cuda_runtime.h>

namespace fa {

// Sequences of a call and places for requests at most: what a block's shared memory holds.
constexpr int kMaxSequences = 4096;
constexpr int kMaxRequests = 16384;

// Pool: the number of free pages, a word that is zero between calls, the stack of free pages.
constexpr int kPoolHead = 2;

struct TablesParams {
  const int* requests;    // [S]
  const int* lens;        // [S] new tokens; keys that are kept (null: none)
  const int* kept_pages;  // [R] or null
  int* request_lens;      // [R]
  int* request_table;     // [R, max_pages]
  int* pool;              // [kPoolHead + num_pages]
  int* cu_seqlens;        // [S + 1]
  int* kv_lens;           // [S]
  int* page_table;        // [S, max_pages]
  int* positions;         // [T] or null
  long long* slots;       // [T] or null
  int T, S, R, num_pages, page_log2, max_pages;
  int* status;
};

cudaError_t launch_paged_extend(const TablesParams& p, int sms, cudaStream_t stream);
cudaError_t launch_paged_release(const TablesParams& p, int sms, cudaStream_t stream);

}  // namespace fa
