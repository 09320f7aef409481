// Launch interface of the norm-and-rotation kernels (fa_norm_rope.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>

namespace fa {

// Rows of one tensor: element (b, n, h, c) at p + b sb + n sn + h sh + c.
struct HeadRows {
  const void* p;
  long long sb, sn, sh;
};

// Division of n < 2^31 by a fixed d: q = (mulhi(n, m) + n) >> l with
// l = ceil(log2 d), m = floor(2^32 (2^l - d) / d) + 1 (Granlund and Montgomery).
struct FastDiv {
  unsigned m, l, d;
  FastDiv() = default;
  explicit FastDiv(unsigned d_) : m(0), l(0), d(d_) {
    while ((1ull << l) < d) ++l;
    m = (unsigned)(((1ull << 32) * ((1ull << l) - d)) / d + 1);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ unsigned div(unsigned n) const { return (__umulhi(n, m) + n) >> l; }
#endif
};

struct NormRopeParams {
  int d, dr;               // head dimension; rotated columns (0: no rotation)
  int interleaved;         // pairs (2i, 2i + 1) instead of (i, i + dr / 2)
  int norm;                // 0: rotation only
  int weights_f32;         // weights are fp32 (else bf16)
  const void* w[2];        // weights of queries and keys, [d], or null (ones)
  float eps;
  const float* rope;       // [rope_len, dr]: cosines, then sines
  int rope_len;
  int* status;
};

struct NormRopeLaunch {
  NormRopeParams p;
  HeadRows in[2];          // queries, keys (strided)
  void* out[2];            // forward: [B, H, N, d] contiguous
  int H[2];
  int B, N;
  const int* positions;    // [B, N] or null (n)
  int walk;                // tokens a warp takes
  FastDiv by_n, by_chunks;
  unsigned q_blocks;       // row by row: CTAs of the queries
  FastDiv by_h[2];
  // backward: dout is what `out` was, dx is strided
  const void* dout[2];
  HeadRows dx[2];
  float* dw[2];            // [d] fp32 or null
  float* partial;          // [grid, d] fp32
  int sms;
};

struct AppendLaunch {
  NormRopeParams p;
  HeadRows in[3];          // queries, keys, values: (sn = token stride, sh = head stride; sb unused)
  void* q_out;             // [T, Hq, d] contiguous
  void* pages[2];          // key and value pages
  long long page_sp[2], page_sh[2], page_sr[2];  // strides of page, head, row
  const int* page_table;   // [S, max_pages]
  const int* cu_seqlens;   // [S + 1]
  const int* kv_lens;      // [S]
  int T, S, Hq, Hk, num_pages, page_log2, max_pages;
  FastDiv by_chunks;
  int span, sms;
};

// Heads of a tensor at most, and CTAs of the backward kernel at most (the rows of
// its partial sums): at least one for every chunk of heads of either tensor.
constexpr int kNormRopeMaxHeads = 2048;
constexpr int kNormRopeMaxCtas = 2048;

cudaError_t launch_norm_rope(const NormRopeLaunch& a, cudaStream_t stream);
cudaError_t launch_norm_rope_bwd(const NormRopeLaunch& a, cudaStream_t stream);
cudaError_t launch_paged_append(const AppendLaunch& a, cudaStream_t stream);

}  // namespace fa
