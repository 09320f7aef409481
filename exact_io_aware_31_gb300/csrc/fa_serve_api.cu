// C ABI entry points around the attention kernels: per-head norm with position
// rotation, and the paged key/value cache.  Argument validation and launch
// set-up only; no device memory is allocated here.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/fa.h"
#include "fa_host.h"
#include "fa_norm_rope.cuh"
#include "fa_paged.cuh"

namespace fa {
namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool flag(int v) { return v == 0 || v == 1; }

// Strides are 16-byte steps.  Where a size is 1 the stride means nothing: it is
// not looked at, and none is taken.
//
// An input's stride: zero allowed (a broadcast dimension).
bool stride_in(long long* s, long long size) {
  if (size <= 1) *s = 0;
  return *s >= 0 && *s % 8 == 0;
}

// An output's: rows of d elements must not overlap.
bool stride_out(long long* s, long long size, int d) { return stride_in(s, size) && (size <= 1 || *s >= d); }

// One that is written into a tensor map: positive even where it means nothing.
bool stride_map(long long* s, long long size, int d, long long below) {
  if (size <= 1) *s = d;
  return *s >= d && *s % 8 == 0 && *s < below;
}

int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return FA_OK;
  cudaGetLastError();
  return FA_ERR_CUDA;
}

// The arguments that the norm-and-rotation calls share.  `longest` is the
// number of positions taken without a positions array (0: none are).
int check_norm_rope(NormRopeParams* p, int d, int norm, const void* qw, const void* kw, int weights_f32, float eps,
                    const float* rope, int rope_len, int rope_dim, int interleaved, int longest) {
  if (!flag(norm) || !flag(weights_f32) || !flag(interleaved)) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || eps < 0.f) return FA_ERR_INVALID_ARG;
  if (rope_dim < 0 || rope_dim % 16 != 0) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (rope_dim > d) return FA_ERR_INVALID_ARG;
  if (rope_dim > 0 && (!aligned16(rope) || rope_len < 1 || longest > rope_len)) return FA_ERR_INVALID_ARG;
  if ((qw && !aligned16(qw)) || (kw && !aligned16(kw))) return FA_ERR_INVALID_ARG;
  p->d = d;
  p->dr = rope_dim;
  p->interleaved = interleaved;
  p->norm = norm;
  p->weights_f32 = weights_f32;
  p->w[0] = qw;
  p->w[1] = kw;
  p->eps = eps;
  p->rope = rope;
  p->rope_len = rope_len;
  return FA_OK;
}

bool sizes_ok(int B, int Hq, long long Hk, int N) {
  // (the last bound keeps the launch grid below its limit)
  return B >= 1 && N >= 1 && Hq >= 1 && Hk >= 1 && Hq <= kNormRopeMaxHeads && Hk <= 2 * kNormRopeMaxHeads &&
         (long long)B * N <= INT_MAX && (long long)B * N * (Hq + Hk) < (1ll << 34);
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" int fa_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out, int B, int Hq, int Hk, int N,
                               int d, long long q_stride_b, long long q_stride_h, long long q_stride_n,
                               long long k_stride_b, long long k_stride_h, long long k_stride_n, int norm,
                               const void* q_weight, const void* k_weight, int weights_f32, float eps,
                               const float* rope, int rope_len, int rope_dim, int interleaved, const int* positions,
                               cudaStream_t stream) {
  if (!sizes_ok(B, Hq, Hk, N) || Hk > kNormRopeMaxHeads) return FA_ERR_INVALID_ARG;
  NormRopeLaunch a = {};
  int st = check_norm_rope(&a.p, d, norm, q_weight, k_weight, weights_f32, eps, rope, rope_len, rope_dim, interleaved,
                           positions ? 0 : N);
  if (st != FA_OK) return st;
  if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out) || !aligned4(positions))
    return FA_ERR_INVALID_ARG;
  if (!stride_in(&q_stride_b, B) || !stride_in(&q_stride_h, Hq) || !stride_in(&q_stride_n, N) ||
      !stride_in(&k_stride_b, B) || !stride_in(&k_stride_h, Hk) || !stride_in(&k_stride_n, N))
    return FA_ERR_INVALID_ARG;
  DeviceInfo dev;
  if ((st = device_info(&dev)) != FA_OK) return st;
  a.p.status = dev.status;
  a.in[0] = {q, q_stride_b, q_stride_n, q_stride_h};
  a.in[1] = {k, k_stride_b, k_stride_n, k_stride_h};
  a.out[0] = q_out;
  a.out[1] = k_out;
  a.H[0] = Hq;
  a.H[1] = Hk;
  a.B = B;
  a.N = N;
  a.positions = positions;
  a.sms = dev.sms;
  return cuda_status(launch_norm_rope(a, stream));
}

extern "C" size_t fa_qk_norm_rope_bwd_workspace_size(int d) {
  if (d != 64 && d != 128) return 0;
  return (size_t)kNormRopeMaxCtas * d * sizeof(float);
}

extern "C" int fa_qk_norm_rope_bwd(const void* dq_out, const void* dk_out, const void* q, const void* k, void* dq,
                                   void* dk, float* dq_weight, float* dk_weight, int B, int Hq, int Hk, int N, int d,
                                   long long q_stride_b, long long q_stride_h, long long q_stride_n,
                                   long long k_stride_b, long long k_stride_h, long long k_stride_n,
                                   long long dq_stride_b, long long dq_stride_h, long long dq_stride_n,
                                   long long dk_stride_b, long long dk_stride_h, long long dk_stride_n, int norm,
                                   const void* q_weight, const void* k_weight, int weights_f32, float eps,
                                   const float* rope, int rope_len, int rope_dim, int interleaved,
                                   const int* positions, void* workspace, size_t workspace_bytes,
                                   cudaStream_t stream) {
  if (!sizes_ok(B, Hq, Hk, N) || Hk > kNormRopeMaxHeads) return FA_ERR_INVALID_ARG;
  NormRopeLaunch a = {};
  int st = check_norm_rope(&a.p, d, norm, q_weight, k_weight, weights_f32, eps, rope, rope_len, rope_dim, interleaved,
                           positions ? 0 : N);
  if (st != FA_OK) return st;
  if (!aligned16(dq_out) || !aligned16(dk_out) || !aligned16(dq) || !aligned16(dk) || !aligned16(q) ||
      !aligned16(k) || !aligned4(positions) || !aligned4(dq_weight) || !aligned4(dk_weight))
    return FA_ERR_INVALID_ARG;
  if (!stride_in(&q_stride_b, B) || !stride_in(&q_stride_h, Hq) || !stride_in(&q_stride_n, N) ||
      !stride_in(&k_stride_b, B) || !stride_in(&k_stride_h, Hk) || !stride_in(&k_stride_n, N))
    return FA_ERR_INVALID_ARG;
  if (!stride_out(&dq_stride_b, B, d) || !stride_out(&dq_stride_h, Hq, d) || !stride_out(&dq_stride_n, N, d) ||
      !stride_out(&dk_stride_b, B, d) || !stride_out(&dk_stride_h, Hk, d) || !stride_out(&dk_stride_n, N, d))
    return FA_ERR_INVALID_ARG;
  const bool weights = dq_weight != nullptr || dk_weight != nullptr;
  if (weights && !norm) return FA_ERR_INVALID_ARG;
  if (weights && (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
                  workspace_bytes < fa_qk_norm_rope_bwd_workspace_size(d)))
    return FA_ERR_WORKSPACE;
  DeviceInfo dev;
  if ((st = device_info(&dev)) != FA_OK) return st;
  a.p.status = dev.status;
  a.in[0] = {q, q_stride_b, q_stride_n, q_stride_h};
  a.in[1] = {k, k_stride_b, k_stride_n, k_stride_h};
  a.dout[0] = dq_out;
  a.dout[1] = dk_out;
  a.dx[0] = {dq, dq_stride_b, dq_stride_n, dq_stride_h};
  a.dx[1] = {dk, dk_stride_b, dk_stride_n, dk_stride_h};
  a.dw[0] = dq_weight;
  a.dw[1] = dk_weight;
  a.partial = weights ? static_cast<float*>(workspace) : nullptr;
  a.H[0] = Hq;
  a.H[1] = Hk;
  a.B = B;
  a.N = N;
  a.positions = positions;
  a.sms = dev.sms;
  return cuda_status(launch_norm_rope_bwd(a, stream));
}

namespace fa {
namespace {

// The cache arguments that every paged call shares (T, S >= 1 here).
int check_cache(const void* k_pages, const void* v_pages, const int* page_table, const int* cu_seqlens,
                const int* kv_lens, int Hk, int d, int num_pages, int page_size, int max_pages, long long* sp,
                long long* sh, long long* sr) {
  if (num_pages < 1 || max_pages < 1) return FA_ERR_INVALID_ARG;
  if (page_size < 16 || page_size > 65536 || (page_size & (page_size - 1)) != 0) return FA_ERR_INVALID_ARG;
  if ((long long)max_pages * page_size > (1 << 30)) return FA_ERR_INVALID_ARG;
  if (!aligned16(k_pages) || !aligned16(v_pages)) return FA_ERR_INVALID_ARG;
  if (!page_table || !cu_seqlens || !kv_lens || !aligned4(page_table) || !aligned4(cu_seqlens) || !aligned4(kv_lens))
    return FA_ERR_INVALID_ARG;
  for (int i = 0; i < 2; ++i)
    if (!stride_map(&sp[i], num_pages, d, 1ll << 38) || !stride_map(&sh[i], Hk, d, 1ll << 38) ||
        !stride_map(&sr[i], page_size, d, 1ll << 38))
      return FA_ERR_INVALID_ARG;
  return FA_OK;
}

}  // namespace
}  // namespace fa

extern "C" int fa_paged_append(const void* q, const void* k, const void* v, void* q_out, void* k_pages,
                               void* v_pages, const int* page_table, const int* cu_seqlens, const int* kv_lens,
                               int T, int S, int Hq, int Hk, int d, int num_pages, int page_size, int max_pages,
                               long long q_stride_t, long long q_stride_h, long long k_stride_t, long long k_stride_h,
                               long long v_stride_t, long long v_stride_h, long long kp_stride_p,
                               long long kp_stride_h, long long kp_stride_r, long long vp_stride_p,
                               long long vp_stride_h, long long vp_stride_r, int norm, const void* q_weight,
                               const void* k_weight, int weights_f32, float eps, const float* rope, int rope_len,
                               int rope_dim, int interleaved, cudaStream_t stream) {
  if (T < 0 || S < 0 || !sizes_ok(1, Hq, 2ll * Hk, T > 0 ? T : 1)) return FA_ERR_INVALID_ARG;
  AppendLaunch a = {};
  int st = check_norm_rope(&a.p, d, norm, q_weight, k_weight, weights_f32, eps, rope, rope_len, rope_dim, interleaved,
                           0);
  if (st != FA_OK) return st;
  if (T == 0 || S == 0) return FA_OK;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out)) return FA_ERR_INVALID_ARG;
  if (!stride_in(&q_stride_t, T) || !stride_in(&q_stride_h, Hq) || !stride_in(&k_stride_t, T) ||
      !stride_in(&k_stride_h, Hk) || !stride_in(&v_stride_t, T) || !stride_in(&v_stride_h, Hk))
    return FA_ERR_INVALID_ARG;
  long long sp[2] = {kp_stride_p, vp_stride_p}, sh[2] = {kp_stride_h, vp_stride_h},
            sr[2] = {kp_stride_r, vp_stride_r};
  st = check_cache(k_pages, v_pages, page_table, cu_seqlens, kv_lens, Hk, d, num_pages, page_size, max_pages, sp, sh,
                   sr);
  if (st != FA_OK) return st;
  DeviceInfo dev;
  if ((st = device_info(&dev)) != FA_OK) return st;
  a.p.status = dev.status;
  a.in[0] = {q, 0, q_stride_t, q_stride_h};
  a.in[1] = {k, 0, k_stride_t, k_stride_h};
  a.in[2] = {v, 0, v_stride_t, v_stride_h};
  a.q_out = q_out;
  a.pages[0] = k_pages;
  a.pages[1] = v_pages;
  for (int i = 0; i < 2; ++i) {
    a.page_sp[i] = sp[i];
    a.page_sh[i] = sh[i];
    a.page_sr[i] = sr[i];
  }
  a.page_table = page_table;
  a.cu_seqlens = cu_seqlens;
  a.kv_lens = kv_lens;
  a.T = T;
  a.S = S;
  a.Hq = Hq;
  a.Hk = Hk;
  a.num_pages = num_pages;
  while ((1 << a.page_log2) < page_size) ++a.page_log2;
  a.max_pages = max_pages;
  a.sms = dev.sms;
  return cuda_status(launch_paged_append(a, stream));
}

namespace fa {
namespace {

struct PagedWorkspace {
  size_t ml, o, total;
};

PagedWorkspace paged_workspace(int sms, int d) {
  const size_t rows = (size_t)sms * 2 * kPagedRows;
  PagedWorkspace w;
  w.ml = round256((size_t)sms * kPagedHdr * sizeof(int));
  w.o = w.ml + round256(rows * 2 * sizeof(float));
  w.total = w.o + round256(rows * d * sizeof(float));
  return w;
}

// A pool [pages, Hk, page_size, d] of any strides: boxes of 64 columns by the
// rows of a page, at most a key tile's 128 (128-byte swizzle).
int make_pool_map(CUtensorMap* m, const void* base, int pages, int Hk, int page_size, int d, long long sp,
                  long long sh, long long sr) {
  cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)page_size, (cuuint64_t)Hk, (cuuint64_t)pages};
  cuuint64_t strides[3] = {(cuuint64_t)sr * 2, (cuuint64_t)sh * 2, (cuuint64_t)sp * 2};
  cuuint32_t box[4] = {64, (cuuint32_t)(page_size < 128 ? page_size : 128), 1, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return tensor_map_encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, es,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? FA_OK
             : FA_ERR_CUDA;
}

// Queries [T, Hk, G, d]: boxes of 64 columns x one key head's G heads x `tokens`.
int make_ragged_map(CUtensorMap* m, const void* base, int T, int Hk, int G, int d, int tokens, long long st,
                    long long sh) {
  cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)G, (cuuint64_t)Hk, (cuuint64_t)T};
  cuuint64_t strides[3] = {(cuuint64_t)sh * 2, (cuuint64_t)sh * G * 2, (cuuint64_t)st * 2};
  cuuint32_t box[4] = {64, (cuuint32_t)G, 1, (cuuint32_t)tokens};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return tensor_map_encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, es,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? FA_OK
             : FA_ERR_CUDA;
}

}  // namespace
}  // namespace fa

extern "C" size_t fa_fwd_paged_workspace_size(int d) {
  if (d != 64 && d != 128) return 0;
  DeviceInfo dev;
  if (device_info(&dev) != FA_OK) return 0;
  return paged_workspace(dev.sms, d).total;
}

extern "C" int fa_fwd_paged(const void* q, const void* k_pages, const void* v_pages, void* o, float* lse,
                            const int* page_table, const int* cu_seqlens, const int* kv_lens, int T, int S, int Hq,
                            int Hk, int d, int num_pages, int page_size, int max_pages, long long q_stride_t,
                            long long q_stride_h, long long kp_stride_p, long long kp_stride_h, long long kp_stride_r,
                            long long vp_stride_p, long long vp_stride_h, long long vp_stride_r, float scale,
                            int causal, int max_q, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (T < 0 || S < 0 || T >= (1 << 30) || Hq < 1 || Hk < 1 || Hq % Hk != 0 || max_q < 0 || !flag(causal) ||
      !std::isfinite(scale))
    return FA_ERR_INVALID_ARG;
  if (Hq >= (1 << 15)) return FA_ERR_INVALID_ARG;
  const int G = Hq / Hk;
  if ((d != 64 && d != 128) || G > 128) return FA_ERR_UNSUPPORTED;
  if (T == 0 || S == 0) return FA_OK;
  if (!aligned16(q) || !aligned16(o) || !aligned4(lse)) return FA_ERR_INVALID_ARG;
  if (!stride_map(&q_stride_t, T, d, 1ll << 31) || !stride_map(&q_stride_h, Hq, d, 1ll << 31))
    return FA_ERR_INVALID_ARG;
  long long sp[2] = {kp_stride_p, vp_stride_p}, sh[2] = {kp_stride_h, vp_stride_h},
            sr[2] = {kp_stride_r, vp_stride_r};
  int st = check_cache(k_pages, v_pages, page_table, cu_seqlens, kv_lens, Hk, d, num_pages, page_size, max_pages, sp,
                       sh, sr);
  if (st != FA_OK) return st;
  if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return FA_ERR_WORKSPACE;
  DeviceInfo dev;
  if ((st = device_info(&dev)) != FA_OK) return st;
  const PagedWorkspace w = paged_workspace(dev.sms, d);
  if (workspace_bytes < w.total) return FA_ERR_WORKSPACE;
  PagedLaunch a = {};
  a.d = d;
  a.grid = dev.sms;
  PagedParams& p = a.p;
  p.tile_tokens = 128 / G;
  p.copy_tokens = 32 / G;
  // Chunks whose rows for one key head fit a quarter of a tile take the kernel
  // that has no other form.
  a.is_short = max_q > 0 && max_q <= p.copy_tokens;
  p.o = o;
  p.lse = lse;
  p.page_table = page_table;
  p.cu_seqlens = cu_seqlens;
  p.kv_lens = kv_lens;
  p.T = T;
  p.S = S;
  p.Hk = Hk;
  p.G = G;
  p.g_inverse = 65536 / G + 1;
  p.num_pages = num_pages;
  p.page_log2 = 0;
  while ((1 << p.page_log2) < page_size) ++p.page_log2;
  p.max_pages = max_pages;
  p.causal = causal;
  p.c2 = log2_scale(scale);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.hdr = reinterpret_cast<int*>(ws);
  p.part_ml = reinterpret_cast<float*>(ws + w.ml);
  p.part_o = reinterpret_cast<float*>(ws + w.o);
  p.status = dev.status;
  if (make_ragged_map(&a.tm_q, q, T, Hk, G, d, p.tile_tokens, q_stride_t, q_stride_h) ||
      make_ragged_map(&a.tm_q4, q, T, Hk, G, d, p.copy_tokens > 0 ? p.copy_tokens : 1, q_stride_t, q_stride_h) ||
      make_pool_map(&a.tm_k, k_pages, num_pages, Hk, page_size, d, sp[0], sh[0], sr[0]) ||
      make_pool_map(&a.tm_v, v_pages, num_pages, Hk, page_size, d, sp[1], sh[1], sr[1]))
    return FA_ERR_CUDA;
  return cuda_status(launch_paged(a, stream));
}
