// Norm of queries and keys for each head with the position rotation in the
// same pass: forward, backward, and the serving form that writes keys and
// values into a paged cache.
//
// Mathematics, for one head row x[0..d) at position p:
//   r = 1 / sqrt(mean(x^2) + eps),  y = w * x * r           (norm)
//   z_a = y_a c - y_b s,  z_b = y_b c + y_a s                (rotation)
// for each pair (a, b) of the first dr columns, c and s the cosine and sine of
// the pair's angle at p; the other columns pass through.  Backward, given dz:
//   dy = R^T dz (the rotation by -angle),  dw = sum over rows of dy * x r,
//   g = dy * w,  dx = r (g - x r mean(g x r)).
//
// About ten operations an element against 4 bytes (forward) or 6 (backward):
// bound by device memory, so each element is read once and written once, 16
// bytes a thread.  d / 8 lanes share a row (a thread holds 8 neighbouring
// columns; the sum of squares and a split rotation's partner columns come by
// shuffle), a warp takes 32 / (d / 8) rows at once and kSteps such steps per
// item: an item is one token's run of up to kSteps * rows heads, so that the
// token's cosines and sines are loaded once for all of them and four 16-byte
// loads a thread are in flight.  The input may be any strided view (a slice
// of the projection's output); the output is the contiguous [B, H, N, d] that
// the attention kernels read, so the transposition costs no pass of its own.
// Everything between load and store is fp32; the one rounding is the stored
// bf16 (the weights' gradient stays fp32).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/fa.h"
#include "fa_norm_rope.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSteps = 4;

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(v[i] << 16);
    x[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

__device__ __forceinline__ void load_weights(const NormRopeParams& p, int which, int l, float (&w)[8]) {
  const void* src = p.w[which];
  if (src == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.f;
  } else if (p.weights_f32) {
    load8(static_cast<const float*>(src) + 8 * l, w);
  } else {
    unpack8(__ldg(static_cast<const uint4*>(src) + l), w);
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int off = LPR / 2; off > 0; off /= 2) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// The cosines and sines of this lane's 8 columns (lane l of a row), and how
// the row turns.  Split pairs (i, i + dr / 2): lanes l and l + dr / 16 hold
// partner columns and the same angles.  Neighbouring pairs: four angles a lane.
struct Turn {
  float c[8], s[8];  // interleaved: the first four
  int mode;          // 0: columns pass, 1: split pairs, first half, 2: second half, 3: neighbouring pairs
  int hl;            // lanes between split partners
};

__device__ __forceinline__ void load_turn(const NormRopeParams& p, int pos, int l, Turn& t) {
  const int half = p.dr / 2;
  t.hl = p.dr / 16;
  t.mode = 0;
  if (8 * l >= p.dr) return;
  const float* row = p.rope + (size_t)pos * p.dr;
  if (p.interleaved) {
    t.mode = 3;
    const float4 a = __ldg(reinterpret_cast<const float4*>(row) + l);
    const float4 b = __ldg(reinterpret_cast<const float4*>(row + half) + l);
    t.c[0] = a.x, t.c[1] = a.y, t.c[2] = a.z, t.c[3] = a.w;
    t.s[0] = b.x, t.s[1] = b.y, t.s[2] = b.z, t.s[3] = b.w;
  } else {
    t.mode = l < t.hl ? 1 : 2;
    const int at = 8 * (l < t.hl ? l : l - t.hl);
    load8(row + at, t.c);
    load8(row + half + at, t.s);
  }
}

// Rotate the row's 8 columns of this lane by the angle (BACK: by minus the
// angle).  Every lane of the warp calls it.
template <bool BACK>
__device__ __forceinline__ void turn_row(const NormRopeParams& p, const Turn& t, float (&y)[8]) {
  if (p.dr == 0) return;
  if (p.interleaved) {
    if (t.mode == 3) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float s = BACK ? -t.s[i] : t.s[i];
        const float a = y[2 * i], b = y[2 * i + 1];
        y[2 * i] = a * t.c[i] - b * s;
        y[2 * i + 1] = b * t.c[i] + a * s;
      }
    }
    return;
  }
  const int lane = threadIdx.x & 31;
  const int src = t.mode == 1 ? lane + t.hl : t.mode == 2 ? lane - t.hl : lane;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float other = __shfl_sync(0xffffffffu, y[i], src);
    if (t.mode != 0) {
      const float s = (t.mode == 1) != BACK ? -t.s[i] : t.s[i];
      y[i] = y[i] * t.c[i] + other * s;
    }
  }
}

// One item: a token's heads [h0, h0 + kSteps * 32 / LPR) of one tensor.
template <int D>
struct Item {
  static constexpr int LPR = D / 8;          // lanes a row
  static constexpr int RPW = 32 / LPR;       // rows a warp and step
  static constexpr int kRows = RPW * kSteps; // heads an item
};

// ----------------------------------------------------------------- forward ---
template <int D>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const NormRopeLaunch a) {
  using I = Item<D>;
  const int lane = threadIdx.x & 31, l = lane % I::LPR, sub = lane / I::LPR;
  const int cq = (a.H[0] + I::kRows - 1) / I::kRows, ck = (a.H[1] + I::kRows - 1) / I::kRows;
  const long long item = (long long)blockIdx.x * kWarps + threadIdx.x / 32;
  const long long token = item / (cq + ck);
  if (token >= (long long)a.B * a.N) return;
  const int chunk = (int)(item - token * (cq + ck));
  const int which = chunk >= cq;
  const int h0 = (which ? chunk - cq : chunk) * I::kRows, H = a.H[which];
  const int b = (int)(token / a.N), n = (int)(token - (long long)b * a.N);
  const HeadRows in = a.in[which];
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(in.p) + b * in.sb + n * in.sn + 8 * l;
  uint4 raw[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int h = h0 + i * I::RPW + sub;
    raw[i] = h < H ? __ldg(reinterpret_cast<const uint4*>(src + h * in.sh)) : make_uint4(0, 0, 0, 0);
  }
  const int pos = a.positions ? __ldg(a.positions + token) : n;
  const bool bad = a.p.dr > 0 && (pos < 0 || pos >= a.p.rope_len);
  Turn t;
  load_turn(a.p, bad ? 0 : pos, l, t);
  float w[8];
  load_weights(a.p, which, l, w);
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out[which]) + (((size_t)b * H) * a.N + n) * D + 8 * l;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int h = h0 + i * I::RPW + sub;
    float y[8];
    unpack8(raw[i], y);
    if (a.p.norm) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
      const float r = rsqrtf(row_sum<I::LPR>(ss) * (1.f / D) + a.p.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = y[e] * r * w[e];
    }
    turn_row<false>(a.p, t, y);
    if (h < H)
      *reinterpret_cast<uint4*>(dst + (size_t)h * a.N * D) = bad ? make_uint4(0, 0, 0, 0) : pack8(y);
  }
  if (bad && lane == 0) atomicExch(a.p.status, FA_ERR_DEVICE_INDEX);
}

// ---------------------------------------------------------------- backward ---
// A warp walks the items with a grid stride and keeps the weights' gradients
// of its 8 columns in registers (queries and keys apart); a CTA adds up its
// warps and writes one row of partial sums, and a second kernel adds those in
// a fixed order: no atomics, the same bits on every run.
template <int D>
__global__ void __launch_bounds__(kThreads) norm_rope_bwd_kernel(const NormRopeLaunch a) {
  using I = Item<D>;
  const int lane = threadIdx.x & 31, l = lane % I::LPR, sub = lane / I::LPR;
  const int cq = (a.H[0] + I::kRows - 1) / I::kRows, ck = (a.H[1] + I::kRows - 1) / I::kRows;
  const long long items = (long long)a.B * a.N * (cq + ck);
  float dw[2][8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[0][e] = dw[1][e] = 0.f;
  for (long long item = (long long)blockIdx.x * kWarps + threadIdx.x / 32; item < items;
       item += (long long)gridDim.x * kWarps) {
    const long long token = item / (cq + ck);
    const int chunk = (int)(item - token * (cq + ck));
    const int which = chunk >= cq;
    const int h0 = (which ? chunk - cq : chunk) * I::kRows, H = a.H[which];
    const int b = (int)(token / a.N), n = (int)(token - (long long)b * a.N);
    const HeadRows in = a.in[which], dx = a.dx[which];
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(in.p) + b * in.sb + n * in.sn + 8 * l;
    const __nv_bfloat16* dsrc =
        static_cast<const __nv_bfloat16*>(a.dout[which]) + (((size_t)b * H) * a.N + n) * D + 8 * l;
    uint4 raw[kSteps], draw[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int h = h0 + i * I::RPW + sub;
      raw[i] = h < H && a.p.norm ? __ldg(reinterpret_cast<const uint4*>(src + h * in.sh)) : make_uint4(0, 0, 0, 0);
      draw[i] = h < H ? __ldg(reinterpret_cast<const uint4*>(dsrc + (size_t)h * a.N * D)) : make_uint4(0, 0, 0, 0);
    }
    const int pos = a.positions ? __ldg(a.positions + token) : n;
    const bool bad = a.p.dr > 0 && (pos < 0 || pos >= a.p.rope_len);
    Turn t;
    load_turn(a.p, bad ? 0 : pos, l, t);
    float w[8];
    load_weights(a.p, which, l, w);
    __nv_bfloat16* dst =
        static_cast<__nv_bfloat16*>(const_cast<void*>(dx.p)) + b * dx.sb + n * dx.sn + 8 * l;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int h = h0 + i * I::RPW + sub;
      float g[8];
      unpack8(draw[i], g);
      turn_row<true>(a.p, t, g);
      if (a.p.norm) {
        float x[8];
        unpack8(raw[i], x);
        float ss = 0.f, sg = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ss = fmaf(x[e], x[e], ss);
          sg = fmaf(x[e] * w[e], g[e], sg);
        }
#pragma unroll
        for (int off = I::LPR / 2; off > 0; off /= 2) {
          ss += __shfl_xor_sync(0xffffffffu, ss, off);
          sg += __shfl_xor_sync(0xffffffffu, sg, off);
        }
        const float r = rsqrtf(ss * (1.f / D) + a.p.eps);
        const float k = sg * (1.f / D) * r * r;  // mean(g x r) r, per unit of x
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float xr = x[e] * r;
          if (!bad) {  // a row without a position has no gradient
            if (which)
              dw[1][e] = fmaf(g[e], xr, dw[1][e]);
            else
              dw[0][e] = fmaf(g[e], xr, dw[0][e]);
          }
          g[e] = r * (g[e] * w[e] - x[e] * k);
        }
      }
      if (h < H) *reinterpret_cast<uint4*>(dst + h * dx.sh) = bad ? make_uint4(0, 0, 0, 0) : pack8(g);
    }
    if (bad && lane == 0) atomicExch(a.p.status, FA_ERR_DEVICE_INDEX);
  }
  if (a.partial == nullptr) return;
  // rows of the warp, then the warps of the CTA
  __shared__ float acc[kWarps][2][D];
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float v = dw[q][e];
#pragma unroll
      for (int off = I::LPR; off < 32; off *= 2) v += __shfl_xor_sync(0xffffffffu, v, off);
      if (sub == 0) acc[threadIdx.x / 32][q][8 * l + e] = v;
    }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * D; c += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int wp = 0; wp < kWarps; ++wp) v += acc[wp][c / D][c % D];
    a.partial[(size_t)blockIdx.x * 2 * D + c] = v;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Adds the rows of partial sums: one block per 32 columns, 32 threads a column.
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const float* __restrict__ partial, int rows, int d,
                                                            float* dqw, float* dkw) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ float acc[32][33];
  const int x = threadIdx.x % 32, y = threadIdx.x / 32;
  const int col = blockIdx.x * 32 + x;  // of 2 d columns
  float v = 0.f;
  for (int r = y; r < rows; r += 32) v += partial[(size_t)r * 2 * d + col];
  acc[y][x] = v;
  __syncthreads();
  float u = acc[x][y];  // warp y adds column y
#pragma unroll
  for (int off = 16; off > 0; off /= 2) u += __shfl_xor_sync(0xffffffffu, u, off);
  const int c = blockIdx.x * 32 + y;
  if (x == 0) {
    float* out = c < d ? dqw : dkw;
    if (out) out[c < d ? c : c - d] = u;
  }
}

// ----------------------------------------------------------- serving form ----
// The sequence of token t: the last s with cu[s] <= t, found 32 ways at a time
// (whole warp).  -1 in front of the first sequence, S behind the last.
__device__ __forceinline__ int find_sequence(const int* cu, int S, int t) {
  int lo = 0, hi = S + 1;  // the count of entries <= t lies in [lo, hi]
  const int lane = threadIdx.x & 31;
  while (hi - lo > 0) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + (lane + 1) * step - 1;
    const bool below = i < hi && __ldg(cu + i) <= t;
    const int k = __popc(__ballot_sync(0xffffffffu, below));  // whole steps that are <= t
    const int nlo = min(lo + k * step, hi);
    hi = min(nlo + step - 1, hi);
    lo = nlo;
  }
  return lo - 1;
}

// Tokens of a ragged batch: queries to q_out, keys (normed, rotated) and
// values into their pages.  A token's position is its place in its sequence;
// one without a slot (in front of position 0, behind the page table or the
// rotation table, or in a page outside the pool) is not cached, and its query
// row is zero where it has no position.
template <int D>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const AppendLaunch a) {
  using I = Item<D>;
  const int lane = threadIdx.x & 31, l = lane % I::LPR, sub = lane / I::LPR;
  const int cq = (a.Hq + I::kRows - 1) / I::kRows, ck = (a.Hk + I::kRows - 1) / I::kRows;
  const long long item = (long long)blockIdx.x * kWarps + threadIdx.x / 32;
  const long long tok = item / (cq + 2 * ck);
  if (tok >= a.T) return;
  const int t = (int)tok;
  const int chunk = (int)(item - tok * (cq + 2 * ck));
  const int which = chunk < cq ? 0 : chunk < cq + ck ? 1 : 2;  // queries, keys, values
  const int h0 = (chunk - (which == 0 ? 0 : which == 1 ? cq : cq + ck)) * I::kRows;
  const int H = which ? a.Hk : a.Hq;
  const HeadRows in = a.in[which];
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(in.p) + t * in.sn + 8 * l;
  uint4 raw[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int h = h0 + i * I::RPW + sub;
    raw[i] = h < H ? __ldg(reinterpret_cast<const uint4*>(src + h * in.sh)) : make_uint4(0, 0, 0, 0);
  }
  const int s = find_sequence(a.cu_seqlens, a.S, t);
  if (s < 0 || s >= a.S) return;  // a row of no sequence: left as it was
  const long long pos = (long long)__ldg(a.kv_lens + s) - __ldg(a.cu_seqlens + s + 1) + t;
  const bool bad = pos < 0 || pos >= (long long)a.max_pages * a.page_size || (a.p.dr > 0 && pos >= a.p.rope_len);
  __nv_bfloat16* dst = nullptr;
  long long step = 0;
  bool lost = bad;  // no place to write
  if (which == 0) {
    dst = static_cast<__nv_bfloat16*>(a.q_out) + (size_t)t * a.Hq * D + 8 * l;
    step = D;
    lost = false;
  } else if (!bad) {
    const int page = __ldg(a.page_table + (size_t)s * a.max_pages + pos / a.page_size);
    lost = page < 0 || page >= a.num_pages;
    if (!lost) {
      const int kv = which - 1;
      dst = static_cast<__nv_bfloat16*>(a.pages[kv]) + page * a.page_sp[kv] + (pos % a.page_size) * a.page_sr[kv] +
            8 * l;
      step = a.page_sh[kv];
    }
  }
  if ((bad || lost) && lane == 0) atomicExch(a.p.status, FA_ERR_DEVICE_INDEX);
  if (lost) return;
  if (which == 2) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int h = h0 + i * I::RPW + sub;
      if (h < H) *reinterpret_cast<uint4*>(dst + h * step) = raw[i];
    }
    return;
  }
  Turn tn;
  load_turn(a.p, bad ? 0 : (int)pos, l, tn);
  float w[8];
  load_weights(a.p, which, l, w);
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int h = h0 + i * I::RPW + sub;
    float y[8];
    unpack8(raw[i], y);
    if (a.p.norm) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
      const float r = rsqrtf(row_sum<I::LPR>(ss) * (1.f / D) + a.p.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = y[e] * r * w[e];
    }
    turn_row<false>(a.p, tn, y);
    if (h < H) *reinterpret_cast<uint4*>(dst + h * step) = bad ? make_uint4(0, 0, 0, 0) : pack8(y);
  }
}

template <int D>
long long item_blocks(long long tokens, int chunks) {
  return (tokens * chunks + kWarps - 1) / kWarps;
}

template <int D>
int chunks_of(int H) {
  return (H + Item<D>::kRows - 1) / Item<D>::kRows;
}

template <int D>
cudaError_t launch_norm_rope_t(const NormRopeLaunch& a, cudaStream_t stream) {
  const long long blocks = item_blocks<D>((long long)a.B * a.N, chunks_of<D>(a.H[0]) + chunks_of<D>(a.H[1]));
  norm_rope_kernel<D><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_norm_rope_bwd_t(const NormRopeLaunch& a, cudaStream_t stream) {
  const long long blocks = item_blocks<D>((long long)a.B * a.N, chunks_of<D>(a.H[0]) + chunks_of<D>(a.H[1]));
  const long long most = 4ll * a.sms < kNormRopeMaxCtas ? 4ll * a.sms : kNormRopeMaxCtas;
  const int grid = (int)(blocks < most ? blocks : most);
  norm_rope_bwd_kernel<D><<<grid, kThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.partial == nullptr) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * D / 32);
  cfg.blockDim = dim3(1024);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_rope_dw_kernel, static_cast<const float*>(a.partial), grid, D, a.dw[0],
                            a.dw[1]);
}

template <int D>
cudaError_t launch_paged_append_t(const AppendLaunch& a, cudaStream_t stream) {
  const long long blocks = item_blocks<D>(a.T, chunks_of<D>(a.Hq) + 2 * chunks_of<D>(a.Hk));
  paged_append_kernel<D><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeLaunch& a, cudaStream_t stream) {
  return a.p.d == 64 ? launch_norm_rope_t<64>(a, stream) : launch_norm_rope_t<128>(a, stream);
}

cudaError_t launch_norm_rope_bwd(const NormRopeLaunch& a, cudaStream_t stream) {
  return a.p.d == 64 ? launch_norm_rope_bwd_t<64>(a, stream) : launch_norm_rope_bwd_t<128>(a, stream);
}

cudaError_t launch_paged_append(const AppendLaunch& a, cudaStream_t stream) {
  return a.p.d == 64 ? launch_paged_append_t<64>(a, stream) : launch_paged_append_t<128>(a, stream);
}

}  // namespace fa
