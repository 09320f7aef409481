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
// shuffle), a warp takes 32 / (d / 8) rows at once and STEPS such steps: a
// chunk of one token's heads, so that the token's cosines and sines are loaded
// once for all of them.  A CTA takes one chunk of neighbouring tokens (its
// warps one after the other, each a few), the CTAs of a token's chunks are
// neighbours, so its table row comes from the caches after the first.  Many
// short CTAs: a grid of resident ones that walk all tokens measured 91 to 111
// us, with loads in flight through registers or cp.async, against 85 (0.54 GB,
// 79 us at the copy rate).
// The input may be any strided view (a slice of the projection's output); the
// output is the contiguous [B, H, N, d] that the attention kernels read, so the
// transposition costs no pass of its own.  Everything between load and store is
// fp32; the one rounding is the stored bf16 (the weights' gradient stays fp32).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_norm_rope.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// A thread's 8 columns of a row as four pairs (one instruction for two elements).
using Row = uint64_t[4];

__device__ __forceinline__ uint64_t unpack2(uint32_t v) {
  return f2_pack(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}

__device__ __forceinline__ void unpack8(const uint4& u, Row& x) {
  x[0] = unpack2(u.x), x[1] = unpack2(u.y), x[2] = unpack2(u.z), x[3] = unpack2(u.w);
}

__device__ __forceinline__ uint32_t pack2(uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  return pack_bf16x2(lo, hi);
}

__device__ __forceinline__ uint4 pack8(const Row& x) {
  return make_uint4(pack2(x[0]), pack2(x[1]), pack2(x[2]), pack2(x[3]));
}

__device__ __forceinline__ void load8(const float* p, Row& x) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = f2_pack(a.x, a.y), x[1] = f2_pack(a.z, a.w), x[2] = f2_pack(b.x, b.y), x[3] = f2_pack(b.z, b.w);
}

// Weights of the 8 columns of lane l of a row.
__device__ __forceinline__ void load_weights(const NormRopeParams& p, int which, int l, Row& w) {
  const void* src = p.w[which];
  if (src == nullptr) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = f2_pack(1.f, 1.f);
  } else if (p.weights_f32) {
    load8(static_cast<const float*>(src) + 8 * l, w);
  } else {
    unpack8(__ldg(static_cast<const uint4*>(src) + l), w);
  }
}

__device__ __forceinline__ float pair_sum(uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  return lo + hi;
}

// Where a lane stands in its row.  The rotation is z = y * c + other * s:
// `other` is the partner column's element (dr / 16 lanes away for split pairs
// (i, i + dr / 2), the neighbour within the pair for (2i, 2i + 1): INTER), and
// s carries a sign.  Columns that pass have c = 1, s = 0 and an `other` of zero.
template <int D, bool INTER>
struct Lane {
  int l;         // of the row's D / 8
  int partner;   // the lane that holds the partner columns
  int angle;     // its first angle
  bool turned, first;
  __device__ __forceinline__ Lane(const NormRopeParams& p, int lane) {
    const int hl = p.dr / 16;
    l = lane % (D / 8);
    turned = 8 * l < p.dr;
    first = l < hl;
    partner = INTER || !turned ? l : first ? l + hl : l - hl;
    angle = INTER ? 4 * l : 8 * (first ? l : l - hl);
  }
};

constexpr uint64_t kSign2 = 0x8000000080000000ull;

// Cosines and sines of the 8 columns at a table row, without sign.
template <int D, bool INTER>
__device__ __forceinline__ void load_angles(const NormRopeParams& p, const Lane<D, INTER>& ln, int pos, Row& c,
                                            Row& s) {
  if (!ln.turned) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = f2_pack(1.f, 1.f), s[i] = 0;
    return;
  }
  const float* row = p.rope + (size_t)pos * p.dr + ln.angle;
  const float* sines = row + p.dr / 2;
  if constexpr (INTER) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(row)), b = __ldg(reinterpret_cast<const float4*>(sines));
    c[0] = f2_pack(a.x, a.x), c[1] = f2_pack(a.y, a.y), c[2] = f2_pack(a.z, a.z), c[3] = f2_pack(a.w, a.w);
    s[0] = f2_pack(b.x, b.x), s[1] = f2_pack(b.y, b.y), s[2] = f2_pack(b.z, b.z), s[3] = f2_pack(b.w, b.w);
  } else {
    load8(row, c);
    load8(sines, s);
  }
}

// What the sines are multiplied with: the sign of z_a = y_a c - y_b s, z_b = y_b c + y_a s
// (BACK: the other one) times `w`, the partner columns' weights.
template <int D, bool INTER, bool BACK>
__device__ __forceinline__ void signed_row(const Lane<D, INTER>& ln, Row& w) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] ^= INTER ? (BACK ? 0x8000000000000000ull : 0x80000000ull) : ln.first != BACK ? kSign2 : 0;
}

// The partner columns of 8 bf16 columns (every lane of the warp calls it).
template <int D, bool INTER>
__device__ __forceinline__ uint4 partner_of(const NormRopeParams& p, const Lane<D, INTER>& ln, const uint4& v) {
  uint4 o;
  if constexpr (INTER) {
    o = make_uint4(__byte_perm(v.x, 0, 0x1032), __byte_perm(v.y, 0, 0x1032), __byte_perm(v.z, 0, 0x1032),
                   __byte_perm(v.w, 0, 0x1032));
  } else {
    o.x = __shfl_sync(0xffffffffu, v.x, ln.partner, D / 8);
    o.y = __shfl_sync(0xffffffffu, v.y, ln.partner, D / 8);
    o.z = __shfl_sync(0xffffffffu, v.z, ln.partner, D / 8);
    o.w = __shfl_sync(0xffffffffu, v.w, ln.partner, D / 8);
  }
  if (p.dr < D && !ln.turned) o = make_uint4(0, 0, 0, 0);
  return o;
}

// The norm's weights folded into the rotation, z = r (x c + other s): c is
// multiplied with the columns' weights, s with its sign and the partner columns'.
template <int D, bool INTER>
struct Factors {
  Row w, o;
  __device__ __forceinline__ void load(const NormRopeParams& p, const Lane<D, INTER>& ln, int which) {
    if (p.norm) {
      load_weights(p, which, ln.l, w);
      load_weights(p, which, ln.partner, o);
      if constexpr (INTER) {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = (o[i] << 32) | (o[i] >> 32);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = o[i] = f2_pack(1.f, 1.f);
    }
    signed_row<D, INTER, false>(ln, o);
  }
  __device__ __forceinline__ void fold(Row& c, Row& s) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = f2_mul(c[i], w[i]), s[i] = f2_mul(s[i], o[i]);
  }
};

// 1 / rms of STEPS (one, two or four) rows at once.  The lanes of a row exchange
// halves of the sums instead of all of them: after one or two rounds each lane
// goes on with one row's, so the reduction and the root are done once.
template <int D, int STEPS>
__device__ __forceinline__ void inverse_rms(const uint4 (&raw)[STEPS], int l, float eps, float (&r)[STEPS]) {
  static_assert(STEPS == 1 || STEPS == 2 || STEPS == 4, "one, two or four rows");
  float v[STEPS];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    Row x;
    unpack8(raw[i], x);
    uint64_t ss = f2_mul(x[0], x[0]);
#pragma unroll
    for (int e = 1; e < 4; ++e) ss = f2_fma(x[e], x[e], ss);
    v[i] = pair_sum(ss);
  }
  const bool b0 = l & 1, b1 = l & 2;
  float u;
  if constexpr (STEPS == 4) {
    const float t0 = (b0 ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, b0 ? v[0] : v[2], 1);
    const float t1 = (b0 ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, b0 ? v[1] : v[3], 1);
    u = (b1 ? t1 : t0) + __shfl_xor_sync(0xffffffffu, b1 ? t0 : t1, 2);  // row 2 b0 + b1
  } else if constexpr (STEPS == 2) {
    u = (b0 ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, b0 ? v[0] : v[1], 1);  // row b0
    u += __shfl_xor_sync(0xffffffffu, u, 2);
  } else {
    u = v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
    u += __shfl_xor_sync(0xffffffffu, u, 2);
  }
#pragma unroll
  for (int off = 4; off < D / 8; off *= 2) u += __shfl_xor_sync(0xffffffffu, u, off);
  u = rsqrtf(u * (1.f / D) + eps);
#pragma unroll
  for (int i = 0; i < STEPS; ++i)
    r[i] = STEPS == 1 ? u : __shfl_sync(0xffffffffu, u, STEPS == 4 ? (i >> 1) | ((i & 1) << 1) : i, D / 8);
}

// A row's 8 columns of this lane, turned and scaled (c and s folded).
template <int D, bool INTER>
__device__ __forceinline__ uint4 turn_row(const NormRopeParams& p, const Lane<D, INTER>& ln, const Row& c, const Row& s,
                                          const uint4& raw, float r) {
  Row x, o;
  unpack8(raw, x);
  unpack8(partner_of<D, INTER>(p, ln, raw), o);
  const uint64_t r2 = f2_pack(r, r);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = f2_mul(f2_fma(o[i], s[i], f2_mul(x[i], c[i])), r2);
  return pack8(x);
}

// The gradient of a row's 8 columns: dz -> dx (c and s of minus the angle), and its part of dw added to `dw` if it
// counts.  One that does not, without a position or not there at all, comes with zeros for x and dz: then only its
// 1 / rms may be infinite (eps = 0), and is left out.
template <int D, bool INTER>
__device__ __forceinline__ uint4 turn_row_back(const NormRopeParams& p, const Lane<D, INTER>& ln, const Row& c,
                                               const Row& s, const Row& w, const uint4& raw, const uint4& dz,
                                               bool counts, Row& dw) {
  Row g, o;
  unpack8(dz, g);
  unpack8(partner_of<D, INTER>(p, ln, dz), o);
#pragma unroll
  for (int e = 0; e < 4; ++e) g[e] = f2_fma(o[e], s[e], f2_mul(g[e], c[e]));  // dy
  if (p.norm) {
    Row x, gw;
    unpack8(raw, x);
    uint64_t ss2 = 0, sg2 = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      gw[e] = f2_mul(g[e], w[e]);
      ss2 = f2_fma(x[e], x[e], ss2);
      sg2 = f2_fma(x[e], gw[e], sg2);
    }
    float ss = pair_sum(ss2), sg = pair_sum(sg2);
    // both sums at once: even lanes go on with one, odd lanes with the other
    const bool odd = ln.l & 1;
    float v = (odd ? sg : ss) + __shfl_xor_sync(0xffffffffu, odd ? ss : sg, 1);
#pragma unroll
    for (int off = D / 16; off > 1; off /= 2) v += __shfl_xor_sync(0xffffffffu, v, off);
    const float u = __shfl_xor_sync(0xffffffffu, v, 1);
    ss = odd ? u : v;
    sg = odd ? v : u;
    const float r = rsqrtf(ss * (1.f / D) + p.eps);
    const float k = -sg * (1.f / D) * r * r * r;  // -mean(g x r) r^2, per unit of x
    const float rw = counts ? r : 0.f;
    const uint64_t r2 = f2_pack(r, r), k2 = f2_pack(k, k), rw2 = f2_pack(rw, rw);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      dw[e] = f2_fma(g[e], f2_mul(x[e], rw2), dw[e]);
      g[e] = f2_fma(x[e], k2, f2_mul(gw[e], r2));
    }
  }
  return pack8(g);
}

// A CTA's sums of the weights' gradients: rows of the warp, then its warps.
template <int D>
__device__ __forceinline__ void store_partial(const Row& dw, int l, int sub, float* partial) {
  constexpr int LPR = D / 8;
  __shared__ float acc[kWarps][D];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float lo, hi;
    f2_unpack(dw[e], lo, hi);
#pragma unroll
    for (int off = LPR; off < 32; off *= 2) {
      lo += __shfl_xor_sync(0xffffffffu, lo, off);
      hi += __shfl_xor_sync(0xffffffffu, hi, off);
    }
    if (sub == 0) acc[threadIdx.x / 32][8 * l + 2 * e] = lo, acc[threadIdx.x / 32][8 * l + 2 * e + 1] = hi;
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float v = 0.f;
#pragma unroll
    for (int wp = 0; wp < kWarps; ++wp) v += acc[wp][threadIdx.x];
    partial[(size_t)blockIdx.x * D + threadIdx.x] = v;
  }
}

// A chunk: up to kRows heads of one token.
template <int D, int STEPS>
struct Chunk {
  static constexpr int LPR = D / 8;           // lanes a row
  static constexpr int RPW = 32 / LPR;        // rows a warp and step
  static constexpr int kRows = RPW * STEPS;   // heads a chunk
  __host__ __device__ static int of(int H) { return (H + kRows - 1) / kRows; }
};
// CTAs an SM of the forward: 80 registers at three, in which the kernels of split
// pairs do not spill (those of neighbouring pairs 4 to 12 bytes a thread); four and
// five measured 89 and 110 us against 85 (B = 64, N = 1024, 16 + 16 heads, d = 64).
constexpr int kFwdCtas = 3;

// ----------------------------------------------------------------- forward ---
template <int D, bool INTER, int STEPS>
__global__ void __launch_bounds__(kThreads, kFwdCtas) norm_rope_kernel(const NormRopeLaunch a) {
  using I = Chunk<D, STEPS>;
  const int lane = threadIdx.x & 31, sub = lane / I::LPR;
  const Lane<D, INTER> ln(a.p, lane);
  const unsigned cq = I::of(a.H[0]);
  const unsigned group = a.by_chunks.div(blockIdx.x), chunk = blockIdx.x - group * a.by_chunks.d;
  const int which = chunk >= cq, H = a.H[which];
  const int h0 = (which ? chunk - cq : chunk) * I::kRows + sub;  // this lane's first head
  const HeadRows in = a.in[which];
  const __nv_bfloat16* base = static_cast<const __nv_bfloat16*>(in.p) + h0 * in.sh + 8 * ln.l;
  const long long hop = in.sh * I::RPW;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out[which]) + (size_t)h0 * a.N * D + 8 * ln.l;
  const size_t out_hop = (size_t)a.N * D * I::RPW;
  Factors<D, INTER> f;
  f.load(a.p, ln, which);
  unsigned token = group * a.walk * kWarps + threadIdx.x / 32;
#pragma unroll 1
  for (int k = 0; k < a.walk; ++k, token += kWarps) {
    if (token >= (unsigned)a.B * a.N) return;
    const unsigned b = a.by_n.div(token), n = token - b * a.N;
    const __nv_bfloat16* src = base + b * in.sb + n * in.sn;
    uint4 raw[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i, src += hop)
      raw[i] = h0 + i * I::RPW < H ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
    const int pos = a.positions ? __ldg(a.positions + token) : (int)n;
    const bool bad = a.p.dr > 0 && (pos < 0 || pos >= a.p.rope_len);
    Row c, s;
    load_angles<D, INTER>(a.p, ln, bad ? 0 : pos, c, s);
    f.fold(c, s);
    float r[STEPS];
    if (a.p.norm) inverse_rms<D, STEPS>(raw, ln.l, a.p.eps, r);
    __nv_bfloat16* dst = out + ((size_t)b * H * a.N + n) * D;
#pragma unroll
    for (int i = 0; i < STEPS; ++i, dst += out_hop) {
      const uint4 z = turn_row<D, INTER>(a.p, ln, c, s, raw[i], a.p.norm ? r[i] : 1.f);
      if (h0 + i * I::RPW < H) *reinterpret_cast<uint4*>(dst) = bad ? make_uint4(0, 0, 0, 0) : z;
    }
    if (bad && lane == 0) record_index(a.p.status);
  }
}

// ---------------------------------------------------------------- backward ---
// Bound by the loads in flight: the rows of x and dz of four steps take 119 registers
// a thread, two CTAs an SM (B = 64, N = 1024, 16 + 16 heads, d = 64: 153 us, 5.3 of
// 6.8 TB/s; two steps and three CTAs an SM, which spill 28 to 40 bytes a thread, are
// slower for many heads, steps_for()).
// The weights' gradients of a thread's 8 columns stay in registers over all its
// tokens; a CTA adds up its warps and writes one row of partial sums, and a
// second kernel adds those in a fixed order: no atomics, the same bits on every
// run.
template <int D, bool INTER, int STEPS>
__global__ void __launch_bounds__(kThreads, STEPS == 4 ? 2 : 3) norm_rope_bwd_kernel(const NormRopeLaunch a) {
  using I = Chunk<D, STEPS>;
  const int lane = threadIdx.x & 31, sub = lane / I::LPR;
  const Lane<D, INTER> ln(a.p, lane);
  const unsigned cq = I::of(a.H[0]);
  const unsigned group = a.by_chunks.div(blockIdx.x), chunk = blockIdx.x - group * a.by_chunks.d;
  const int which = chunk >= cq, H = a.H[which];
  const int h0 = (which ? chunk - cq : chunk) * I::kRows + sub;
  const HeadRows in = a.in[which], dx = a.dx[which];
  const __nv_bfloat16* base = static_cast<const __nv_bfloat16*>(in.p) + h0 * in.sh + 8 * ln.l;
  const __nv_bfloat16* dbase = static_cast<const __nv_bfloat16*>(a.dout[which]) + (size_t)h0 * a.N * D + 8 * ln.l;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(const_cast<void*>(dx.p)) + h0 * dx.sh + 8 * ln.l;
  const long long hop = in.sh * I::RPW, out_hop = dx.sh * I::RPW;
  const size_t dhop = (size_t)a.N * D * I::RPW;
  Row w, dw = {0, 0, 0, 0};
  load_weights(a.p, which, ln.l, w);
  unsigned token = group * a.walk * kWarps + threadIdx.x / 32;
#pragma unroll 1
  for (int k = 0; k < a.walk && token < (unsigned)a.B * a.N; ++k, token += kWarps) {
    const unsigned b = a.by_n.div(token), n = token - b * a.N;
    const __nv_bfloat16* src = base + b * in.sb + n * in.sn;
    const __nv_bfloat16* dsrc = dbase + ((size_t)b * H * a.N + n) * D;
    uint4 raw[STEPS], dz[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i, src += hop, dsrc += dhop) {
      const bool row = h0 + i * I::RPW < H;
      raw[i] = row && a.p.norm ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
      dz[i] = row ? __ldg(reinterpret_cast<const uint4*>(dsrc)) : make_uint4(0, 0, 0, 0);
    }
    const int pos = a.positions ? __ldg(a.positions + token) : (int)n;
    const bool bad = a.p.dr > 0 && (pos < 0 || pos >= a.p.rope_len);
    Row c, s;
    load_angles<D, INTER>(a.p, ln, bad ? 0 : pos, c, s);
    signed_row<D, INTER, true>(ln, s);
    if (bad) {  // whatever these rows hold (NaN, if nothing was written there) is not part of any sum
#pragma unroll
      for (int i = 0; i < STEPS; ++i) raw[i] = dz[i] = make_uint4(0, 0, 0, 0);
    }
    __nv_bfloat16* dst = out + b * dx.sb + n * dx.sn;
#pragma unroll
    for (int i = 0; i < STEPS; ++i, dst += out_hop) {
      const uint4 g = turn_row_back<D, INTER>(a.p, ln, c, s, w, raw[i], dz[i],
                                                         !bad && h0 + i * I::RPW < H, dw);
      if (h0 + i * I::RPW < H) *reinterpret_cast<uint4*>(dst) = bad ? make_uint4(0, 0, 0, 0) : g;
    }
    if (bad && lane == 0) record_index(a.p.status);
  }
  if (a.partial != nullptr) store_partial<D>(dw, ln.l, sub, a.partial);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ------------------------------------------------------- few heads a token ---
// The same two passes where a chunk of heads would leave most of a warp idle
// (one query and one key head fill 2 of 32 rows at d = 64: 597 us where the
// copy rate allows 60): the rows of a tensor in order of token and head, a warp
// takes neighbouring ones of any tokens, and each row loads its own angles.
// The first q_blocks CTAs take the queries, the others the keys.
constexpr int kRowSteps = 2;

template <int D>
struct RowWalk {
  static constexpr int RPW = 256 / D;                            // rows a warp and step
  static constexpr int kBlockRows = kWarps * RPW * kRowSteps;    // a CTA and turn
  long long rows;      // of the tensor
  long long first;     // this CTA's first row
  long long token0;    // its token
  unsigned head0;      // and head
  __device__ __forceinline__ RowWalk(const NormRopeLaunch& a, int which, unsigned block) {
    rows = (long long)a.B * a.N * a.H[which];
    first = (long long)block * a.walk * kBlockRows;
    token0 = first / a.H[which];
    head0 = (unsigned)(first - token0 * a.H[which]);
  }
};

template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads, 3) norm_rope_rows_kernel(const NormRopeLaunch a) {
  using W = RowWalk<D>;
  const int lane = threadIdx.x & 31, sub = lane / (D / 8);
  const Lane<D, INTER> ln(a.p, lane);
  const int which = blockIdx.x >= a.q_blocks;
  const W walk(a, which, which ? blockIdx.x - a.q_blocks : blockIdx.x);
  const HeadRows in = a.in[which];
  const int H = a.H[which];
  Factors<D, INTER> f;
  f.load(a.p, ln, which);
#pragma unroll 1
  for (int k = 0; k < a.walk; ++k) {
    const unsigned at = (k * kWarps + threadIdx.x / 32) * (W::RPW * kRowSteps) + sub;  // behind walk.first
    if (walk.first + at - sub >= walk.rows) return;
    uint4 raw[kRowSteps];
    int pos[kRowSteps];
    size_t to[kRowSteps];
    bool there[kRowSteps], bad[kRowSteps];
#pragma unroll
    for (int i = 0; i < kRowSteps; ++i) {
      const unsigned o = at + i * W::RPW;
      there[i] = walk.first + o < walk.rows;
      const unsigned t = a.by_h[which].div(walk.head0 + o);
      const unsigned h = walk.head0 + o - t * H, token = there[i] ? (unsigned)(walk.token0 + t) : 0;
      const unsigned b = a.by_n.div(token), n = token - b * a.N;
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(in.p) + b * in.sb + n * in.sn + h * in.sh + 8 * ln.l;
      raw[i] = there[i] ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
      pos[i] = a.positions ? __ldg(a.positions + token) : (int)n;
      to[i] = (((size_t)b * H + h) * a.N + n) * D + 8 * ln.l;
    }
    float r[kRowSteps];
    if (a.p.norm) inverse_rms<D, kRowSteps>(raw, ln.l, a.p.eps, r);
#pragma unroll
    for (int i = 0; i < kRowSteps; ++i) {
      bad[i] = a.p.dr > 0 && (pos[i] < 0 || pos[i] >= a.p.rope_len);
      Row c, s;
      load_angles<D, INTER>(a.p, ln, bad[i] ? 0 : pos[i], c, s);
      f.fold(c, s);
      const uint4 z = turn_row<D, INTER>(a.p, ln, c, s, raw[i], a.p.norm ? r[i] : 1.f);
      if (!there[i]) continue;
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out[which]) + to[i]) =
          bad[i] ? make_uint4(0, 0, 0, 0) : z;
      if (bad[i] && ln.l == 0) record_index(a.p.status);
    }
  }
}

template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads, 3) norm_rope_rows_bwd_kernel(const NormRopeLaunch a) {
  using W = RowWalk<D>;
  const int lane = threadIdx.x & 31, sub = lane / (D / 8);
  const Lane<D, INTER> ln(a.p, lane);
  const int which = blockIdx.x >= a.q_blocks;
  const W walk(a, which, which ? blockIdx.x - a.q_blocks : blockIdx.x);
  const HeadRows in = a.in[which], dx = a.dx[which];
  const int H = a.H[which];
  Row w, dw = {0, 0, 0, 0};
  load_weights(a.p, which, ln.l, w);
#pragma unroll 1
  for (int k = 0; k < a.walk; ++k) {
    const unsigned at = (k * kWarps + threadIdx.x / 32) * (W::RPW * kRowSteps) + sub;
    if (walk.first + at - sub >= walk.rows) break;
    uint4 raw[kRowSteps], dz[kRowSteps];
    int pos[kRowSteps];
    __nv_bfloat16* to[kRowSteps];
    bool there[kRowSteps];
#pragma unroll
    for (int i = 0; i < kRowSteps; ++i) {
      const unsigned o = at + i * W::RPW;
      there[i] = walk.first + o < walk.rows;
      const unsigned t = a.by_h[which].div(walk.head0 + o);
      const unsigned h = walk.head0 + o - t * H, token = there[i] ? (unsigned)(walk.token0 + t) : 0;
      const unsigned b = a.by_n.div(token), n = token - b * a.N;
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(in.p) + b * in.sb + n * in.sn + h * in.sh + 8 * ln.l;
      const __nv_bfloat16* dsrc =
          static_cast<const __nv_bfloat16*>(a.dout[which]) + (((size_t)b * H + h) * a.N + n) * D + 8 * ln.l;
      raw[i] = there[i] && a.p.norm ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
      dz[i] = there[i] ? __ldg(reinterpret_cast<const uint4*>(dsrc)) : make_uint4(0, 0, 0, 0);
      pos[i] = a.positions ? __ldg(a.positions + token) : (int)n;
      to[i] = static_cast<__nv_bfloat16*>(const_cast<void*>(dx.p)) + b * dx.sb + n * dx.sn + h * dx.sh + 8 * ln.l;
    }
#pragma unroll
    for (int i = 0; i < kRowSteps; ++i) {
      const bool bad = a.p.dr > 0 && (pos[i] < 0 || pos[i] >= a.p.rope_len);
      Row c, s;
      load_angles<D, INTER>(a.p, ln, bad ? 0 : pos[i], c, s);
      signed_row<D, INTER, true>(ln, s);
      if (bad) raw[i] = dz[i] = make_uint4(0, 0, 0, 0);  // as in norm_rope_bwd_kernel
      const uint4 g = turn_row_back<D, INTER>(a.p, ln, c, s, w, raw[i], dz[i], !bad && there[i], dw);
      if (!there[i]) continue;
      *reinterpret_cast<uint4*>(to[i]) = bad ? make_uint4(0, 0, 0, 0) : g;
      if (bad && ln.l == 0) record_index(a.p.status);
    }
  }
  if (a.partial != nullptr) store_partial<D>(dw, ln.l, sub, a.partial);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Adds the rows of partial sums, those of the queries' CTAs and those of the
// keys': row r is a query row if r mod `period` < `cq`.  8 columns a block, 128
// threads a column.
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const float* __restrict__ partial, int rows, int d,
                                                            int cq, int period, float* dqw, float* dkw) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ float acc[32][8];
  const int x = threadIdx.x % 8, y = threadIdx.x / 8;
  const int col = blockIdx.x * 8 + x, which = blockIdx.y;
  const int first = which ? cq : 0, width = which ? period - cq : cq;
  const int count = rows / period * width;
  float v = 0.f;
#pragma unroll 4
  for (int i = y; i < count; i += 128) v += partial[(size_t)(i / width * period + first + i % width) * d + col];
#pragma unroll
  for (int off = 8; off < 32; off *= 2) v += __shfl_xor_sync(0xffffffffu, v, off);
  if (threadIdx.x % 32 < 8) acc[threadIdx.x / 32][x] = v;
  __syncthreads();
  if (threadIdx.x < 8) {
    float u = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) u += acc[i][x];
    float* out = which ? dkw : dqw;
    if (out) out[col] = u;
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
// A warp takes one token: one chunk of its heads, or (`span`) all of them, so
// that the search for its sequence and slot is made once.  8207 tokens, 32 + 8 heads,
// d = 128, pages of 16 take 39 us (5.2 TB/s; the copy rate allows 30): issue slots,
// part of them for what is done again for each chunk of a token's heads (angles and
// weights loaded and folded; at four steps 60 to 68 bytes a thread spilled at the 64
// registers of four CTAs an SM), and a chunk's rows are asked for only behind the
// stores of the last.  64 single tokens take 3.9 us, the chain search - page entry - row.
template <int D, bool INTER, int STEPS>
__global__ void __launch_bounds__(kThreads, 4) paged_append_kernel(const AppendLaunch a) {
  using I = Chunk<D, STEPS>;
  const int lane = threadIdx.x & 31, sub = lane / I::LPR;
  const Lane<D, INTER> ln(a.p, lane);
  const unsigned cq = I::of(a.Hq), ck = I::of(a.Hk);
  const unsigned group = a.span ? blockIdx.x : a.by_chunks.div(blockIdx.x);
  const unsigned token = group * kWarps + threadIdx.x / 32;
  if (token >= (unsigned)a.T) return;
  const int t = (int)token;
  uint4 raw[STEPS];
  auto load = [&](unsigned chunk) {  // 0 .. cq: queries, then keys, then values
    const int which = chunk < cq ? 0 : chunk < cq + ck ? 1 : 2;
    const int h0 = (chunk - (which == 0 ? 0 : which == 1 ? cq : cq + ck)) * I::kRows + sub, H = which ? a.Hk : a.Hq;
    const HeadRows in = a.in[which];
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(in.p) + t * in.sn + h0 * in.sh + 8 * ln.l;
    const long long hop = in.sh * I::RPW;
#pragma unroll
    for (int i = 0; i < STEPS; ++i, src += hop)
      raw[i] = h0 + i * I::RPW < H ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
  };
  unsigned chunk = a.span ? 0 : blockIdx.x - group * a.by_chunks.d;
  const unsigned end = a.span ? cq + 2 * ck : chunk + 1;
  load(chunk);
  const int sq = find_sequence(a.cu_seqlens, a.S, t);
  if (sq < 0 || sq >= a.S) return;  // a row of no sequence: left as it was
  const long long pos = (long long)__ldg(a.kv_lens + sq) - __ldg(a.cu_seqlens + sq + 1) + t;
  const int cap = a.max_pages << a.page_log2;
  const bool bad = pos < 0 || pos >= cap || (a.p.dr > 0 && pos >= a.p.rope_len);
  const int at = bad ? 0 : (int)pos;
  const int page = bad || end <= cq ? -1 : __ldg(a.page_table + (size_t)sq * a.max_pages + (at >> a.page_log2));
  const bool lost = page < 0 || page >= a.num_pages;  // no slot
  if ((bad || (lost && end > cq)) && lane == 0) record_index(a.p.status);
#pragma unroll 1
  while (true) {
    const int which = chunk < cq ? 0 : chunk < cq + ck ? 1 : 2;
    const int h0 = (chunk - (which == 0 ? 0 : which == 1 ? cq : cq + ck)) * I::kRows + sub, H = which ? a.Hk : a.Hq;
    if (which > 0 && lost) return;
    __nv_bfloat16* dst;
    long long hop;
    if (which == 0) {
      dst = static_cast<__nv_bfloat16*>(a.q_out) + (size_t)t * a.Hq * D;
      hop = D;
    } else {
      dst = static_cast<__nv_bfloat16*>(a.pages[which - 1]) + page * a.page_sp[which - 1] +
            (at & ((1 << a.page_log2) - 1)) * a.page_sr[which - 1];
      hop = a.page_sh[which - 1];
    }
    dst += h0 * hop + 8 * ln.l;
    hop *= I::RPW;
    if (which == 2) {
#pragma unroll
      for (int i = 0; i < STEPS; ++i, dst += hop)
        if (h0 + i * I::RPW < H) *reinterpret_cast<uint4*>(dst) = raw[i];
    } else {
      Row c, s;
      load_angles<D, INTER>(a.p, ln, at, c, s);
      Factors<D, INTER> f;
      f.load(a.p, ln, which);
      f.fold(c, s);
      float r[STEPS];
      if (a.p.norm) inverse_rms<D, STEPS>(raw, ln.l, a.p.eps, r);
#pragma unroll
      for (int i = 0; i < STEPS; ++i, dst += hop) {
        const uint4 z = turn_row<D, INTER>(a.p, ln, c, s, raw[i], a.p.norm ? r[i] : 1.f);
        if (h0 + i * I::RPW < H) *reinterpret_cast<uint4*>(dst) = bad ? make_uint4(0, 0, 0, 0) : z;
      }
    }
    if (++chunk == end) return;
    load(chunk);
  }
}

unsigned token_groups(long long tokens) { return (unsigned)((tokens + kWarps - 1) / kWarps); }

// Tokens a warp of the forward walks: up to four, as long as the device gets
// two rounds of CTAs.  One token a warp spends as much on its own set-up as on
// the rows: 94 us against 85 at four (the sizes above); more leave a tail.
int forward_walk(unsigned groups, int chunks, int sms) {
  int walk = 1;
  while (walk < 4 && (long long)groups * chunks >= 2ll * walk * 2 * kFwdCtas * sms) walk *= 2;
  return walk;
}

// Steps of a chunk (4, 2 or 1), or 0 for row by row: the cheapest for these
// heads.  Costs of a chunk and of a step of the row kernels, from times with
// 1 to 40 heads at d = 64 and 128 (nanoseconds x 100 a warp's chunk on the
// whole device): a chunk's set-up weighs more than its rows, so empty rows cost
// little at four steps, and few heads gain by fewer steps or none.  16 + 16 heads,
// d = 64, 32000 tokens: 45 us at four steps, 61 at two, 77 row by row; 1 + 1 heads,
// 400000 tokens: 365, 319, 72.
template <int D>
int steps_for(int Hq, int Hk, int keys, const int (&cost)[4]) {  // of 4, 2, 1 steps, of a row step (0: not built)
  const int of[3] = {Chunk<D, 4>::of(Hq) + keys * Chunk<D, 4>::of(Hk), Chunk<D, 2>::of(Hq) + keys * Chunk<D, 2>::of(Hk),
                     Chunk<D, 1>::of(Hq) + keys * Chunk<D, 1>::of(Hk)};
  int best = 0, least = cost[3] > 0 ? cost[3] * (Hq + Hk) / RowWalk<D>::RPW : 1 << 30;
  for (int i = 0; i < 3; ++i)
    if (cost[i] > 0 && cost[i] * of[i] <= least) least = cost[i] * of[i], best = 4 >> i;
  return best;
}

// Turns of a CTA that walks rows: `most` CTAs at most, the first q_blocks for the queries.
template <int D>
unsigned row_blocks(NormRopeLaunch* a, long long most, int max_walk) {
  const long long tokens = (long long)a->B * a->N, turns = RowWalk<D>::kBlockRows;
  auto blocks = [&](int which, long long walk) {
    return (tokens * a->H[which] + walk * turns - 1) / (walk * turns);
  };
  long long walk = 1;
  while (blocks(0, walk) + blocks(1, walk) > most && (max_walk == 0 || walk < max_walk)) walk *= 2;
  a->walk = (int)walk;
  a->q_blocks = (unsigned)blocks(0, walk);
  a->by_n = FastDiv(a->N);
  a->by_h[0] = FastDiv(a->H[0]);
  a->by_h[1] = FastDiv(a->H[1]);
  return (unsigned)(a->q_blocks + blocks(1, walk));
}

template <int D, bool INTER, int STEPS>
void launch_chunks(NormRopeLaunch a, cudaStream_t stream) {
  using I = Chunk<D, STEPS>;
  const unsigned chunks = I::of(a.H[0]) + I::of(a.H[1]), groups = token_groups((long long)a.B * a.N);
  a.walk = forward_walk(groups, chunks, a.sms);
  a.by_n = FastDiv(a.N);
  a.by_chunks = FastDiv(chunks);
  norm_rope_kernel<D, INTER, STEPS><<<(groups + a.walk - 1) / a.walk * chunks, kThreads, 0, stream>>>(a);
}

template <int D, bool INTER>
cudaError_t launch_norm_rope_t(NormRopeLaunch a, cudaStream_t stream) {
  constexpr int kCost[4] = {46, 40, 0, 34};
  switch (steps_for<D>(a.H[0], a.H[1], 1, kCost)) {
    case 4:
      launch_chunks<D, INTER, 4>(a, stream);
      break;
    case 2:
      launch_chunks<D, INTER, 2>(a, stream);
      break;
    default:
      const unsigned blocks = row_blocks<D>(&a, 2ll * kFwdCtas * a.sms, 4);
      norm_rope_rows_kernel<D, INTER><<<blocks, kThreads, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

// Launches, and returns the grid; *cq of every *period rows of partial sums are the queries'.
template <int D, bool INTER, int STEPS>
int launch_bwd_chunks(NormRopeLaunch a, int* cq, int* period, cudaStream_t stream) {
  using I = Chunk<D, STEPS>;
  *cq = I::of(a.H[0]);
  *period = *cq + I::of(a.H[1]);
  const unsigned groups = token_groups((long long)a.B * a.N);
  const unsigned runs = kNormRopeMaxCtas / *period;  // of tokens, at most: a row of partial sums for each
  static_assert(2 * kNormRopeMaxHeads / I::kRows <= kNormRopeMaxCtas, "a run at least");
  a.walk = (groups + runs - 1) / runs;
  a.by_n = FastDiv(a.N);
  a.by_chunks = FastDiv(*period);
  const int grid = (groups + a.walk - 1) / a.walk * *period;
  norm_rope_bwd_kernel<D, INTER, STEPS><<<grid, kThreads, 0, stream>>>(a);
  return grid;
}

template <int D, bool INTER>
cudaError_t launch_norm_rope_bwd_t(NormRopeLaunch a, cudaStream_t stream) {
  constexpr int kCost[4] = {110, 65, 40, 46};
  int grid, cq, period;
  switch (steps_for<D>(a.H[0], a.H[1], 1, kCost)) {
    case 4:
      grid = launch_bwd_chunks<D, INTER, 4>(a, &cq, &period, stream);
      break;
    case 2:
      grid = launch_bwd_chunks<D, INTER, 2>(a, &cq, &period, stream);
      break;
    case 1:
      grid = launch_bwd_chunks<D, INTER, 1>(a, &cq, &period, stream);
      break;
    default:
      grid = (int)row_blocks<D>(&a, kNormRopeMaxCtas, 0);
      cq = (int)a.q_blocks;
      period = grid;
      norm_rope_rows_bwd_kernel<D, INTER><<<grid, kThreads, 0, stream>>>(a);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.partial == nullptr) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(D / 8, 2);
  cfg.blockDim = dim3(1024);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_rope_dw_kernel, static_cast<const float*>(a.partial), grid, D, cq, period,
                            a.dw[0], a.dw[1]);
}

template <int D, bool INTER, int STEPS>
void launch_append(AppendLaunch a, cudaStream_t stream) {
  using I = Chunk<D, STEPS>;
  const unsigned groups = token_groups(a.T), chunks = I::of(a.Hq) + 2 * I::of(a.Hk);
  a.by_chunks = FastDiv(chunks);
  // One warp for all of a token's chunks where there are tokens enough to fill
  // the device (16000 tokens, 4 + 4 heads, d = 128: 34 -> 31 us); few tokens are
  // spread chunk by chunk.
  a.span = groups >= 4u * a.sms;
  paged_append_kernel<D, INTER, STEPS><<<a.span ? groups : groups * chunks, kThreads, 0, stream>>>(a);
}

template <int D, bool INTER>
cudaError_t launch_paged_append_t(const AppendLaunch& a, cudaStream_t stream) {
  constexpr int kCost[4] = {100, 78, 62, 0};
  switch (steps_for<D>(a.Hq, a.Hk, 2, kCost)) {
    case 4:
      launch_append<D, INTER, 4>(a, stream);
      break;
    case 2:
      launch_append<D, INTER, 2>(a, stream);
      break;
    default:
      launch_append<D, INTER, 1>(a, stream);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeLaunch& a, cudaStream_t stream) {
  if (a.p.d == 64)
    return a.p.interleaved ? launch_norm_rope_t<64, true>(a, stream) : launch_norm_rope_t<64, false>(a, stream);
  return a.p.interleaved ? launch_norm_rope_t<128, true>(a, stream) : launch_norm_rope_t<128, false>(a, stream);
}

cudaError_t launch_norm_rope_bwd(const NormRopeLaunch& a, cudaStream_t stream) {
  if (a.p.d == 64)
    return a.p.interleaved ? launch_norm_rope_bwd_t<64, true>(a, stream) : launch_norm_rope_bwd_t<64, false>(a, stream);
  return a.p.interleaved ? launch_norm_rope_bwd_t<128, true>(a, stream)
                         : launch_norm_rope_bwd_t<128, false>(a, stream);
}

cudaError_t launch_paged_append(const AppendLaunch& a, cudaStream_t stream) {
  if (a.p.d == 64)
    return a.p.interleaved ? launch_paged_append_t<64, true>(a, stream) : launch_paged_append_t<64, false>(a, stream);
  return a.p.interleaved ? launch_paged_append_t<128, true>(a, stream) : launch_paged_append_t<128, false>(a, stream);
}

}  // namespace fa
