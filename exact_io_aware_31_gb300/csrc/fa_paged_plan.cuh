// How the paged attention kernel divides its work: pure index arithmetic, for
// host and device.
//
// A unit is one key head's block of `ut` new tokens of one sequence, with every
// key tile (128 keys) that the block sees; the units lie one after the other,
// sequence by sequence, key head by key head, block by block, and the row of all
// their key tiles is cut into equal runs, one per CTA.  A role of a CTA walks
// its run as segments, each the part of one unit that lies in the run.
#pragma once

#include "fa_common.cuh"

namespace fa {
namespace paged {

struct Seq {
  int q0, qn, kv;  // first row, new tokens, keys
};

__host__ __device__ inline int imin(int a, int b) { return a < b ? a : b; }
__host__ __device__ inline int imax(int a, int b) { return a > b ? a : b; }

// A sequence's entries, forced into the T rows and the `cap` keys there are.
__host__ __device__ inline Seq make_seq(int begin, int end, int kv, int T, int cap, bool& bad) {
  Seq q;
  q.q0 = imin(imax(begin, 0), T);
  const int q1 = imin(imax(end, q.q0), T);
  q.qn = q1 - q.q0;
  q.kv = imin(imax(kv, 0), cap);
  bad = bad || q.q0 != begin || q1 != end || q.kv != kv;
  return q;
}

// sum of floor((a i + b) / m) over i < n, by the reduction of a and b modulo m
// and the exchange of rows and columns of the lattice points under the line
// (Euclid's steps).
__host__ __device__ inline long long floor_sum(unsigned n, unsigned m, unsigned a, unsigned b) {
  long long sum = 0;
  while (n > 0) {
    sum += (long long)n * (n - 1) / 2 * (a / m) + (long long)n * (b / m);
    a %= m;
    b %= m;
    const unsigned long long top = (unsigned long long)a * n + b;
    if (top < m) break;
    n = (unsigned)(top / m);
    b = (unsigned)(top % m);
    const unsigned t = m;
    m = a;
    a = t;
  }
  return sum;
}

// Key tiles that tokens [.., hi) of the sequence see, at least one (so that
// rows that see no key are written as well).
__host__ __device__ inline int tiles_upto(const Seq& q, int hi, int causal) {
  const int vis = causal ? q.kv - q.qn + hi : q.kv;
  return imax(1, (vis + kTileRows - 1) >> 7);
}

__host__ __device__ inline int unit_tiles(const Seq& q, int b, int ut, int causal) {
  return tiles_upto(q, imin(q.qn, (b + 1) * ut), causal);
}

// Key tiles of blocks [0, b) of one key head, b < blocks of the sequence.
__host__ __device__ inline long long tiles_before(const Seq& q, int b, int ut, int causal) {
  if (!causal) return (long long)b * unit_tiles(q, 0, ut, 0);
  const int c = q.kv - q.qn;  // block i sees c + (i + 1) ut keys
  const int one = 128 - c < 0 ? 0 : imin(b, (128 - c) / ut);  // blocks with a single tile
  return one + floor_sum(b - one, 128, ut, (unsigned)(c + (one + 1) * ut + 127) * (b > one));
}

__host__ __device__ inline long long seq_tiles(const Seq& q, int ut, int causal) {  // of one key head
  const int nb = (q.qn + ut - 1) / ut;
  if (nb == 0) return 0;
  return (nb > 1 ? tiles_before(q, nb - 1, ut, causal) : 0) + unit_tiles(q, nb - 1, ut, causal);
}

// Border c of `ctas` equal runs of `total` tiles.
__host__ __device__ inline long long border(long long total, int c, int ctas) {
  return c >= ctas ? total : total * c / ctas;
}

// Tile x of a sequence (all key heads; `per_head` tiles each): its key head,
// block and key tile.  A tile within `tol` of its unit's border moves there:
// returns the distance moved, and j = the unit's tiles where it moved to the end.
__host__ __device__ inline int place(const Seq& q, long long x, long long per_head, int ut, int causal, long long tol,
                                     int& hk, int& b, int& j) {
  hk = (int)(x / per_head);
  const long long y = x - hk * per_head;
  int lo = 0, hi = (q.qn + ut - 1) / ut;  // tiles_before(lo) <= y < tiles_before(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (tiles_before(q, mid, ut, causal) <= y)
      lo = mid;
    else
      hi = mid;
  }
  b = lo;
  const int at = (int)(y - tiles_before(q, lo, ut, causal)), n = unit_tiles(q, lo, ut, causal);
  j = at <= tol ? 0 : n - at <= tol ? n : at;
  return j - at;
}

// How near to a unit's border a cut moves there: a sixteenth of a run, so that
// runs stay equal within an eighth and fewer units leave partial outputs.
__host__ __device__ inline long long snap_tolerance(long long total, int ctas) {
  return ctas > 0 ? total / ctas / 16 : 0;
}

// A run's segments: parts of units, each walked by every role on its own.
struct Walk {
  long long rem;  // key tiles left
  int s, hk, b, j;
  Seq q;
};

struct Segment {
  int tok0, ntok;  // first token (in the sequence), tokens
  int n, j0, j1;   // key tiles of the unit, of this segment
};

// What a walk needs to know: `seq(s)` gives a sequence, S, Hk, causal.
template <class P>
__host__ __device__ inline void walk_skip(const P& p, Walk& w, int ut) {  // to the next unit
  w.j = 0;
  if (++w.b * ut < w.q.qn) return;
  w.b = 0;
  if (++w.hk < p.Hk) return;
  w.hk = 0;
  while (++w.s < p.S) {
    w.q = p.seq(w.s);
    if (w.q.qn > 0) return;
  }
  w.rem = 0;
}

// `rem` tiles from tile j of block b of key head hk of sequence s on.
template <class P>
__host__ __device__ inline Walk walk_start(const P& p, long long rem, int s, int hk, int b, int j, int ut) {
  Walk w = {s >= p.S ? 0 : rem, s, hk, b, j, {0, 0, 0}};
  if (w.rem > 0) {
    w.q = p.seq(s);
    if (w.j == unit_tiles(w.q, w.b, ut, p.causal)) walk_skip(p, w, ut);
  }
  return w;
}

// The current segment; false at the run's end.
template <class P>
__host__ __device__ inline bool walk_get(const P& p, const Walk& w, int ut, Segment& g) {
  if (w.rem <= 0) return false;
  g.tok0 = w.b * ut;
  g.ntok = imin(ut, w.q.qn - g.tok0);
  g.n = unit_tiles(w.q, w.b, ut, p.causal);
  g.j0 = w.j;
  g.j1 = (int)(w.rem < g.n - w.j ? w.j + w.rem : g.n);
  return true;
}

template <class P>
__host__ __device__ inline void walk_next(const P& p, Walk& w, int ut, const Segment& g) {
  w.rem -= g.j1 - g.j0;
  if (w.rem > 0) walk_skip(p, w, ut);
}

// Key tiles of query tile 0 of a two-tile unit within the segment (tile 1
// sees every one of the unit's).
__host__ __device__ inline int tile0_count(const Seq& q, const Segment& g, int tt, int causal) {
  const int vis = causal ? q.kv - q.qn + g.tok0 + tt : q.kv;
  const int n0 = vis <= 0 ? 0 : imin((vis + kTileRows - 1) >> 7, g.n);
  return imax(0, imin(g.j1, n0) - g.j0);
}

// The key tile that holds a sequence's last key (0 if it has none).
__host__ __device__ inline int last_tile(int kv) { return kv > 0 ? (kv - 1) >> 7 : 0; }

}  // namespace paged
}  // namespace fa
