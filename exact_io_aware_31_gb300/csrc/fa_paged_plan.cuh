// How the paged attention kernels divide their work: pure index arithmetic, for
// host and device.
//
// A unit is one key head's block of `ut` new tokens of one sequence, with every
// key tile (128 keys) that the block sees; the units lie one after the other,
// sequence by sequence, key head by key head, block by block.  Each has a cost,
// and the row of all costs is cut into equal runs, one per CTA.  A role of a CTA
// walks its run as segments, each the part of one unit that lies in the run.
//
// Where sequences share their first keys (fa_paged_shared.cu), the shared keys of
// a group are an entry of their own in front: all of the group's tokens, one after
// the other, against those keys.  The group's sequences then begin behind them.
#pragma once

#include "fa_common.cuh"

namespace fa {
namespace paged {

// Which form a unit takes (fa_paged.cu).
enum Form { kTwoTiles, kOneTile, kFourCopies, kShortCopies };  // (the last: four copies, and no other form there)

// The launch's division: tokens of a unit, of a query tile, of a quarter tile.
struct Shape {
  int ut, tt, t4;
  int causal;
  __host__ __device__ Form form(int tokens) const {
    return tokens <= t4 ? (ut <= t4 ? kShortCopies : kFourCopies) : tokens <= tt ? kOneTile : kTwoTiles;
  }
};

// Cost of a unit: `tile` for each key tile, `unit` for its beginning and end, in
// tenths of a microsecond as traced on GB300 in batches of all forms.  (Four
// copies: what the SM's share of HBM takes for a tile; two tiles: the softmax.)
// The units' share was then moved until mixed batches took least: with too little
// for two tiles and too much for four copies, the CTAs of single tokens ended 15 us
// before the others (d = 128: 45, 35, 24 -> 75, 35, 15 took a step of 2 chunks of
// 509 among 14 single tokens from 64 to 60 us, 3 chunks of 200 among 97 from 208 to
// 197).  The kernels that hold four copies alone have shorter units: 10 and 12 there
// take 64 x 8 tokens, d = 64, from 41.8 to 41.2 us, and in the others 4 chunks of up
// to 225 among 25 single tokens, d = 64, from 31.6 to 35.8.
template <int D>
__host__ __device__ inline int tile_cost(Form f) {
  return D == 128 ? (f == kTwoTiles ? 15 : f == kOneTile ? 10 : 12) : (f == kTwoTiles ? 12 : f == kOneTile ? 7 : 6);
}
template <int D>
__host__ __device__ inline int unit_cost(Form f) {
  return D == 128 ? (f == kTwoTiles ? 75 : f == kOneTile ? 35 : f == kFourCopies ? 15 : 10)
                  : (f == kTwoTiles ? 60 : f == kOneTile ? 30 : f == kFourCopies ? 17 : 12);
}

struct Seq {
  int q0, qn, kv;  // first row, new tokens, keys
};

// An entry of a batch whose sequences share keys.
enum Kind { kAlone, kPrefix, kRest };  // a whole sequence; a group's shared keys; a sequence behind them
struct SharedSeq : Seq {
  int row, page0;  // its pages: entries of this row of the table from page0 on
  int kind;
};

// Whether tokens see only the keys up to their own.
__host__ __device__ inline int causal_in(const Seq&, int causal) { return causal; }
__host__ __device__ inline int causal_in(const SharedSeq& q, int causal) { return causal && q.kind != kPrefix; }

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

__host__ __device__ inline int blocks_of(const Seq& q, int ut) { return (q.qn + ut - 1) / ut; }

// Keys that tokens [.., hi) of the sequence see.
template <class Q>
__host__ __device__ inline int keys_upto(const Q& q, int hi, int causal) {
  return imax(0, causal_in(q, causal) ? q.kv - q.qn + hi : q.kv);
}

// Key tiles of block b, at least one (so that rows that see no key are written as well).
template <class Q>
__host__ __device__ inline int unit_tiles(const Q& q, int b, const Shape& sh) {
  return imax(1, (keys_upto(q, imin(q.qn, (b + 1) * sh.ut), sh.causal) + kTileRows - 1) >> 7);
}

// Cost of a unit that sees `keys` keys, in 128ths of the above: keys + 127
// stand for its tiles, so that sums over blocks are arithmetic series.
template <int D>
__host__ __device__ inline long long cost_of(long long blocks, long long keys, Form f) {
  return tile_cost<D>(f) * (keys + 127 * blocks) + 128 * unit_cost<D>(f) * blocks;
}

// Cost of blocks [0, b) of one key head, all of them full.
template <int D, class Q>
__host__ __device__ inline long long cost_before(const Q& q, int b, const Shape& sh) {
  const Form f = sh.form(sh.ut);
  if (!causal_in(q, sh.causal)) return cost_of<D>(b, (long long)b * q.kv, f);
  const int c = q.kv - q.qn;  // block i sees c + (i + 1) ut keys, or none
  const int z = c >= 0 ? 0 : imin(b, -c / sh.ut);
  const long long keys = (long long)(b - z) * c + (long long)sh.ut * ((long long)b * (b + 1) - (long long)z * (z + 1)) / 2;
  return cost_of<D>(b, keys, f);
}

template <int D, class Q>
__host__ __device__ inline long long cost_of_block(const Q& q, int b, const Shape& sh) {
  const int hi = imin(q.qn, (b + 1) * sh.ut);
  return cost_of<D>(1, keys_upto(q, hi, sh.causal), sh.form(hi - b * sh.ut));
}

// Of one key head.
template <int D, class Q>
__host__ __device__ inline long long cost_of_seq(const Q& q, const Shape& sh) {
  const int nb = blocks_of(q, sh.ut);
  return nb == 0 ? 0 : cost_before<D>(q, nb - 1, sh) + cost_of_block<D>(q, nb - 1, sh);
}

// CTAs that work of this total is given to: each gets more than the dearest
// tile's cost, so that every CTA behind a cut has a tile of the unit.
template <int D>
__host__ __device__ inline int ctas_for(long long total, int grid) {
  const long long most = total / (128 * (tile_cost<D>(kTwoTiles) + 1));
  return most >= grid ? grid : most > 0 ? (int)most : total > 0 ? 1 : 0;
}

// Border c of `ctas` runs of `total`, whose ctas-th part is `part`.
__host__ __device__ inline long long border(long long total, long long part, int c, int ctas) {
  const int rest = (int)(total - part * ctas);
  return c >= ctas ? total : part * c + imin(c, rest);
}

// Key tiles of a unit that place() never cuts: no tile of three is two away from both ends.
constexpr int kNeverCut = 3;

// Whether position y of a key head's cost lies in block b.  Then j is the key
// tile at which the unit is cut: 0 or its number of tiles (no cut) where that is
// a tile away, which costs less than a unit's other beginning and its partial outputs.
template <int D, class Q>
__host__ __device__ inline bool place(const Q& q, long long y, int b, const Shape& sh, int& j) {
  const long long at = y - cost_before<D>(q, b, sh);
  if (at < 0 || at >= cost_of_block<D>(q, b, sh)) return false;
  const Form f = sh.form(imin(q.qn, (b + 1) * sh.ut) - b * sh.ut);
  const int n = unit_tiles(q, b, sh);
  const long long in = at - 128 * unit_cost<D>(f);
  j = in <= 0 ? 0 : imin(n, (int)(in / (128 * tile_cost<D>(f))));
  if (j <= 1)
    j = 0;
  else if (n - j <= 1)
    j = n;
  return true;
}

// A place in the row of units: key tile j of block b of key head hk of sequence s.
struct Spot {
  int s, hk, b, j;
};

// Where a role stands in its walk through the run.
template <class Q>
struct WalkOf {
  Spot at;
  Q q;
};
using Walk = WalkOf<Seq>;

struct Segment {
  int tok0, ntok;  // first token (in the sequence), tokens
  int n, j0, j1;   // key tiles of the unit, of this segment
};

__host__ __device__ inline bool same_unit(const Spot& a, const Spot& b) { return a.s == b.s && a.hk == b.hk && a.b == b.b; }

// To the next unit.  P tells what a walk needs to know: `seq(s)` gives a sequence; S, Hk.
// Empty sequences are passed one by one: four chunks of 75 tokens against 300 keys
// (32 + 8 heads, d = 128) take 18 us, and 49 among 1020 empty ones.  Passing 32 at a
// time gained a quarter of that, but batches without empty ones took 3% more, or long
// chunks 5%: code of the softmax loop.
template <class P, class Q>
__host__ __device__ inline void walk_skip(const P& p, WalkOf<Q>& w, const Shape& sh) {
  w.at.j = 0;
  if (++w.at.b * sh.ut < w.q.qn) return;
  w.at.b = 0;
  if (++w.at.hk < p.Hk) return;
  w.at.hk = 0;
  while (++w.at.s < p.S) {
    w.q = p.seq(w.at.s);
    if (w.q.qn > 0) return;
  }
}

// The current segment of a run up to `end`; false at its end.
template <class P, class Q>
__host__ __device__ inline bool walk_get(const P& p, const WalkOf<Q>& w, const Spot& end, const Shape& sh, Segment& g) {
  if (w.at.s >= p.S) return false;
  const bool last = same_unit(w.at, end);
  if (last && w.at.j >= end.j) return false;
  g.tok0 = w.at.b * sh.ut;
  g.ntok = imin(sh.ut, w.q.qn - g.tok0);
  g.n = unit_tiles(w.q, w.at.b, sh);
  g.j0 = w.at.j;
  g.j1 = last ? end.j : g.n;
  return true;
}

template <class P, class Q>
__host__ __device__ inline void walk_next(const P& p, WalkOf<Q>& w, const Spot& end, const Shape& sh, const Segment& g) {
  if (same_unit(w.at, end))
    w.at.j = g.j1;  // the run's last segment
  else
    walk_skip(p, w, sh);
}

// `q` is sequence at.s (anything for at.s >= S).
template <class P, class Q>
__host__ __device__ inline WalkOf<Q> walk_start(const P& p, const Spot& at, const Spot& end, const Q& q,
                                                const Shape& sh) {
  WalkOf<Q> w = {at, q};
  if (at.s < p.S && !same_unit(at, end) && at.j >= unit_tiles(q, at.b, sh)) walk_skip(p, w, sh);
  return w;
}

// Key tiles of query tile 0 of a two-tile unit within the segment (tile 1
// sees every one of the unit's).
template <class Q>
__host__ __device__ inline int tile0_count(const Q& q, const Segment& g, const Shape& sh) {
  const int vis = keys_upto(q, g.tok0 + sh.tt, sh.causal);
  const int n0 = imin((vis + kTileRows - 1) >> 7, g.n);
  return imax(0, imin(g.j1, n0) - g.j0);
}

// The key tile that holds a sequence's last key (0 if it has none).
__host__ __device__ inline int last_tile(int kv) { return kv > 0 ? (kv - 1) >> 7 : 0; }

// Parts of an SM and fewest keys of one (an entry with few rows of a batch whose sequences
// share keys), and what their keys are multiples of.
constexpr int kPartsASm = 16, kLeastPart = 256, kPartStep = 64;

// Keys of the parts of such an entry that has `before` of all of those entries' `keys` (times
// their heads) in front of it: an eighth of a CTA's share, and half of that for the last fifth
// of the keys, which end when there is nothing else left to take.  With two row tiles (`tiles`)
// parts are twice as long, as there are half as many CTAs and places.
__host__ __device__ inline int part_keys(float before, float keys, int tiles, int sms) {
  const float share = keys / (kPartsASm * sms) * (5.f * before > 4.f * keys ? 0.5f : 1.f) * tiles;
  // (a share beyond all keys that there can be, 2^30, leaves every entry whole)
  const int n = (share < 1073741824.f ? (int)share : 1 << 30) / kPartStep * kPartStep + kPartStep;
  return imax(n, kLeastPart * tiles);
}
// The parts of an entry, as near to `part` keys as equal ones come: how many, and the keys of each
// but the last (64 x 330 keys, 32 + 8 heads, d = 128, took 26.8 us with parts of 256 and 74).
__host__ __device__ inline int parts_of_keys(int keys, int& part) {
  const int parts = imax(1, (keys + part / 2) / part);
  part = imax(1, (keys + parts - 1) / parts + kPartStep - 1) / kPartStep * kPartStep;
  part = imax(part, kPartStep);
  return imax(0, keys - 1) / part + 1;
}

// Parts that there is room for, of kPartRows rows (or half as many of twice the rows).  An entry
// of n keys in several parts of some L has at most 4/3 n / L; with W keys times heads in all and
// part_keys()' lengths these are at most 4/3 * 16 * 0.8 an SM for those that begin in the first
// four fifths, and 4/3 * 32 * 0.2 for the others: 25.6.  (There is room for entries cut at every
// L keys, too, up to 2 n / L parts each, 38.4 an SM, and for sums in fp32 that are off by a
// fifth: at d = 128 26 MB more of workspace than equal parts and exact sums need.)
constexpr int kMaxParts = 46;
constexpr int kPartRows = 16;
inline __host__ __device__ int shared_parts(int sms) { return kMaxParts * sms; }

}  // namespace paged
}  // namespace fa
