"""How the paged attention divides its work (CPU, compiled with g++).

``fa_paged_plan.cuh`` holds the index arithmetic that the CTAs share.  A driver
built from it walks random ragged batches (empty sequences, single tokens, long
chunks, lengths shorter than their chunk, unusual block sizes) and checks that
costs in closed form equal sums over the blocks, that the runs of all CTAs
together visit every key tile of every unit once and in order, that a unit that
is cut is continued by the CTAs right behind until one ends it, and that no run
costs more than its even share and what its two borders may move.
"""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "exact_io_aware_31_gb300", "csrc")

DRIVER = r"""
#include <cstdio>
#include <random>
#include <vector>
#include "fa_paged_plan.cuh"
using namespace fa::paged;
static int fail(const char* what, long long a, long long b, long long c) {
  std::printf("FAIL %s %lld %lld %lld\n", what, a, b, c);
  return 1;
}
struct Batch {
  std::vector<Seq> seqs;
  int S, Hk;
  Seq seq(int s) const { return seqs[s]; }
};
template <int D>
int run() {
  std::mt19937 g(7 + D);
  auto pick = [&](int lo, int hi) { return (int)(lo + g() % (unsigned)(hi - lo + 1)); };
  const int Gs[] = {1, 2, 3, 4, 5, 6, 8, 16, 20, 32, 33, 64, 128};
  for (int round = 0; round < 3000; ++round) {
    Batch p;
    p.S = pick(1, round % 10 ? 12 : 60);
    p.Hk = pick(1, 5);
    const int G = Gs[pick(0, 12)], grid = pick(0, 1) ? 152 : pick(1, 40);
    const bool is_short = G <= 32 && pick(0, 2) == 0;
    Shape sh = {0, 128 / G, 32 / G, pick(0, 3) > 0};
    sh.ut = is_short ? sh.t4 : 2 * sh.tt;
    const int ut = sh.ut;
    const int long_q = pick(0, 2) ? 3 : is_short ? 200 : 3000, long_kv = pick(0, 2) ? 400 : 9000;
    std::vector<long long> before(p.S + 1, 0);
    for (int s = 0; s < p.S; ++s) {
      bool bad = false;
      const int qn = pick(0, 4) ? pick(1, long_q) : 0;
      const int kv = pick(0, 9) ? qn + pick(0, long_kv) : pick(0, long_q);
      Seq q = make_seq(0, qn, kv, 1 << 29, 1 << 30, bad);
      p.seqs.push_back(q);
      long long sum = 0;
      for (int b = 0; b * ut < qn; ++b) {
        if (cost_before<D>(q, b, sh) != sum) return fail("cost_before", s, b, sum);
        int most = 0;  // by the definition, over the block's tokens
        for (int t = b * ut; t < qn && t < (b + 1) * ut; ++t) {
          const int see = sh.causal ? kv - qn + t + 1 : kv;
          most = see > most ? see : most;
        }
        const int n = most > 128 ? (most + 127) / 128 : 1;
        if (unit_tiles(q, b, sh) != n) return fail("unit_tiles", s, b, n);
        if (cost_of_block<D>(q, b, sh) <= 0) return fail("cost", s, b, 0);
        sum += cost_of_block<D>(q, b, sh);
      }
      if (cost_of_seq<D>(q, sh) != sum) return fail("cost_of_seq", s, sum, 0);
      before[s + 1] = before[s] + sum * p.Hk;
    }
    const long long total = before[p.S];
    const int ctas = ctas_for<D>(total, grid);
    if (ctas > grid || (total > 0) != (ctas > 0)) return fail("ctas", ctas, grid, total);
    const long long share = ctas ? total / ctas : 0;
    // every CTA's borders, as the kernel computes them
    Seq found_q = {0, 0, 0};
    auto spot = [&](int c, Spot* out) -> bool {
      const long long x = border(total, share, c, ctas);
      *out = {p.S, 0, 0, 0};
      for (int s = 0; s < p.S; ++s)
        if (x >= before[s] && x < before[s + 1]) {
          const long long per_head = (before[s + 1] - before[s]) / p.Hk;
          const int hk = (int)((x - before[s]) / per_head);
          int found = 0;
          for (int b = 0; b * ut < p.seqs[s].qn; ++b) {
            int j;
            if (!place<D>(p.seqs[s], x - before[s] - hk * per_head, b, sh, j)) continue;
            ++found;
            *out = {s, hk, b, j};
            const int n = unit_tiles(p.seqs[s], b, sh);
            if (n <= kNeverCut && j != 0 && j != n) return false;
            found_q = p.seqs[s];
          }
          return found == 1;
        }
      return x == total;
    };
    int s = 0, hk = 0, b = 0, j = 0;  // the tile that comes next
    bool open = false;                // the unit of the last segment goes on
    auto skip_empty = [&] { while (s < p.S && p.seqs[s].qn == 0) ++s; };
    skip_empty();
    long long dearest = 0;
    for (int s2 = 0; s2 < p.S; ++s2)
      for (int b2 = 0; b2 * ut < p.seqs[s2].qn; ++b2) {
        const Form f = sh.form(p.seqs[s2].qn - b2 * ut < ut ? p.seqs[s2].qn - b2 * ut : ut);
        const long long slack = 128 * (unit_cost<D>(f) + 3 * tile_cost<D>(f)) + 128;
        dearest = slack > dearest ? slack : dearest;
      }
    for (int c = 0; c < ctas; ++c) {
      Spot at, end;
      if (!spot(c + 1, &end) || !spot(c, &at)) return fail("spot", c, ctas, total);
      Walk w = walk_start(p, at, end, found_q, sh);
      Segment e;
      long long cost = 0;
      const bool owed = open;
      int segments = 0;
      while (walk_get(p, w, end, sh, e)) {
        if (w.at.s != s || w.at.hk != hk || w.at.b != b || e.j0 != j) return fail("walk", c, w.at.s, e.j0);
        if (open != (e.j0 > 0)) return fail("continued", c, w.at.s, e.j0);
        if (e.j1 <= e.j0 || e.j1 > e.n) return fail("segment", e.j0, e.j1, e.n);
        if (e.ntok < 1 || e.ntok > ut || e.tok0 + e.ntok > w.q.qn) return fail("tokens", e.tok0, e.ntok, ut);
        const int c0 = tile0_count(w.q, e, sh);
        int want = 0;
        for (int k = e.j0; k < e.j1 && e.ntok > sh.tt; ++k) {
          const int last = sh.causal ? w.q.kv - w.q.qn + e.tok0 + sh.tt - 1 : w.q.kv - 1;
          want += k * 128 <= last;
        }
        if (e.ntok > sh.tt && c0 != want) return fail("tile0_count", c0, want, sh.tt);
        const Form f = sh.form(e.ntok);
        cost += 128 * ((long long)tile_cost<D>(f) * (e.j1 - e.j0) + (e.j0 == 0 ? unit_cost<D>(f) : 0));
        open = e.j1 < e.n;
        ++segments;
        if (open) {
          j = e.j1;
        } else {
          j = 0;
          if (++b * ut >= w.q.qn) {
            b = 0;
            if (++hk == p.Hk) {
              hk = 0;
              ++s;
              skip_empty();
            }
          }
        }
        walk_next(p, w, end, sh, e);
      }
      if (owed && segments == 0) return fail("gap in a unit", c, ctas, total);
      // even shares, but for the two moved borders
      if (cost > share + 2 * dearest) return fail("share", c, cost, share);
    }
    if (s != p.S || open) return fail("cover", s, p.S, open);
  }
  return 0;
}
int main() {
  if (run<64>() || run<128>()) return 1;
  std::printf("OK\n");
  return 0;
}
"""


def test_runs_cover_every_unit_once(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    src = tmp_path / "plan.cpp"
    src.write_text(DRIVER)
    exe = tmp_path / "plan"
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-D__host__=", "-D__device__=", "-I", CSRC, str(src), "-o",
                        str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.strip() == "OK", out.stdout + out.stderr
