"""How the paged attention divides its work (CPU, compiled with g++).

``fa_paged_plan.cuh`` holds the index arithmetic that the CTAs share.  A driver
built from it walks random ragged batches (empty sequences, single tokens, long
chunks, lengths shorter than their chunk, unusual block sizes) and checks that
the tile counts in closed form equal sums over the blocks, that the runs of all
CTAs together visit every key tile of every unit once and in order, that a
unit that is cut is continued by the following CTAs until one ends it, and that
no run exceeds its even share by more than the two moved borders.
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
  int S, Hk, causal;
  Seq seq(int s) const { return seqs[s]; }
};
int main() {
  std::mt19937 g(7);
  auto pick = [&](int lo, int hi) { return (int)(lo + g() % (unsigned)(hi - lo + 1)); };
  for (int i = 0; i < 20000; ++i) {
    const unsigned n = pick(0, 40), m = pick(1, 200), a = pick(0, 400), b = pick(0, 500);
    long long want = 0;
    for (unsigned k = 0; k < n; ++k) want += (a * k + b) / m;
    if (floor_sum(n, m, a, b) != want) return fail("floor_sum", n, m, a);
  }
  const int uts[] = {1, 2, 3, 8, 21, 32, 64, 85, 128, 200, 256};
  for (int round = 0; round < 3000; ++round) {
    Batch p;
    p.S = pick(1, round % 10 ? 12 : 60);
    p.Hk = pick(1, 5);
    p.causal = pick(0, 3) > 0;
    const int ut = uts[pick(0, 10)], grid = pick(0, 1) ? 152 : pick(1, 40);
    const int long_q = pick(0, 2) ? 3 : 3000, long_kv = pick(0, 2) ? 400 : 9000;
    std::vector<long long> before(p.S + 1, 0);
    for (int s = 0; s < p.S; ++s) {
      bool bad = false;
      const int qn = pick(0, 4) ? pick(1, long_q) : 0;
      const int kv = pick(0, 9) ? qn + pick(0, long_kv) : pick(0, long_q);
      Seq q = make_seq(0, qn, kv, 1 << 29, 1 << 30, bad);
      p.seqs.push_back(q);
      long long sum = 0;
      for (int b = 0; b * ut < qn; ++b) {
        if (tiles_before(q, b, ut, p.causal) != sum) return fail("tiles_before", s, b, sum);
        int most = 0;  // by the definition, over the block's tokens
        for (int t = b * ut; t < qn && t < (b + 1) * ut; ++t) {
          const int see = p.causal ? kv - qn + t + 1 : kv;
          most = see > most ? see : most;
        }
        const int n = most > 128 ? (most + 127) / 128 : 1;
        if (unit_tiles(q, b, ut, p.causal) != n) return fail("unit_tiles", s, b, n);
        sum += n;
      }
      if (seq_tiles(q, ut, p.causal) != sum) return fail("seq_tiles", s, sum, 0);
      before[s + 1] = before[s] + sum * p.Hk;
    }
    const long long total = before[p.S];
    const int ctas = (int)(total < grid ? total : grid);
    const long long tol = snap_tolerance(total, ctas);
    // every CTA's run, as the kernel computes it
    struct Run { long long x0, x1; int s, hk, b, j; };
    auto at = [&](int c, Run* r) -> long long {
      const long long x = border(total, c, ctas);
      for (int s = 0; s < p.S; ++s)
        if (x >= before[s] && x < before[s + 1]) {
          int hk, b, j;
          const int moved = place(p.seqs[s], x - before[s], (before[s + 1] - before[s]) / p.Hk, ut, p.causal, tol, hk,
                                  b, j);
          if (r) r->s = s, r->hk = hk, r->b = b, r->j = j;
          return x + moved;
        }
      return total;
    };
    int s = 0, hk = 0, b = 0, j = 0;  // the tile that comes next
    bool open = false;                // the unit of the last segment goes on
    auto skip_empty = [&] { while (s < p.S && p.seqs[s].qn == 0) ++s; };
    skip_empty();
    long long seen = 0;
    for (int c = 0; c < ctas; ++c) {
      Run r = {0, 0, p.S, 0, 0, 0};
      r.x0 = at(c, &r);
      r.x1 = at(c + 1, nullptr);
      if (r.x1 < r.x0) return fail("run order", c, r.x0, r.x1);
      if (r.x1 - r.x0 > total / ctas + 1 + 2 * tol) return fail("run length", c, r.x1 - r.x0, total / ctas);
      Walk w = walk_start(p, r.x1 - r.x0, r.s, r.hk, r.b, r.j, ut);
      Segment e;
      while (walk_get(p, w, ut, e)) {
        if (w.s != s || w.hk != hk || w.b != b || e.j0 != j) return fail("walk", c, w.s, e.j0);
        if (open != (e.j0 > 0)) return fail("continued", c, w.s, e.j0);
        if (e.j1 <= e.j0 || e.j1 > e.n) return fail("segment", e.j0, e.j1, e.n);
        if (e.ntok < 1 || e.ntok > ut || e.tok0 + e.ntok > w.q.qn) return fail("tokens", e.tok0, e.ntok, ut);
        for (int tt = 1; tt < e.ntok; ++tt) {
          const int c0 = tile0_count(w.q, e, tt, p.causal);
          int want = 0;
          for (int k = e.j0; k < e.j1; ++k) {
            const int last = p.causal ? w.q.kv - w.q.qn + e.tok0 + tt - 1 : w.q.kv - 1;
            want += k * 128 <= last;
          }
          if (c0 != want) return fail("tile0_count", c0, want, tt);
        }
        seen += e.j1 - e.j0;
        open = e.j1 < e.n;
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
        walk_next(p, w, ut, e);
      }
    }
    if (seen != total || open) return fail("cover", seen, total, open);
  }
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
