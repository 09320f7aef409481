"""How the attention over shared keys divides its work (CPU, compiled with g++): the driver of tests/test_paged_plan.py
on entries of all kinds, among them a group's shared keys, which every one of its tokens sees."""

import shutil
import subprocess

import pytest

from tests.test_paged_plan import CSRC, DRIVER

CHANGES = [
    ("std::vector<Seq> seqs;", "std::vector<SharedSeq> seqs;"),
    ("Seq seq(int s) const", "SharedSeq seq(int s) const"),
    ("Seq q = make_seq(0, qn, kv, 1 << 29, 1 << 30, bad);",
     "SharedSeq q;\n      static_cast<Seq&>(q) = make_seq(0, qn, kv, 1 << 29, 1 << 30, bad);\n"
     "      q.row = s, q.page0 = 0, q.kind = pick(0, 2);"),
    ("const int see = sh.causal ? kv - qn + t + 1 : kv;",
     "const int see = sh.causal && q.kind != kPrefix ? kv - qn + t + 1 : kv;"),
    ("Seq found_q = {0, 0, 0};", "SharedSeq found_q = {};"),
    ("Walk w = walk_start", "WalkOf<SharedSeq> w = walk_start"),
    ("const int last = sh.causal ? w.q.kv", "const int last = sh.causal && w.q.kind != kPrefix ? w.q.kv"),
]


def test_runs_cover_every_unit_of_every_kind_once(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    text = DRIVER
    for old, new in CHANGES:
        assert text.count(old) == 1, old
        text = text.replace(old, new)
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text(text)
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-D__host__=", "-D__device__=", "-I", CSRC, str(src), "-o",
                        str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.strip() == "OK", out.stdout + out.stderr


PARTS = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "fa_paged_plan.cuh"
using namespace fa::paged;
int main() {
  unsigned long long seed = 1;
  auto next = [&](int n) { return int((seed = seed * 6364136223846793005ull + 1442695040888963407ull) >> 33) % n; };
  for (int round = 0; round < 3000; ++round) {
    const int sms = round % 3 ? 152 : 1 + next(178), tiles = 1 + next(2), heads = 1 << next(6);
    const int n = 1 + next(round % 10 ? 300 : 9000), most = round % 7 == 0 ? 1 << 30 : 1 << (4 + next(22));
    const int form = next(3);
    std::vector<int> keys(n);
    for (int i = 0; i < n; ++i) keys[i] = form == 0 ? most : form == 1 ? next(most) + 1 : next(8) ? next(40) : most;
    float all = 0.f, before = 0.f;
    for (int k : keys) all += (float)k;
    long long places = 0;
    for (int k : keys) {
      const int most_keys = part_keys(before * heads, all * heads, tiles, sms);
      int part = most_keys;
      const int parts = parts_of_keys(k, part);
      if (most_keys < kLeastPart || part % kPartStep || part < kPartStep || parts < 1 || part > most_keys * 3ll / 2 + 64)
        return printf("part %d of %d, %d of them\n", part, most_keys, parts), 1;
      if ((long long)parts * part < k || (parts - 1ll) * part >= (k > 0 ? k : 1))
        return printf("%d parts of %d keys for %d\n", parts, part, k), 1;
      if (parts > 1) places += (long long)parts * heads;
      before += (float)k;
    }
    if (places * tiles > shared_parts(sms))
      return printf("%lld places of %d row tiles (%d SMs, %d heads, %d entries)\n", places, tiles, sms, heads, n), 1;
  }
  puts("OK");
}
"""


def test_parts_of_few_rows_have_room_and_cover_their_keys(tmp_path):
    """Entries from one key to as many as a cache may have, in numbers whose keys are past what one part may hold."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    src, exe = tmp_path / "parts.cpp", tmp_path / "parts"
    src.write_text(PARTS)
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover", "-D__host__=",
                        "-D__device__=", "-I", CSRC, str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.strip() == "OK", out.stdout + out.stderr
