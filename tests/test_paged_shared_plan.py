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
